"""Pins of the float64 oracle of the operators around the projection, each against
something other than the oracle: closed forms, torch's own float64 functions, counts
of samples, finite differences."""

import numpy as np
import pytest
import torch

from oracle import operators as ops


def test_attention_of_equal_keys_is_the_mean_of_the_seen_values():
    rng = np.random.default_rng(1)
    b, n, hq, hkv, d = 1, 4, 4, 2, 16
    q = rng.standard_normal((b, n, hq, d))
    k = np.ones((b, n, hkv, d))
    v = rng.standard_normal((b, n, hkv, d))
    kc = np.ones((3, 2, hkv, d))
    vc = rng.standard_normal((3, 2, hkv, d))
    table = np.array([[2, 0]])
    mask = np.array([[0b1, 0b11, 0b101, 0]])
    out, weight, _ = ops.tree_attention(q, k, v, mask, kc, vc, table, np.array([3]), 0.25)
    cached = [vc[2, 0], vc[2, 1], vc[0, 0]]  # positions 0, 1, 2
    for i, seen in enumerate([[0], [0, 1], [0, 2], []]):
        for h in range(hq):
            rows = np.array([c[h // 2] for c in cached] + [v[0, t, h // 2] for t in seen])
            assert np.allclose(out[0, i, h], rows.mean(0), atol=1e-14)
            assert np.allclose(weight[0, i, h], np.abs(rows).mean(0), atol=1e-14)
    none, _, _ = ops.tree_attention(q, k, v, mask * 0, kc, vc, table, np.array([0]), 0.25)
    assert np.array_equal(none, np.zeros_like(none))


def test_attention_against_torch_float64():
    rng = np.random.default_rng(2)
    b, n, h, d = 2, 5, 3, 32
    q, k, v = (rng.standard_normal((b, n, h, d)) for _ in range(3))
    causal = np.array([[(1 << (i + 1)) - 1 for i in range(n)]] * b)
    got, _, _ = ops.tree_attention(q, k, v, causal, np.zeros((1, 1, h, d)), np.zeros((1, 1, h, d)),
                                   np.zeros((b, 1), int), np.zeros(b, int), d ** -0.5)
    t = [torch.from_numpy(a.transpose(0, 2, 1, 3).copy()) for a in (q, k, v)]
    want = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=True).numpy().transpose(0, 2, 1, 3)
    assert np.abs(got - want).max() < 1e-13


def test_append_places_rows_by_position():
    k = np.arange(2 * 3 * 1 * 2).reshape(2, 3, 1, 2)
    kc, vc = ops.cache_append(k, -k, np.zeros((4, 2, 1, 2), int), np.zeros((4, 2, 1, 2), int),
                              np.array([[1, 3], [2, -1]]), np.array([1, 1]),
                              np.array([[0, 2, -1], [1, 0, 0]]), np.array([2, 3]))
    assert kc[1, 1, 0].tolist() == [0, 1] and kc[3, 0, 0].tolist() == [4, 5]  # sequence 0: nodes 0 and 2
    assert kc[2, 1, 0].tolist() == [8, 9]  # sequence 1: node 1; then a page of -1
    assert np.count_nonzero(kc.any(-1)) == 3 and np.array_equal(vc, -kc)


def test_sample_counts_follow_the_weights():
    w = np.array([0.0, 1.0, 0.0, 3.0, 4.0, 0.0])
    got = [ops.sample(w, (i + 0.5) / 80) for i in range(80)]
    assert [got.count(t) for t in range(6)] == [0, 10, 0, 30, 40, 0]
    assert ops.sample(w, 0.0) == 1 and ops.sample(w, 0.125) == 3 and ops.sample(w, 1.0) == 4
    assert ops.sample(w * 0, 0.5) == -1 and ops.sample(w, np.nan) == 1


def test_weights_against_torch_softmax_and_edges():
    x = np.random.default_rng(3).standard_normal(50) * 5
    w = ops.weights(x, 0.7)
    assert np.allclose(w / w.sum(), torch.softmax(torch.from_numpy(x) / 0.7, 0).numpy(), atol=1e-15)
    assert ops.weights(np.array([1.0, 3.0, 3.0]), 0.0).tolist() == [0, 1, 0]
    assert ops.weights(np.array([1.0, np.nan, np.inf, np.inf]), 1.0).tolist() == [0, 0, 1, 1]
    assert ops.weights(np.array([-np.inf, np.nan]), 1.0).tolist() == [0, 0]


def test_tree_walk_takes_the_first_matching_child():
    logits = np.full((1, 5, 4), -np.inf)
    for node, token in enumerate([2, 1, 3, 0, 0]):
        logits[0, node, token] = 0.0
    tokens = np.array([[9, 1, 2, 2, 3]])
    parents = np.array([[-1, 0, 0, 0, 2]])
    acc, count, after = ops.verify_tree(logits, tokens, parents, np.full((1, 5), 0.5))
    assert acc.tolist() == [[0, 2, 4, -1, -1]] and count.tolist() == [3] and after.tolist() == [0]


def test_chain_sampling_keeps_the_targets_distribution():
    """Drafts from q, accepted or replaced, come out with the target's probabilities: counted
    over an even grid of random numbers."""
    p, q = np.array([0.5, 0.25, 0.25]), np.array([0.25, 0.25, 0.5], np.float32)
    logits = np.log(np.stack([p, p]))[None]
    m = 64
    got = np.zeros(3)
    for x in range(3):
        for i in range(m):
            for j in range(m):
                c, t = ops.verify_chain(logits, np.array([[0, x]]), q[None, None], np.array([[(i + 0.5) / m, (j + 0.5) / m]]))
                got[x if c[0] == 2 else t[0]] += q[x]
    assert np.allclose(got / got.sum(), p, atol=1e-12)


def test_distill_against_torch_and_differences():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 12))
    index = np.array([[3, 7, -1], [0, 0, 11]])
    top = rng.standard_normal((2, 3))
    w = np.array([0.5, 2.0])
    loss, grad, p, t = ops.distill(x, index, top, w, 1.7)
    for r in range(2):
        target = torch.from_numpy(t[r])
        lp = torch.log_softmax(torch.from_numpy(x[r]) / 1.7, 0)
        there = index[r] >= 0
        ty = torch.softmax(torch.from_numpy(top[r][there]) / 1.7, 0)
        want = (ty * ty.log()).sum() - (target * lp).sum()
        assert abs(loss[r] - want.item()) < 1e-14
        for i in range(12):
            step = np.zeros_like(x)
            step[r, i] = 1e-6
            up, down = ops.distill(x + step, index, top, w, 1.7)[0], ops.distill(x - step, index, top, w, 1.7)[0]
            assert abs((up[r] - down[r]) / 2e-6 * w[r] - grad[r, i]) < 1e-8
    empty = ops.distill(x, index * 0 - 1, top, w, 1.0)
    assert not empty[0].any() and not empty[1].any()


@pytest.mark.parametrize("planted", ["mask", "page", "scale"])
def test_planted_mistakes_move_the_oracle(planted):
    rng = np.random.default_rng(5)
    b, n, h, d = 1, 3, 1, 16
    q, k, v = (rng.standard_normal((b, n, h, d)) for _ in range(3))
    kc, vc = rng.standard_normal((2, 4, 2, h, d))
    mask, table, scale = np.array([[1, 3, 5]]), np.array([[1, 0]]), 0.25
    want = ops.tree_attention(q, k, v, mask, kc, vc, table, np.array([3]), scale)[0]
    if planted == "mask":
        mask = mask | 4
    if planted == "page":
        table = table[:, ::-1]
    if planted == "scale":
        scale = 0.26
    got = ops.tree_attention(q, k, v, mask, kc, vc, table, np.array([3]), scale)[0]
    assert np.abs(got - want).max() > 1e-3
