"""Verification of drafted trees and chains on the GPU: whole numbers, equal to the
float64 oracle's. Random numbers are inputs; a drawn border is 64-bit rounding away from
one of them with a chance below 1e-8 a row."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import operators as ops
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def draws(seed, batch, nodes, vocab, dt, tops=4):
    """Logits with a few likely tokens a row, a random tree, tokens that are often right."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((batch, nodes, vocab)) * 2
    likely = r.integers(0, vocab, (batch, nodes, tops))
    for b in range(batch):
        for i in range(nodes):
            x[b, i, likely[b, i]] = 14 - np.arange(tops) + r.standard_normal(tops)
    logits = torch.from_numpy(x).to(DT[dt])
    parents = np.array([[-1] + [int(r.integers(max(0, i - 4), i)) for i in range(1, nodes)] for _ in range(batch)],
                       np.int32).reshape(batch, nodes)
    tokens = np.array([[likely[b, max(parents[b, i], 0), r.integers(0, tops)] for i in range(nodes)] for b in range(batch)],
                      np.int32)
    u = r.random((batch, nodes)).astype(np.float32)
    return logits, tokens, parents, u


def gpu_tree(logits, tokens, parents, u, temperature=None):
    got = tq.verify_tree(logits.cuda(), torch.from_numpy(tokens).cuda(), torch.from_numpy(parents).cuda(),
                         torch.from_numpy(u).cuda(), None if temperature is None else torch.from_numpy(temperature).cuda())
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in got]


def check_tree(logits, tokens, parents, u, temperature=None):
    got = gpu_tree(logits, tokens, parents, u, temperature)
    want = ops.verify_tree(logits.double().numpy(), tokens, parents, u, temperature)
    for g, w in zip(got, want):
        assert np.array_equal(g, w), (g, w)
    return got


def check_chain(logits, tokens, q, u, temperature=None):
    got = tq.verify_chain(logits.cuda(), torch.from_numpy(tokens).cuda(), torch.from_numpy(q).cuda(),
                          torch.from_numpy(u).cuda(), None if temperature is None else torch.from_numpy(temperature).cuda())
    torch.cuda.synchronize()
    want = ops.verify_chain(logits.double().numpy(), tokens, q, u, temperature)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w), (g, w)
    return want


VOCABS = [1, 2, 63, 64, 65, 255, 1000, 1001, 4096, 32003]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_trees(gpu, dt, vocab):
    say(f"tree {dt} {vocab}")
    logits, tokens, parents, u = draws(vocab, 7, 9, vocab, dt)
    t = np.array([0.7, 1.0, 0.0, 1.3, -1.0, 100.0, 0.01], np.float32)
    check_tree(logits, tokens, parents, u)
    check_tree(logits, tokens, parents, u, t)


def chain_of(seed, batch, nodes, vocab, dt):
    logits, tokens, _, u = draws(seed, batch, nodes, vocab, dt)
    r = np.random.default_rng(seed + 1)
    near = logits.double().numpy()[:, :-1] + r.standard_normal((batch, nodes - 1, vocab)) * 0.5
    q = np.exp(near - near.max(-1, keepdims=True))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    for b in range(batch):
        for j in range(nodes - 1):
            tokens[b, j + 1] = r.choice(vocab, p=q[b, j].astype(np.float64) / q[b, j].astype(np.float64).sum())
    return logits, tokens, q, u


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_chains(gpu, dt, vocab):
    say(f"chain {dt} {vocab}")
    logits, tokens, q, u = chain_of(vocab, 8, 6, vocab, dt)
    t = np.array([0.7, 1.0, 0.0, 1.3, -1.0, 100.0, 0.01, 1.0], np.float32)
    check_chain(logits, tokens, q, u)
    check_chain(logits, tokens, q, u, t)


def test_large_vocabulary(gpu):
    logits, tokens, parents, u = draws(1, 3, 8, 129280, "bf16")
    check_tree(logits, tokens, parents, u)
    logits, tokens, q, u = chain_of(2, 3, 4, 129280, "f32")
    check_chain(logits, tokens, q, u)


@pytest.mark.parametrize("nodes", [1, 2, 33, 64, 65, 200, 1024])
def test_node_counts(gpu, nodes):
    say(f"nodes {nodes}")
    logits, tokens, parents, u = draws(nodes, 2, nodes, 50, "f32")
    check_tree(logits, tokens, parents, u)
    logits, tokens, q, u = chain_of(nodes, 2, nodes, 50, "f32")
    check_chain(logits, tokens, q, u)


def test_many_sequences(gpu):
    logits, tokens, parents, u = draws(3, 500, 4, 300, "f16")
    check_tree(logits, tokens, parents, u)
    logits, tokens, q, u = chain_of(3, 500, 4, 300, "f16")
    want = check_chain(logits, tokens, q, u)
    assert len(set(want[0].tolist())) == 4  # every outcome occurs


@pytest.mark.parametrize("vocab", [2048, 2049, 4100, 131072, 300001])
def test_ends_of_the_random_numbers(gpu, vocab):
    """The first and the last place with weight, over one chunk, several, and more than a wave has lanes."""
    say(f"ends {vocab}")
    x = torch.full((1, 4, vocab), -float("inf"))
    x[0, 0, [5, vocab - 1]] = torch.tensor([1.0, 1.5])
    x[0, 1, vocab // 2 : vocab // 2 + 9] = -2.0
    x[0, 2] = torch.randn(vocab, generator=torch.Generator().manual_seed(vocab))
    x[0, 3, vocab - 2] = 0.0
    tokens, parents = np.zeros((1, 1), np.int32), np.full((1, 1), -1, np.int32)
    for value in (0.0, float(np.nextafter(np.float32(1), np.float32(0))), 0.37):
        u = np.full((1, 1), value, np.float32)
        for i in range(4):
            for t in (None, np.full(1, 0.5, np.float32), np.zeros(1, np.float32)):
                check_tree(x[:, i : i + 1].contiguous(), tokens, parents, u, t)


def test_an_empty_batch(gpu):
    x = torch.zeros((0, 3, 50), device=gpu)
    i, u = torch.zeros((0, 3), dtype=torch.int32, device=gpu), torch.zeros((0, 3), device=gpu)
    assert [t.shape for t in tq.verify_tree(x, i, i, u)] == [(0, 3), (0,), (0,)]
    assert [t.shape for t in tq.verify_chain(x, i, torch.zeros((0, 2, 50), device=gpu), u)] == [(0,), (0,)]


def test_ties_and_masked_vocabularies(gpu):
    """Equal logits, rows with a few finite places, with none, with +inf and NaN, at every
    temperature, for random numbers at the ends of their range."""
    vocab = 700
    x = torch.full((1, 8, vocab), -float("inf"))
    x[0, 0] = 3.0
    x[0, 1, 699] = -5.0
    x[0, 2, [5, 600]] = 1.0
    x[0, 4, [7, 300, 650]] = float("inf")
    x[0, 4, 8] = 1e30
    x[0, 5, 100:500] = float("nan")
    x[0, 5, [50, 450, 550]] = 2.0
    x[0, 6] = torch.linspace(-3e38, 3e38, vocab)
    x[0, 7, 0] = -3.4e38
    tokens = np.zeros((1, 8), np.int32)
    parents = np.full((1, 8), -1, np.int32)
    for dt in ("f32", "bf16"):
        for value in (0.0, 0.5, 0.999, float(np.nextafter(np.float32(1), np.float32(0))), 1.0, 2.0, -1.0, float("nan")):
            u = np.full((1, 8), value, np.float32)
            for t in (None, np.zeros(1, np.float32), np.full(1, 0.3, np.float32), np.full(1, np.nan, np.float32)):
                rows = x.to(DT[dt])
                for i in range(8):  # each row as the tree's root
                    check_tree(rows[:, i : i + 1].contiguous(), tokens[:, :1], parents[:, :1], u[:, :1], t)


def test_tree_shapes(gpu):
    """Twins, padding nodes, forward and cyclic parents, tokens outside the vocabulary."""
    vocab = 40
    logits = torch.full((1, 8, vocab), -20.0)
    for node, token in enumerate([3, 5, 7, 9, 3, 5, 3, 1]):
        logits[0, node, token] = 20.0
    u = np.full((1, 8), 0.5, np.float32)
    for parents, tokens, path in [
        ([-1, 0, 0, 0, 1, 2, 2, 3], [0, 4, 3, 3, 5, 7, 7, 9], [0, 2, 5]),  # the first twin wins
        ([-1, -1, -1, -1, -1, -1, -1, -1], [3] * 8, [0]),
        ([0, 1, 2, 3, 4, 5, 6, 7], [3] * 8, [0]),  # a node under itself is under nobody
        ([7, 7, 7, 7, 7, 7, 7, 0], [3] * 8, [0, 7]),  # a parent behind its child is none
        ([-1, 0, 1, 2, 3, 4, 5, 6], [0, 3, 5, 7, 9, 3, 5, 3], [0, 1, 2, 3, 4, 5, 6, 7]),
        ([2 ** 31 - 1, 0, 2 ** 31 - 1, -(2 ** 31), 1, 4, 5, 6], [-1, 3, -1, 2 ** 31 - 1, 5, -1, 5, 3], [0, 1, 4]),
    ]:
        got = check_tree(logits, np.array([tokens], np.int32), np.array([parents], np.int32), u)
        assert got[0][0, : got[1][0]].tolist() == path


def test_chain_edges(gpu):
    vocab = 30
    logits = torch.zeros((6, 2, vocab))
    q = np.full((6, 1, vocab), 1 / vocab, np.float32)
    tokens = np.array([[0, 3], [0, -1], [0, vocab], [0, 2 ** 31 - 1], [0, 3], [0, 4]], np.int32)
    u = np.full((6, 2), 0.999, np.float32)
    q[0] = 1.0  # over p everywhere: no residual, so p itself
    logits[4] = -float("inf")  # nothing to sample: -1
    q[5, 0] = np.nan
    want = check_chain(logits, tokens, q, u)
    assert want[1][4] == -1
    u[:] = 0.0
    check_chain(logits, tokens, q, u)


def test_strided_rows(gpu):
    logits, tokens, parents, u = draws(5, 3, 4, 257, "bf16")
    wide = torch.zeros((3, 8, 300), dtype=torch.bfloat16, device=gpu)
    wide[:, ::2, 3:260] = logits.cuda()
    got = tq.verify_tree(wide[:, ::2, 3:260], torch.from_numpy(tokens).cuda(), torch.from_numpy(parents).cuda(),
                         torch.from_numpy(u).cuda())
    for g, w in zip(got, ops.verify_tree(logits.double().numpy(), tokens, parents, u)):
        assert np.array_equal(g.cpu().numpy(), w)
    logits, tokens, q, u = chain_of(6, 3, 4, 257, "f32")
    wide = torch.zeros((3, 8, 300), device=gpu)
    wide[:, ::2, 3:260] = logits.cuda()
    wq = torch.zeros((3, 6, 259), device=gpu)
    wq[:, ::2, 1:258] = torch.from_numpy(q).cuda()
    got = tq.verify_chain(wide[:, ::2, 3:260], torch.from_numpy(tokens).cuda(), wq[:, ::2, 1:258], torch.from_numpy(u).cuda())
    for g, w in zip(got, ops.verify_chain(logits.double().numpy(), tokens, q, u)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_graph_replays_and_another_stream(gpu):
    sets = [draws(7 + i, 4, 6, 5000, "bf16") for i in range(4)]
    chains = [chain_of(17 + i, 4, 6, 5000, "bf16") for i in range(4)]
    a = [x.cuda() if torch.is_tensor(x) else torch.from_numpy(x).cuda() for x in sets[0]]
    c = [x.cuda() if torch.is_tensor(x) else torch.from_numpy(x).cuda() for x in chains[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.verify_tree(*a)
        tq.verify_chain(*c)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tree, chain = tq.verify_tree(*a), tq.verify_chain(*c)
    for i in (1, 2, 3, 0):
        for have, new in zip(a + c, sets[i] + chains[i]):
            have.copy_(new if torch.is_tensor(new) else torch.from_numpy(new))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ops.verify_tree(sets[i][0].double().numpy(), *sets[i][1:])
        want += ops.verify_chain(chains[i][0].double().numpy(), *chains[i][1:])
        for g, w in zip(tree + chain, want):
            assert np.array_equal(g.cpu().numpy(), w)
