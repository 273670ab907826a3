"""Attention of packed prompts on the GPU, against the float64 oracle. Tolerances as derived in
test_gpu_tree_attention: roundings of the weights and the output, fp32 sums over the head and over the keys."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import rows as oracle
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def bound(dt, dim, keys, want, weight, spread):
    h, f = torch.finfo(DT[dt]).eps / 2, 2.0 ** -24
    tol = h * np.abs(want) + (h + (2 * (dim + 2) * spread[..., None] + keys + 64) * f) * weight
    return tol + (2.0 ** -24 if dt == "f16" else 2.0 ** -133)


def rows_of(seed, dt, tokens, hq, hkv, dim, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((tokens, hq + 2 * hkv, dim), generator=g) * spread).to(DT[dt])


def check(got, qkv, heads, offsets, dt, scale=None, before=0.0):
    q, k, v = (t.double().numpy() for t in qkv.split(heads, dim=1))
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, weight, spread, seen = oracle.prompt_attention(q, k, v, offsets, scale)
    keys = max([b - a for a, b in zip(offsets, offsets[1:])], default=0)
    got = got.double().cpu().numpy()
    assert (got[~seen] == before).all(), "a row outside of all sequences was written"
    assert np.isfinite(got[seen]).all()
    over = (np.abs(got - want) - bound(dt, q.shape[2], keys, want, weight, spread))[seen]
    if over.size:
        assert over.max() <= 0, f"{over.max():.3g} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


def run(seed, dt, lengths, hq, hkv, dim, *, front=0, behind=0, spread=1.0, scale=None):
    offsets = [front]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    heads = [hq, hkv, hkv]
    qkv = rows_of(seed, dt, offsets[-1] + behind, hq, hkv, dim, spread)
    g = qkv.cuda()
    out = torch.full((qkv.shape[0], hq, dim), 7.0, dtype=DT[dt], device="cuda")
    got = tq.prompt_attention(*g.split(heads, dim=1), torch.tensor(offsets, dtype=torch.int32, device="cuda"), scale=scale, out=out)
    torch.cuda.synchronize()
    assert got is out
    check(out, qkv, heads, offsets, dt, scale, 7.0)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257])
def test_every_length(gpu, dt, dim, length):
    say(f"{dt} {dim} {length}")
    run(length, dt, [length], 2, 1, dim)


@pytest.mark.parametrize("dim", [16, 32, 48, 80, 96, 112, 144, 160, 192, 208, 240])
def test_every_head_size(gpu, dim):
    say(f"dim {dim}")
    run(dim, "bf16" if dim % 32 else "f16", [70, 5, 140], 4, 2, dim)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (8, 8), (5, 1), (12, 2), (40, 8), (16, 4), (24, 3)])
def test_every_group(gpu, hq, hkv):
    say(f"heads {hq} {hkv}")
    run(hq, "bf16", [90, 33], hq, hkv, 64)


@pytest.mark.parametrize("lengths", [[0], [0, 0, 0], [1] * 200, [0, 1, 0, 0, 130, 0], [3, 0, 100, 1, 1, 64, 64, 0, 31],
                                     [127, 1, 128, 2], [129, 129], [17] * 20, [1, 300], [300, 1]])
@pytest.mark.parametrize("front,behind", [(0, 0), (3, 0), (0, 5), (130, 200)])
def test_packed_batches(gpu, lengths, front, behind):
    say(f"{lengths[:8]} {front} {behind}")
    if sum(lengths) + front + behind == 0:
        front = 1
    run(len(lengths), "bf16", lengths, 4, 2, 128, front=front, behind=behind)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [48, 64, 96, 128])
@pytest.mark.parametrize("lengths", [[400], [1, 130, 0, 200, 69], [3] * 20 + [64, 33, 128, 115]])
def test_two_row_tiles(gpu, dt, dim, lengths):
    """So many heads that a wave takes two row tiles; a few of them are looked at."""
    say(f"two row tiles {dt} {dim} {lengths[:5]}")
    hq, hkv, front, behind = 352, 176, 2, 5
    offsets = np.cumsum([front, *lengths]).tolist()
    qkv = rows_of(dim, dt, offsets[-1] + behind, hq, hkv, dim)
    qkv[offsets[-1]:] = float("nan")
    out = torch.full((qkv.shape[0], hq, dim), 7.0, dtype=DT[dt], device="cuda")
    tq.prompt_attention(*qkv.cuda().split([hq, hkv, hkv], dim=1), torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
    for h in (0, 3, 175, 350):
        some = qkv[:, [h, hq + h // 2, hq + hkv + h // 2]]
        check(out[:, [h]], some, [1, 1, 1], offsets, dt, None, 7.0)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_odd_values_under_two_row_tiles(gpu, dt, dim):
    """Infinities among the values: rows that do not see them keep their bits, others get them."""
    hq, n = 352, 400
    offsets = torch.tensor([0, 150, n], dtype=torch.int32, device="cuda")
    qkv = rows_of(dim + 1, dt, n, hq, hq, dim).cuda()
    clean = tq.prompt_attention(*qkv.split([hq] * 3, dim=1), offsets)
    qkv[100, 2 * hq + 7, 3] = float("inf")
    qkv[390, 2 * hq + 7, 5] = -float("inf")
    out = tq.prompt_attention(*qkv.split([hq] * 3, dim=1), offsets)
    changed = torch.zeros((n, hq, dim), dtype=torch.bool, device="cuda")
    changed[100:150, 7, 3] = True
    changed[390:, 7, 5] = True
    assert torch.equal(out[~changed], clean[~changed])
    assert (out[100:150, 7, 3] == float("inf")).all() and (out[390:, 7, 5] == -float("inf")).all()


def test_many_sequences(gpu):
    """More of them than a wave has lanes, some empty."""
    run(4, "f16", [(7 * b) % 11 for b in range(300)], 2, 1, 64)


@pytest.mark.parametrize("dt,dim,hq", [("bf16", 128, 4), ("f16", 64, 2), ("bf16", 256, 2)])
def test_longer(gpu, dt, dim, hq):
    say(f"longer {dt} {dim}")
    run(dim, dt, [1021, 513], hq, 2, dim, behind=40)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("spread", [0.01, 4.0, 12.0])
def test_score_sizes(gpu, dt, spread):
    run(11, dt, [200, 61], 4, 2, 64, spread=spread)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 3.0])
def test_scales(gpu, scale):
    run(12, "bf16", [100, 40], 2, 1, 64, scale=scale)


def test_rising_scores(gpu):
    """Each key scores above all before it, so every tile raises the base."""
    for dt in DT:
        n, dim = 400, 64
        qkv = torch.zeros((n, 3, dim))
        qkv[:, 0, 0] = 8.0
        qkv[:, 1, 0] = torch.arange(n) * 0.25
        qkv[:, 2] = torch.randn((n, dim), generator=torch.Generator().manual_seed(1))
        qkv = qkv.to(DT[dt])
        out = tq.prompt_attention(*qkv.cuda().split(1, dim=1), torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        check(out, qkv, [1, 1, 1], [0, n], dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_none_reach_only_rows_that_see_them(gpu, dt, bad):
    """In keys and in values, of a row's own sequence behind it, of other sequences, and in rows of none."""
    lengths, dim, behind = [70, 130, 20], 128, 9
    offsets = [0, 70, 200, 220]
    qkv = rows_of(5, dt, 220 + behind, 4, 2, dim)
    spoiled = qkv.clone()
    for at in (69, 150, 219):
        spoiled[at, 5, 3] = bad   # a key of kv head 1
        spoiled[at, 7, 17] = bad  # a value of kv head 1
    spoiled[220:] = bad
    out = torch.zeros((229, 4, dim), dtype=DT[dt], device="cuda")
    tq.prompt_attention(*spoiled.cuda().split([4, 2, 2], dim=1), torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
    clean = tq.prompt_attention(*qkv.cuda().split([4, 2, 2], dim=1), torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    sees = torch.zeros(220, dtype=torch.bool)
    sees[69], sees[150:200], sees[219] = True, True, True
    out, clean = out[:220].cpu(), clean[:220].cpu()
    assert torch.equal(out[:, :2], clean[:, :2])
    assert torch.equal(out[~sees], clean[~sees])
    assert not torch.isfinite(out[sees][:, 2:]).all(-1).any()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_an_infinite_value_that_a_row_sees(gpu, dt):
    n, dim = 100, 64
    qkv = rows_of(6, dt, n, 2, 1, dim)
    qkv[80, 3, 5], qkv[90, 3, 6] = float("inf"), -float("inf")
    out = tq.prompt_attention(*qkv.cuda().split([2, 1, 1], dim=1), torch.tensor([0, n], dtype=torch.int32, device="cuda")).cpu()
    assert torch.isfinite(out[:80]).all()
    assert (out[80:, :, 5] == float("inf")).all() and (out[90:, :, 6] == -float("inf")).all()
    rest = torch.ones(dim, dtype=torch.bool)
    rest[5] = rest[6] = False
    assert torch.isfinite(out[:, :, rest]).all()


def test_a_key_that_no_row_weighs(gpu):
    """Scores of -inf leave nothing of their keys; a row of nothing else gets zeros."""
    n, dim = 40, 64
    qkv = torch.randn((n, 3, dim), generator=torch.Generator().manual_seed(2))
    qkv[:, 0] = qkv[:, 0].abs() + 0.1
    qkv[3:5, 1] = -float("inf")
    qkv = qkv.bfloat16()
    out = tq.prompt_attention(*qkv.cuda().split(1, dim=1), torch.tensor([0, 3, 4, n], dtype=torch.int32, device="cuda")).cpu()
    assert torch.isfinite(out).all() and not out[3].any() and not out[4].any()


def test_strides(gpu):
    """Heads first, rows apart, results likewise."""
    lengths, heads, dim = [50, 77], [4, 2, 2], 64
    qkv = rows_of(8, "bf16", 127, 4, 2, dim)
    offsets = torch.tensor([0, 50, 127], dtype=torch.int32, device="cuda")
    q, k, v = (t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in qkv.split(heads, dim=1))
    wide = torch.zeros((127, 9, dim + 8), dtype=torch.bfloat16, device="cuda")
    out = wide[:, 2:6, :dim]
    tq.prompt_attention(q, k, v, offsets, out=out)
    check(out, qkv, heads, [0, 50, 127], "bf16")
    wide[:, 2:6, :dim] = 0
    assert not wide.any()


@pytest.mark.parametrize("offsets", [[-5, 40, 90], [0, 40, 5000], [60, 20, 90], [90, 0], [2 ** 31 - 1, -2 ** 31], [50, 50]])
def test_offsets_out_of_range_stay_in_the_buffers(gpu, offsets):
    """What the rows hold is not stated where offsets do not ascend; the guards around out stay."""
    n, dim = 90, 64
    qkv = rows_of(9, "bf16", n, 2, 1, dim).cuda()
    room = torch.full((n + 256, 2, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    tq.prompt_attention(*qkv.split([2, 1, 1], dim=1), torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=room[128:128 + n])
    torch.cuda.synchronize()
    assert (room[:128] == 7).all() and (room[128 + n:] == 7).all()


def test_same_bits_and_other_offsets_in_a_graph(gpu):
    """A captured call, replayed over other offsets and other rows, with eager work in between."""
    n, dim, heads = 300, 128, [8, 2, 2]
    qkv = rows_of(10, "bf16", n, 8, 2, dim).cuda()
    offsets = torch.tensor([0, 300, 300, 300], dtype=torch.int32, device="cuda")
    out = torch.zeros((n, 8, dim), dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        tq.prompt_attention(*qkv.split(heads, dim=1), offsets, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tq.prompt_attention(*qkv.split(heads, dim=1), offsets, out=out)
    for seed, ends in ((1, [0, 300, 300, 300]), (2, [0, 10, 200, 290]), (3, [7, 7, 8, 300]), (1, [0, 300, 300, 300])):
        qkv.copy_(rows_of(seed, "bf16", n, 8, 2, dim))
        offsets.copy_(torch.tensor(ends, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = tq.prompt_attention(*qkv.split(heads, dim=1), offsets, out=torch.zeros_like(out))
        assert torch.equal(out, eager)


def test_no_tokens_and_no_sequences(gpu):
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert tq.prompt_attention(e, e, e, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 2, 64)
    x = torch.randn((5, 2, 64), device="cuda").bfloat16()
    out = torch.ones_like(x)
    tq.prompt_attention(x, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 1).all()


def test_gradient_is_refused_when_asked_for(gpu):
    x = torch.randn((5, 2, 64), device="cuda").bfloat16().requires_grad_()
    out = tq.prompt_attention(x, x, x, torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError, match="prompt_attention has no gradient"):
        out.float().sum().backward()
