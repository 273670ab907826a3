"""Tree attention over a paged cache on the GPU, against the float64 oracle.

Tolerance, per output o = sum p_j V_j / sum p_j with A = sum p_j |V_j| / sum p_j:
  half an ulp of the output type for the last rounding            h |o|
  half an ulp of the type for each probability                    h A
  the score's fp32 sum (dim products) and the scale's rounding    2 (dim + 2) 2^-24 S A
  exponential, fp32 sums over the keys and joining of parts       (keys + 64) 2^-24 A
with h = finfo(type).eps / 2 and S the largest scale * sum |q_d K_d| of the row (a score's
error moves a probability by at most twice its own relative amount). fp16 adds half a
subnormal step for each of the two roundings."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import operators as ops
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def tree_mask(parents):
    """[nodes] masks of a tree: a node sees itself and what is above it."""
    masks = []
    for i, p in enumerate(parents):
        masks.append((1 << i) | (masks[p] if p >= 0 else 0))
    return masks


def signed64(masks):
    return np.array(masks, dtype=np.uint64).view(np.int64)


class Case:
    """Inputs on the CPU in their own type; the cache's unused slots and pages hold NaN."""

    def __init__(self, seed, dt, lengths, nodes, hq, hkv, dim, page, *, heads_first=False, masks=None, spread=1.0, room=None):
        g = torch.Generator().manual_seed(seed)
        t = DT[dt]
        self.batch, self.nodes, self.dim, self.dt = len(lengths), nodes, dim, dt
        self.lengths = np.array(lengths, np.int32)
        qkv = torch.randn((self.batch, nodes, hq + 2 * hkv, dim), generator=g) * spread
        self.q, self.k, self.v = qkv.to(t).split([hq, hkv, hkv], dim=2)
        need = [-(-int(n) // page) for n in lengths]
        cols = max(max(need), 1) if room is None else room
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).tolist()
        self.kc, self.vc = (torch.full((pages, page, hkv, dim), float("nan"), dtype=t) for _ in range(2))
        self.table = np.full((self.batch, cols), -7, np.int32)  # entries behind a sequence's length are never used
        for b, n in enumerate(lengths):
            for c in range(need[b]):
                p = order.pop()
                self.table[b, c] = p
                fill = min(page, int(n) - c * page)
                for cache in (self.kc, self.vc):
                    cache[p, :fill] = (torch.randn((fill, hkv, dim), generator=g) * spread).to(t)
        if masks is None:
            r = np.random.default_rng(seed)
            masks = [tree_mask([-1] + [int(r.integers(max(0, i - 5), i)) for i in range(1, nodes)]) for _ in lengths]
        self.mask = signed64(masks)
        self.heads_first = heads_first
        self.scale = dim ** -0.5

    def gpu(self):
        out = dict(q=self.q, k=self.k, v=self.v, mask=torch.from_numpy(self.mask), table=torch.from_numpy(self.table),
                   lengths=torch.from_numpy(self.lengths))
        out = {n: x.cuda() for n, x in out.items()}
        rows = torch.cat([self.q, self.k, self.v], 2).cuda()  # q, k, v as views of one projection's rows
        hq, hkv = self.q.shape[2], self.k.shape[2]
        out["q"], out["k"], out["v"] = rows.split([hq, hkv, hkv], dim=2)
        for n, c in (("k_cache", self.kc), ("v_cache", self.vc)):
            out[n] = c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.heads_first else c.cuda()
        return out

    def oracle(self):
        f = [x.double().numpy() for x in (self.q, self.k, self.v)]
        return ops.tree_attention(*f, self.mask, self.kc.double().numpy(), self.vc.double().numpy(), self.table,
                                  self.lengths, self.scale)


def bound(case, want, weight, spread):
    h = torch.finfo(DT[case.dt]).eps / 2
    keys = int(case.lengths.max()) + case.nodes
    f = 2.0 ** -24
    tol = h * np.abs(want) + (h + (2 * (case.dim + 2) * spread[..., None] + keys + 64) * f) * weight
    return tol + (2.0 ** -24 if case.dt == "f16" else 2.0 ** -133)


def check(case, got, rows=None):
    want, weight, spread = case.oracle()
    got = got.double().cpu().numpy()
    over = np.abs(got - want) - bound(case, want, weight, spread)
    if rows is not None:
        over = over[rows]
    assert np.isfinite(got if rows is None else got[rows]).all()
    assert over.max() <= 0, f"{over.max():.3g} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


def run(case, **kw):
    out = tq.tree_attention(**case.gpu(), scale=case.scale, **kw)
    torch.cuda.synchronize()
    return out


LENGTHS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1021]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_length(gpu, dt, dim):
    say(f"lengths {dt} {dim}")
    case = Case(dim, dt, LENGTHS, 3, 4, 2, dim, 16)
    check(case, run(case))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 64, 100, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_every_page(gpu, page, heads_first):
    say(f"page {page} {heads_first}")
    case = Case(page, "bf16", [page, 2 * page - 1, 2 * page + 1, 333, 0], 5, 5, 1, 128, page, heads_first=heads_first)
    check(case, run(case))


@pytest.mark.parametrize("nodes", [1, 2, 7, 8, 16, 31, 32, 33, 47, 63, 64])
@pytest.mark.parametrize("group", [1, 6])
def test_every_tree(gpu, nodes, group):
    say(f"nodes {nodes} group {group}")
    case = Case(nodes, "bf16" if nodes % 2 else "f16", [100, 0, 40], nodes, 2 * group, 2, 128, 16)
    check(case, run(case))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (12, 1), (40, 8), (16, 16), (24, 2), (71, 1)])
def test_every_group(gpu, hq, hkv):
    say(f"heads {hq} {hkv}")
    case = Case(hq, "bf16", [200, 77], 9, hq, hkv, 64, 24)
    check(case, run(case))


@pytest.mark.parametrize("dim", [16, 32, 48, 80, 96, 112, 144, 160, 192, 224, 240])
def test_every_head_size(gpu, dim):
    say(f"dim {dim}")
    case = Case(dim, "f16", [97, 31], 6, 6, 2, dim, 16, heads_first=dim % 32 == 0)
    check(case, run(case))


@pytest.mark.parametrize("dt,dim,nodes,hq", [("bf16", 128, 1, 8), ("f16", 128, 16, 8), ("bf16", 64, 64, 4), ("f16", 256, 20, 4)])
def test_long_sequences(gpu, dt, dim, nodes, hq):
    """Ragged batches long enough that a sequence is split and joined, and that one part spans sequences."""
    say(f"long {dt} {dim} {nodes}")
    case = Case(dim + nodes, dt, [9001, 1, 4500, 0, 13000, 300], nodes, hq, 2, dim, 64)
    check(case, run(case))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [700, 2100, 2600, 3300, 4500, 6200, 7000, 9000, 12500])
def test_one_row_over_many_pieces(gpu, dim, length):
    """Few rows over one sequence: as many workgroups as its tiles allow, joined into each row."""
    say(f"pieces {dim} {length}")
    case = Case(length + dim, "bf16", [length], 1, 3, 1, dim, 64)
    check(case, run(case))


def test_many_sequences(gpu):
    case = Case(9, "bf16", [(7 * b) % 50 for b in range(300)], 2, 2, 1, 64, 16)
    check(case, run(case))


def test_more_sequences_than_are_split(gpu):
    case = Case(21, "bf16", [(11 * b) % 90 for b in range(1500)], 1, 2, 1, 64, 16)
    check(case, run(case))


@pytest.mark.parametrize("scale", [0.0, -0.11, 0.7, 1e-30, -3.0])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_scales(gpu, scale, dt):
    say(f"scale {scale} {dt}")
    case = Case(22, dt, [700, 0, 33], 5, 4, 2, 64, 16, spread=0.5)
    case.scale = scale
    check(case, run(case))


def test_caches_of_different_layouts(gpu):
    """Keys by [page][slot][head], values by [page][head][slot], and a table that is part of a wider one."""
    case = Case(23, "bf16", [300, 41, 900], 4, 4, 2, 128, 24)
    a = case.gpu()
    a["v_cache"] = a["v_cache"].transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.full((3, case.table.shape[1] + 5), 2 ** 31 - 1, dtype=torch.int32, device=gpu)
    wide[:, : case.table.shape[1]] = a["table"]
    a["table"] = wide[:, : case.table.shape[1]]
    check(case, tq.tree_attention(**a, scale=case.scale))


def test_pages_four_gib_apart(gpu):
    case = Case(24, "f16", [20], 3, 4, 2, 64, 16)
    a = case.gpu()
    pages, far = a["k_cache"].shape[0], 1 << 31
    for n in ("k_cache", "v_cache"):
        small = a[n]
        big = torch.empty(((pages - 1) * far + small[0].numel(),), dtype=torch.float16, device=gpu)
        a[n] = big.as_strided(small.shape, (far, *small.stride()[1:]))
        a[n].copy_(small)
    check(case, tq.tree_attention(**a, scale=case.scale))


def test_no_pages_at_all(gpu):
    case = Case(25, "bf16", [0, 0], 6, 4, 2, 64, 16)
    a = case.gpu()
    a["table"] = torch.empty((2, 0), dtype=torch.int32, device=gpu)
    a["lengths"] = torch.tensor([9, -9], dtype=torch.int32, device=gpu)  # taken as the table's room: none
    check(case, tq.tree_attention(**a, scale=case.scale))


def test_an_empty_batch(gpu):
    case = Case(26, "bf16", [5], 2, 4, 2, 64, 16)
    a = {n: (x if n.endswith("cache") else x[:0]) for n, x in case.gpu().items()}
    assert tq.tree_attention(**a).shape == (0, 2, 4, 64)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 12.0])
def test_flat_and_peaked_scores(gpu, spread):
    """Scores that are all equal, and scores hundreds apart."""
    say(f"spread {spread}")
    case = Case(11, "bf16", [500, 64], 8, 8, 2, 128, 32, spread=spread)
    check(case, run(case))


def test_rows_that_see_nothing_are_zero(gpu):
    masks = [[0, 0b1, 0b110, 0]] * 2
    case = Case(12, "bf16", [0, 40], 4, 4, 2, 64, 16, masks=masks)
    got = run(case)
    check(case, got)
    assert not got[0, 0].any() and not got[0, 3].any()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("nodes", [6, 40])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_no_row_sees_stay_out(gpu, value, nodes, dim):
    """Padding nodes hold infinities or NaN in keys and values; they see themselves, the real
    ones do not see them. Slots behind the lengths and unused pages hold NaN in every test."""
    say(f"unseen {value} {nodes} {dim}")
    real = nodes - 2
    masks = [tree_mask([-1] + [i - 1 for i in range(1, real)]) + [1 << real, 1 << (real + 1)]]
    case = Case(13, "bf16", [77], nodes, 4, 2, dim, 16, masks=masks)
    case.k[:, real:] = value
    case.v[:, real:] = value
    check(case, run(case), rows=np.s_[:, :real])


def test_a_seen_infinity_reaches_its_rows_only(gpu):
    masks = [tree_mask([-1, 0, 0, 1, 2, 3])]
    case = Case(14, "bf16", [50], 6, 2, 1, 64, 16, masks=masks)
    case.v[:, 2, :, 5] = float("inf")  # seen by nodes 2 and 4
    got = run(case).float().cpu()
    hit = torch.isinf(got).any(-1).any(-1)[0]
    assert hit.tolist() == [False, False, True, False, True, False]
    assert torch.isinf(got[0, 2, :, 5]).all() and torch.isfinite(got[0, 2, :, :5]).all()
    want, weight, spread = case.oracle()
    fine = np.isfinite(want)
    over = np.abs(got.double().numpy() - want)[fine] - bound(case, want, weight, spread)[fine]
    assert over.max() <= 0


def test_lengths_outside_the_table(gpu):
    """A negative length is 0, one past the table's room is the room."""
    case = Case(15, "bf16", [64, 0, 33], 3, 4, 2, 128, 32, room=2)
    case.table[2, 1] = case.table[0, 0]  # sequence 2 may read its whole room
    inside = run(case)
    a = case.gpu()
    a["lengths"] = torch.tensor([1 << 30, -5, 33], dtype=torch.int32, device="cuda")
    got = tq.tree_attention(**a, scale=case.scale)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), inside.view(torch.int16))


def test_bad_pages_touch_no_other_sequence(gpu):
    """Page numbers outside the cache are read as page 0; the other sequences keep their values."""
    case = Case(16, "bf16", [100, 90, 80], 4, 4, 2, 64, 16)
    a = case.gpu()
    a["k_cache"].nan_to_num_(0.0)
    a["v_cache"].nan_to_num_(0.0)
    a["table"][1, 1], a["table"][1, 2], a["table"][1, 3] = 2 ** 31 - 1, -(2 ** 31), a["k_cache"].shape[0]
    got = tq.tree_attention(**a, scale=case.scale)
    torch.cuda.synchronize()
    assert torch.isfinite(got).all()
    check(case, got, rows=np.s_[[0, 2]])


def test_offsets_past_32_bits(gpu):
    """Pages beyond 4 GiB of a cache's bytes, and beyond 2^32 elements."""
    page, hkv, dim = 64, 4, 128
    pages = (1 << 33) // (page * hkv * dim * 2) * 9 // 8 + 1  # 9 GiB a cache
    case = Case(17, "bf16", [130, 70], 2, 4, hkv, dim, page)
    a = case.gpu()
    far = [pages - 1, pages // 2 + 3, pages - 7, pages * 9 // 10, 5]
    big = [torch.empty((pages, page, hkv, dim), dtype=torch.bfloat16, device=gpu) for _ in range(2)]
    used = sorted({int(p) for b in range(2) for p in case.table[b] if p >= 0})
    move = dict(zip(used, far))
    for src, dst in move.items():
        for small, large in zip((a["k_cache"], a["v_cache"]), big):
            large[dst] = small[src]
    a["k_cache"], a["v_cache"] = big
    a["table"] = torch.tensor([[move.get(int(p), -1) for p in row] for row in case.table], dtype=torch.int32, device=gpu)
    got = tq.tree_attention(**a, scale=case.scale)
    torch.cuda.synchronize()
    check(case, got)


def test_strided_output_and_another_stream(gpu):
    case = Case(18, "f16", [300, 20], 5, 8, 2, 128, 16)
    a = case.gpu()
    want = tq.tree_attention(**a, scale=case.scale)
    wide = torch.full((2, 5, 16, 128), 3.0, dtype=torch.float16, device=gpu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = tq.tree_attention(**a, scale=case.scale, out=wide[:, :, ::2])
    torch.cuda.synchronize()
    assert out.data_ptr() == wide.data_ptr()
    assert torch.equal(wide[:, :, ::2], want) and (wide[:, :, 1::2] == 3.0).all()


def test_the_same_call_gives_the_same_bits(gpu):
    case = Case(19, "bf16", [9000, 5000, 12], 16, 8, 2, 128, 64)
    a = case.gpu()
    first = tq.tree_attention(**a)
    for _ in range(5):
        assert torch.equal(tq.tree_attention(**a).view(torch.int16), first.view(torch.int16))


def test_graph_replays_follow_the_inputs(gpu):
    """A captured call replayed with other queries, lengths and pages, eager work between."""
    cases = [Case(20 + i, "bf16", n, 8, 8, 2, 128, 16, room=80) for i, n in
             enumerate([[1200, 3], [0, 900], [64, 64], [1, 1279]])]
    a = cases[0].gpu()
    pages = max(c.kc.shape[0] for c in cases)
    for n in ("k_cache", "v_cache"):
        a[n] = torch.cat([a[n], a[n].new_zeros((pages - a[n].shape[0], *a[n].shape[1:]))])
    out = torch.empty_like(a["q"].contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.tree_attention(**a, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tree_attention(**a, out=out)
    for case in cases[1:] + cases[:1]:
        b = case.gpu()
        for n in a:
            if n.endswith("cache"):
                a[n][: b[n].shape[0]].copy_(b[n])
            else:
                a[n].copy_(b[n])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(case, out)
        assert torch.equal(out.view(torch.int16), tq.tree_attention(**a).view(torch.int16))
