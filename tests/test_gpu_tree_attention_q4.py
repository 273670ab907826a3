"""Tree attention over a paged cache in 4 bits on the GPU, against the float64 oracle over the
values that the cache stands for; tolerances as derived in test_gpu_tree_attention."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import rows as q4
from tests.gpu_util import say
from tests.test_gpu_tree_attention import Case, check

pytestmark = pytest.mark.gpu


class Case4(Case):
    """The same inputs with the cache in 4 bits; unused slots and pages hold bytes of NaN scales."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.bytes = []
        for name in ("kc", "vc"):
            x = getattr(self, name).float().numpy()
            there = ~np.isnan(x).any(-1)
            packed = np.full((*x.shape[:3], x.shape[3] // 8 * 5), 0xFF, np.uint8)
            packed[there] = q4.q4_pack(x[there])
            values = np.full(x.shape, np.nan)
            values[there] = q4.round_to(q4.q4_unpack(packed[there]), self.dt)
            setattr(self, name, torch.from_numpy(values))
            self.bytes.append(torch.from_numpy(packed))

    def gpu(self):
        out = super().gpu()
        for n, c in zip(("k_cache", "v_cache"), self.bytes):
            out[n] = c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.heads_first else c.cuda()
        return out


def run(case, **kw):
    out = tq.tree_attention_q4(**case.gpu(), scale=case.scale, **kw)
    torch.cuda.synchronize()
    return out


LENGTHS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1021]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_length(gpu, dt, dim):
    say(f"lengths {dt} {dim}")
    case = Case4(dim, dt, LENGTHS, 3, 4, 2, dim, 16)
    check(case, run(case))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("rows", [3, 14, 30, 50, 100, 200])
def test_every_head_size_and_row_tile(gpu, dt, dim, rows):
    say(f"dim {dim} {dt} rows {rows}")
    nodes = min(rows, 50)
    case = Case4(dim + rows, dt, [97, 31, 200], nodes, 2 * (rows // nodes), 2, dim, 16, heads_first=dim % 64 == 0)
    check(case, run(case))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("nodes,hq", [(9, 4), (16, 4), (12, 6), (16, 8), (33, 2), (50, 8), (64, 4)])
def test_many_rows_of_long_tables(gpu, dt, dim, nodes, hq):
    """Tables with so much room that a wave takes two or four row tiles, with short and empty sequences in them."""
    say(f"long tables {dt} {dim} {nodes} {hq}")
    case = Case4(dim + nodes, dt, [97, 0, 700, 131], nodes, hq, 2, dim, 64, heads_first=dim % 64 == 0, room=800)
    check(case, run(case))


@pytest.mark.parametrize("dt,dim,nodes", [("bf16", 128, 16), ("f16", 64, 20), ("bf16", 64, 8), ("f16", 128, 40), ("bf16", 256, 9)])
def test_many_rows_of_many_sequences(gpu, dt, dim, nodes):
    """Groups that one workgroup takes as a whole, with two or four row tiles."""
    say(f"many sequences {dt} {dim} {nodes}")
    case = Case4(dim, dt, [(37 * b) % 300 for b in range(260)], nodes, 8, 2, dim, 16, room=64)
    got = run(case)
    some = [0, 1, 7, 130, 259]
    for name in ("q", "k", "v", "mask", "table", "lengths"):
        setattr(case, name, getattr(case, name)[some])
    check(case, got[some])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_sequences_of_many_rows(gpu, dt, dim):
    """Pieces that begin and end within a sequence, with two or four row tiles."""
    say(f"long, many rows {dt} {dim}")
    case = Case4(dim + 1, dt, [5001, 1, 2500, 300], 16, 8, 2, dim, 64, room=900)
    check(case, run(case))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("nodes", [16, 40])
def test_nodes_that_some_of_many_rows_see(gpu, bad, nodes):
    masks = [[1 << min(i, nodes - 2) for i in range(nodes)]] * 2
    case = Case4(6, "bf16", [30, 64], nodes, 4, 2, 128, 64, masks=masks, room=2000)
    want = run(case)
    case.k[:, nodes - 1], case.v[:, nodes - 1] = bad, bad
    assert torch.equal(run(case), want)
    case.v[:, 3, 1, 7] = float("inf")
    got = run(case)
    assert (got[:, 3, 2:, 7] == float("inf")).all()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[:, 3, 2:, 7] = False
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 64, 100, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_every_page(gpu, page, heads_first):
    say(f"page {page} {heads_first}")
    case = Case4(page, "bf16", [page, 2 * page - 1, 2 * page + 1, 333, 0], 5, 5, 1, 128, page, heads_first=heads_first)
    check(case, run(case))


@pytest.mark.parametrize("nodes", [1, 2, 7, 8, 16, 31, 32, 33, 47, 63, 64])
@pytest.mark.parametrize("group", [1, 6])
def test_every_tree(gpu, nodes, group):
    say(f"nodes {nodes} group {group}")
    case = Case4(nodes, "bf16" if nodes % 2 else "f16", [100, 0, 40], nodes, 2 * group, 2, 128, 16)
    check(case, run(case))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (12, 1), (40, 8), (24, 2)])
def test_every_group(gpu, hq, hkv):
    say(f"heads {hq} {hkv}")
    case = Case4(hq, "bf16", [200, 77], 9, hq, hkv, 64, 24)
    check(case, run(case))


@pytest.mark.parametrize("dt,dim,nodes,hq", [("bf16", 128, 1, 8), ("f16", 128, 16, 8), ("bf16", 64, 64, 4), ("f16", 256, 20, 4)])
def test_long_sequences(gpu, dt, dim, nodes, hq):
    say(f"long {dt} {dim} {nodes}")
    case = Case4(dim + nodes, dt, [5001, 1, 2500, 0, 300], nodes, hq, 2, dim, 64)
    check(case, run(case))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [700, 2600, 6200])
def test_one_row_over_many_pieces(gpu, dim, length):
    say(f"pieces {dim} {length}")
    case = Case4(length + dim, "bf16", [length], 1, 3, 1, dim, 64)
    check(case, run(case))


def test_many_sequences(gpu):
    case = Case4(9, "bf16", [(7 * b) % 50 for b in range(300)], 2, 2, 1, 64, 16)
    check(case, run(case))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("spread", [0.01, 3.0, 20.0])
def test_score_sizes(gpu, dt, spread):
    case = Case4(13, dt, [200, 31], 6, 4, 2, 128, 16, spread=spread)
    check(case, run(case))


def test_masks_that_see_nothing(gpu):
    masks = [[0, 1, 0b110, 0], [0, 0, 0, 0b1111]]
    case = Case4(5, "bf16", [0, 20], 4, 4, 2, 64, 16, masks=masks)
    out = run(case)
    check(case, out)
    assert not out[0, 0].any() and not out[0, 3].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nodes_that_no_row_sees(gpu, bad):
    """What such a node's key and value hold reaches no row."""
    masks = [[0b001, 0b010, 0b010]] * 2
    case = Case4(6, "f16", [30, 64], 3, 4, 2, 128, 16, masks=masks)
    want = run(case)
    case.k[:, 2], case.v[:, 2] = bad, bad
    assert torch.equal(run(case), want)


def test_a_value_that_only_some_rows_see(gpu):
    masks = [[0b001, 0b011, 0b101]]
    case = Case4(7, "bf16", [70], 3, 4, 2, 64, 16, masks=masks)
    want = run(case)
    case.v[0, 1, 0, 5] = float("inf")
    got = run(case)
    assert torch.equal(got[:, [0, 2]], want[:, [0, 2]])
    assert (got[0, 1, :2, 5] == float("inf")).all() and torch.equal(got[0, 1, 2:], want[0, 1, 2:])


def test_out_and_wide_strides(gpu):
    case = Case4(8, "bf16", [50, 20], 5, 4, 2, 64, 16)
    a = case.gpu()
    for n in ("k_cache", "v_cache"):  # pages and slots apart by more than they hold
        wide = torch.zeros((a[n].shape[0], 20, 3, 44), dtype=torch.uint8, device="cuda")
        view = wide[:, :16, :2, :40]
        view.copy_(a[n])
        a[n] = view
    room = torch.zeros((2, 7, 6, 72), dtype=torch.bfloat16, device="cuda")
    out = room[:, 1:6, 2:, :64]
    got = tq.tree_attention_q4(**a, scale=case.scale, out=out)
    assert got is out
    check(case, out)
    out.zero_()
    assert not room.any()


def test_caches_of_different_strides(gpu):
    case = Case4(14, "bf16", [50, 20, 300], 5, 4, 2, 128, 16)
    a = case.gpu()
    a["v_cache"] = case.bytes[1].transpose(1, 2).contiguous().cuda().transpose(1, 2)
    check(case, tq.tree_attention_q4(**a, scale=case.scale))


def test_bad_lengths_and_pages_stay_in_the_buffers(gpu):
    case = Case4(9, "bf16", [40, 40, 40], 2, 4, 2, 64, 16)
    a = case.gpu()
    a["lengths"] = torch.tensor([-7, 2 ** 31 - 1, 40], dtype=torch.int32, device="cuda")
    a["table"][1] = torch.tensor([2 ** 31 - 1, -2 ** 31, 10 ** 6], dtype=torch.int32)
    out = tq.tree_attention_q4(**a, scale=case.scale)
    torch.cuda.synchronize()
    case.lengths = np.array([0, 0, 40], np.int32)
    check(case, out, rows=[0, 2])


def test_in_a_graph(gpu):
    case = Case4(10, "bf16", [500, 0, 900], 4, 8, 2, 128, 16, room=64)
    a = case.gpu()
    tq.tree_attention_q4(**a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tq.tree_attention_q4(**a)
    for lengths in ([500, 0, 900], [3, 0, 64], [100, 0, 899], [500, 0, 900]):
        a["lengths"].copy_(torch.tensor(lengths, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, tq.tree_attention_q4(**a))


def test_gradient_is_refused_when_asked_for(gpu):
    case = Case4(15, "bf16", [20], 2, 2, 1, 64, 16)
    a = case.gpu()
    a["q"] = a["q"].detach().requires_grad_()
    out = tq.tree_attention_q4(**a)
    with pytest.raises(RuntimeError, match="tree_attention_q4 has no gradient"):
        out.float().sum().backward()

