"""Tree attention over a cache in 4 bits: the line of many sequences cut into pieces, and rows far behind the caches'
beginnings. Against the float64 oracle, tolerances as derived in test_gpu_tree_attention."""

import ctypes

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.gpu_util import say
from tests.test_gpu_tree_attention import check
from tests.test_gpu_tree_attention_q4 import Case4, run
from trellis_quantized_linear_tf_amd import _lib

pytestmark = pytest.mark.gpu

PAGE, ROOM = 64, 40  # 20 tiles of 128 positions and one for the nodes: more than any group is taken whole for


def ragged(batch):
    """Mostly short sequences, empty ones among them, and a few that fill many tiles."""
    lengths = [(37 * b) % 150 if b % 5 else 0 for b in range(batch)]
    for b, n in ((1, 1300), (batch // 2, 2400), (batch - 1, PAGE * ROOM)):
        lengths[b] = n
    return lengths


def workspace(dt, batch, nodes, hq, hkv, dim):
    a = _lib.TreeAttentionArgs({"f16": 1, "bf16": 2}[dt], batch, nodes, hq, hkv, dim, 1, PAGE, ROOM)
    return _lib.load().tf_exl3_tree_attention_q4_workspace(ctypes.byref(a))


def only(case, some):
    for name in ("q", "k", "v", "mask", "table", "lengths"):
        setattr(case, name, getattr(case, name)[some])


# One, two and four row tiles a wave by the rule on rows and tiles; sequences that are looked at 64 at a time.
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("batch,nodes,hq", [(65, 3, 2), (100, 16, 2), (128, 8, 1), (200, 30, 2)])
def test_pieces_of_many_sequences(gpu, dt, batch, nodes, hq):
    say(f"pieces of {batch} sequences {dt} {nodes} {hq}")
    assert workspace(dt, batch, nodes, hq, 1, 64) > batch * 24 + 64  # more than the places of the sequences: cut
    case = Case4(batch + nodes, dt, ragged(batch), nodes, hq, 1, 64, PAGE, heads_first=batch % 2 == 0, room=ROOM)
    got = run(case)
    assert torch.equal(run(case), got)
    some = [0, 1, 2, 63, 64, batch // 2 - 1, batch // 2, batch // 2 + 1, batch - 2, batch - 1]
    only(case, some)
    check(case, got[some])
    alone = run(case)
    check(case, alone)


def test_all_sequences_empty_or_full(gpu):
    """The line's sequences of nodes only (but for the last), and all of them longer than a tile."""
    say("70 empty")
    case = Case4(3, "bf16", [0] * 70 + [1], 5, 2, 1, 64, PAGE, room=ROOM)
    check(case, run(case))
    say("66 long")
    case = Case4(4, "bf16", [129] * 66, 5, 2, 1, 64, PAGE, room=ROOM)
    check(case, run(case))


def moved(case, pages, page_bytes=None):
    """The caches with `pages` pages, the used ones spread over them to the last."""
    a = case.gpu()
    used = sorted({int(p) for row in case.table for p in row if p >= 0})
    to = dict(zip(used, [pages - 1, *(pages * (i + 1) // (len(used) + 1) for i in range(len(used) - 1))]))
    for n in ("k_cache", "v_cache"):
        small = a[n]
        step = page_bytes or small[0].numel()
        big = torch.empty(((pages - 1) * step + small[0].numel(),), dtype=torch.uint8, device="cuda")
        a[n] = big.as_strided((pages, *small.shape[1:]), (step, *small.stride()[1:]))
        a[n][[to[p] for p in used]] = small[used]
    a["table"] = torch.tensor([[to.get(int(p), -1) for p in row] for row in case.table], dtype=torch.int32, device="cuda")
    return a


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("room", [None, 200])
def test_far_pages(gpu, dt, room):
    """Rows up to 5 GiB behind the caches' beginnings, taken whole and in pieces."""
    say(f"far pages {dt} {room}")
    case = Case4(21, dt, [130, 70, 0, 1000], 9, 4, 2, 64, PAGE, room=room)
    a = moved(case, 5 * (1 << 30) // (PAGE * 2 * 40))
    check(case, tq.tree_attention_q4(**a, scale=case.scale))


def test_pages_almost_four_gib_apart(gpu):
    case = Case4(22, "bf16", [100], 3, 4, 2, 64, PAGE)
    a = moved(case, 3, (1 << 32) - 4)
    assert a["k_cache"].stride(0) == (1 << 32) - 4
    check(case, tq.tree_attention_q4(**a, scale=case.scale))


def test_no_pages_at_all(gpu):
    case = Case4(25, "bf16", [1, 0], 6, 4, 2, 64, 16)
    a = case.gpu()
    case.lengths[:] = 0
    a["table"] = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    a["lengths"] = torch.tensor([9, -9], dtype=torch.int32, device="cuda")  # taken as the table's room: none
    check(case, tq.tree_attention_q4(**a, scale=case.scale))


def test_replays_over_many_sequences(gpu):
    """A captured call over a cut line, replayed over other lengths, with eager work in between."""
    case = Case4(30, "bf16", ragged(100), 4, 2, 1, 64, PAGE, room=ROOM)
    a = case.gpu()
    a["table"].clamp_(min=0)
    a["k_cache"].zero_(), a["v_cache"].random_(0, 50)  # numbers of any page
    run_one = lambda: tq.tree_attention_q4(**a)  # noqa: E731
    run_one()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_one()
    full = torch.from_numpy(case.lengths).cuda()
    for lengths in (full, full // 3, torch.zeros_like(full), full.flip(0), full):
        a["lengths"].copy_(lengths)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run_one())


def test_oracle_of_some_sequences_is_that_of_all():
    """What `only` leaves is the same case."""
    case = Case4(1, "bf16", [3, 0, 20], 2, 2, 1, 64, 16)
    want = case.oracle()[0]
    only(case, [2, 0])
    assert np.array_equal(case.oracle()[0], want[[2, 0]])
