"""Tree attention where sequences are cut into pieces and joined, beside the same where one workgroup takes a
sequence whole. Which of both a call does goes by the room in its table, not by its lengths, so each case
runs with a table as wide as its lengths and with one of 1280 positions or more. Tolerances are those of
test_gpu_tree_attention."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.gpu_util import say
from tests.test_gpu_tree_attention import Case, bound, check, run, tree_mask

pytestmark = pytest.mark.gpu

WIDE = 160  # pages of 16
ROOMS = [None, WIDE]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("nodes,group", [(1, 1), (3, 4), (16, 1), (16, 2), (33, 1), (20, 3), (20, 6), (33, 6), (64, 1), (64, 6)])
def test_every_shape_in_pieces(gpu, dt, dim, nodes, group):
    """All forms (rows of 16 to 192 a workgroup) with sequences of no, one and many tiles."""
    say(f"pieces {dt} {dim} {nodes} {group}")
    case = Case(nodes + group, dt, [700, 0, 40, 64, 1290], nodes, 2 * group, 2, dim, 16, room=WIDE)
    check(case, run(case))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lengths", [[1500, 700, 0, 2600, 63], [5000], [9, 3300]])
def test_wide_trees_over_ragged_sequences(gpu, dt, dim, lengths):
    """64 nodes of 6 query heads a kv head: two row tiles of 192, several of both in a piece."""
    say(f"wide {dt} {dim} {lengths}")
    case = Case(len(lengths) + dim, dt, lengths, 64, 12, 2, dim, 64)
    check(case, run(case))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim,nodes,hq", [(64, 4, 4), (128, 64, 12), (256, 64, 4), (256, 40, 2)])
@pytest.mark.parametrize("room", ROOMS)
def test_rows_that_see_no_key(gpu, dt, dim, nodes, hq, room):
    """At 256 columns a tile has 32 positions, so that 64 nodes without a cache are two pieces without a key."""
    say(f"no key {dt} {dim} {nodes} {room}")
    half = [0] * (nodes // 2) + [(1 << (nodes - 1)) | 1] * (nodes - nodes // 2)
    case = Case(31, dt, [0, 40, 512, 0], nodes, hq, 2, dim, 16, masks=[half, half, [0] * nodes, [0] * nodes],
                room=room)
    got = run(case)
    check(case, got)
    assert not got[0, : nodes // 2].any() and not got[3].any()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim,nodes,hq,length", [(64, 6, 4, 77), (128, 40, 12, 300), (128, 64, 12, 700), (256, 40, 4, 77)])
@pytest.mark.parametrize("room", ROOMS)
def test_values_that_no_row_sees(gpu, dt, value, dim, nodes, hq, length, room):
    say(f"unseen {dt} {value} {dim} {nodes} {room}")
    real = nodes - 2
    masks = [tree_mask([-1] + [i - 1 for i in range(1, real)]) + [1 << real, 1 << (real + 1)]]
    case = Case(33, dt, [length], nodes, hq, 2, dim, 16, masks=masks, room=room)
    case.k[:, real:] = value
    case.v[:, real:] = value
    check(case, run(case), rows=np.s_[:, :real])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim,nodes,hq,length", [(64, 6, 2, 50), (128, 6, 12, 640), (128, 64, 12, 900), (256, 24, 4, 333)])
@pytest.mark.parametrize("room", ROOMS)
def test_seen_values_reach_their_rows_only(gpu, dt, dim, nodes, hq, length, room):
    """Infinities of both signs and NaN in a node's values: in their columns, for the rows that see the node."""
    say(f"seen {dt} {dim} {nodes} {room}")
    masks = [tree_mask([-1, 0, 0, 1, 2, 3] + list(range(5, nodes - 1)))]
    case = Case(34, dt, [length], nodes, hq, 2, dim, 16, masks=masks, room=room)
    for column, value in ((5, float("inf")), (6, -float("inf")), (dim - 1, float("nan"))):
        case.v[:, 2, :, column] = value
    got = run(case).double().cpu().numpy()
    want, weight, spread = case.oracle()
    sees = np.array([(int(m) >> 2) & 1 for m in case.mask[0]], bool)
    fine = np.isfinite(want)
    assert (~fine[0, sees]).sum(-1).min() == 3 and fine[0, ~sees].all()
    assert np.array_equal(np.isfinite(got), fine)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True)
    with np.errstate(invalid="ignore"):
        over = np.abs(got - want) - bound(case, np.where(fine, want, 0), np.where(fine, weight, 0), spread)
    assert over[fine].max() <= 0


def test_pieces_and_whole_sequences_agree(gpu):
    """One call as a whole and in pieces: equal up to the order of fp32 sums, so within a unit of bf16."""
    case = Case(35, "bf16", [250, 31], 8, 8, 2, 128, 16)
    a = case.gpu()
    whole = tq.tree_attention(**a, scale=case.scale)
    table = torch.full((2, 400), -1, dtype=torch.int32, device=gpu)
    table[:, : a["table"].shape[1]] = a["table"]
    cut = tq.tree_attention(**{**a, "table": table}, scale=case.scale)
    check(case, whole)
    check(case, cut)
