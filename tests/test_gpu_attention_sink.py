"""Attention whose weight stands at one key with values of 0: what the other keys leave, each with a
weight of 2^-14 to 2^-26 of that key's, is the whole output.

Tolerance: as in test_gpu_tree_attention (half a unit of the type for each weight and for the output,
fp32 elsewhere). fp16 has half a subnormal step of the output on top, 2^-25, and for each weight below its
smallest normal number half a subnormal step of the weight, which the header gives as 2^-38 of the row's largest:
keys 2^-38 max |V|."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.gpu_util import say
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def sink(dt, lengths, nodes, hq, dim, gap, at, up, same):
    """A batch whose scores are `gap` at position `at` of each sequence and, elsewhere, in [0, 1/2) or all 0."""
    case = Case(int(gap * 4) + dim + at, dt, lengths, nodes, hq, 2, dim, 64, masks=[[0] * nodes] * len(lengths))
    case.scale = 1.0
    g = torch.Generator().manual_seed(dim)
    case.q[:] = 0
    case.q[..., 0] = 1
    free = torch.isnan(case.kc[..., :1])
    score = torch.rand(case.kc.shape[:3], generator=g) / 2 * (not same)
    case.kc[..., 0] = torch.where(free[..., 0], float("nan"), score).to(DT[dt])
    case.vc.copy_(torch.where(free, float("nan"), up * (1 + 0.25 * case.vc.float())).to(DT[dt]))
    for b in range(len(lengths)):
        page, slot = case.table[b, at // 64], at % 64
        case.kc[page, slot, :, 0] = gap
        case.vc[page, slot] = 0
    return case


@pytest.mark.parametrize("gap", [0.0, 10.0, 12.0, 14.0, 15.0, 16.0, 16.5, 17.0, 17.5, 18.0])
@pytest.mark.parametrize("dt,dim,nodes,hq", [("f16", 128, 1, 2), ("f16", 64, 8, 8), ("f16", 128, 9, 12), ("f16", 128, 16, 16),
                                             ("f16", 256, 3, 4), ("bf16", 128, 1, 2)])
def test_what_stands_beside_one_dominant_key(gpu, dt, dim, nodes, hq, gap):
    """One to 128 rows a kv head; the key that counts comes first, in the middle and last."""
    say(f"sink {dt} {dim} {nodes} {hq} {gap}")
    lengths = [4096, 13000] if nodes < 9 else [4096]
    for at, up, same in ((0, 1.0, False), (2000, 8.0, False), (4095, 0.25, True)):
        case = sink(dt, lengths, nodes, hq, dim, gap, at, up, same)
        got = tq.tree_attention(**case.gpu(), scale=1.0).double().cpu().numpy()
        want, weight, spread = case.oracle()
        h, keys = torch.finfo(DT[dt]).eps / 2, max(lengths)
        tol = h * np.abs(want) + (h + (2 * (dim + 2) * spread[..., None] + keys + 64) * 2.0 ** -24) * weight
        tol += 2.0 ** -25 + keys * 2.0 ** -38 * 4 * up if dt == "f16" else 2.0 ** -133
        over = np.abs(got - want) - tol
        worst = np.unravel_index(over.argmax(), over.shape)
        assert over.max() <= 0, f"key {at}: {got[worst]:.6g} for {want[worst]:.6g}, {over.max():.3g} over the bound"


@pytest.mark.parametrize("dt,size", [("f16", 2.0 ** 4), ("f16", 2.0 ** 14), ("f16", 2.0 ** 15), ("bf16", 2.0 ** 15),
                                     ("bf16", 2.0 ** 30), ("bf16", 2.0 ** 100)])
@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0078125])
@pytest.mark.parametrize("dim,nodes,hq", [(64, 1, 2), (128, 9, 12), (128, 40, 12), (256, 24, 8)])
def test_scores_beyond_what_fp32_resolves(gpu, dt, size, scale, dim, nodes, hq):
    """Scores are exact products, a few units of `size` apart at up to 20000 of them and more than 1000
    apart after the scale: the largest alone has weight (or two that are equal, half each)."""
    say(f"far scores {dt} {size} {scale} {dim} {nodes}")
    case = Case(dim, dt, [900, 257], nodes, hq, 2, dim, 64, masks=[[0] * nodes] * 2)
    case.scale = scale
    case.q[:] = 0
    case.q[..., 0] = size * (2048 if dt == "f16" and size < 2 ** 10 else 1)
    g = torch.Generator().manual_seed(dim)
    unit = 32.0 if dt == "f16" else 128.0
    for b, n in enumerate(case.lengths):
        rank = torch.randperm(int(n), generator=g) % (100 if b else 200)  # sequence 0 has every rank more than once
        if b:
            rank[torch.randint(0, int(n), (1,), generator=g)] = 105  # sequence 1 one largest
        else:
            top = (rank == rank.max()).nonzero()[:, 0]
            rank[top[2:]] = 0
        for p in range(int(n)):
            case.kc[case.table[b, p // 64], p % 64, :, 0] = (unit * rank[p] + 64 * unit if dt == "f16" else unit * (rank[p] + 1)) * (
                1 if scale > 0 else -1)
    got = tq.tree_attention(**case.gpu(), scale=scale).double().cpu().numpy()
    want, _, _ = case.oracle()
    h = torch.finfo(DT[dt]).eps / 2
    assert (np.abs(got - want) <= (h + 2.0 ** -20) * np.abs(want) + 2.0 ** -25).all()
