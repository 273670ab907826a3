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
