"""Verification next to a border: rows of two places whose weights exp(-a / T) and 1 put the border between
them 8e-15 to 2e-14 of the lighter weight beside the random number, found by search in 80 bits. A running sum that
is as exact as stated (3e-15 of itself) stands on the right side of each; float64's own exp does too."""

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_verify import check_chain, check_tree

pytestmark = pytest.mark.gpu

# a, T, u: the lighter place's share exp(-a / T) / (1 + exp(-a / T)) is above u, or below it.
ABOVE = [
    ("0x1.9108f2p+1", "0x1.013450p+0", "0x1.5af6cep-5"), ("0x1.1f2744p+2", "0x1.70490ap+0", "0x1.5ad4d6p-5"),
    ("0x1.4d3d1ap+1", "0x1.abad04p-1", "0x1.5b8554p-5"), ("0x1.b08714p-1", "0x1.f3a854p-2", "0x1.34105cp-3"),
    ("0x1.2b37eap+1", "0x1.59dd96p+0", "0x1.3455eep-3"), ("0x1.3ffeb4p-1", "0x1.cda802p+0", "0x1.a827a8p-2"),
    ("0x1.215faap-1", "0x1.167266p-1", "0x1.0b9140p-2"), ("0x1.167ff6p+2", "0x1.cb6026p+0", "0x1.4cf050p-4"),
    ("0x1.16e842p-2", "0x1.9889ecp-1", "0x1.a9742cp-2"), ("0x1.1455e2p-1", "0x1.946122p+0", "0x1.a95f18p-2"),
]
BELOW = [
    ("0x1.2561dep-2", "0x1.a753ecp-1", "0x1.a82b12p-2"), ("0x1.b0f6dap-1", "0x1.f3c518p-2", "0x1.33b56ap-3"),
    ("0x1.93d350p-3", "0x1.250ba2p-1", "0x1.a8ab0ap-2"), ("0x1.6cc4a6p-3", "0x1.048faap-1", "0x1.a74ecap-2"),
]


@pytest.mark.parametrize("above", [True, False])
def test_both_sides_of_a_border(gpu, above):
    say(f"borders {above}")
    a, t, u = (np.array([float.fromhex(c[i]) for c in (ABOVE if above else BELOW)]) for i in range(3))
    a, t, u = (x.astype(np.float32) for x in (a, t, u))
    n = len(a)
    share = np.exp(-np.float64(a) / np.float64(t))
    share = share / (1 + share)
    assert ((share > u) == above).all() and (np.abs(share / u - 1) > 7e-15).all()
    logits = torch.full((n, 2, 5000), -float("inf"))
    logits[:, :, 7] = torch.from_numpy(-a)[:, None]
    logits[:, :, 4000] = 0.0  # of another chunk
    logits[::2, :, 4000], logits[::2, :, 9] = -float("inf"), 0.0  # of the same one
    tokens = np.full((n, 2), 7, np.int32)
    tree = check_tree(logits, tokens, np.array([[-1, 0]] * n, np.int32), np.stack([u, u], 1), t)
    assert (tree[1] == (2 if above else 1)).all()
    q = np.ones((n, 1, 5000), np.float32)
    count, _ = check_chain(logits, tokens, q, np.stack([u, u], 1), t)
    assert (count == (2 if above else 1)).all()
