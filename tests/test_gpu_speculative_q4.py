"""The speculative example over a cache in 4 bits: it runs, and tokens come out."""

import pytest
import torch

from examples import speculative_decode as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("trees", [False, True])
def test_it_decodes(gpu, trees):
    model = ex.Model()
    prompt = torch.randint(0, ex.VOCAB, (3, 21), generator=torch.Generator().manual_seed(5)).to(model.device)
    out, steps, _ = ex.decode(model, prompt, 8, trees=trees, cache_bits=4)
    assert steps > 0 and all(len(o) >= 8 and all(0 <= t < ex.VOCAB for t in o) for o in out)
