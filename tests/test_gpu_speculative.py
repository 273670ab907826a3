"""The operators together: greedy decoding by trees of drafts gives the tokens of decoding one
by one, and the drafter learns while it drafts."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("speculative_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trees_of_drafts_decode_as_one_by_one(gpu, example):
    model = example.Model()
    prompt = torch.randint(0, example.VOCAB, (3, 37), generator=torch.Generator().manual_seed(2)).to(gpu)
    plain, steps, _ = example.decode(model, prompt, 20, trees=False)
    assert steps == 20 and all(len(t) == 20 for t in plain)
    drafter = example.Drafter(gpu)
    first, _, losses = example.decode(model, prompt, 20, drafter=drafter)
    assert [t[:20] for t in first] == plain
    for _ in range(2):
        again, steps, later = example.decode(model, prompt, 20, drafter=drafter)
        assert [t[:20] for t in again] == plain
    assert later[-1] < 0.5 * losses[0]
    assert steps < 20  # drafts were accepted


def test_sampling_follows_the_given_numbers(gpu, example):
    model = example.Model(seed=2)
    prompt = torch.randint(0, example.VOCAB, (2, 9), generator=torch.Generator().manual_seed(4)).to(gpu)
    a, _, _ = example.decode(model, prompt, 8, temperature=0.9)
    b, _, _ = example.decode(model, prompt, 8, temperature=0.9)
    c, _, _ = example.decode(model, prompt, 8, temperature=0.9, seed=4)
    assert a == b and a != c
    assert all(0 <= t < example.VOCAB for row in a for t in row)
