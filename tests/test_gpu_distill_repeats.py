"""Distillation where many of a teacher's entries have one place: the result, and that the time stays near that
of entries apart. An entry list of n entries is walked a few times, not n times: 1024 entries are
n^2 / n = 1024 times too slow otherwise, and the bounds below leave a factor of 20 or more to both sides."""

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.gpu_util import say
from tests.test_gpu_distill import check, inputs

pytestmark = pytest.mark.gpu

K = 1024


def repeated(kind, vocab, rows):
    """Entries all apart; 24 of them and then place 0 with no mass, as a padded teacher has it; all at one place."""
    x, index, top, w = inputs(vocab, rows, vocab, K, "bf16", "f32", missing=False)
    if kind == "padded":
        index[:, 24:], top[:, 24:] = 0, -float("inf")
    if kind == "one place":
        index[:] = vocab // 3
    if kind == "one piece":
        index[:] = vocab // 3 // 8 * 8 + torch.arange(K, dtype=torch.int32) % 8
    return x, index, top, w


def compare(x, index, top, w):
    """Entries without mass against the same row with them left out, which is the same by the formula (and
    the bound has no infinities in it then)."""
    a = [t.cuda() for t in (x, index, top, w)]
    loss, grad = tq.distill(*a)
    assert torch.equal(tq.distill_loss(*a[:3]), loss) and torch.equal(tq.distill_grad(*a), grad)
    check(x, torch.where(top == -float("inf"), -1, index), top, w, got=(loss, grad))


@pytest.mark.parametrize("vocab", [3001, 50257, 129280])
@pytest.mark.parametrize("kind", ["apart", "padded", "one place", "one piece"])
def test_values(gpu, vocab, kind):
    say(f"repeats {vocab} {kind}")
    compare(*repeated(kind, vocab, 3))


def test_entries_without_mass_leave_the_others_alone(gpu):
    """Entries of mass 0 at the places of others, and at places of their own."""
    x, index, top, w = inputs(5, 4, 700, 60, "f32", missing=False)
    top[:, 20:] = -float("inf")
    index[0, 20:] = index[0, :40] % 700
    index[1, 20:] = index[1, 0]
    index[2, 20:] = 699
    compare(x, index, top, w)


@pytest.mark.parametrize("vocab,rows", [(50257, 64), (129280, 16), (129280, 512)])
@pytest.mark.parametrize("kind,most", [("padded", 3), ("one place", 40), ("one piece", 60)])
def test_time(gpu, vocab, rows, kind, most):
    def took(which):
        a = [t.cuda() for t in repeated(which, vocab, 2)]
        a = [t.repeat((rows // 2,) + (1,) * (t.dim() - 1)) for t in a]
        best = float("inf")
        for _ in range(6):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            tq.distill(*a)
            end.record()
            torch.cuda.synchronize()
            best = min(best, begin.elapsed_time(end) * 1e3)
        return best

    apart, other = took("apart"), took(kind)
    say(f"repeats {kind} {vocab} x {rows}: {other:.0f} us, apart {apart:.0f} us")
    assert other < most * apart
