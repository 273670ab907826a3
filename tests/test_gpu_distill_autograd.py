"""The distillation loss under autograd: what backward leaves is the gradient that the formula gives for
the weights that reach each row's loss. Tolerances are those of test_gpu_distill."""

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.gpu_util import say
from tests.test_gpu_distill import DT, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab,temperature", [(1, 9, 1.0), (7, 1021, 2.0), (40, 20000, 0.5), (3, 140001, 1.0)])
def test_backward(gpu, dt, rows, vocab, temperature):
    say(f"backward {dt} {rows} {vocab}")
    x, index, top, w = inputs(rows, rows, vocab, min(vocab, 12), dt, "f32")
    wide = torch.zeros((rows, vocab + 3), dtype=DT[dt], device=gpu)
    wide[:, 1 : vocab + 1] = x.cuda()
    wide.requires_grad_()
    loss = tq.distill_loss(wide[:, 1 : vocab + 1], index.cuda(), top.cuda(), temperature)
    (loss * w.cuda()).sum().backward()
    assert not wide.grad[:, 0].any() and not wide.grad[:, vocab + 1 :].any()
    check(x, index, top, w, temperature, got=(loss.detach(), wide.grad[:, 1 : vocab + 1]))


def test_beside_another_loss(gpu):
    """Cross entropy and distillation of one student: its weights get the gradients of both."""
    g = torch.Generator().manual_seed(3)
    h = torch.randn((16, 32), generator=g).cuda()
    weight = (torch.randn((32, 700), generator=g) * 0.3).cuda().requires_grad_()
    _, index, top, _ = inputs(4, 16, 700, 10, "f32")
    target = torch.randint(0, 700, (16,), generator=g).cuda()
    logits = h @ weight
    ce = torch.nn.functional.cross_entropy(logits, target)
    own = tq.distill_loss(logits, index.cuda(), top.cuda(), 2.0).mean()
    of_ce, = torch.autograd.grad(ce, weight, retain_graph=True)
    of_both, = torch.autograd.grad(ce + own, weight, retain_graph=True)
    each = torch.full((16,), 1 / 16, device=gpu)
    want = h.t() @ tq.distill_grad(logits.detach(), index.cuda(), top.cuda(), each, 2.0)
    # The same kernel and product on the same numbers, then one sum: a few half units of fp32.
    assert (of_both - of_ce - want).abs().max() <= 8 * 2.0 ** -24 * (of_ce.abs() + want.abs()).max()
    assert want.abs().max() > 0.01


def test_both_results_and_a_second_backward(gpu):
    x, index, top, w = (t.cuda() for t in inputs(9, 5, 300, 8, "f32"))
    x.requires_grad_()
    loss, grad = tq.distill(x, index, top, w)
    (loss * w).sum().backward()
    assert torch.equal(x.grad, grad) and not grad.requires_grad
    with torch.no_grad():
        x.add_(1.0)
    again = tq.distill_loss(x, index, top).sum()
    with torch.no_grad():
        x.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        again.backward()


@pytest.mark.parametrize("both", [False, True])
def test_the_backward_pass_takes_the_gradients_memory_alone(gpu, both):
    """No gradient of the gradient's size beside it."""
    x, index, top, w = (t.cuda() for t in inputs(11, 64, 50257, 20, "bf16"))
    x.requires_grad_()
    loss = tq.distill(x, index, top, w)[0] if both else tq.distill_loss(x, index, top)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    loss.sum().backward()
    torch.cuda.synchronize()
    size = x.numel() * x.element_size()
    assert torch.cuda.max_memory_allocated() - before < 1.5 * size


def test_a_loss_that_nothing_uses(gpu):
    x, index, top, _ = (t.cuda() for t in inputs(12, 3, 100, 5, "f32"))
    x.requires_grad_()
    tq.distill_loss(x, index, top)
    y = (x * 2).sum()
    y.backward()
    assert (x.grad == 2).all()
