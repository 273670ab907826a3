"""What autograd sees of the operators, on the host: a loss has its gradient, an operator without one fails
where a gradient is asked for, and nothing is dropped without a word. The library and the tensors' place
are stand-ins, as in test_other_gpu_host; the values are the GPU tests' matter."""

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from trellis_quantized_linear_tf_amd import _ops
from tests.test_other_gpu_host import attention, far, machine, rows  # noqa: F401


@pytest.fixture(autouse=True)
def anywhere(monkeypatch):
    """What autograd passes on are plain tensors of the host."""
    monkeypatch.setattr(_ops, "_one_gpu", lambda *tensors: None)


@pytest.mark.parametrize("which", [0, 1, 2, 4, 5])
def test_attention_has_no_backward_pass(machine, which):  # noqa: F811
    a = list(attention())
    a[which].requires_grad_()
    out = tq.tree_attention(*a)
    assert out.requires_grad
    with pytest.raises(RuntimeError, match="tree_attention has no gradient"):
        (out.float().sum() + a[which].float().sum()).backward()
    with torch.no_grad():
        assert not tq.tree_attention(*a).requires_grad
    a[which].requires_grad_(False)
    assert not tq.tree_attention(*a).requires_grad


def test_attention_into_a_buffer_leaves_the_buffer_plain(machine):  # noqa: F811
    a = list(attention())
    a[0].requires_grad_()
    out = far(*a[0].shape, dtype=a[0].dtype)
    got = tq.tree_attention(*a, out=out)
    assert got.data_ptr() == out.data_ptr() and got.requires_grad and not out.requires_grad


@pytest.mark.parametrize("both", [False, True])
def test_the_loss_has_a_gradient(machine, both):  # noqa: F811
    x, index, top, weight = rows()
    x.requires_grad_()
    got = tq.distill(x, index, top, weight, 2.0) if both else (tq.distill_loss(x, index, top, 2.0), None)
    assert got[0].requires_grad and (not both or not got[1].requires_grad)
    assert len(machine.calls) == 1
    got[0].mean().backward()
    assert len(machine.calls) == 2 and x.grad.shape == x.shape
    with torch.no_grad():
        assert not tq.distill_loss(x, index, top).requires_grad


def test_the_loss_has_one_backward_pass_and_none_for_the_teacher(machine):  # noqa: F811
    x, index, top, _ = rows()
    x.requires_grad_()
    g, = torch.autograd.grad(tq.distill_loss(x, index, top).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    top.requires_grad_()
    for logits in (x, x.detach()):
        loss = tq.distill_loss(logits, index, top)
        with pytest.raises(RuntimeError, match="teacher"):
            loss.sum().backward()


@pytest.mark.parametrize("call", ["attention", "loss"])
def test_forward_mode_is_refused(machine, call):  # noqa: F811
    from torch.autograd import forward_ad

    with forward_ad.dual_level():
        if call == "attention":
            a = [t.as_subclass(torch.Tensor) if i == 0 else t for i, t in enumerate(attention())]
            a[0] = forward_ad.make_dual(a[0], torch.ones_like(a[0])).as_subclass(type(a[1]))
            with pytest.raises(NotImplementedError):
                tq.tree_attention(*a)
            assert not tq.tree_attention(*attention()).requires_grad
        else:
            x, index, top, _ = rows()
            plain = x.as_subclass(torch.Tensor)
            with pytest.raises(NotImplementedError):
                tq.distill_loss(forward_ad.make_dual(plain, torch.ones_like(plain)).as_subclass(type(x)), index, top)
