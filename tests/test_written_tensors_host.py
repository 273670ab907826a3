"""What autograd knows of the tensors that a call writes into, on the host: one that it follows is refused, for its
graph would go on as if nothing had been written. The library and the tensors' place are stand-ins, as in
test_other_gpu_host."""

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.test_argument_checks_host import Near
from tests.test_argument_checks_host import attention as attention16
from tests.test_other_gpu_host import machine  # noqa: F401
from tests.test_rows_host import append, attention, packed, prompt, rotate
from trellis_quantized_linear_tf_amd import _ops, _rows

INTO = {"norm_rotate": (tq.norm_rotate, rotate), "norm_rotate packed": (tq.norm_rotate, packed),
        "prompt_attention": (tq.prompt_attention, prompt), "tree_attention_q4": (tq.tree_attention_q4, attention),
        "tree_attention": (tq.tree_attention, attention16)}


@pytest.fixture(autouse=True)
def anywhere(monkeypatch):
    """What autograd passes on are plain tensors of the host."""
    for module in (_ops, _rows):
        monkeypatch.setattr(module, "_one_gpu", lambda *tensors: None)


def near(make):
    """A call's arguments, with a buffer to write into."""
    a = {n: t.as_subclass(Near) for n, t in make().items()}
    return a if "out" in a else a | dict(out=tuple(torch.zeros_like(a[n]) for n in "qk"))


@pytest.mark.parametrize("name", INTO)
@pytest.mark.parametrize("leaf", [False, True])
def test_into_a_tensor_that_autograd_follows(machine, name, leaf):  # noqa: F811
    call, make = INTO[name]
    for which in range(2 if "rotate" in name else 1):
        a = near(make)
        outs = list(a["out"]) if isinstance(a["out"], tuple) else [a["out"]]
        outs[which].requires_grad_()
        if not leaf:
            outs[which] = outs[which] * 2
        a["out"] = tuple(outs) if isinstance(a["out"], tuple) else outs[0]
        with pytest.raises(ValueError, match="autograd follows"):
            call(**a)
        assert not machine.calls
        with torch.no_grad():  # as torch's own functions
            call(**a)
        assert machine.calls.pop()


@pytest.mark.parametrize("which", ["q", "k"])
def test_rows_turned_where_they_stand(machine, which):  # noqa: F811
    """q = 2 w, turned in place: q's graph would still say 2 w."""
    a = near(rotate)
    a[which] = a[which].requires_grad_() * 2
    with pytest.raises(ValueError, match="autograd follows"):
        tq.norm_rotate(**dict(a, out=(a["q"], a["k"])))
    assert not machine.calls


@pytest.mark.parametrize("name,inputs", [("norm_rotate", ("q", "k", "q_weight", "k_weight")), ("prompt_attention", ("q", "k", "v")),
                                         ("tree_attention_q4", ("q", "k", "v"))])
def test_followed_inputs_into_a_buffer(machine, name, inputs):  # noqa: F811
    """The buffer would hold results without the graph that they belong to."""
    call, make = INTO[name]
    for n in inputs:
        a = near(make)
        a[n].requires_grad_()
        with pytest.raises(ValueError, match="autograd follows"):
            call(**a)
        assert not machine.calls
        with torch.no_grad():
            call(**a)
        assert machine.calls.pop()
        del a["out"]
        out = call(**a)
        assert any(o.requires_grad for o in (out if isinstance(out, tuple) else (out,)))
        machine.calls.clear()


def test_one_buffer_of_two(machine):  # noqa: F811
    a = near(rotate)
    into = a["out"][1]
    a["q"].requires_grad_()
    with pytest.raises(ValueError, match="autograd follows"):
        tq.norm_rotate(**dict(a, out=(None, into)))
    a["q"].requires_grad_(False)
    assert tq.norm_rotate(**dict(a, out=(None, into)))[1] is into


# ---------------------------------------------------------------- versions


def append_args():
    a = attention16()
    return {n: a[n] for n in ("k", "v", "k_cache", "v_cache", "table", "lengths")}


WRITERS = {**INTO, "cache_append": (tq.cache_append, append_args), "cache_append_q4": (tq.cache_append_q4, append)}


@pytest.mark.parametrize("name", WRITERS)
def test_what_is_written_is_known_to_have_changed(machine, name):  # noqa: F811
    call, make = WRITERS[name]
    a = near(make) if name in INTO else {n: t.as_subclass(Near) for n, t in make().items()}
    outs = a.get("out", (a.get("k_cache"), a.get("v_cache")))
    outs = outs if isinstance(outs, tuple) else (outs,)
    others = [t for n, t in a.items() if n != "out" and all(t is not o for o in outs)]
    before, still = [o._version for o in outs], [t._version for t in others]
    call(**a)
    assert all(o._version > n for o, n in zip(outs, before)) and [t._version for t in others] == still


def test_a_backward_pass_that_needs_overwritten_rows_fails(machine):  # noqa: F811
    """s = sum q q keeps q, and q is turned in place before s's backward pass."""
    a = near(rotate)
    w = torch.ones_like(a["q"]).requires_grad_()
    s = (w * a["q"]).sum()
    tq.norm_rotate(**dict(a, out=(a["q"], a["k"])))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        s.backward()


def test_buffers_of_inference_mode(machine):  # noqa: F811
    """They have no version."""
    with torch.inference_mode():
        for name in WRITERS:
            call, make = WRITERS[name]
            call(**(near(make) if name in INTO else {n: t.as_subclass(Near) for n, t in make().items()}))
    assert len(machine.calls) == len(WRITERS)


@pytest.mark.parametrize("name", ["norm_rotate", "norm_rotate packed"])
@pytest.mark.parametrize("which", ["q", "k", "frequencies", "q_weight", "k_weight"])
def test_rotation_has_no_backward_pass(machine, name, which):  # noqa: F811
    call, make = INTO[name]
    a = near(make)
    into = a.pop("out")
    a[which].requires_grad_()
    out = call(**a)
    assert [o.requires_grad for o in out] == [which not in ("k", "k_weight"), which not in ("q", "q_weight")]
    with pytest.raises(RuntimeError, match="norm_rotate has no gradient"):
        sum(o.float().sum() for o in out).backward()
    with pytest.raises(ValueError, match="autograd follows"):
        call(**a, out=into)
    with torch.no_grad():
        assert not any(o.requires_grad for o in call(**a))
