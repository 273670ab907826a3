"""The operators look their arguments over with one chain of comparisons, and one by one only if that fails. Here
both answer the same arguments, changed at random: tensors that say they are on a GPU meet the chain first,
the same tensors on the host never pass it. What the one accepts, the other refuses for its place alone, and what
the one refuses, the other refuses for the same reason. The library is a stand-in."""

import random

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from tests.test_other_gpu_host import Far, machine  # noqa: F401

bf, i32 = torch.bfloat16, torch.int32


class Near(Far):
    def get_device(self):
        return 0


def attention():
    q, k = torch.zeros(2, 3, 4, 64, dtype=bf), torch.zeros(2, 3, 2, 64, dtype=bf)
    cache = torch.zeros(5, 16, 2, 64, dtype=bf)
    return dict(q=q, k=k, v=k.clone(), mask=torch.zeros(2, 3, dtype=torch.int64), k_cache=cache, v_cache=cache.clone(),
                table=torch.zeros(2, 2, dtype=i32), lengths=torch.zeros(2, dtype=i32), out=q.clone())


def append():
    a = attention()
    return {n: a[n] for n in ("k", "v", "k_cache", "v_cache", "table", "lengths")} | dict(
        nodes=torch.zeros(2, 3, dtype=i32), counts=torch.zeros(2, dtype=i32))


def tree():
    return dict(logits=torch.zeros(2, 3, 50), tokens=torch.zeros(2, 3, dtype=i32), parents=torch.zeros(2, 3, dtype=i32),
                u=torch.zeros(2, 3), temperature=torch.zeros(2))


def chain():
    a = tree()
    del a["parents"]
    return a | dict(q=torch.zeros(2, 2, 50))


def loss():
    return dict(logits=torch.zeros(3, 50), index=torch.zeros(3, 5, dtype=i32), top=torch.zeros(3, 5))


def both():
    return loss() | dict(weight=torch.zeros(3))


CALLS = {"tree_attention": (tq.tree_attention, attention), "cache_append": (tq.cache_append, append),
         "verify_tree": (tq.verify_tree, tree), "verify_chain": (tq.verify_chain, chain), "distill": (tq.distill, both),
         "distill_loss": (tq.distill_loss, loss), "distill_grad": (tq.distill_grad, both)}
DTYPES = [torch.float32, torch.float16, bf, torch.float64, i32, torch.int64, torch.uint8, torch.int8]


def change(r, t):
    """A tensor that differs from t in one way."""
    kind = r.choice(["dtype", "size", "none", "fewer", "more", "gaps", "turned", "spread", "rows apart", "empty"])
    d = r.randrange(t.dim())
    if kind == "dtype":
        return t.to(r.choice(DTYPES))
    if kind == "size":
        shape = list(t.shape)
        shape[d] = max(1, shape[d] + r.choice([-1, 1]))
        return t.new_zeros(shape)
    if kind == "none" or t.numel() == 0:
        return None
    if kind == "fewer":
        return t.select(d, 0)
    if kind == "more":
        return t.unsqueeze(d)
    if kind == "gaps":
        return t.new_zeros((*t.shape[:-1], 2 * t.shape[-1]))[..., ::2]
    if kind == "turned":
        return t.transpose(0, -1).contiguous().transpose(0, -1)
    if kind == "spread":
        return t.select(d, 0).unsqueeze(d).expand(t.shape)
    if kind == "rows apart":
        return t.new_zeros((*t.shape[:-1], t.shape[-1] + 8))[..., : t.shape[-1]]
    return t.narrow(d, 0, 0)


def refusal(call, args):
    try:
        call(**args)
    except ValueError as e:
        return str(e)
    return None


@pytest.mark.parametrize("name", CALLS)
def test_the_chain_accepts_what_the_checks_accept(machine, name):  # noqa: F811
    call, make = CALLS[name]
    r = random.Random(name)
    seen = {True: 0, False: 0}
    for _ in range(600):
        plain = make()
        for _ in range(r.choice([0, 1, 1, 1, 2])):
            n = r.choice([n for n, t in plain.items() if t is not None and t.dim() > 0])
            plain[n] = change(r, plain[n])
        said = {n: None if t is None else t.as_subclass(Near) for n, t in plain.items()}
        what = {n: None if t is None else (t.dtype, tuple(t.shape), t.stride()) for n, t in plain.items()}
        mine, its = refusal(call, said), refusal(call, plain)
        assert its is not None
        assert mine == (None if "must live on the GPU" in its else its), what
        seen[mine is None] += 1
    assert min(seen.values()) > 50


@pytest.mark.parametrize("name", CALLS)
def test_one_tensor_elsewhere(machine, name):  # noqa: F811
    call, make = CALLS[name]
    for n in make():
        for elsewhere, message in ((Far, "one GPU"), (torch.Tensor, "on the GPU")):
            args = {m: t.as_subclass(elsewhere if m == n else Near) for m, t in make().items()}
            assert message in (refusal(call, args) or ""), n


def near(make, **change):
    return {n: t.as_subclass(Near) for n, t in (make() | change).items()}


def test_sizes_beyond_32_bits(machine):  # noqa: F811
    cache = torch.zeros(1, 16, 2, 64, dtype=bf).expand(2 ** 31, 16, 2, 64)
    for call, make in ((tq.tree_attention, attention), (tq.cache_append, append)):
        with pytest.raises(ValueError, match="range"):
            call(**near(make, k_cache=cache, v_cache=cache))
    far_row = torch.empty(1, 1, 2 ** 32 + 50, dtype=torch.float16)  # never touched
    small = dict(tokens=torch.zeros(1, 1, dtype=i32), u=torch.zeros(1, 1))
    with pytest.raises(ValueError, match="below 2"):
        tq.verify_tree(**near(dict, logits=far_row, parents=torch.zeros(1, 1, dtype=i32), **small))
    with pytest.raises(ValueError, match="below 2"):
        tq.verify_chain(**near(dict, logits=far_row, q=torch.empty(1, 0, 2 ** 32 + 50), **small))
    for call, make in ((tq.distill, both), (tq.distill_loss, loss), (tq.distill_grad, both)):
        args = {n: t[:1] for n, t in make().items()} | dict(logits=far_row[0])
        with pytest.raises(ValueError, match="below 2"):
            call(**near(dict, **args))
    assert machine.calls == []
