"""Distillation from a teacher's top logits on the GPU, against the float64 oracle.

Tolerances, with f = 2^-24 (half an ulp of fp32), R the largest |x - max| / T among what
enters a figure and n = vocab / 256 + 64 (the longest chain of fp32 sums of the simplest
split, and room for the joins):
  ln p, ln t: the difference, its scaling and the logarithm's own   (4 R + 2 |ln| + n + 16) f
  p, t:       the exponent's rounding, the exponential, the sum     (4 R + n + 16) f, relative
  loss:       sum of t (ln t - ln p) and its own sum of K terms
  gradient:   half an ulp of its type, and w / T times what p and t are off"""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import operators as ops
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F = 2.0 ** -24


def inputs(seed, rows, vocab, k, dt, top_dt=None, missing=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, vocab), generator=g)
    at = torch.stack([torch.randperm(vocab, generator=g)[:k] if k <= vocab else torch.randint(0, vocab, (k,), generator=g)
                      for _ in range(rows)]) if rows else torch.zeros((0, k), dtype=torch.long)
    top = torch.randn((rows, k), generator=g) * 2 + 8
    x.scatter_(1, at, top + torch.randn((rows, k), generator=g))
    if missing:
        at = torch.where(torch.arange(k) < torch.randint((k + 1) // 2, k + 1, (rows, 1), generator=g), at, -1)
    w = torch.rand((rows,), generator=g) + 0.1
    return x.to(DT[dt]), at.to(torch.int32), top.to(DT[top_dt or dt]), w


def check(x, index, top, w, temperature=1.0, got=None):
    if got is None:
        a = [t.cuda() for t in (x, index, top, w)]
        loss, grad = tq.distill(*a, temperature=temperature)
        alone = tq.distill_loss(*a[:3], temperature=temperature)
        apart = tq.distill_grad(*a, temperature=temperature)
        torch.cuda.synchronize()
        assert torch.equal(loss, alone) and torch.equal(grad, apart)
    else:
        loss, grad = got
    x64 = x.double().numpy()
    y64, idx, w64 = top.double().numpy(), index.numpy(), w.double().numpy()
    want, want_grad, p, t = ops.distill(x64, idx, y64, w64, temperature)
    rows, vocab = x64.shape
    there = (idx >= 0) & (idx < vocab)
    n = vocab / 256 + 64
    xs, ys = x64 / temperature, np.where(there, y64 / temperature, 0.0)
    top_x = xs.max(1, keepdims=True)
    top_y = np.where(there, ys, -np.inf).max(1, keepdims=True)
    rx = np.where(there, top_x - np.take_along_axis(xs, np.where(there, idx, 0), 1), 0.0)
    ry = np.where(there, np.where(np.isfinite(top_y), top_y, 0.0) - ys, 0.0)
    far = np.maximum(rx, ry).max(1)
    reach = far + np.log(vocab) + 20
    tol = (8 * far + 4 * reach + 2 * n + 32 + index.shape[1] / 64) * F * (1 + reach)
    off = np.abs(loss.double().cpu().numpy() - want)
    assert (off <= tol).all(), (off.max(), tol[off.argmax()])
    scale = (np.abs(w64) / temperature)[:, None]
    h = torch.finfo(x.dtype).eps / 2
    dx = top_x - xs
    dp = np.where(p > 0, p * (4 * np.where(p > 0, dx, 0) + n + 16) * F, 0.0)  # -inf has exactly no probability
    dt_ = t * (4 * ry.max(1, keepdims=True) + n + 16 + index.shape[1]) * F
    tol = scale * (dp + dt_ + 4 * F * (p + t)) * (1 + h) + h * np.abs(want_grad)
    tol += {"torch.float16": 2.0 ** -24, "torch.bfloat16": 2.0 ** -126, "torch.float32": 2.0 ** -126}[str(x.dtype)]
    off = np.abs(grad.double().cpu().numpy() - want_grad) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


VOCABS = [1, 2, 7, 8, 9, 63, 64, 65, 257, 1000, 4096, 8191, 50257]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_vocabularies(gpu, dt, vocab):
    say(f"distill {dt} {vocab}")
    check(*inputs(vocab, 5, vocab, min(20, vocab), dt))


@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 200, 255, 257, 1024])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 2.0])
def test_entries_and_temperatures(gpu, k, temperature):
    say(f"entries {k} at {temperature}")
    check(*inputs(k, 4, 3001, k, "bf16", "f32"), temperature)


@pytest.mark.parametrize("temperature", [0.1, 0.3, 0.7, 1.3, 3.0, 7.0, 1.4426950216293335])
@pytest.mark.parametrize("rows,vocab", [(3, 777), (3, 20011), (200, 20011)])
def test_temperatures_that_round_either_way(gpu, temperature, rows, vocab):
    """log2(e) / T is above its fp32 value for some and below for others; rows hold -inf."""
    say(f"temperature {temperature} {rows} {vocab}")
    x, index, top, w = inputs(rows, rows, vocab, 12, "f16", "f32", missing=False)
    x[:, 700:740] = -float("inf")
    index[:] = torch.arange(12, dtype=torch.int32) * 50
    check(x, index, top, w, temperature)


@pytest.mark.parametrize("rows", [0, 1, 2, 15, 16, 17, 255, 300, 1025])
def test_row_counts(gpu, rows):
    say(f"rows {rows}")
    x, index, top, w = inputs(rows + 1, rows, 515, 9, "f16")
    if rows == 0:
        loss, grad = tq.distill(x.cuda(), index.cuda(), top.cuda(), w.cuda())
        assert loss.shape == (0,) and grad.shape == (0, 515)
        return
    check(x, index, top, w)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [2, 300])
def test_the_heads_vocabulary(gpu, dt, rows):
    say(f"head {dt} {rows}")
    x, index, top, w = inputs(rows, min(rows, 4), 129280, 64, dt)
    if rows > 4:  # enough rows for another split of the work; the first ones are compared
        many = [t.cuda().repeat((rows // 4,) + (1,) * (t.dim() - 1)) for t in (x, index, top, w)]
        loss, grad = tq.distill(*many)
        torch.cuda.synchronize()
        assert torch.equal(grad[:4], grad[-4:]) and torch.equal(loss[:4], loss[-4:])
        check(x, index, top, w, got=(loss[:4], grad[:4]))
    else:
        check(x, index, top, w)


@pytest.mark.parametrize("top_dt", ["f32", "bf16", "f16"])
def test_teachers_type_is_its_own(gpu, top_dt):
    check(*inputs(3, 6, 1003, 30, "bf16", top_dt))


def test_the_same_place_more_than_once(gpu):
    x, index, top, w = inputs(5, 4, 300, 40, "f32", missing=False)
    index[0] = 7
    index[1, ::2] = 11
    index[2, 30:] = index[2, :10]
    index[3, 5], index[3, 39] = index[3, 0], index[3, 0]
    check(x, index, top, w)


@pytest.mark.parametrize("vocab", [13, 20011, 140001])
@pytest.mark.parametrize("k", [3, 9, 300])
def test_many_entries_of_few_places(gpu, vocab, k):
    """Every entry of a row at one of a few places, the last ones of the row among them."""
    say(f"few places {vocab} {k}")
    x, index, top, w = inputs(vocab + k, 3, vocab, k, "bf16", "f32", missing=False)
    g = torch.Generator().manual_seed(k)
    places = torch.tensor([0, 1, 7, vocab // 2, vocab - 3, vocab - 1])
    index = places[torch.randint(0, 6, (3, k), generator=g)].to(torch.int32)
    index[2] = vocab - 1
    check(x, index, top, w)


def test_a_few_very_long_rows(gpu):
    check(*inputs(31, 2, 3_000_017, 40, "f32"))


def test_rows_without_a_teacher_or_weight(gpu):
    x, index, top, w = inputs(6, 5, 700, 8, "bf16")
    index[1] = -1
    index[2] = torch.tensor([-5, 700, 2 ** 31 - 1, -(2 ** 31), 3, 701, -1, -2], dtype=torch.int32)
    w[3] = 0.0
    check(x, index, top, w)
    x[3, 5] = float("nan")  # a row of weight 0 has no gradient, whatever it holds
    a = [t.cuda() for t in (x, index, top, w)]
    loss, grad = tq.distill(*a)
    torch.cuda.synchronize()
    assert not grad[1].any() and loss[1] == 0 and not grad[3].any() and torch.isnan(loss[3])
    assert torch.equal(tq.distill_grad(*a), grad)


def test_masked_and_extreme_logits(gpu):
    x, index, top, w = inputs(7, 4, 600, 6, "f32", missing=False)
    x[0, 100:400] = -float("inf")  # a masked part of the vocabulary
    index[0] = torch.tensor([1, 2, 3, 4, 5, 6], dtype=torch.int32)
    x[1] = torch.finfo(torch.float32).min
    x[1, 9] = 0.0
    index[1] = 9
    top[2, 3:] = -float("inf")  # entries that the teacher gives no mass
    x[3] *= 1e4
    index[3] = x[3].argmax()
    a = [t.cuda() for t in (x, index, top, w)]
    loss, grad = tq.distill(*a)
    torch.cuda.synchronize()
    want, want_grad, _, _ = ops.distill(x.double().numpy(), index.numpy(), top.double().numpy(), w.double().numpy(), 1.0)
    assert np.isfinite(want).all()
    assert np.abs(loss.double().cpu().numpy() - want).max() < 1e-4  # 64 * 2^-24 * (20 + the largest logit, 10)
    assert np.abs(grad.double().cpu().numpy() - want_grad).max() < 1e-4
    index[0, 0] = 200  # mass on a place that the student cannot give
    loss = tq.distill_loss(x.cuda(), index.cuda(), top.cuda())
    assert torch.isinf(loss[0]) and loss[0] > 0


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_gradient_against_differences(gpu, dt):
    """Central differences of the kernel's own loss. The gradient is of size 1; the step of
    2^-5 leaves (2^-5)^2 / 6 of the third derivative (below 1), and the loss, about 5 with
    some hundred roundings of 2^-24, over the step: 2^-9 in all."""
    x, index, top, _ = inputs(8, 1, 64, 5, dt, "f32", missing=False)
    x = (x * 0.5).half().to(DT[dt])
    step = 2.0 ** -5
    places = torch.arange(64)
    up, down = x.repeat(64, 1).float(), x.repeat(64, 1).float()
    up[places, places] += step
    down[places, places] -= step
    up, down = up.to(DT[dt]), down.to(DT[dt])
    width = (up.double() - down.double())[places, places]
    many = [t.repeat(64, 1).cuda() for t in (index, top)]
    lu, ld = (tq.distill_loss(z.cuda(), *many).double().cpu() for z in (up, down))
    grad = tq.distill_grad(x.cuda(), index.cuda(), top.cuda(), torch.ones(1, device=gpu))[0].double().cpu()
    assert ((lu - ld) / width - grad).abs().max() < 2.0 ** -9 + (2.0 ** -10 if dt == "f16" else 0)


def test_strided_rows_at_odd_addresses(gpu):
    for dt in ("bf16", "f32"):
        x, index, top, w = inputs(9, 6, 1021, 10, dt)
        wide = torch.full((6, 1030), 50.0, dtype=DT[dt], device=gpu)
        for shift in (0, 1, 3, 8):
            wide.fill_(50.0)
            wide[:, shift : shift + 1021] = x.cuda()
            a = (wide[:, shift : shift + 1021], index.cuda(), top.cuda(), w.cuda())
            loss, grad = tq.distill(*a)
            torch.cuda.synchronize()
            check(x, index, top, w, got=(loss, grad))


def test_graph_replays_and_another_stream(gpu):
    sets = [inputs(20 + i, 8, 20000, 30, "bf16") for i in range(4)]
    a = [t.cuda() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.distill(*a)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grad = tq.distill(*a)
    for i in (1, 2, 3, 0):
        for have, new in zip(a, sets[i]):
            have.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(*sets[i], got=(loss, grad))
        again = tq.distill(*a)
        assert torch.equal(again[0], loss) and torch.equal(again[1], grad)
