"""Norm and rotation of query and key rows on the GPU, against the float64 oracle.

Tolerance, with f = 2^-24, h = finfo(type).eps / 2 and size = |y1| + |y2| of the pair an element is made of:
  the squares' sum (16 products in a lane, 5 joins), its mean, eps, root and reciprocal: half of 22 f, and 3 f
  the products with it and with the weight                                      2 f
  cosine and sine: 2 units in the last place, the part of a turn (pi f)         6 f
  the two products of the rotation and their sum                                2 f
together below 32 f size; the angle t in 64 bits (product, product with 1 / 2 pi, that constant) 2^-51 |t| size;
the last rounding h |out|, of fp16's subnormals 2^-25."""

import numpy as np
import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from oracle import rows as oracle
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def inputs(seed, dt, tokens, hq, hkv, dim, rotary, *, weights="same", far=1000, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((*tokens, hq + 2 * hkv, dim), generator=g) * spread).to(DT[dt])
    q, k, _ = x.split([hq, hkv, hkv], dim=-2)
    pos = torch.randint(0, far, tokens, generator=g).to(torch.int32)
    freq = 10000.0 ** (-torch.arange(0, rotary, 2) / max(rotary, 1)) if rotary else None
    w = [None, None]
    if weights:
        w = [(1 + 0.3 * torch.randn(dim, generator=g)).to(DT[dt if weights == "same" else weights]) for _ in range(2)]
    return x, q, k, pos, freq, w


def check(got, x, w, pos, freq, eps, interleaved, dt):
    x64 = x.double().numpy()
    freqs = [] if freq is None else freq.float().numpy()
    want, size = oracle.norm_rotate(x64, None if w is None else w.double().numpy(), pos.numpy(), freqs, eps, interleaved)
    f, h = 2.0 ** -24, torch.finfo(DT[dt]).eps / 2
    t = np.abs(pos.numpy().astype(np.float64))[..., None, None] * (max(np.abs(freqs)) if len(freqs) else 0)
    tol = h * np.abs(want) + (32 * f + 2.0 ** -51 * t) * size + (2.0 ** -25 if dt == "f16" else 2.0 ** -130)
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - want) - tol
    assert over.max() <= 0, f"{over.max():.3g} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


def run(dt, tokens, hq, hkv, dim, rotary, *, interleaved=False, eps=1e-6, seed=0, **kw):
    x, q, k, pos, freq, w = inputs(seed + dim, dt, tokens, hq, hkv, dim, rotary, **kw)
    xg = x.cuda()
    qg, kg, _ = xg.split([hq, hkv, hkv], dim=-2)
    wg = [None if a is None else a.cuda() for a in w]
    out = tq.norm_rotate(qg, kg, pos.cuda(), None if freq is None else freq.cuda(), *wg, eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(xg.cpu(), x)
    for got, a, b in zip(out, (q, k), w):
        assert got.dtype == a.dtype and got.shape == a.shape
        check(got, a, b, pos, freq, eps, interleaved, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rotary", [(16, 16), (32, 16), (48, 48), (64, 64), (80, 32), (96, 96), (112, 112), (128, 128),
                                        (128, 64), (160, 160), (192, 64), (256, 256), (320, 160), (512, 512), (512, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes(gpu, dt, dim, rotary, interleaved):
    say(f"{dt} {dim} {rotary} {interleaved}")
    run(dt, (2, 5), 3, 2, dim, rotary, interleaved=interleaved)


@pytest.mark.parametrize("tokens", [(1,), (7,), (1000,), (1, 1), (1, 300), (300, 1), (3, 2051), (5, 413)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (40, 8)])
def test_tokens_and_heads(gpu, tokens, hq, hkv):
    say(f"{tokens} {hq} {hkv}")
    run("bf16", tokens, hq, hkv, 64, 32)


@pytest.mark.parametrize("weights", [None, "f32", "f16", "bf16"])
def test_weights(gpu, weights):
    for dt in DT:
        run(dt, (3, 4), 4, 2, 128, 128, weights=weights)


def test_one_weight(gpu):
    x, q, k, pos, freq, w = inputs(3, "bf16", (9,), 4, 2, 64, 64)
    out = tq.norm_rotate(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), None, w[1].cuda())
    check(out[0], q, None, pos, freq, 1e-6, False, "bf16")
    check(out[1], k, w[1], pos, freq, 1e-6, False, "bf16")


def test_norm_alone_and_rotation_alone(gpu):
    run("f32", (4, 6), 4, 2, 128, 0)
    run("f32", (4, 6), 4, 2, 128, 96, eps=None, weights=None)
    run("f16", (4, 6), 4, 2, 96, 32, eps=None, weights=None, interleaved=True)


@pytest.mark.parametrize("far", [1 << 16, 1 << 20, 1 << 27])
def test_far_positions(gpu, far):
    run("f32", (2, 64), 2, 1, 128, 128, far=far)


def test_negative_positions(gpu):
    x, q, k, pos, freq, _ = inputs(3, "f32", (9,), 4, 2, 64, 64)
    out = tq.norm_rotate(q.cuda(), k.cuda(), (-pos).cuda(), freq.cuda())
    check(out[0], q, None, -pos, freq, 1e-6, False, "f32")


@pytest.mark.parametrize("spread", [1e-4, 100.0])
def test_small_and_large_rows(gpu, spread):
    run("bf16", (2, 9), 4, 2, 128, 128, spread=spread)


def test_rows_of_zeros(gpu):
    z = torch.zeros((3, 4, 64), device="cuda")
    freq = torch.ones(16, device="cuda")
    out = tq.norm_rotate(z, z[:, :2], torch.arange(3, dtype=torch.int32, device="cuda"), freq)
    assert not out[0].any() and not out[1].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_in_place(gpu, dt):
    """The fused projection's rows turned where they stand; its values stay."""
    x, q, k, pos, freq, w = inputs(5, dt, (3, 17), 4, 2, 128, 64)
    xg = x.cuda()
    views = xg.split([4, 2, 2], dim=-2)
    out = tq.norm_rotate(*views[:2], pos.cuda(), freq.cuda(), *(a.cuda() for a in w), out=views[:2])
    assert out[0].data_ptr() == xg.data_ptr()
    check(xg[..., :4, :], q, w[0], pos, freq, 1e-6, False, dt)
    check(xg[..., 4:6, :], k, w[1], pos, freq, 1e-6, False, dt)
    assert torch.equal(xg[..., 6:, :].cpu(), x[..., 6:, :])


def test_rows_at_odd_addresses(gpu):
    """Rows that begin at any element, heads apart by odd strides, results of the same kind."""
    x, q, k, pos, freq, w = inputs(7, "bf16", (2, 5), 4, 2, 64, 64)

    def odd(t):
        wide = torch.zeros((*t.shape[:2], t.shape[2], 67), dtype=t.dtype, device="cuda")
        view = wide.flatten()[1:1 + wide.numel() - 3].as_strided(t.shape, wide.stride())
        view.copy_(t)
        return view

    outs = odd(torch.zeros_like(q)), odd(torch.zeros_like(k))
    tq.norm_rotate(odd(q), odd(k), pos.cuda(), freq.cuda(), *(a.cuda() for a in w), out=outs)
    for got, a, b in zip(outs, (q, k), w):
        check(got, a, b, pos, freq, 1e-6, False, "bf16")


def test_a_nan_stays_in_its_row(gpu):
    x, q, k, pos, freq, w = inputs(9, "bf16", (6,), 4, 2, 64, 64)
    a = q.cuda().clone()
    a[2, 1, 5] = float("nan")
    out = tq.norm_rotate(a, k.cuda(), pos.cuda(), freq.cuda())[0]
    bad = out.isnan().any(-1).cpu()
    assert bad[2, 1] and bad.sum() == 1


def test_no_tokens(gpu):
    e = torch.empty((0, 4, 64), device="cuda")
    out = tq.norm_rotate(e, e[:, :1], torch.empty(0, dtype=torch.int32, device="cuda"), torch.ones(8, device="cuda"))
    assert out[0].shape == (0, 4, 64) and out[1].shape == (0, 1, 64)


def test_gradient_is_refused_when_asked_for(gpu):
    x, q, k, pos, freq, _ = inputs(9, "f32", (6,), 4, 2, 64, 64)
    a = q.cuda().requires_grad_()
    out = tq.norm_rotate(a, k.cuda(), pos.cuda(), freq.cuda())
    assert out[0].requires_grad
    with pytest.raises(RuntimeError, match="norm_rotate has no gradient"):
        out[0].sum().backward()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_heads_first_rows_in_place(gpu, dt):
    """[batch][heads][tokens][dim] of a fused projection, a sequence's queries, then its keys, then its values."""
    x, q, k, pos, freq, w = inputs(6, dt, (3, 17), 4, 2, 128, 64)
    xg = x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    views = xg.split([4, 2, 2], dim=-2)
    tq.norm_rotate(*views[:2], pos.cuda(), freq.cuda(), *(a.cuda() for a in w), out=views[:2])
    check(xg[..., :4, :], q, w[0], pos, freq, 1e-6, False, dt)
    check(xg[..., 4:6, :], k, w[1], pos, freq, 1e-6, False, dt)
    assert torch.equal(xg[..., 6:, :].cpu(), x[..., 6:, :])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("spread", [1e-36, 1e-30, 1e-24, 1e-20, 1e-18, 1e17, 1e19, 1e24, 1e30, 1e36])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-6])
def test_rows_whose_squares_leave_fp32(gpu, dt, spread, eps):
    run(dt, (2, 9), 4, 2, 128, 64, spread=spread, eps=eps)


@pytest.mark.parametrize("dim", [16, 64, 256, 512])
def test_rows_of_many_sizes_beside_each_other(gpu, dim):
    """Rows of every size share a wave with rows of others."""
    x, q, k, pos, freq, w = inputs(8, "f32", (40,), 4, 2, dim, 16)
    sizes = 10.0 ** torch.linspace(-36, 36, 40)[torch.randperm(40, generator=torch.Generator().manual_seed(1))]
    x = x * sizes[:, None, None]
    q, k, _ = x.split([4, 2, 2], dim=-2)
    out = tq.norm_rotate(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), *(a.cuda() for a in w), eps=0.0)
    check(out[0], q, w[0], pos, freq, 0.0, False, "f32")
    check(out[1], k, w[1], pos, freq, 0.0, False, "f32")


@pytest.mark.parametrize("tokens", [(1, 1), (4, 300)])
def test_in_a_graph(gpu, tokens):
    """A captured call in place and one with results of its own, replayed over other rows and positions, with
    eager work in between."""
    x, q, k, pos, freq, w = inputs(11, "bf16", tokens, 4, 2, 128, 64)
    xg, posg, freqg, wg = torch.empty_like(x, device="cuda"), pos.cuda(), freq.cuda(), [a.cuda() for a in w]
    views = xg.split([4, 2, 2], dim=-2)[:2]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        xg.copy_(x)
        tq.norm_rotate(*views, posg, freqg, *wg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        apart = tq.norm_rotate(*views, posg, freqg, *wg)
        tq.norm_rotate(*views, posg, freqg, *wg, out=views)
    for seed in (11, 12, 13, 11):
        x, q, k, pos, _, _ = inputs(seed, "bf16", tokens, 4, 2, 128, 64)
        xg.copy_(x)
        posg.copy_(pos)
        eager = tq.norm_rotate(*views, posg, freqg, *wg)
        graph.replay()
        torch.cuda.synchronize()
        for got, there, want in zip(apart, views, eager):
            assert torch.equal(got, want) and torch.equal(there, want)
        check(eager[0], q, w[0], pos, freq, 1e-6, False, "bf16")
        assert torch.equal(xg[..., 6:, :].cpu(), x[..., 6:, :])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rotary", [(32, 24), (48, 24), (48, 40), (64, 24), (64, 56), (80, 72), (96, 24), (96, 88), (128, 24), (128, 120),
                                        (160, 40), (256, 24), (256, 248), (320, 72), (512, 24), (512, 504)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_sizes_between_pieces(gpu, dt, dim, rotary, interleaved):
    say(f"{dt} {dim} {rotary} {interleaved}")
    run(dt, (2, 5), 3, 2, dim, rotary, interleaved=interleaved)
    run(dt, (700,), 5, 1, dim, rotary, interleaved=interleaved, weights="f32" if dt == "f16" else None)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rotary_sizes_between_pieces_in_place(gpu, dt, interleaved):
    x, q, k, pos, freq, w = inputs(5, dt, (3, 417), 4, 2, 96, 24)
    xg = x.cuda()
    views = xg.split([4, 2, 2], dim=-2)
    tq.norm_rotate(*views[:2], pos.cuda(), freq.cuda(), *(a.cuda() for a in w), interleaved=interleaved, out=views[:2])
    check(xg[..., :4, :], q, w[0], pos, freq, 1e-6, interleaved, dt)
    check(xg[..., 4:6, :], k, w[1], pos, freq, 1e-6, interleaved, dt)
    assert torch.equal(xg[..., 6:, :].cpu(), x[..., 6:, :])


def test_infinities_beside_the_turned_part(gpu):
    """What lies behind rotary_dim is not multiplied by any sine."""
    for interleaved in (False, True):
        x = torch.ones((3, 2, 96))
        x[..., 24:32] = float("inf")
        out = tq.norm_rotate(x.cuda(), x.cuda(), torch.arange(3, dtype=torch.int32).cuda(), torch.ones(12, device="cuda"), eps=None,
                             interleaved=interleaved)[0].cpu()
        assert torch.equal(out[..., 24:], x[..., 24:]) and out[..., :24].isfinite().all()
