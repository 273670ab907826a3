"""Pins of the oracle's operators between the projection's rows and the cache."""

import math

import numpy as np
import pytest

from oracle import rows


def test_codes_of_a_ramp():
    """0 .. 31 times 15 / 31: the codes are the nearest of 16 steps of the scale."""
    x = np.arange(32, dtype=np.float32) * np.float32(0.5) - 3
    codes, scale, low = rows.q4_codes(x)
    assert low[0] == -3 and scale[0] == np.float16(np.float32(15.5) / 15)
    steps = (x.astype(np.float64) + 3) / float(scale[0])
    assert np.abs(codes - steps).max() <= 0.5 and codes[0] == 0 and codes[-1] == 15


def test_ties_go_to_even():
    x = np.zeros(32, np.float32)
    x[:5] = 15, 0.5, 1.5, 2.5, 3.5  # a scale of 1
    assert list(rows.q4_codes(x)[0][:5]) == [15, 0, 2, 2, 4]


@pytest.mark.parametrize("value", [0.0, -7.25, 65408.0, 1e-7])
def test_equal_numbers_stand_for_themselves(value):
    """Code and scale of 0, the minimum in fp16."""
    x = np.full(64, value, np.float32)
    codes, scale, _ = rows.q4_codes(x)
    assert not codes.any() and not scale.any()
    assert (rows.q4_unpack(rows.q4_pack(x)) == float(np.float16(value))).all()


def test_numbers_that_are_none():
    x = np.linspace(-1, 1, 32).astype(np.float32)
    x[3], x[4], x[5] = np.nan, np.inf, -np.inf
    codes, scale, low = rows.q4_codes(x)
    assert low[0] == -65408 and scale[0] == np.float16(np.float32(130816) / 15)
    assert codes[4] == 15 and codes[5] == 0 and codes[3] in (7, 8)


@pytest.mark.parametrize("low", [-65504.0, -65408.0, -3e4, 0.0, 65000.0])
def test_the_largest_numbers_stay_finite_in_fp16(low):
    for high in (65504.0, 65408.0, 65376.0, 64000.0, 3e38):
        x = np.linspace(low, high, 32).astype(np.float32)
        assert np.isfinite(rows.round_to(rows.q4_unpack(rows.q4_pack(x)), "f16")).all()


def test_bytes_of_a_row():
    """Eight codes of a word: the even ones in the lower half; a pair (scale, low) behind the codes."""
    x = np.zeros(32, np.float32)
    x[:8] = 1, 2, 3, 4, 5, 6, 7, 15
    b = rows.q4_pack(x)
    assert b.shape == (20,)
    assert b[:4].view("<u4")[0] == 0x1 | 0x3 << 4 | 0x5 << 8 | 0x7 << 12 | 0x2 << 16 | 0x4 << 20 | 0x6 << 24 | 0xF << 28
    assert list(b[16:].view(np.float16)) == [1, 0]
    assert (rows.q4_unpack(b) == x).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_quarter_turn(interleaved):
    x = np.arange(1.0, 5.0)[None, None]  # one token, one head, two pairs
    out, size = rows.norm_rotate(x, None, np.array([1]), [math.pi / 2, 0.0], None, interleaved)
    want = [-2, 1, 3, 4] if interleaved else [-3, 2, 1, 4]
    assert np.abs(out[0, 0] - want).max() < 1e-6
    assert list(size[0, 0]) == ([3, 3, 7, 7] if interleaved else [4, 6, 4, 6])


def test_norm():
    out, _ = rows.norm_rotate(np.array([[[3.0, 4.0]]]), [1.0, 2.0], np.array([0]), [], 0.5, False)
    assert np.allclose(out[0, 0], np.array([3, 8]) / math.sqrt(13))


def test_prompts_do_not_see_each_other():
    r = np.random.default_rng(3)
    q, k, v = r.standard_normal((7, 4, 8)), r.standard_normal((7, 2, 8)), r.standard_normal((7, 2, 8))
    out, _, _, seen = rows.prompt_attention(q, k, v, [1, 1, 4, 6], 0.3)
    assert list(seen) == [False] + [True] * 5 + [False]
    one, _, _, _ = rows.prompt_attention(q[4:6], k[4:6], v[4:6], [0, 2], 0.3)
    assert np.allclose(out[4:6], one) and np.allclose(out[1, 3], v[1, 1]) and not out[[0, 6]].any()


def test_rounding():
    x = np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -20, -3.0])
    assert list(rows.round_to(x, "bf16")) == [1, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -3]
