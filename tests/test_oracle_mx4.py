"""Pins of the microscaled 4-bit oracle: hand-worked blocks and closed forms."""

import numpy as np
import pytest

from oracle import mx4
from oracle import mxfp4 as mx


def test_hand_worked_block():
    """A block whose largest value is 7: exponent 2, scale 2^0 (byte 127)."""
    v = np.zeros((1, 32))
    v[0, :12] = [7.0, -6.0, 5.0, 4.99, 3.5, -2.5, 1.75, 1.25, 0.75, 0.25, -0.0, 0.26]
    packed, scale = mx4.quantize_ref(v)
    assert scale.tolist() == [[127]]
    got = mx4.values_ref(packed, scale)[0, :12]
    # ties go to the even code: 5 -> 4, 3.5 -> 4, 2.5 -> 2, 1.75 -> 2, 1.25 -> 1, 0.75 -> 1, 0.25 -> 0
    assert got.tolist() == [6.0, -6.0, 4.0, 4.0, 4.0, -2.0, 2.0, 1.0, 1.0, 0.0, 0.0, 0.5]
    assert packed[0, 5] & 15 == 8  # the sign of -0.0 stays
    # without saturation 7 > 6 doubles the scale: 3.5 -> 4 (tie to even), 8 in all
    packed, scale = mx4.quantize_ref(v, saturate=False)
    assert scale.tolist() == [[128]]
    assert mx4.values_ref(packed, scale)[0, 0] == 8.0


@pytest.mark.parametrize("saturate", [True, False])
def test_scale_bytes(saturate):
    f = lambda t: mx4.block_scale_byte(t, saturate)  # noqa: E731
    assert f(0.0) == 0 and f(2.0**-149) == 0 and f(2.0**-125) == 0 and f(np.inf) == 255 and f(np.nan) == 255
    assert f(4.0) == 127 and f(6.0) == 127 and f(np.nextafter(6.0, 7.0)) == (127 if saturate else 128)
    assert f(2.0**127) == 252 and f(float(np.finfo(np.float32).max)) == (252 if saturate else 253)


def test_representable_values_survive():
    """Values of a microscaled matrix quantise to themselves (blocks that hold a 4 or a 6)."""
    g = np.random.default_rng(5)
    packed = g.integers(0, 256, (40, 32), dtype=np.uint8)
    packed[:, 0] = 0x76  # codes 6 and 7 first in every second block
    packed[:, 16] = 0x76
    scale = g.integers(1, 253, (40, 2), dtype=np.uint8)
    v = mx4.values_ref(packed, scale)
    for saturate in (True, False):
        p, s = mx4.quantize_ref(v, saturate)
        assert np.array_equal(s, scale) and np.array_equal(mx4.values_ref(p, s), v)


def test_values_match_the_codec_oracle():
    g = np.random.default_rng(6)
    packed = g.integers(0, 256, (7, 48), dtype=np.uint8)
    scale = g.integers(0, 255, (7, 3), dtype=np.uint8)
    assert np.array_equal(mx4.values_ref(packed, scale), mx.decode_ct(packed, scale))


@pytest.mark.parametrize("saturate", [True, False])
def test_error_bound(saturate):
    """Rounding moves a value by at most a quarter of its binade's upper end (one step of E2M1 is half the
    value's power of two, at least half the block unit), and clamping only happens with saturation."""
    g = np.random.default_rng(7)
    v = g.standard_normal((64, 96)) * np.exp(g.standard_normal((64, 96)))
    p, s = mx4.quantize_ref(v, saturate)
    q = mx4.values_ref(p, s)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    a = np.abs(v) / unit
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    inside = a <= 6
    assert np.all(np.abs(q - v)[inside] <= (0.5 * step * unit)[inside])
    assert saturate or inside.all()
    assert np.all(np.abs(q)[~inside] == (6 * unit)[~inside])


def test_nonfinite_block():
    v = np.ones((1, 64))
    v[0, 40] = np.nan
    p, s = mx4.quantize_ref(v)
    assert s.tolist() == [[125, 255]] and set(p[0, 16:].tolist()) == {0x77}
    assert np.isnan(mx4.values_ref(p, s)[0, 32:]).all()


def test_product_closed_form():
    """All codes 1.0 at scale 2^-1 against all codes 2.0 at 2^3: every entry is K * (0.5 * 16)."""
    a = np.full((3, 48), 0x22, dtype=np.uint8)
    w = np.full((5, 48), 0x44, dtype=np.uint8)
    out = mx4.product_ref(a, np.full((3, 3), 126, np.uint8), w, np.full((5, 3), 130, np.uint8))
    assert out.shape == (3, 5) and np.all(out == 96 * 0.5 * 16)
