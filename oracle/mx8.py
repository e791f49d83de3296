"""fp64 oracle of microscaled 8-bit rounding, the norm in front of it, and products with microscaled 4-bit weights.

Written from the definitions (OCP Microscaling Formats specification 1.0: one E8M0 scale per 32 elements, shared
exponent floor(log2(max |v|)) less the element type's largest exponent, 8 for E4M3; elements rounded to nearest even and
clamped); shares no code with the GPU path.
"""

from __future__ import annotations

import numpy as np

from oracle import mx4


def magnitudes() -> np.ndarray:
    """The 127 magnitudes of E4M3 (codes 0 .. 126), exponent bias 7."""
    c = np.arange(127)
    ex, man = c >> 3, c & 7
    return np.where(ex == 0, man / 8.0 * 2.0**-6, (1 + man / 8.0) * np.exp2(ex - 7.0))


MAGNITUDES = magnitudes()


def quantize_ref(x: np.ndarray, saturate: bool = True):
    """x [R, K] (any float values, long double included) -> (codes u8 [R, K], scale u8 [R, K/32])."""
    v = np.asarray(x)
    v = v if v.dtype == np.longdouble else v.astype(np.float64)
    R, K = v.shape
    v = v.reshape(R, K // 32, 32)
    top = np.abs(v).max(-1) if v.size else np.zeros((R, K // 32))
    top = np.where(np.isnan(v).any(-1), np.nan, top)
    scale = np.zeros(top.shape, np.int64)
    for i, t in np.ndenumerate(top):
        if not np.isfinite(t):
            scale[i] = 255
        elif t > 0:
            _, ex = np.frexp(t)  # t = f * 2^ex, 0.5 <= f < 1
            e = max(int(ex) - 1 - 8, -127)
            e += int(not saturate and t > 448 * np.ldexp(type(t)(1), e))
            scale[i] = min(e + 127, 255)
    unit = np.ldexp(np.ones((), v.dtype), scale - 127)[..., None]
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.minimum(np.where(np.isfinite(v), np.abs(v), 0) / unit, 1e6)
    hi = np.clip(np.searchsorted(MAGNITUDES, a), 1, 126)
    dl, dh = a - MAGNITUDES[hi - 1], MAGNITUDES[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, hi - 1).astype(np.uint8)
    code |= np.signbit(v).astype(np.uint8) << 7
    code[scale == 255] = 127
    return code.reshape(R, K), scale.astype(np.uint8)


def values_ref(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """fp64 values [R, K] of a microscaled 8-bit pair."""
    table = np.append(MAGNITUDES, np.nan)
    v = table[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    unit = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(unit, 32, axis=1)


def product_ref(codes, scale, w_packed, w_scale) -> np.ndarray:
    """fp64 A [M, K] times W [N, K] transposed."""
    return values_ref(codes, scale) @ mx4.values_ref(w_packed, w_scale).T


def norm_ref(x, residual, gamma, eps):
    """(v, y) of the norm in long double; None for an absent residual or gamma."""
    v = np.asarray(x, dtype=np.longdouble)
    if residual is not None:
        v = v + np.asarray(residual, dtype=np.longdouble)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = v / np.sqrt((v * v).mean(-1, keepdims=True) + np.longdouble(eps))
        if gamma is not None:
            y = y * np.asarray(gamma, dtype=np.longdouble)
    return v, y
