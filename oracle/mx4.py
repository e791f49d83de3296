"""fp64 oracle of microscaled 4-bit quantisation and products.

Written from the definitions (OCP Microscaling Formats specification 1.0: one
E8M0 scale per 32 elements, shared exponent floor(log2(max |v|)) less the
element type's largest exponent, E2M1 elements rounded to nearest even and
clamped); shares no code with the GPU path.
"""

from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def block_scale_byte(top: float, saturate: bool) -> int:
    """E8M0 byte of a block whose largest magnitude is `top`."""
    if not np.isfinite(top):
        return 255
    if top == 0.0:
        return 0
    _, ex = np.frexp(np.float64(top))  # top = f * 2^ex, 0.5 <= f < 1
    e = max(int(ex) - 1 - 2, -127)
    if not saturate and top > 6.0 * 2.0**e:
        e += 1
    return e + 127


def nearest_code(a: float) -> int:
    """Magnitude code of a >= 0: the nearest magnitude, ties to the even code."""
    d = np.abs(MAGNITUDES - a)
    best = np.flatnonzero(d == d.min())
    return int(best[0]) if len(best) == 1 else int([c for c in best if c % 2 == 0][0])


def quantize_ref(x: np.ndarray, saturate: bool = True):
    """x [R, K] (any float values) -> (packed u8 [R, K/2], scale u8 [R, K/32])."""
    v = np.asarray(x, dtype=np.float64)
    R, K = v.shape
    v = v.reshape(R, K // 32, 32)
    top = np.abs(v).max(-1) if v.size else np.zeros((R, K // 32))
    top = np.where(np.isnan(v).any(-1), np.nan, top)
    scale = np.array([block_scale_byte(t, saturate) for t in top.ravel()], dtype=np.uint8).reshape(R, K // 32)
    unit = np.ldexp(1.0, scale.astype(np.int64) - 127)[..., None]
    with np.errstate(invalid="ignore"):
        a = np.abs(v) / unit
    # distance to every magnitude; ties resolved by a second key that prefers even codes
    d = np.abs(a[..., None] - MAGNITUDES)
    near = d == np.nanmin(np.where(np.isnan(d), np.inf, d), axis=-1, keepdims=True)
    key = np.where(near, np.arange(8) % 2, 2)
    code = key.argmin(-1).astype(np.uint8)
    code = code | (np.signbit(v).astype(np.uint8) << 3)
    code[scale == 255] = 7
    code = code.reshape(R, K)
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8), scale


def values_ref(packed: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """fp64 values [R, K] of a microscaled pair; NaN where the scale byte is 255."""
    R, half = packed.shape
    code = np.empty((R, 2 * half), dtype=np.uint8)
    code[:, 0::2] = packed & 15
    code[:, 1::2] = packed >> 4
    v = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    unit = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(unit, 32, axis=1)


def product_ref(a_packed, a_scale, w_packed, w_scale) -> np.ndarray:
    """fp64 A [M, K] times W [N, K] transposed."""
    return values_ref(a_packed, a_scale) @ values_ref(w_packed, w_scale).T
