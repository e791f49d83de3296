"""GPU parity of the microscaled calls in their rarer variants: every product tile
with both output types and with every way in which K can end, 16-bit inputs over
their whole range, and more elements than one pass over the grid covers."""

import numpy as np
import pytest
import torch

from oracle import mx4

pytestmark = pytest.mark.gpu


def matrix(g, rows, K, scale):
    r = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return r(rows, K // 2), r(rows, K // 32) % 2 + scale


# 256-row tiles: from 256 tiles of 256 x 256; 128-row tiles: from 256 of 128 x 128 where those are fewer; else 64.
# K in whole 512 columns (one to four groups of scales), and ending in one to four more steps of 128.
TILES = {256: (4000, 4200), 128: (2000, 2100), 64: (300, 500)}


@pytest.mark.parametrize("side", sorted(TILES))
@pytest.mark.parametrize("K", [512, 1024, 1536, 2048, 32, 128, 256, 384, 480, 640, 768, 896, 992, 1504])
def test_every_tile_and_end_of_k(k3, side, K):
    """Scale bytes of two neighbouring values on either side and K <= 29127: every partial sum is exact in fp32, in
    any order, so both outputs are compared for equality (bf16: one rounding of the exact sum)."""
    M, N = TILES[side]
    g = torch.Generator(device="cuda").manual_seed(side + K)
    a, w = matrix(g, M, K, 126), matrix(g, N, K, 127)
    want = k3.mxfp4_unpack(*a).double() @ k3.mxfp4_unpack(*w).double().t().contiguous()
    assert torch.equal(k3.mxfp4_matmul(*a, *w), want.float())
    assert torch.equal(k3.mxfp4_matmul(*a, *w, out_dtype=torch.bfloat16), want.float().bfloat16())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("saturate", [True, False])
def test_quantize_every_16_bit_value(k3, dtype, saturate):
    """Each finite value of the type as a block's largest, beside its halves and neighbours of both signs (subnormals
    among them), and each finite value beside the largest of its binade and the two above."""
    bits = np.arange(1 << 15, dtype=np.uint16)
    top = bits[(bits >> 7) < 255] if dtype == torch.bfloat16 else bits[(bits >> 10) < 31]
    step = np.uint16(1 << (7 if dtype == torch.bfloat16 else 10))
    most = top.max()
    blocks = np.zeros((2 * len(top), 32), np.uint16)
    own, other = blocks[: len(top)], blocks[len(top):]
    for i in range(32):  # the value, then down by quarters of a binade, signs by turns
        own[:, i] = np.maximum(top.astype(np.int64) - i * int(step) // 4, 0).astype(np.uint16) | (0x8000 if i % 2 else 0)
    for i in range(32):  # neighbours of the value under a larger top
        other[:, i] = np.clip(top.astype(np.int64) + i - 16, 0, int(most)).astype(np.uint16) | (0x8000 if i % 3 == 0 else 0)
    other[:, 0] = np.minimum((top | (step - 1)).astype(np.int64) + int(step) * (np.arange(len(top)) % 3), int(most)).astype(np.uint16)
    x = torch.from_numpy(blocks.view(np.int16)).view(dtype)
    ref_p, ref_s = mx4.quantize_ref(x.double().numpy(), saturate)
    p, s = k3.mxfp4_quantize(x.cuda(), saturate=saturate)
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(p.cpu().numpy(), ref_p)


@pytest.mark.slow
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_than_2_to_32_elements(k3, dtype):
    """Offsets beyond 32 bits, and more elements than a pass of the largest grid (2^32): the rows repeat, so do the codes."""
    K, period = 1024, 4096
    R = (2**32 + 2**25) // K + 1
    g = torch.Generator(device="cuda").manual_seed(5)
    base = torch.randn((period, K), generator=g, device="cuda").to(dtype)
    x = torch.empty((R, K), dtype=dtype, device="cuda")
    for r in range(0, R, period):
        x[r: r + period] = base[: min(period, R - r)]
    p, s = k3.mxfp4_quantize(x)
    bp, bs = k3.mxfp4_quantize(base)
    v = k3.mxfp4_unpack(bp, bs, dtype)
    del x
    out = k3.mxfp4_unpack(p, s, dtype)
    for r in range(0, R, period):
        n = min(period, R - r)
        assert torch.equal(p[r: r + n], bp[:n]) and torch.equal(s[r: r + n], bs[:n]) and torch.equal(out[r: r + n], v[:n]), r
    del p, s, out
    torch.cuda.empty_cache()
