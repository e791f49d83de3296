"""GPU parity of the microscaled 8-bit calls (quantise, unpack, norm, product) against the oracle.

Rounding is exact, so codes and scales are compared bit for bit, the norm's too: its fp64 arithmetic (relative error
about 1e-15) moves no random value across a border.  Products are compared for equality where every partial sum is
exact in fp32, and else with the bound of an fp32 sum of the products.
"""

import numpy as np
import pytest
import torch

from oracle import mx4, mx8
from tests.gpu_util import to_dev_u8

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def assert_quantized(k3, x, saturate, what):
    ref_c, ref_s = mx8.quantize_ref(x.double().numpy(), saturate)
    c, s = k3.mxfp8_quantize(x.cuda(), saturate=saturate)
    assert np.array_equal(s.cpu().numpy(), ref_s), what
    assert np.array_equal(c.cpu().numpy(), ref_c), what


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("saturate", [True, False])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (1, 7168), (5, 1056), (257, 96), (1000, 32)])
def test_quantize(k3, dtype, saturate, R, K):
    g = torch.Generator().manual_seed(R * K + saturate)
    x = torch.randn((R, K), generator=g) * torch.exp2(torch.randint(-9, 9, (R, 1), generator=g).float())
    assert_quantized(k3, x.to(TORCH[dtype]), saturate, (dtype, R, K))


@pytest.mark.parametrize("saturate", [True, False])
def test_quantize_every_exponent(k3, saturate):
    """Block maxima of every fp32 exponent, at, just below and just above the mantissa of 1.75, and what lies below them."""
    rows = []
    for E in range(255):
        for mant in (0, 1, 0x5FFFFF, 0x600000, 0x600001, 0x67FFFF, 0x680000, 0x7FFFFF):
            b = np.zeros(32, np.uint32)
            b[7] = np.uint32(E << 23 | mant)
            for i in range(1, 12):
                if E - i > 0:
                    b[8 + 2 * i] = np.uint32((E - i) << 23 | mant)
                    b[9 + 2 * i] = np.uint32((E - i) << 23 | 0x700000) | np.uint32(1 << 31)
            rows.append(b)
    assert_quantized(k3, torch.from_numpy(np.stack(rows).view(np.float32)), saturate, "exponents")


def test_quantize_ties_and_signs(k3):
    """Every midpoint between two magnitudes, both signs, with neighbours on both sides."""
    m = mx8.MAGNITUDES
    mid = np.float32((m[1:] + m[:-1]) / 2)
    v = np.concatenate([mid, np.nextafter(mid, np.float32(999)), np.nextafter(mid, np.float32(0)), np.float32(m), np.float32([0.0, 2.0**-30])])
    v = np.concatenate([v, -v])
    n = -(-len(v) // 31)
    x = np.full((n, 32), 448.0, np.float32)  # 448 in every block: scale 2^0
    x[:, 1:] = np.resize(v, n * 31).reshape(n, 31)
    assert_quantized(k3, torch.from_numpy(x), True, "ties")


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_nonfinite(k3, bad, dtype):
    x = torch.ones((2, 128))
    x[0, 37], x[1, 127] = bad, bad
    c, s = k3.mxfp8_quantize(x.to(TORCH[dtype]).cuda())
    assert s.tolist() == [[119, 255, 119, 119], [119, 119, 119, 255]]
    assert set(c[0, 32:64].tolist()) == {127} and set(c[1, 96:].tolist()) == {127} and set(c[0, :32].tolist()) == {0x78}
    v = k3.mxfp8_unpack(c, s)
    assert torch.isnan(v[0, 32:64]).all() and torch.isnan(v[1, 96:]).all() and int(torch.isnan(v).sum()) == 64


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_unpack_every_code_and_scale(k3, out):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scale = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, axis=1)
    ref = torch.from_numpy(mx8.values_ref(codes, scale)).float().to(TORCH[out])
    got = k3.mxfp8_unpack(to_dev_u8(codes), to_dev_u8(scale), TORCH[out]).cpu()
    nan = torch.isnan(ref)
    assert torch.equal(nan, torch.isnan(got))
    it = torch.int32 if out == "f32" else torch.int16
    assert torch.equal(ref[~nan].view(it), got[~nan].view(it))  # bits: signs of zeros, subnormals, infinities


def test_leading_dims_and_buffers(k3):
    x = torch.randn((2, 3, 4, 64), device="cuda")
    c, s = k3.mxfp8_quantize(x)
    assert c.shape == x.shape and s.shape == (2, 3, 4, 2)
    c2, s2 = torch.empty_like(c), torch.empty_like(s)
    r = k3.mxfp8_quantize(x, codes=c2, scale=s2)
    assert r[0] is c2 and torch.equal(c, c2) and torch.equal(s, s2)
    e = k3.mxfp8_quantize(x[:0].contiguous())
    assert e[0].shape == (0, 3, 4, 64) and k3.mxfp8_unpack(*e).shape == (0, 3, 4, 64)
    n = k3.mxfp8_rms_norm(x, residual=x, normed=True)
    assert all(t.shape[:3] == (2, 3, 4) for t in n)


def assert_norm(k3, x, gamma, residual, eps, saturate, what):
    n64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    v, y = mx8.norm_ref(n64(x), n64(residual), n64(gamma), eps)
    ref_c, ref_s = mx8.quantize_ref(y, saturate)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    c, s, total, ny = k3.mxfp8_rms_norm(dev(x), dev(gamma), dev(residual), eps=eps, saturate=saturate, normed=True)
    assert np.array_equal(s.cpu().numpy(), ref_s), what
    assert np.array_equal(c.cpu().numpy(), ref_c), what
    # rounded once: half a step of the type (of its subnormals near zero; the fp64 value's own error is far below)
    for got, ref in ((ny, y), (total, v)):
        if got is None:
            continue
        f = torch.finfo(x.dtype)
        tiny = float(f.tiny) * float(f.eps)
        err = np.abs(got.cpu().double().numpy() - ref.astype(np.float64))
        assert (err <= np.maximum(np.abs(ref.astype(np.float64)) * (f.eps / 2), tiny / 2) * (1 + 1e-6)).all(), what
    return c, s, total, ny


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,K", [(1, 32), (2, 64), (7, 480), (3, 512), (5, 544), (1, 7168), (33, 4128), (300, 96), (2, 8192), (2, 16416), (1, 70016)])
def test_norm(k3, dtype, R, K):
    g = torch.Generator().manual_seed(R + K)
    t = TORCH[dtype]
    x = torch.randn((R, K), generator=g).to(t)
    r = (3 * torch.randn((R, K), generator=g)).to(t)
    gamma = (1 + 0.3 * torch.randn((K,), generator=g)).to(t)
    assert_norm(k3, x, gamma, r, 1e-5, True, (dtype, R, K))


@pytest.mark.parametrize("gamma_type", ["f32", "bf16", "f16", None])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("res", [False, True])
def test_norm_variants(k3, gamma_type, dtype, res):
    g = torch.Generator().manual_seed(5)
    K = 1504
    x = torch.randn((4, K), generator=g).to(TORCH[dtype])
    r = torch.randn((4, K), generator=g).to(TORCH[dtype]) if res else None
    gamma = None if gamma_type is None else torch.randn((K,), generator=g).to(TORCH[gamma_type])
    assert_norm(k3, x, gamma, r, 0.0, False, (gamma_type, dtype, res))


def test_norm_wide_range(k3):
    """Channels far above the rest, rows of tiny and of huge values, blocks of zeros."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn((6, 1024), generator=g)
    x[0, 17] = 3e4
    x[1] *= 1e-30
    x[2] *= 1e30
    x[3, 64:128] = 0.0
    x[4] = 0.0
    x[5, ::2] *= 2.0**-60
    assert_norm(k3, x, None, None, 1e-6, True, "f32")
    assert_norm(k3, x[[0, 3, 4]].bfloat16(), torch.full((1024,), 1e3), x[[3, 0, 5]].bfloat16(), 1e-6, False, "bf16")


def test_norm_nonfinite_rows_stay_alone(k3):
    x = torch.randn((4, 256))
    x[1, 40], x[2, 40] = float("nan"), float("inf")
    c, s, _, y = k3.mxfp8_rms_norm(x.cuda(), normed=True)
    rc, rs = mx8.quantize_ref(mx8.norm_ref(x.double().numpy(), None, None, 1e-5)[1])
    assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)
    assert torch.isnan(y[1]).all() and int(torch.isnan(y[2]).sum()) == 1 and not torch.isnan(y[[0, 3]]).any()
    c, s, _, y = k3.mxfp8_rms_norm(torch.zeros((1, 64), device="cuda"), eps=0.0, normed=True)  # 0 / 0
    assert torch.isnan(y).all() and s.tolist() == [[255, 255]]


@pytest.mark.parametrize("K", [64, 2080, 70016])
def test_norm_in_place(k3, K):
    x, r = torch.randn((3, K), device="cuda").bfloat16(), torch.randn((3, K), device="cuda").bfloat16()
    want = k3.mxfp8_rms_norm(x, residual=r, normed=True)
    for target in ("x", "residual"):
        x2, r2 = x.clone(), r.clone()
        got = k3.mxfp8_rms_norm(x2, residual=r2, normed=True, total=x2 if target == "x" else r2)
        for a, b in zip(got, want):
            assert torch.equal(a, b), target
        assert torch.equal(r2 if target == "x" else x2, r if target == "x" else x)


def test_norm_feeds_what_quantize_gives(k3):
    """Codes only, y only and both agree; the codes are those of the unrounded y (quantize of an f32 y differs at most where y's rounding crossed a border)."""
    x, g = torch.randn((9, 512), device="cuda"), torch.rand((512,), device="cuda")
    c, s, total, y = k3.mxfp8_rms_norm(x, g)
    assert total is None and y is None
    c2, s2, _, y = k3.mxfp8_rms_norm(x, g, normed=True)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    c3, _ = k3.mxfp8_quantize(y)
    assert (c3.int() - c.int()).abs().max() <= 1 and (c3 != c).float().mean() < 1e-3


# ---------------------------------------------------------------------------
# products

SHAPES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (3, 33, 512), (16, 64, 544), (7, 100, 4128), (16, 1003, 1024), (5, 2000, 8192),
          (1, 5000, 3584), (17, 1, 32), (17, 64, 128), (31, 65, 160), (64, 64, 480), (65, 130, 512), (77, 1003, 1056),
          (130, 257, 1504), (128, 512, 2048), (33, 7, 2080), (300, 300, 96), (16, 40, 16384), (3, 20, 100000), (2, 300, 163840)]


def rows8(g, M, K, lo, hi, e0, e1):
    """Codes with exponent fields lo .. hi, signs, and scale bytes e0 .. e1."""
    c = (g.integers(lo, hi + 1, (M, K)) << 3 | g.integers(0, 8, (M, K)) | g.integers(0, 2, (M, K)) << 7).astype(np.uint8)
    return c, g.integers(e0, e1 + 1, (M, K // 32), dtype=np.uint8)


def weights4(g, N, K, e0, e1):
    return g.integers(0, 256, (N, K // 2), dtype=np.uint8), g.integers(e0, e1 + 1, (N, K // 32), dtype=np.uint8)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_exact(k3, M, N, K):
    """Magnitudes 0.5 .. 3.75, so on both sides of 2: products are multiples of 2^-6 up to 11.25 (720 units), scales of
    one value; sums up to 720 K units stay within 2^24 for K <= 23301, and for longer K codes are thinned out."""
    g = np.random.default_rng([M, N, K])
    (ac, as_), (wp, ws) = rows8(g, M, K, 6, 8, 127, 127), weights4(g, N, K, 126, 126)
    if K > 23301:
        ac[g.random((M, K)) < 1 - 20000 / K] = 0
    a = mx8.values_ref(ac, as_)
    assert np.abs(a).sum(1).max() * 3 * 2**6 <= 2**24
    ref = torch.from_numpy(a @ mx4.values_ref(wp, ws).T).float()
    dev = [to_dev_u8(t) for t in (ac, as_, wp, ws)]
    assert torch.equal(k3.mxfp8_matmul(*dev).cpu(), ref)
    assert torch.equal(k3.mxfp8_matmul(*dev, out_dtype=torch.bfloat16).cpu(), ref.bfloat16())


@pytest.mark.parametrize("M,N,K", [(4096, 4224, 512), (2100, 8300, 544), (1100, 4100, 1024), (4200, 4097, 96), (2048, 2048, 1600)])
def test_matmul_large_tiles_exact(k3, M, N, K):
    """The largest tiles, ragged at every edge; the reference is a double product on the device."""
    g = np.random.default_rng([M, N, K])
    ac, as_, wp, ws = [to_dev_u8(t) for p in (rows8(g, M, K, 6, 8, 126, 127), weights4(g, N, K, 126, 127)) for t in p]
    ref = k3.mxfp8_unpack(ac, as_).double() @ k3.mxfp4_unpack(wp, ws).double().t()
    assert torch.equal(k3.mxfp8_matmul(ac, as_, wp, ws).double(), ref)


@pytest.mark.parametrize("M,N,K", [(64, 7200, 2048), (31, 9000, 1504), (97, 3000, 2560), (17, 20001, 1056), (32, 16448, 3584),
                                   (150, 4200, 2080), (130, 3500, 2048), (150, 7000, 2080), (160, 6400, 2048), (1000, 2000, 544),
                                   (1000, 2000, 512), (640, 1600, 2560), (1900, 2040, 1536), (1920, 2048, 1056), (1920, 2048, 3584),
                                   (1037, 7000, 1024), (2048, 7168, 512), (2047, 7100, 1536), (500, 800, 32),
                                   (1530, 7160, 1024), (1900, 6100, 1056), (2300, 4800, 2080), (3900, 4090, 1024), (4096, 3584, 512),
                                   (1000, 10000, 1536)])
def test_matmul_tile_sides_exact(k3, M, N, K):
    """One and several tiles of 32 x 64, of 64 and of 128 a CU and one of 256, whole and ragged, of whole and ragged groups of scales."""
    g = np.random.default_rng([3, M, N, K])
    ac, as_, wp, ws = [to_dev_u8(t) for p in (rows8(g, M, K, 6, 8, 126, 127), weights4(g, N, K, 126, 127)) for t in p]
    ref = k3.mxfp8_unpack(ac, as_).double() @ k3.mxfp4_unpack(wp, ws).double().t()
    assert torch.equal(k3.mxfp8_matmul(ac, as_, wp, ws).double(), ref)
    assert torch.equal(k3.mxfp8_matmul(ac, as_, wp, ws, torch.bfloat16), ref.float().bfloat16())


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_matmul_keeps_small_elements_beside_large_ones(k3, M):
    """Blocks of one 448 and 31 elements down to 2^-9: the sum is a multiple of 2^-10 below 2^14 (two blocks of K), so exact in fp32."""
    g = np.random.default_rng(M)
    N, K = 300, 64
    ac, as_ = rows8(g, M, K, 0, 3, 127, 127)
    ac[:, 3], ac[:, 40] = 0x7E, 0xFE  # 448, -448
    wp, ws = weights4(g, N, K, 127, 127)
    ref = torch.from_numpy(mx8.product_ref(ac, as_, wp, ws)).float()
    assert torch.equal(k3.mxfp8_matmul(*[to_dev_u8(t) for t in (ac, as_, wp, ws)]).cpu(), ref)


@pytest.mark.parametrize("M,N,K", [(1, 500, 7168), (12, 333, 4128), (16, 100, 9600), (70, 200, 1056), (200, 400, 2048), (1100, 4100, 1024)])
def test_matmul_full_range(k3, M, N, K):
    """Every code and scales apart: an fp32 sum of two parts per block, each addition off by at most 2^-23 (whether it rounds or
    truncates) of the sum of magnitudes."""
    g = np.random.default_rng([7, M, N, K])
    (ac, as_), (wp, ws) = rows8(g, M, K, 0, 15, 110, 130), weights4(g, N, K, 100, 130)
    ac[(ac & 127) == 127] = 0
    a, w = mx8.values_ref(ac, as_), mx4.values_ref(wp, ws)
    got = k3.mxfp8_matmul(*[to_dev_u8(t) for t in (ac, as_, wp, ws)]).cpu().double().numpy()
    bound = (2 * K // 32 + 16) * 2.0**-23 * (np.abs(a) @ np.abs(w).T)
    assert (np.abs(got - a @ w.T) <= bound).all()


@pytest.mark.parametrize("M", [3, 100, 1100])
def test_matmul_nan_stays_in_its_row_and_column(k3, M):
    g = np.random.default_rng(M)
    N, K = 4100 if M > 1000 else 50, 544
    (ac, as_), (wp, ws) = rows8(g, M, K, 6, 8, 127, 127), weights4(g, N, K, 126, 126)
    ac[1, 70] = 0xFF
    as_[2, 16] = 255
    ws[5, 3] = 255
    out = k3.mxfp8_matmul(*[to_dev_u8(t) for t in (ac, as_, wp, ws)]).cpu()
    nan = torch.zeros((M, N), dtype=torch.bool)
    nan[1:3] = True
    nan[:, 5] = True
    assert torch.equal(torch.isnan(out), nan)


@pytest.mark.parametrize("M,N,K", [(9, 300, 4096), (40, 300, 1024), (60, 7000, 1024), (150, 4200, 2048), (1000, 2000, 512),
                                   (1900, 2040, 1536), (1530, 7160, 1024), (2048, 7168, 512), (3900, 4090, 1024)])
def test_matmul_nan_beside_whole_groups_of_scales(k3, M, N, K):
    """A NaN code, a NaN scale of A and one of W: their rows and column, and nothing else."""
    g = np.random.default_rng([5, M, N, K])
    ac, as_, wp, ws = [to_dev_u8(t) for p in (rows8(g, M, K, 6, 8, 126, 127), weights4(g, N, K, 126, 127)) for t in p]
    ref = k3.mxfp8_matmul(ac, as_, wp, ws)
    ac[M // 2, K - 1], as_[M - 1, 0], ws[N - 2, K // 32 - 1] = 127, 255, 255
    ref[M // 2], ref[M - 1], ref[:, N - 2] = (float("nan"),) * 3
    assert torch.equal(torch.nan_to_num(k3.mxfp8_matmul(ac, as_, wp, ws), nan=1e30), torch.nan_to_num(ref, nan=1e30))


def test_matmul_matches_linear_by_four_bits(k3):
    """Rows that hold E2M1 values: the 8-bit product gives what the 4-bit one gives."""
    g = np.random.default_rng(3)
    M, N, K = 9, 200, 1024
    wp, ws = weights4(g, N, K, 125, 126)
    ap, as_ = weights4(g, M, K, 126, 126)
    v = k3.mxfp4_unpack(to_dev_u8(ap), to_dev_u8(as_))
    c, s = k3.mxfp8_quantize(v)
    assert torch.equal(k3.mxfp8_unpack(c, s), v)
    w = (to_dev_u8(wp), to_dev_u8(ws))
    assert torch.equal(k3.mxfp8_matmul(c, s, *w), k3.mxfp4_matmul(to_dev_u8(ap), to_dev_u8(as_), *w))


def test_empty_products(k3):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    assert k3.mxfp8_matmul(u8(0, 64), u8(0, 2), u8(5, 32), u8(5, 2)).shape == (0, 5)
    assert k3.mxfp8_matmul(u8(5, 64), u8(5, 2), u8(0, 32), u8(0, 2)).shape == (5, 0)


def test_streams_and_graph(k3):
    """Norm and product captured together and replayed on new inputs, with eager work between."""
    g = np.random.default_rng(11)
    x = torch.randn((5, 1024), device="cuda").bfloat16()
    w = [to_dev_u8(t) for t in weights4(g, 333, 1024, 120, 122)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    k3.mxfp8_matmul(*k3.mxfp8_rms_norm(x)[:2], *w)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c, s, _, y = k3.mxfp8_rms_norm(x, residual=x, normed=True)
        out = k3.mxfp8_matmul(c, s, *w)
    for rep in range(3):
        x.copy_(torch.randn((5, 1024), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ec, es, _, ey = k3.mxfp8_rms_norm(x, residual=x, normed=True)
        assert torch.equal(y, ey) and torch.equal(out, k3.mxfp8_matmul(ec, es, *w)), rep
