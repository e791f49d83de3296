"""GPU parity of the microscaled 4-bit calls (quantise, unpack, matmul, linear)
against the fp64 oracle.

Quantisation and decode are exact, so they are compared bit for bit.  Products
are compared for equality wherever every partial sum is exact in fp32: with
scale bytes of two neighbouring values on each side, products are multiples of
2^-2 * 2^(smallest scales) and bounded by 36 * 2^2 of that unit's scales, so K *
36 * 4 * 4 <= 2^24, that is K <= 29127, makes every partial sum exact in any order.
"""

import numpy as np
import pytest
import torch

from oracle import mx4
from tests.gpu_util import to_dev_u8

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def pair(g, R, K, lo, hi):
    """Random microscaled matrix on the host."""
    return g.integers(0, 256, (R, K // 2), dtype=np.uint8), g.integers(lo, hi + 1, (R, K // 32), dtype=np.uint8)


def gpu_quantize(k3, x, saturate):
    p, s = k3.mxfp4_quantize(x, saturate=saturate)
    return p.cpu().numpy(), s.cpu().numpy()


def assert_quantized(k3, x, saturate, what):
    ref_p, ref_s = mx4.quantize_ref(x.double().numpy(), saturate)
    p, s = gpu_quantize(k3, x.cuda(), saturate)
    assert np.array_equal(s, ref_s), what
    assert np.array_equal(p, ref_p), what


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("saturate", [True, False])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (1, 7168), (5, 1056), (257, 96), (1000, 32)])
def test_quantize(k3, dtype, saturate, R, K):
    g = torch.Generator().manual_seed(R * K + saturate)
    x = torch.randn((R, K), generator=g) * torch.exp2(torch.randint(-9, 9, (R, 1), generator=g).float())
    assert_quantized(k3, x.to(TORCH[dtype]), saturate, (dtype, R, K))


@pytest.mark.parametrize("saturate", [True, False])
def test_quantize_every_exponent(k3, saturate):
    """Block maxima of every fp32 exponent (subnormals too), at, just below and just above the mantissa of 1.5."""
    rows = []
    for E in range(255):
        for mant in (0, 1, 0x3FFFFF, 0x400000, 0x400001, 0x7FFFFF):
            top = np.uint32(E << 23 | mant)
            b = np.zeros(32, np.uint32)
            b[7] = top
            for i, sh in enumerate(range(1, 9)):  # values one binade apart, down from the top, with both signs
                if E - sh > 0:
                    b[8 + 2 * i] = np.uint32((E - sh) << 23 | mant)
                    b[9 + 2 * i] = np.uint32((E - sh) << 23 | 0x400000) | np.uint32(1 << 31)
            rows.append(b)
    x = torch.from_numpy(np.stack(rows).view(np.float32))
    assert_quantized(k3, x, saturate, "exponents")


def test_quantize_ties_and_signs(k3):
    """Every quarter step of the E2M1 range, both signs, with neighbours on both sides of each tie."""
    base = np.arange(0, 33, dtype=np.float32) / 4
    v = np.unique(np.concatenate([base, np.nextafter(base, np.float32(9)), np.nextafter(base, np.float32(-9))]))
    v = np.concatenate([v, -v, np.float32([0.0, -0.0])]).astype(np.float32)
    v = v[np.abs(v) < 8]
    n = -(-len(v) // 31)
    x = np.full((n, 32), 7.0, np.float32)  # 7 in every block: scale 2^0
    x[:, 1:].ravel()[:0] = 0
    flat = np.resize(v, n * 31).reshape(n, 31)
    x[:, 1:] = flat
    assert_quantized(k3, torch.from_numpy(x), True, "ties")


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_nonfinite(k3, bad, dtype):
    x = torch.ones((2, 128))
    x[0, 37], x[1, 127] = bad, bad
    p, s = gpu_quantize(k3, x.to(TORCH[dtype]).cuda(), True)
    assert s.tolist() == [[125, 255, 125, 125], [125, 125, 125, 255]]
    assert set(p[0, 16:32].tolist()) == {0x77} and set(p[1, 48:].tolist()) == {0x77} and set(p[0, :16].tolist()) == {0x66}
    v = k3.mxfp4_unpack(to_dev_u8(p), to_dev_u8(s)).cpu()
    assert torch.isnan(v[0, 32:64]).all() and torch.isnan(v[1, 96:]).all() and int(torch.isnan(v).sum()) == 64
    # through the 17-byte blocks the same elements are infinite, none is a plain number
    b = k3.mxfp4_dequant(k3.mxfp4_repack(to_dev_u8(p), to_dev_u8(s))).cpu()
    assert torch.isinf(b[0, 32:64]).all() and torch.isinf(b[1, 96:]).all() and int(torch.isinf(b).sum()) == 64


def test_quantize_leading_dims_and_buffers(k3):
    x = torch.randn((2, 3, 4, 64), device="cuda")
    p, s = k3.mxfp4_quantize(x)
    assert p.shape == (2, 3, 4, 32) and s.shape == (2, 3, 4, 2)
    p2, s2 = torch.empty_like(p), torch.empty_like(s)
    r = k3.mxfp4_quantize(x.reshape(-1, 64), packed=p2.view(-1, 32), scale=s2.view(-1, 2))
    assert r[0].data_ptr() == p2.data_ptr() and torch.equal(p, p2) and torch.equal(s, s2)
    e = k3.mxfp4_quantize(x[:0].contiguous())
    assert e[0].shape == (0, 3, 4, 32) and k3.mxfp4_unpack(*e).shape == (0, 3, 4, 64)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_unpack_every_code_and_scale(k3, out):
    packed = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scale = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    ref = torch.from_numpy(mx4.values_ref(packed, scale)).float().to(TORCH[out])  # exact but for overflow to inf
    got = k3.mxfp4_unpack(to_dev_u8(packed), to_dev_u8(scale), TORCH[out]).cpu()
    nan = torch.isnan(ref)
    assert torch.equal(nan, torch.isnan(got)) and int(nan.sum()) == 512
    it = torch.int32 if out == "f32" else torch.int16
    assert torch.equal(ref[~nan].view(it), got[~nan].view(it))  # bits: signs of zeros, subnormals, infinities


def test_round_trip_feeds_the_expert_layout(k3):
    """quantise -> repack -> dequant gives the values unpack gives."""
    x = torch.randn((48, 1024), device="cuda")
    p, s = k3.mxfp4_quantize(x, saturate=False)
    assert torch.equal(k3.mxfp4_dequant(k3.mxfp4_repack(p, s)), k3.mxfp4_unpack(p, s) + 0.0)


SHAPES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (3, 33, 512), (16, 64, 544), (7, 100, 4128), (16, 1003, 1024), (5, 2000, 8192),
          (1, 5000, 3584), (17, 1, 32), (17, 64, 128), (31, 65, 160), (64, 64, 480), (65, 130, 512), (77, 1003, 1056),
          (130, 257, 1504), (128, 512, 2048), (33, 7, 2080), (300, 300, 96)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_exact(k3, M, N, K):
    g = np.random.default_rng([M, N, K])
    (ap, as_), (wp, ws) = pair(g, M, K, 126, 127), pair(g, N, K, 127, 128)
    ref = torch.from_numpy(mx4.product_ref(ap, as_, wp, ws)).float()
    dev = [to_dev_u8(t) for t in (ap, as_, wp, ws)]
    assert torch.equal(k3.mxfp4_matmul(*dev).cpu(), ref)
    assert torch.equal(k3.mxfp4_matmul(*dev, out_dtype=torch.bfloat16).cpu(), ref.bfloat16())


@pytest.mark.parametrize("M,N,K", [(4096, 4224, 512), (2100, 8300, 544), (1100, 4100, 1024), (4200, 4097, 96)])
def test_matmul_large_tiles_exact(k3, M, N, K):
    """The largest tiles, ragged at every edge; the reference is a double product on the device."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    rnd = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    ap, wp = rnd(M, K // 2), rnd(N, K // 2)
    as_, ws = rnd(M, K // 32) % 2 + 126, rnd(N, K // 32) % 2 + 127
    ref = k3.mxfp4_unpack(ap, as_).double() @ k3.mxfp4_unpack(wp, ws).double().t()
    assert torch.equal(k3.mxfp4_matmul(ap, as_, wp, ws).double(), ref)


@pytest.mark.parametrize("M,N,K", [(4, 40, 7168), (16, 50, 1056), (40, 40, 7168), (200, 130, 1056)])
def test_matmul_wide_scales(k3, M, N, K):
    """Scales over 60 binades: fp32 sums of K products are off by at most K roundings of the sum of magnitudes
    (2^-24 each); results below the smallest normal number are not reached."""
    g = np.random.default_rng([M, N, K, 1])
    (ap, as_), (wp, ws) = pair(g, M, K, 97, 157), pair(g, N, K, 97, 157)
    a, w = mx4.values_ref(ap, as_), mx4.values_ref(wp, ws)
    got = k3.mxfp4_matmul(*[to_dev_u8(t) for t in (ap, as_, wp, ws)]).cpu().double().numpy()
    assert np.all(np.abs(got - a @ w.T) <= K * 2.0**-24 * (np.abs(a) @ np.abs(w).T))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_matmul_nan_scale_stays_in_its_row_and_column(k3, M):
    g = np.random.default_rng(M)
    N, K = 150, 672
    (ap, as_), (wp, ws) = pair(g, M, K, 126, 127), pair(g, N, K, 127, 128)
    ref = torch.from_numpy(mx4.product_ref(ap, as_, wp, ws)).float()
    as_[M - 1, 20], ws[5, 0] = 255, 255
    got = k3.mxfp4_matmul(*[to_dev_u8(t) for t in (ap, as_, wp, ws)]).cpu()
    nan = torch.zeros((M, N), dtype=torch.bool)
    nan[M - 1], nan[:, 5] = True, True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], ref[~nan])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 7168), (8, 333, 1056), (16, 64, 32), (17, 100, 4128), (16, 20, 8192), (200, 300, 544)])
@pytest.mark.parametrize("saturate", [True, False])
def test_linear_is_quantize_then_matmul(k3, dtype, M, N, K, saturate):
    g = np.random.default_rng([M, N, K, 2])
    wp, ws = (to_dev_u8(t) for t in pair(g, N, K, 120, 124))
    x = torch.from_numpy(g.standard_normal((M, K))).to(TORCH[dtype]).cuda()
    p, s = k3.mxfp4_quantize(x, saturate=saturate)
    for out in (torch.float32, torch.bfloat16):
        want = k3.mxfp4_matmul(p, s, wp, ws, out_dtype=out)
        ws_bytes = k3.mxfp4_linear_workspace_size(M, N, K)
        work = torch.full((max(ws_bytes, 1),), 255, dtype=torch.uint8, device="cuda")
        got = k3.mxfp4_linear(x, wp, ws, saturate=saturate, out_dtype=out, workspace=work)
        assert torch.equal(got, want)


def test_outputs_stay_inside(k3):
    """Rows behind the outputs keep what they held."""
    g = np.random.default_rng(9)
    for M, N, K in ((3, 50, 96), (70, 70, 160)):
        dev = [to_dev_u8(t) for p in (pair(g, M, K, 126, 127), pair(g, N, K, 127, 128)) for t in p]
        buf = torch.full((M * N + 1000,), 7.5, device="cuda")
        k3.mxfp4_matmul(*dev, out=buf[: M * N].view(M, N))
        assert bool((buf[M * N:] == 7.5).all()) and not bool((buf[: M * N] == 7.5).all())
    x = torch.randn((5, 96), device="cuda")
    p, s = torch.full((6, 48), 9, dtype=torch.uint8, device="cuda"), torch.full((48,), 9, dtype=torch.uint8, device="cuda")
    k3.mxfp4_quantize(x, packed=p[:5], scale=s[:15].view(5, 3))
    assert bool((p[5] == 9).all()) and bool((s[15:] == 9).all())


def test_streams_and_graph(k3):
    """On a side stream, and captured: replays see the buffers' new contents."""
    g = np.random.default_rng(10)
    N, K = 200, 1024
    wp, ws = (to_dev_u8(t) for t in pair(g, N, K, 120, 124))
    for M in (4, 40):
        x = torch.randn((M, K), device="cuda")
        out = torch.zeros((M, N), device="cuda")
        work = torch.empty(max(1, k3.mxfp4_linear_workspace_size(M, N, K)), dtype=torch.uint8, device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            k3.mxfp4_linear(x, wp, ws, out=out, workspace=work)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(out, k3.mxfp4_linear(x, wp, ws))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            k3.mxfp4_linear(x, wp, ws, out=out, workspace=work)
        for i in range(4):
            x.copy_(torch.randn((M, K), device="cuda"))
            work.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, k3.mxfp4_linear(x, wp, ws)), i


@pytest.mark.parametrize("M,N,K", [(17, 40, 4096), (33, 100, 4128), (77, 60, 7168), (64, 4, 8192), (48, 260, 4160), (200, 17, 4096)])
def test_rows_sixteen_at_a_time_exact(k3, M, N, K):
    """More than 16 rows of a long K and few columns: 16 rows side by side, ragged at the last ones and at N."""
    test_matmul_exact(k3, M, N, K)


@pytest.mark.parametrize("M,N,K", [(5, 33, 6592), (12, 100, 4128), (16, 50, 7168), (9, 40, 32768), (40, 70, 5120)])
def test_linear_rows_quantised_first(k3, M, N, K):
    test_linear_is_quantize_then_matmul(k3, "bf16", M, N, K, True)


@pytest.mark.parametrize("M,N,K", [(300, 500, 1024), (513, 2100, 512), (140, 8300, 1536), (2100, 4200, 512), (2049, 4100, 544)])
def test_matmul_tiles_exact(k3, M, N, K):
    """Every tile size, with the scales of whole 512 columns and of shorter ones."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    rnd = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    ap, wp, as_, ws = rnd(M, K // 2), rnd(N, K // 2), rnd(M, K // 32) % 2 + 126, rnd(N, K // 32) % 2 + 127
    ref = (k3.mxfp4_unpack(ap, as_).double() @ k3.mxfp4_unpack(wp, ws).double().t().contiguous()).float()
    assert torch.equal(k3.mxfp4_matmul(ap, as_, wp, ws), ref)


@pytest.mark.parametrize("M,K", [(3, 672), (16, 7168), (40, 7168)])
def test_nonfinite_blocks_of_few_rows(k3, M, K):
    """A block that is not a number gives NaN in its row or column alone, also where K's last piece is short."""
    g = np.random.default_rng(M + K)
    N = 70
    (ap, as_), (wp, ws) = pair(g, M, K, 126, 127), pair(g, N, K, 127, 128)
    ref = torch.from_numpy(mx4.product_ref(ap, as_, wp, ws)).float()
    as_[M - 1, K // 32 - 1], ws[N - 1, K // 32 - 1], ws[5, 0] = 255, 255, 255
    got = k3.mxfp4_matmul(*(to_dev_u8(t) for t in (ap, as_, wp, ws))).cpu()
    nan = torch.zeros((M, N), dtype=torch.bool)
    nan[M - 1], nan[:, N - 1], nan[:, 5] = True, True, True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], ref[~nan])
