"""The norm's y and sum are rounded once, bit for bit, also where fp32 on the way would round before the type does: y below
the normal range, and elements whose v / sqrt(..) is below it while gamma takes y back above."""

import numpy as np
import pytest
import torch

from oracle import mx8

pytestmark = pytest.mark.gpu

# significant bits, exponent of the smallest normal number
FORMS = {torch.float32: (24, -126), torch.bfloat16: (8, -126), torch.float16: (11, -14)}


def rounded(v, dtype):
    """Long double v rounded once to dtype, to nearest, ties to even: the bits as integers (of -0.0 those of -0.0)."""
    bits, least = FORMS[dtype]
    with np.errstate(over="ignore"):
        _, e = np.frexp(v)
        step = np.ldexp(np.ones((), np.longdouble), np.maximum(e - 1, least) - (bits - 1))
        r = np.copysign(np.rint(v / step) * step, v)
    # (exact in fp64; r is a number of the type, which torch's conversion keeps)
    return bits_of(torch.from_numpy(r.astype(np.float64)).to(dtype))


def bits_of(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def check(k3, x, gamma, residual, eps, saturate=True):
    n64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    v, y = mx8.norm_ref(n64(x), n64(residual), n64(gamma), eps)
    rc, rs = mx8.quantize_ref(y, saturate)
    c, s, total, ny = k3.mxfp8_rms_norm(dev(x), dev(gamma), dev(residual), eps=eps, saturate=saturate, normed=True)
    assert torch.equal(bits_of(ny.cpu()), rounded(y, x.dtype))
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(c.cpu().numpy(), rc)
    if total is not None:
        assert torch.equal(bits_of(total.cpu()), rounded(v, x.dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,K", [(3, 64), (5, 1504), (300, 2080), (2, 16416), (1, 33024)])
def test_ordinary_rows(k3, dtype, R, K):
    g = torch.Generator().manual_seed(K)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    check(k3, n(R, K).to(dtype), 1 + 0.3 * n(K), (4 * n(R, K)).to(dtype), 1e-5)


@pytest.mark.parametrize("K", [64, 1024, 9216, 40960])
def test_bf16_below_the_normal_range_beside_ties(k3, K):
    """eps = 1 and rows of 2^-130 have 1 / sqrt(..) = 1, so y = 2^-130 gamma exactly: m + 1/2 steps of 2^-133, and 2^-17 or
    nothing of a step more or less. fp32's own subnormals (2^-149, 2^-16 steps) are coarser than that."""
    m = torch.arange(K) % 127
    off = torch.tensor([2.0**-17, -(2.0**-17), 0.0], dtype=torch.float64)[torch.arange(K) % 3]
    gamma = (m.double() + 0.5 + off) / 8
    gamma[K // 2:] *= -1
    assert torch.equal(gamma, gamma.float().double())
    x = torch.full((2, K), 2.0**-130).bfloat16()
    x[1] *= -1
    check(k3, x, gamma.float(), None, 1.0)
    check(k3, x / 2, gamma.float(), x / 2, 1.0, saturate=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [64, 1024, 9216, 40960])
def test_random_below_the_normal_range(k3, dtype, K):
    """y over the last binades of the type, and below its smallest number."""
    bits, least = FORMS[dtype]
    g = torch.Generator().manual_seed(K)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    gamma = torch.exp2(torch.randint(-bits - 6, 6, (K,), generator=g).float()) * n(K) * 2.0 ** (least + 4 if dtype == torch.float16 else -20)
    x = n(3, K) * (1.0 if dtype == torch.float16 else 2.0 ** (least + 20))
    check(k3, x.to(dtype), gamma, None, 1.0)


@pytest.mark.parametrize("K", [64, 1024, 9216, 40960])
@pytest.mark.parametrize("eps", [3.0, 3.0 * 2.0**16, 5.0 * 2.0**20])
def test_bf16_that_gamma_takes_back_above(k3, K, eps):
    """A 1 in every block, which keeps its scale ordinary, beside elements whose v / sqrt(..) holds only a few of fp32's bits
    below 2^-126, times a gamma of 2^17 to 2^19."""
    g = torch.Generator().manual_seed(K)
    k = torch.randint(1, 128, (4, K), generator=g).float() * torch.exp2(torch.randint(0, 8, (4, K), generator=g).float())
    x = (k * 2.0**-133).bfloat16()
    x[:, ::32] = 1.0
    gamma = torch.exp2(17 + 2 * torch.rand((K,), generator=g)).clamp(max=2.0**19 - 1)
    check(k3, x, gamma, None, eps)
    check(k3, x / 2, -gamma, x / 2, eps, saturate=False)
