"""GPU parity of the microscaled products at the largest counts of rows and
columns that the header allows (2^31 - 1; 40 to 110 GB on the device).

The long operand repeats a short one, so the result repeats, too; the scales are
those for which every partial sum is exact, so results are compared for equality
with a double product of the unpacked short operand."""

import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

MOST = 2**31 - 1
PERIOD = 2**20
K = 32


def matrix(g, rows, scale):
    r = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return r(rows, K // 2), r(rows, K // 32) % 2 + scale


def longest(pair):
    """The pair's rows over and over, MOST of them."""
    out = []
    for t in pair:
        b = torch.empty((2048, *t.shape), dtype=torch.uint8, device="cuda")
        b.copy_(t)
        out.append(b.view(2048 * PERIOD, t.shape[1])[:MOST])
    return out


@pytest.fixture(autouse=True)
def room():
    """Memory that earlier tests left in torch's cache goes back first, and this test's after it."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 130 * 2**30:
        pytest.skip("needs 130 GB of free device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,dtype", [(1, torch.float32), (16, torch.bfloat16), (17, torch.bfloat16)])
def test_most_columns(k3, M, dtype):
    """Few rows (groups of 16 columns) and tiles; the last group or tile is one short of whole."""
    g = torch.Generator(device="cuda").manual_seed(M)
    a, w = matrix(g, M, 126), matrix(g, PERIOD, 127)
    want = (k3.mxfp4_unpack(*a).double() @ k3.mxfp4_unpack(*w).double().t().contiguous()).to(dtype)
    buf = torch.full((M * MOST + 1000,), 7.25, dtype=dtype, device="cuda")
    out = buf[: M * MOST].view(M, MOST)
    k3.mxfp4_matmul(*a, *longest(w), out_dtype=dtype, out=out)
    torch.cuda.synchronize()
    for m in range(M):
        whole = out[m, : 2047 * PERIOD].view(2047, PERIOD)
        assert all(bool((whole[i: i + 256] == want[m]).all()) for i in range(0, 2047, 256)), m
        assert torch.equal(out[m, 2047 * PERIOD:], want[m, :-1]), m
    assert bool((buf[M * MOST:] == 7.25).all())


def test_most_rows(k3):
    g = torch.Generator(device="cuda").manual_seed(3)
    a, w = matrix(g, PERIOD, 126), matrix(g, 3, 127)
    want = k3.mxfp4_unpack(*a) @ k3.mxfp4_unpack(*w).t().contiguous()
    buf = torch.full((3 * MOST + 1000,), 7.25, device="cuda")
    out = buf[: 3 * MOST].view(MOST, 3)
    k3.mxfp4_matmul(*longest(a), *w, out=out)
    torch.cuda.synchronize()
    whole = out[: 2047 * PERIOD].view(2047, PERIOD, 3)
    assert all(bool((whole[i: i + 256] == want).all()) for i in range(0, 2047, 256))
    assert torch.equal(out[2047 * PERIOD:], want[:-1])
    assert bool((buf[3 * MOST:] == 7.25).all())
