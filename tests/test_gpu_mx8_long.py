"""Products of up to 16 rows of 8 bits over a long K, in chunks of rows and in tiles: exact."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(16, 6140, 9216), (16, 6150, 9216), (12, 12280, 16416), (16, 12290, 16416), (12, 4090, 33792), (9, 4100, 33792),
                                   (16, 7168, 33792), (16, 1530, 65536), (16, 1540, 65536), (3, 12290, 65568)])
def test_products_on_both_sides(k3, M, N, K):
    """Magnitudes 0.5 .. 3.75 and one scale, thinned out so that sums up to 720 units an element stay within 2^24: exact in fp32."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    r = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    ac = (r(3, M, K) + 6) * 8 + r(8, M, K) + 128 * r(2, M, K)
    if K > 23301:
        ac[torch.rand((M, K), generator=g, device="cuda") < 1 - 20000 / K] = 0
    as_ = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
    wp, ws = r(256, N, K // 2), torch.full((N, K // 32), 126, dtype=torch.uint8, device="cuda")
    a = k3.mxfp8_unpack(ac, as_).double()
    assert float(a.abs().sum(1).max()) * 3 * 2**6 <= 2**24
    ref = torch.empty((M, N), dtype=torch.float64, device="cuda")
    for n in range(0, N, 1024):
        ref[:, n: n + 1024] = a @ k3.mxfp4_unpack(wp[n: n + 1024], ws[n: n + 1024]).double().t()
    assert torch.equal(k3.mxfp8_matmul(ac, as_, wp, ws).double(), ref)
    assert torch.equal(k3.mxfp8_matmul(ac, as_, wp, ws, torch.bfloat16), ref.float().bfloat16())
