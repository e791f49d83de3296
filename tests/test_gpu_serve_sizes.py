"""The 8-bit calls at the largest counts: more than 2^32 elements, 2^31 - 1 rows or columns, more rows than a launch has
workgroups (up to 130 GB on the device). Long operands repeat short ones, so results repeat, too."""

import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

MOST = 2**31 - 1
PERIOD = 2**20
K = 32


@pytest.fixture(autouse=True)
def room():
    """Memory that earlier tests left in torch's cache goes back first, and this test's after it."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 * 2**30:
        pytest.skip("needs 150 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def longest(t):
    """The rows of t [PERIOD, n] over and over, MOST of them."""
    b = torch.empty((2048, *t.shape), dtype=torch.uint8, device="cuda")
    b.copy_(t)
    return b.view(2048 * PERIOD, t.shape[1])[:MOST]


def weights(g, rows):
    r = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return r(rows, K // 2), r(rows, K // 32) % 2 + 126


def rows8(g, rows):
    """Magnitudes 0.5 .. 3.75 and scales 2^-1, 2^0: products are multiples of 2^-8, sums of 32 exact."""
    r = lambda n, *s: torch.randint(0, n, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return (r(3, rows, K) + 6) * 8 + r(8, rows, K) + 128 * r(2, rows, K), r(2, rows, K // 32) + 126


@pytest.mark.parametrize("M,dtype", [(1, torch.float32), (16, torch.bfloat16), (17, torch.bfloat16)])
def test_most_columns(k3, M, dtype):
    g = torch.Generator(device="cuda").manual_seed(M)
    a, w = rows8(g, M), weights(g, PERIOD)
    want = (k3.mxfp8_unpack(*a).double() @ k3.mxfp4_unpack(*w).double().t().contiguous()).to(dtype)
    buf = torch.full((M * MOST + 1000,), 7.25, dtype=dtype, device="cuda")
    out = buf[: M * MOST].view(M, MOST)
    k3.mxfp8_matmul(*a, *[longest(t) for t in w], out_dtype=dtype, out=out)
    torch.cuda.synchronize()
    for m in range(M):
        whole = out[m, : 2047 * PERIOD].view(2047, PERIOD)
        assert all(bool((whole[i: i + 256] == want[m]).all()) for i in range(0, 2047, 256)), m
        assert torch.equal(out[m, 2047 * PERIOD:], want[m, :-1]), m
    assert bool((buf[M * MOST:] == 7.25).all())


def test_most_rows(k3):
    g = torch.Generator(device="cuda").manual_seed(3)
    a, w = rows8(g, PERIOD), weights(g, 3)
    want = (k3.mxfp8_unpack(*a).double() @ k3.mxfp4_unpack(*w).double().t().contiguous()).float()
    buf = torch.full((3 * MOST + 1000,), 7.25, device="cuda")
    out = buf[: 3 * MOST].view(MOST, 3)
    k3.mxfp8_matmul(*[longest(t) for t in a], *w, out=out)
    torch.cuda.synchronize()
    whole = out[: 2047 * PERIOD].view(2047, PERIOD, 3)
    assert all(bool((whole[i: i + 256] == want).all()) for i in range(0, 2047, 256))
    assert torch.equal(out[2047 * PERIOD:], want[:-1])
    assert bool((buf[3 * MOST:] == 7.25).all())


@pytest.mark.parametrize("P,copies,Kc", [(4096, 257, 8192), (4099, 257, 544), (65536, 2100, 32)])
def test_long_rounding_and_norm(k3, P, copies, Kc):
    """Beyond 2^32 elements, beyond 2^20 workgroups of long rows, and 137 million rows that share waves."""
    x = torch.randn((P, Kc), device="cuda").bfloat16()
    gamma = torch.rand((Kc,), device="cuda")
    R = P * copies - 3
    big = torch.empty((copies, P, Kc), dtype=torch.bfloat16, device="cuda")
    big.copy_(x)
    big = big.view(-1, Kc)[:R]

    def same(long, short):
        whole = long[: (copies - 1) * P].view(copies - 1, *short.shape)
        return all(bool((whole[i: i + 64] == short).all()) for i in range(0, copies - 1, 64)) and torch.equal(long[(copies - 1) * P:], short[:-3])

    c, s = k3.mxfp8_quantize(x)
    lc, ls = k3.mxfp8_quantize(big)
    assert same(lc, c) and same(ls, s)
    assert same(k3.mxfp8_unpack(lc, ls, torch.bfloat16), k3.mxfp8_unpack(c, s, torch.bfloat16))
    c, s, t, y = k3.mxfp8_rms_norm(x, gamma, residual=x, normed=True)
    del lc, ls
    lc, ls, lt, ly = k3.mxfp8_rms_norm(big, gamma, residual=big, normed=True)
    assert same(lc, c) and same(ls, s) and same(lt, t) and same(ly, y)


def test_long_verification_and_routing(k3):
    """More than 2^32 logits (rows beyond 2^32 bytes apart), and 5 million tokens routed."""
    S, W, V = 4, 3, 163841
    copies = 2300
    l = torch.randn((S, W, V), device="cuda").bfloat16()
    d = torch.randint(0, V, (S, W - 1), device="cuda", dtype=torch.int32)
    d[:, 0] = l[:, 0].argmax(-1).int()
    u, v = torch.rand((S, W - 1), device="cuda") * 1e-3, torch.rand((S,), device="cuda")
    q = torch.full((S, W - 1, V), 1.0 / V, device="cuda")
    want = k3.moe_verify_draft(l, d, u, v, draft_probs=q)
    big = [t.repeat(copies, *[1] * (t.dim() - 1)) for t in (l, d, u, v)]
    assert big[0].numel() > 2**32
    got = k3.moe_verify_draft(*big)
    one = k3.moe_verify_draft(l, d, u, v)
    assert all(torch.equal(a, b.repeat(copies, *[1] * (b.dim() - 1))) for a, b in zip(got, one))
    del big
    few = [t.repeat(600, *[1] * (t.dim() - 1)) for t in (l, d, u, v, q)]
    got = k3.moe_verify_draft(*few[:4], draft_probs=few[4])
    assert all(torch.equal(a, b.repeat(600, *[1] * (b.dim() - 1))) for a, b in zip(got, want))
    del few
    z = torch.randn((1000, 896), device="cuda")
    ids, w = k3.moe_route_groups(z, None, 16, 16, 5, score="softmax")
    li, lw = k3.moe_route_groups(z.repeat(5000, 1), None, 16, 16, 5, score="softmax")
    assert torch.equal(li, ids.repeat(5000, 1)) and torch.equal(lw, w.repeat(5000, 1))


def test_most_sequences(k3):
    """2^24 - 1 sequences of one row of two entries: the first where the uniform is below its probability (fp64, apart by more
    than rounding: uniforms are multiples of 2^-24, p0 of 16-bit logits)."""
    S = 2**24 - 1
    l = torch.randn((S, 1, 2), device="cuda").half()
    u = torch.rand((S,), device="cuda")
    n, t, a = k3.moe_verify_draft(l, None, None, u)
    p0 = torch.softmax(l.double(), -1)[:, 0, 0]
    clear = (u.double() - p0).abs() > 1e-12
    assert torch.equal(t[clear, 0], (u >= p0)[clear].int()) and int(n.abs().max()) == 0 and clear.float().mean() > 0.999
    with pytest.raises(k3.K3MoeError):
        k3.moe_verify_draft(torch.zeros((2**24, 1, 1), device="cuda"), None, None, torch.zeros(2**24, device="cuda"))
