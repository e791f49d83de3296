"""GPU parity of grouped routing against the fp64 oracle: ids equal, weights within one fp32 step of it."""

import numpy as np
import pytest
import torch

from oracle.groups import route_groups_ref

pytestmark = pytest.mark.gpu

# E, groups, keep, k
SHAPES = [(8, 2, 1, 2), (1, 1, 1, 1), (64, 64, 5, 5), (60, 4, 4, 3), (96, 3, 2, 64), (256, 8, 4, 8), (896, 8, 4, 16), (896, 16, 5, 16), (1000, 125, 30, 24),
          (1024, 32, 1, 32), (1100, 11, 3, 10), (1540, 20, 7, 24), (5000, 1, 1, 6), (4096, 4096, 40, 40), (130, 130, 64, 64), (62, 31, 30, 33), (8192, 8192, 3, 3), (130, 130, 100, 64), (900, 300, 70, 64),
          (330, 10, 4, 12), (500, 4, 2, 9), (640, 5, 2, 7), (768, 24, 11, 40)]


def check(k3, z, bias, k, groups, keep, what=None, **kw):
    ref_i, ref_w = route_groups_ref(z, bias, k, groups, keep, **kw)
    ids, w = k3.moe_route_groups(torch.from_numpy(z).cuda(), None if bias is None else torch.from_numpy(bias).cuda(), k, groups, keep, **kw)
    assert np.array_equal(ids.cpu().numpy(), ref_i), (what, kw)
    got = w.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref_w))
    # fp64 arithmetic rounded once: off by an fp32 step at most, where a rounding border lies within about 1e-15
    assert np.allclose(got, ref_w, rtol=2.0**-23, atol=1e-44, equal_nan=True), (what, kw)


@pytest.mark.parametrize("E,groups,keep,k", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_shapes(k3, E, groups, keep, k, score):
    g = np.random.default_rng([E, groups, k])
    for T, bias, top, norm in ((1, True, 2, True), (37, False, 1, False), (5, True, 1, True), (9, False, 2, True)):
        z = g.standard_normal((T, E)).astype(np.float32) * 2
        b = (g.standard_normal(E) * (0.1 if score == "sigmoid" else 0.3 / E)).astype(np.float32) if bias else None
        check(k3, z, b, k, groups, keep, (E, T), score=score, group_top=top, normalize=norm, route_scale=2.5)


def test_one_group_is_the_plain_router(k3):
    z, b = torch.randn((50, 896), device="cuda"), 0.1 * torch.randn(896, device="cuda")
    for norm in (True, False):
        a = k3.moe_route_topk(z, b, 16, norm, 1.5)
        c = k3.moe_route_groups(z, b, 16, 1, 1, normalize=norm, route_scale=1.5)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties(k3, score):
    """Equal scores everywhere, in pairs, and groups of equal score: the lower index wins, of groups as of experts."""
    g = np.random.default_rng(1)
    for E, groups, keep, k in ((64, 8, 3, 9), (896, 16, 5, 16), (1540, 20, 7, 24)):
        same = np.zeros((3, E), np.float32)
        few = g.integers(0, 3, (40, E)).astype(np.float32)
        mirrored = np.tile(g.standard_normal((5, E // groups)).astype(np.float32), (1, groups))
        for z in (same, few, mirrored):
            for top in (1, 2):
                check(k3, z, None, k, groups, keep, score=score, group_top=top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_near_ties(k3, score):
    """Neighbouring fp32 logits: scores apart by fp64 steps only matter where fp64 says so (and group sums of such)."""
    z = np.full((8, 256), 0.75, np.float32)
    g = np.random.default_rng(2)
    for t in range(8):
        i = g.integers(0, 256, 40)
        z[t, i] = np.nextafter(np.float32(0.75), np.float32(9 if t % 2 else -9))
    check(k3, z, None, 12, 16, 4, score=score)
    check(k3, z, (g.integers(-1, 2, 256) * 2.0**-30).astype(np.float32), 12, 16, 4, score=score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,groups,keep,k", [(64, 16, 5, 9), (256, 8, 4, 8), (896, 16, 5, 16), (1024, 64, 20, 64)])
def test_groups_that_differ_in_fp64_only(k3, score, top, E, groups, keep, k):
    """Every group has two clear best experts; their scores (and sums) differ by 1e-7 and less from group to group, some not at all."""
    g = np.random.default_rng([E, top])
    n = E // groups
    for T, bias in ((40, False), (40, True)):
        z = (-2.0 - g.random((T, groups, n))).astype(np.float32)
        steps = g.integers(-2, 3, (T, groups, 2))
        z[:, :, 0] = 1.0 + steps[..., 0] * np.float32(2.0**-23)
        z[:, :, 1] = 0.5 - steps[..., 1] * np.float32(2.0**-24)
        z = np.take_along_axis(z, np.argsort(g.random((T, groups, n)), -1), -1).reshape(T, E)
        b = (g.integers(-1, 2, E) * 2.0**-28).astype(np.float32) if bias else None
        check(k3, z, b, k, groups, keep, score=score, group_top=top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,keep,k", [(64, 8, 3, 9), (896, 16, 5, 16), (1540, 20, 7, 24)])
def test_masked_infinite_and_nan(k3, score, E, groups, keep, k):
    g = np.random.default_rng(E)
    z = g.standard_normal((12, E)).astype(np.float32)
    low = np.finfo(np.float32).min
    z[0, ::2] = -np.inf
    z[1] = -np.inf
    z[2, 5:] = -np.inf
    z[3] = low
    z[4, 1:] = low
    z[5, 7] = np.nan
    z[6] = np.nan
    z[7, 3:] = np.nan
    z[8, 9] = np.inf
    z[9, [1, 2, E - 1]] = np.inf
    z[10, :] = np.inf
    z[11, 4], z[11, 6] = np.nan, np.inf
    for norm in (True, False):
        check(k3, z, None, k, groups, keep, score=score, normalize=norm)
    b = np.zeros(E, np.float32)
    b[::3] = -np.inf
    b[1::3] = 1e30
    check(k3, z, b, k, groups, keep, score=score)
    b[5], b[8] = np.inf, np.nan
    check(k3, z, b, k, groups, keep, score=score)


def test_empty_and_buffers(k3):
    z = torch.randn((6, 64), device="cuda")
    ids, w = k3.moe_route_groups(z[:0], None, 4, 8, 2)
    assert ids.shape == w.shape == (0, 4)
    ids, w = torch.empty((6, 4), dtype=torch.int32, device="cuda"), torch.empty((6, 4), device="cuda")
    r = k3.moe_route_groups(z, None, 4, 8, 2, ids=ids, weights=w)
    assert r[0] is ids and r[1] is w
    with pytest.raises(k3.K3MoeError):
        k3.moe_route_groups(z, None, 17, 8, 2)
    with pytest.raises(k3.K3MoeError):
        k3.moe_route_groups(z, None, 4, 7, 2)
    with pytest.raises(ValueError):
        k3.moe_route_groups(z, None, 4, 8, 2, score="tanh")


def test_graph_replays_on_new_logits(k3):
    z = torch.randn((20, 896), device="cuda")
    k3.moe_route_groups(z, None, 16, 8, 4, score="softmax")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = k3.moe_route_groups(z, None, 16, 8, 4, score="softmax")
    for _ in range(3):
        z.copy_(torch.randn((20, 896), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        e = k3.moe_route_groups(z, None, 16, 8, 4, score="softmax")
        assert torch.equal(ids, e[0]) and torch.equal(w, e[1])
