"""The third header's entry points without a GPU: symbols, host-side argument checks, workspace sizes. Every call fails (or
is a no-op) in the host checks."""

import os
import re

import pytest
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "k3moe_serve.h")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
A = 0x10000  # an aligned fake device address (never dereferenced)
F32, BF16, F16 = 0, 1, 2


def test_library_exports_every_declared_symbol(k3):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", text, flags=re.M)))
    assert set(names) == {"mxfp8_quantize", "mxfp8_unpack", "mxfp8_rms_norm", "mxfp8_matmul", "moe_route_groups", "moe_verify_draft",
                          "moe_verify_draft_workspace_size"}
    for n in names:
        assert hasattr(k3.lib, n) and n in k3.__all__, n


def test_quantize_and_unpack_checks(k3):
    f, u = k3.lib.mxfp8_quantize, k3.lib.mxfp8_unpack
    for K in (33, 0, -32, (1 << 20) + 32):
        assert f(A, F32, 4, K, 1, A, A, None) == u(A, A, 4, K, F32, A, None) == ERR_SHAPE
    assert f(A, F32, -1, 32, 1, A, A, None) == f(A, F32, 1 << 41, 64, 1, A, A, None) == ERR_SHAPE
    assert f(A, 3, 4, 32, 1, A, A, None) == u(A, A, 4, 32, F16, A, None) == ERR_UNSUPPORTED
    assert f(None, F16, 0, 32, 1, None, None, None) == u(None, None, 0, 32, F32, None, None) == OK
    for i in range(3):
        p = [A] * 3
        p[i] = None
        assert f(p[0], BF16, 4, 32, 1, p[1], p[2], None) == u(p[0], p[1], 4, 32, BF16, p[2], None) == ERR_NULL
        p[i] = A + 8
        assert f(p[0], BF16, 4, 32, 1, p[1], p[2], None) == u(p[0], p[1], 4, 32, BF16, p[2], None) == ERR_ALIGN


def test_norm_checks(k3):
    def f(x=A, res=A, gamma=A, xt=BF16, gt=F32, R=4, K=64, eps=1e-5, total=A, y=A, codes=A, scale=A):
        return k3.lib.mxfp8_rms_norm(x, res, gamma, xt, gt, R, K, eps, 1, total, y, codes, scale, None)

    assert f(K=48) == f(K=0) == f(R=-1) == f(eps=-1.0) == f(eps=float("nan")) == f(R=1 << 41, K=64) == ERR_SHAPE
    assert f(xt=5) == f(gt=-1) == ERR_UNSUPPORTED
    assert f(x=None) == f(codes=None) == f(scale=None) == f(codes=None, scale=None, y=None) == ERR_NULL
    assert f(x=None, R=0) == OK
    for name in ("x", "res", "gamma", "total", "y", "codes", "scale"):
        assert f(**{name: A + 4}) == ERR_ALIGN, name


def test_matmul_checks(k3):
    f = k3.lib.mxfp8_matmul
    for M, N, K in ((4, 4, 40), (-1, 4, 32), (1 << 31, 4, 32), ((1 << 31) - 1, (1 << 31) - 1, 32), (4, 4, (1 << 20) + 32)):
        assert f(A, A, A, A, M, N, K, F32, A, None) == ERR_SHAPE
    assert f(A, A, A, A, 4, 4, 32, F16, A, None) == ERR_UNSUPPORTED
    assert f(None, None, None, None, 0, 4, 32, F32, None, None) == f(None, None, None, None, 4, 0, 32, F32, None, None) == OK
    for i in range(5):
        p = [A] * 5
        p[i] = None
        assert f(*p[:4], 4, 4, 32, F32, p[4], None) == ERR_NULL
        p[i] = A + 8
        assert f(*p[:4], 4, 4, 32, F32, p[4], None) == ERR_ALIGN


def test_route_groups_checks(k3):
    def f(z=A, b=A, T=4, E=64, groups=8, keep=2, top=2, k=16, score=0, ids=A, w=A):
        return k3.lib.moe_route_groups(z, b, T, E, groups, keep, top, k, score, 1, 1.0, ids, w, None)

    for bad in (dict(T=-1), dict(E=0), dict(E=8200, groups=8), dict(groups=0), dict(groups=7), dict(groups=65), dict(groups=-8), dict(keep=0),
                dict(keep=9), dict(k=0), dict(k=17), dict(k=65, keep=8, groups=8, E=128)):
        assert f(**bad) == ERR_SHAPE, bad
    assert f(score=2) == f(score=-1) == f(top=0) == f(top=3) == ERR_UNSUPPORTED
    assert f(T=0, z=None, ids=None, w=None) == OK
    assert f(z=None) == f(ids=None) == f(w=None) == ERR_NULL
    assert f(z=A + 4) == f(b=A + 4) == f(ids=A + 4) == f(w=A + 4) == ERR_ALIGN


def test_verify_draft_checks_and_workspace(k3):
    size = k3.moe_verify_draft_workspace_size
    S, W, V = 3, 8, 10000
    need = size(S, W, V)
    assert need >= S * W * 3 * 16 + S * 3 * 8 + S * 4
    assert size(0, W, V) == size(S, 0, V) == size(S, 65, V) == size(S, W, 0) == size(S, W, (1 << 24) + 1) == size(1 << 24, 1, 1) == 0

    names = ("draft", "probs", "length", "temp", "ua", "us", "n", "tokens", "chance", "ws")

    def f(z=A, dtype=F32, S=S, W=W, V=V, bytes=need, **kw):
        p = {n: kw.get(n, A) for n in names}
        return k3.lib.moe_verify_draft(z, dtype, p["draft"], p["probs"], p["length"], p["temp"], p["ua"], p["us"], S, W, V, p["n"], p["tokens"],
                                       p["chance"], p["ws"], bytes, None)

    for bad in (dict(S=-1), dict(W=0), dict(W=65), dict(V=0), dict(V=(1 << 24) + 1), dict(S=1 << 24, W=1, V=1), dict(S=1 << 20, W=16)):
        assert f(**bad) == ERR_SHAPE, bad
    assert f(dtype=3) == ERR_UNSUPPORTED
    assert f(S=0, z=None, ws=None) == OK
    for n in ("draft", "ua", "us", "n", "tokens", "ws"):
        assert f(**{n: None}) == ERR_NULL, n
    assert f(z=None) == ERR_NULL and f(W=1, us=None) == ERR_NULL
    assert f(z=A + 4) == ERR_ALIGN
    for n in names:
        assert f(**{n: A + 4}) == ERR_ALIGN, n
    assert f(bytes=need - 1) == ERR_WORKSPACE


def test_binding_refuses(k3):
    x, u8 = torch.zeros((4, 64)), torch.zeros((4, 64), dtype=torch.uint8)
    for call in (lambda: k3.mxfp8_quantize(x), lambda: k3.mxfp8_unpack(u8, u8[:, :2]), lambda: k3.mxfp8_rms_norm(x),
                 lambda: k3.mxfp8_matmul(u8, u8[:, :2], u8, u8), lambda: k3.moe_route_groups(x, None, 4, 8, 2),
                 lambda: k3.moe_verify_draft(x[None], None, None, x[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        k3.mxfp8_quantize(x.double())
    with pytest.raises(TypeError):
        k3.mxfp8_rms_norm(x.int())
