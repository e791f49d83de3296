"""The second header's entry points without a GPU: symbols, host-side argument
checks, workspace sizes. Every call fails (or is a no-op) in the host checks."""

import os
import re

import pytest
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "k3moe_ops.h")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
A = 0x10000  # an aligned fake device address (never dereferenced)
F32, BF16, F16 = 0, 1, 2


def test_library_exports_every_declared_symbol(k3):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(\w+)\s*\(", text, flags=re.M)))
    assert {"mxfp4_quantize", "mxfp4_unpack", "mxfp4_matmul", "mxfp4_linear", "mxfp4_linear_workspace_size"} <= set(names)
    for n in names:
        assert hasattr(k3.lib, n), n
        assert n in k3.__all__ or n.endswith("_profiled"), n


def test_quantize_checks(k3):
    f = k3.lib.mxfp4_quantize
    assert f(A, F32, 4, 33, 1, A, A, None) == ERR_SHAPE
    assert f(A, F32, 4, 0, 1, A, A, None) == ERR_SHAPE
    assert f(A, F32, -1, 32, 1, A, A, None) == ERR_SHAPE
    assert f(A, F32, 4, (1 << 20) + 32, 1, A, A, None) == ERR_SHAPE
    assert f(A, F32, 1 << 41, 64, 1, A, A, None) == ERR_SHAPE
    assert f(A, 3, 4, 32, 1, A, A, None) == ERR_UNSUPPORTED
    assert f(None, F16, 0, 32, 1, None, None, None) == OK
    for args in ((None, A, A), (A, None, A), (A, A, None)):
        assert f(args[0], BF16, 4, 32, 1, args[1], args[2], None) == ERR_NULL
    for args in ((A + 4, A, A), (A, A + 8, A), (A, A, A + 1)):
        assert f(args[0], BF16, 4, 32, 1, args[1], args[2], None) == ERR_ALIGN


def test_unpack_checks(k3):
    f = k3.lib.mxfp4_unpack
    assert f(A, A, 4, 16, F32, A, None) == ERR_SHAPE
    assert f(A, A, 4, 32, F16, A, None) == ERR_UNSUPPORTED
    assert f(None, None, 0, 32, F32, None, None) == OK
    assert f(A, None, 4, 32, F32, A, None) == ERR_NULL
    assert f(A, A, 4, 32, F32, A + 2, None) == ERR_ALIGN


def test_matmul_checks(k3):
    f = k3.lib.mxfp4_matmul
    assert f(A, A, A, A, 4, 4, 40, F32, A, None) == ERR_SHAPE
    assert f(A, A, A, A, -1, 4, 32, F32, A, None) == ERR_SHAPE
    assert f(A, A, A, A, 1 << 31, 4, 32, F32, A, None) == ERR_SHAPE
    assert f(A, A, A, A, (1 << 31) - 1, (1 << 31) - 1, 32, F32, A, None) == ERR_SHAPE  # too many tiles
    assert f(A, A, A, A, 4, 4, 32, F16, A, None) == ERR_UNSUPPORTED
    assert f(None, None, None, None, 0, 4, 32, F32, None, None) == OK
    assert f(None, None, None, None, 4, 0, 32, F32, None, None) == OK
    for i in range(4):
        p = [A] * 4
        p[i] = None
        assert f(*p, 4, 4, 32, F32, A, None) == ERR_NULL
        p[i] = A + 8
        assert f(*p, 4, 4, 32, F32, A, None) == ERR_ALIGN
    assert f(A, A, A, A, 4, 4, 32, F32, None, None) == ERR_NULL


def test_linear_checks_and_workspace(k3):
    f, size = k3.lib.mxfp4_linear, k3.mxfp4_linear_workspace_size
    assert size(1, 100, 7168) == 0 and size(16, 100, 2048) == 0 and size(0, 5, 32) == 0 and size(4, 4, 33) == 0
    assert size(16, 100, 2080) > 0  # beyond 32 Ki elements the rows are quantised by a launch of their own
    assert size(17, 100, 7168) == 17 * 3584 + -(17 * 3584) % 256 + 17 * 224 + -(17 * 224) % 256
    assert size(16, 8, 65536) >= 16 * 65536 // 2  # codes of 16 such rows do not fit in LDS
    assert f(A, F32, A, A, 40, 4, 64, 1, F32, A, None, 0, None) == ERR_NULL
    assert f(A, F32, A, A, 40, 4, 64, 1, F32, A, A, size(40, 4, 64) - 1, None) == ERR_WORKSPACE
    assert f(A, F32, A, A, 40, 4, 64, 1, F32, A, A + 8, 1 << 20, None) == ERR_ALIGN
    assert f(A, 7, A, A, 40, 4, 64, 1, F32, A, A, 1 << 20, None) == ERR_UNSUPPORTED
    assert f(A, F32, A, A, 40, 4, 64, 1, F16, A, A, 1 << 20, None) == ERR_UNSUPPORTED
    assert f(A, F32, A, A, 40, 4, 48, 1, F32, A, A, 1 << 20, None) == ERR_SHAPE
    assert f(None, F32, None, None, 0, 4, 64, 1, F32, None, None, 0, None) == OK


def test_binding_refuses(k3):
    """The Python binding's own checks (host tensors are refused before any pointer is taken)."""
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        k3.mxfp4_quantize(x)
    with pytest.raises(TypeError):
        k3.mxfp4_quantize(x.double())
    u8 = torch.zeros((4, 32), dtype=torch.uint8)
    with pytest.raises(ValueError):
        k3.mxfp4_matmul(u8, u8[:, :2], u8, u8[:, :2])
    with pytest.raises(ValueError):
        k3.mxfp4_linear(x, u8, u8[:, :2])


def test_layer_checks_and_workspace(k3):
    f, size = k3.lib.moe_mxfp4_layer, k3.moe_mxfp4_layer_workspace_size
    T, D, I, E, k = 3, 64, 96, 8, 2
    need = size(T, D, I, E, k)
    assert need > 0 and size(0, D, I, E, k) == 0 and size(17, D, I, E, k) == 0 and size(T, 65, I, E, k) == 0
    call = lambda p, T=T, D=D, I=I, E=E, k=k, act=0, out=A, ids=A, w=A, ws=A, n=need: f(  # noqa: E731
        *p, T, D, I, E, k, 1, 1.0, act, out, ids, w, ws, n, None)
    ok = [A] * 6  # x, logits, bias, w1, w3, w2
    for i in (0, 1, 3, 4, 5):
        assert call(ok[:i] + [None] + ok[i + 1:]) == ERR_NULL
    for i in range(6):
        assert call(ok[:i] + [A + 4] + ok[i + 1:]) == ERR_ALIGN
    assert call(ok, out=None) == ERR_NULL and call(ok, ws=None) == ERR_NULL
    assert call(ok, out=A + 4) == call(ok, ids=A + 4) == call(ok, w=A + 4) == call(ok, ws=A + 8) == ERR_ALIGN
    assert call(ok, n=need - 1) == ERR_WORKSPACE
    assert call(ok, act=1) == ERR_UNSUPPORTED
    for bad in (dict(T=17), dict(T=-1), dict(D=48), dict(I=0), dict(D=65536 + 32), dict(E=0), dict(k=9), dict(k=0), dict(E=8193)):
        assert call(ok, **bad) == ERR_SHAPE, bad
    assert call([None] * 6, T=0, out=None, ids=None, w=None, ws=None, n=0) == OK


def test_short_workspace_message_names_no_other_call(k3):
    """One status for every call that takes a workspace: its text sends the caller to that call's own size function."""
    text = k3.status_str(ERR_WORKSPACE)
    assert "workspace" in text and "moe_mxfp4_ffn_workspace_size" not in text
    assert text in str(k3.K3MoeError("mxfp4_linear", ERR_WORKSPACE))
