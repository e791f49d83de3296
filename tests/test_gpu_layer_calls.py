"""Calls of moe_mxfp4_layer and mxfp4_linear that the header allows beside the
plain ones: no outputs of the routing, graphs that take turns on one workspace,
a captured call with the router's own launch, operands 16 bytes into a buffer."""

import numpy as np
import pytest
import torch

import moe_inputs
from moe_inputs.device import upload_experts
from tests.gpu_util import expert_blocks

pytestmark = pytest.mark.gpu

BASE = moe_inputs.TINY


def layer(k3, T, E, k, D, I):
    cfg = BASE.with_(T=T, E=E, k=k, D=D, I=I, config_id=120)
    g = torch.Generator().manual_seed(T * E)
    return cfg, upload_experts(cfg, expert_blocks(k3)), torch.randn((T, D), generator=g).bfloat16().cuda(), torch.randn((T, E), generator=g).cuda()


@pytest.mark.parametrize("T,E", [(1, 8), (5, 40), (1, 1100), (7, 1100)])
def test_routing_kept_in_the_workspace(k3, T, E):
    """ids, weights, or both NULL: the same output, and what is asked for is written."""
    cfg, dev, x, z = layer(k3, T, E, 4, 64, 96)
    want, ids, w = k3.moe_mxfp4_layer(x, z, None, dev.w1, dev.w3, dev.w2, 4)
    n = k3.moe_mxfp4_layer_workspace_size(T, 64, 96, E, 4)
    for use_ids in (False, True):
        for use_w in (False, True):
            work = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            out = torch.full_like(want, float("nan"))
            i2, w2 = torch.full_like(ids, -7), torch.full_like(w, -7)
            st = k3.lib.moe_mxfp4_layer(x.data_ptr(), z.data_ptr(), None, dev.w1.data_ptr(), dev.w3.data_ptr(), dev.w2.data_ptr(), T, 64, 96, E, 4, 1, 1.0, 0,
                                        out.data_ptr(), i2.data_ptr() if use_ids else None, w2.data_ptr() if use_w else None, work.data_ptr(), n,
                                        torch.cuda.current_stream().cuda_stream)
            assert st == 0 and torch.equal(out, want), (use_ids, use_w)
            assert torch.equal(i2, ids) if use_ids else bool((i2 == -7).all())
            assert torch.equal(w2, w) if use_w else bool((w2 == -7).all())


def test_graphs_take_turns_on_one_workspace(k3):
    """Two sizes captured on the same workspace, replayed by turns with eager calls on it between; and the three-launch form."""
    a, b, c = layer(k3, 3, 16, 4, 512, 544), layer(k3, 16, 9, 3, 96, 64), layer(k3, 2, 1100, 8, 64, 64)
    sizes = [k3.moe_mxfp4_layer_workspace_size(v[0].T, v[0].D, v[0].I, v[0].E, v[0].k) for v in (a, b, c)]
    work = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    call = lambda v, **kw: k3.moe_mxfp4_layer(v[2], v[3], None, v[1].w1, v[1].w3, v[1].w2, v[0].k, **kw)  # noqa: E731
    outs = [torch.empty((v[0].T, v[0].D), device="cuda") for v in (a, b, c)]
    graphs = []
    for v, out in zip((a, b, c), outs):
        call(v, out=out, workspace=work)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(v, out=out, workspace=work)
        graphs.append(graph)
    for i in range(5):
        for v in (a, b, c):
            v[2].copy_(torch.randn_like(v[2], dtype=torch.float32).bfloat16())
            v[3].copy_(torch.randn_like(v[3]))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for v, out in zip((a, b, c), outs):
            assert torch.equal(out, call(v)[0]), (i, v[0].T)
            call(v, workspace=work)


@pytest.mark.parametrize("M,N,K", [(1, 40, 512), (3, 33, 1056), (16, 64, 2048), (17, 50, 4160), (70, 130, 544), (300, 260, 1024)])
def test_operands_at_16_bytes(k3, M, N, K):
    """Every operand, output and workspace 16 bytes into its buffer: the bits of aligned ones, nothing written around them."""
    g = np.random.default_rng([M, N, K])

    def at16(t):
        buf = torch.full((t.numel() * t.element_size() + 64,), 165, dtype=torch.uint8, device="cuda")
        v = buf[16: 16 + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        v.copy_(t)
        return buf, v

    x = torch.from_numpy(g.standard_normal((M, K))).bfloat16().cuda()
    wp = torch.from_numpy(g.integers(0, 256, (N, K // 2), dtype=np.uint8)).cuda()
    ws = torch.from_numpy(g.integers(120, 125, (N, K // 32), dtype=np.uint8)).cuda()
    want = k3.mxfp4_linear(x, wp, ws)
    p, s = k3.mxfp4_quantize(x)
    parts = [at16(t) for t in (x, wp, ws, torch.zeros_like(want), torch.zeros(max(1, k3.mxfp4_linear_workspace_size(M, N, K)), dtype=torch.uint8, device="cuda"),
                               torch.zeros_like(p), torch.zeros_like(s), torch.zeros((M, K), dtype=torch.float32, device="cuda"))]
    vx, vp, vs, out, work, qp, qs, val = (v for _, v in parts)
    assert all(v.data_ptr() % 32 == 16 for _, v in parts)
    k3.mxfp4_linear(vx, vp, vs, out=out, workspace=work)
    assert torch.equal(out, want)
    k3.mxfp4_quantize(vx, packed=qp, scale=qs)
    assert torch.equal(qp, p) and torch.equal(qs, s)
    out.zero_()
    k3.mxfp4_matmul(qp, qs, vp, vs, out=out)
    assert torch.equal(out, want)
    k3.mxfp4_unpack(qp, qs, out=val)
    assert torch.equal(val, k3.mxfp4_unpack(p, s))
    for buf, v in parts:
        n = v.numel() * v.element_size()
        assert bool((buf[:16] == 165).all()) and bool((buf[16 + n:] == 165).all())
