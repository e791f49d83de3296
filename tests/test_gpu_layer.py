"""GPU parity of moe_mxfp4_layer (a few tokens, two launches) against the fp64
oracle, element by element.

Bound, with u = 2^-24 (half a step of fp32), every product summed in some order
in fp32: a sum of n products is off by at most n u times the sum of their
magnitudes.  x enters as base-32 digits relative to its 32-block, for which the
bound allows four (the layer takes five): with
8 * 2^s <= max |x| the last digit's half step is 2^s * 32^-3 / 2 <= 2^-19 max |x|
of the block; h as five, 2^-24 max |h|.  The digits' magnitudes add up to at most
the value's plus one step of each (|d0| <= |q| + 1/2, later ones below 1/32 of
the step before), so the sums' magnitudes are taken as |v| + 2^-3 blockmax / 2.
For one expert, X = |x| + blockmax(x) / 16 (H likewise):
  |dg| <= (D + 8) u (|W1| X) + 2^-19 |W1| blockmax(x),  |du| likewise with W3
  h = silu(g) up: |silu'| <= 1.1, and exp, add, divide and two products are
  good to 4 u together with the argument's rounding (2 u |g|, |silu'| again):
  |dh| <= 1.1 |dg| |up| + |silu(g)| |du| + 1.1 |dg| |du| + (8 + 4 |g|) u |h|
  |dy| <= |W2| |dh| + (I + 8) u |W2| H + 2^-24 |W2| blockmax(h)
and the k weighted outputs add (k + 2) u sum |w y| (weights rounded once).
"""

import numpy as np
import pytest
import torch

import moe_inputs
from moe_inputs.device import upload_experts
from oracle.ffn import bf16_bits_to_f64
from oracle.mxfp4 import decode_ct
from oracle.route import route_ref
from tests.gpu_util import assert_ffn_close, bf16_dev, expert_blocks

pytestmark = pytest.mark.gpu

U = 2.0**-24
BASE = moe_inputs.TINY


def blockmax(v):
    """The largest magnitude of each 32-block, repeated over the block."""
    return np.repeat(np.abs(v).reshape(v.shape[0], -1, 32).max(-1), 32, axis=1)


def layer_ref(x_bits, ids, w, experts):
    """fp64 result and the error bound above."""
    x = bf16_bits_to_f64(x_bits)
    T, D = x.shape
    out, bound = np.zeros((T, D)), np.zeros((T, D))
    mag = np.zeros((T, D))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        w1, w3, w2 = (decode_ct(*m) for m in experts[int(e)])
        I = w1.shape[0]
        xe, xm = x[t], blockmax(x[t])
        g, up = xe @ w1.T, xe @ w3.T
        silu = g / (1 + np.exp(-g))
        h = silu * up
        dg, du = ((D + 8) * U * ((np.abs(xe) + xm / 16) @ np.abs(m).T) + 2.0**-19 * (xm @ np.abs(m).T) for m in (w1, w3))
        dh = 1.1 * dg * np.abs(up) + np.abs(silu) * du + 1.1 * dg * du + (8 + 4 * np.abs(g)) * U * np.abs(h)
        y, hm = h @ w2.T, blockmax(np.abs(h) + dh)
        dy = dh @ np.abs(w2).T + (I + 8) * U * ((np.abs(h) + hm / 16) @ np.abs(w2).T) + 2.0**-24 * (hm @ np.abs(w2).T)
        we = w[t, j].astype(np.float64)[:, None]
        np.add.at(out, t, we * y)
        np.add.at(bound, t, np.abs(we) * dy)
        np.add.at(mag, t, np.abs(we * y))
    return out, bound + (ids.shape[1] + 2) * U * mag


def inputs(cfg, same=False):
    batch = moe_inputs.make_batch(cfg)
    z = np.repeat(batch.z[:1], cfg.T, axis=0) if same else batch.z  # same: every token takes the same experts
    return batch, np.ascontiguousarray(z), batch.b


def run(k3, dev, x, z, b, k, **kw):
    zd = torch.from_numpy(z).cuda()
    bd = None if b is None else torch.from_numpy(b).cuda()
    return k3.moe_mxfp4_layer(x, zd, bd, dev.w1, dev.w3, dev.w2, k, **kw)


def check(k3, cfg, same=False, normalize=True, route_scale=1.0, bias=True, dev=None):
    what = f"T={cfg.T} E={cfg.E} k={cfg.k} D={cfg.D} I={cfg.I} same={same}"
    print(f"[layer] {what}", flush=True)
    dev = dev or upload_experts(cfg, expert_blocks(k3))
    batch, z, b = inputs(cfg, same)
    b = b if bias else None
    out, ids, w = run(k3, dev, bf16_dev(batch.x), z, b, cfg.k, normalize=normalize, route_scale=route_scale)
    rid, _ = route_ref(z, b, cfg.k, normalize, route_scale)
    assert np.array_equal(ids.cpu().numpy(), rid), what
    rids, rw = k3.moe_route_topk(torch.from_numpy(z).cuda(), None if b is None else torch.from_numpy(b).cuda(), cfg.k, normalize,
                                 route_scale)
    assert torch.equal(ids, rids) and torch.equal(w, rw), what  # the router's bits
    ref, bound = layer_ref(batch.x, rid, w.cpu().numpy(), batch.experts)
    got = out.cpu().double().numpy()
    err = np.abs(got - ref)
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    print(f"   rel_l2 {rel:.2e}, worst error / bound {np.max(err / bound):.3f}", flush=True)
    assert np.all(err <= bound), what
    return dev, batch, z, b, out


def test_tiny(k3):
    check(k3, BASE.with_(T=1, config_id=101))


@pytest.mark.parametrize("T", [2, 3, 4, 5, 8, 15, 16])
def test_tokens(k3, T):
    check(k3, BASE.with_(T=T, E=16, k=4, D=512, I=512, config_id=102))


@pytest.mark.parametrize("D,I", [(32, 32), (64, 96), (512, 544), (544, 512), (1056, 736), (1024, 1536), (992, 1504)])
def test_sizes(k3, D, I):
    """Block counts that end inside a stage of 16, and less than one stage."""
    check(k3, BASE.with_(T=3, E=5, k=2, D=D, I=I, config_id=103))


@pytest.mark.parametrize("T", [4, 5, 9, 16])
def test_every_token_takes_the_same_experts(k3, T):
    """Several gate/up tiles per expert, and k = E."""
    check(k3, BASE.with_(T=T, E=9, k=3, D=544, I=256, config_id=104), same=True)
    check(k3, BASE.with_(T=T, E=3, k=3, D=128, I=96, config_id=105))


@pytest.mark.parametrize("E,k", [(1, 1), (64, 64), (65, 7), (129, 16), (257, 5), (513, 16), (1025, 8)])
def test_expert_counts(k3, E, k):
    """Every variant of the plan; more than 1024 experts are routed by their own launch."""
    check(k3, BASE.with_(T=6, E=E, k=k, D=64, I=64, config_id=106))


@pytest.mark.parametrize("normalize,route_scale,bias", [(False, 1.0, True), (False, 2.5, False), (True, 2.5, False), (True, 0.0, True)])
def test_routing_options(k3, normalize, route_scale, bias):
    if route_scale == 0.0:  # every gate weight zero: zeros out
        cfg = BASE.with_(T=2, config_id=107)
        dev = upload_experts(cfg, expert_blocks(k3))
        batch, z, b = inputs(cfg)
        out, _, w = run(k3, dev, bf16_dev(batch.x), z, b, cfg.k, normalize=normalize, route_scale=route_scale)
        assert not bool(w.any()) and not bool(out.any())
    else:
        check(k3, BASE.with_(T=4, E=12, k=3, config_id=107), normalize=normalize, route_scale=route_scale, bias=bias)


def test_workspace_contents_do_not_matter_and_results_repeat(k3):
    cfg = BASE.with_(T=7, E=20, k=4, D=544, I=544, config_id=108)
    dev, batch, z, b, want = check(k3, cfg)
    x = bf16_dev(batch.x)
    need = k3.moe_mxfp4_layer_workspace_size(cfg.T, cfg.D, cfg.I, cfg.E, cfg.k)
    work = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 1, 127):
        work.fill_(fill)
        out = torch.full((cfg.T + 1, cfg.D), float("nan"), device="cuda")
        run(k3, dev, x, z, b, cfg.k, workspace=work[:need], out=out[:-1])
        assert torch.equal(out[:-1], want)
        assert bool(torch.isnan(out[-1]).all()) and bool((work[need:] == fill).all())  # nothing written past the ends
    with pytest.raises(k3.K3MoeError):
        run(k3, dev, x, z, b, cfg.k, workspace=work[: need - 256])


def test_close_to_route_and_ffn(k3):
    """The two calls it stands for, on their own bar."""
    cfg = BASE.with_(T=8, E=24, k=6, D=1024, I=512, config_id=109)
    dev, batch, z, b, out = check(k3, cfg)
    ids, w = k3.moe_route_topk(torch.from_numpy(z).cuda(), torch.from_numpy(b).cuda(), cfg.k)
    ffn = k3.moe_mxfp4_ffn(bf16_dev(batch.x), ids, w, dev.w1, dev.w3, dev.w2)
    assert_ffn_close(ffn.cpu().numpy(), out.cpu().double().numpy(), "ffn against layer")


def test_nonfinite_values_stay_in_their_token(k3):
    cfg = BASE.with_(T=5, E=8, k=2, D=128, I=256, config_id=110)
    dev, batch, z, b, want = check(k3, cfg)
    x = bf16_dev(batch.x)
    x[3, 17] = float("nan")
    out, _, _ = run(k3, dev, x, z, b, cfg.k)
    assert bool(torch.isnan(out[3]).all()) and torch.equal(out[[0, 1, 2, 4]], want[[0, 1, 2, 4]])
    z2 = z.copy()
    z2[1] = np.nan  # every score ranks last: the lowest experts, NaN weights
    out, ids, w = run(k3, dev, bf16_dev(batch.x), z2, b, cfg.k)
    assert ids[1].tolist() == [0, 1] and bool(torch.isnan(w[1]).all()) and bool(torch.isnan(out[1]).all())
    assert torch.equal(out[[0, 2, 3, 4]], want[[0, 2, 3, 4]])


def test_zero_tokens_and_binding_checks(k3):
    cfg = BASE.with_(T=2, config_id=111)
    dev = upload_experts(cfg, expert_blocks(k3))
    x = torch.zeros((2, cfg.D), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((2, cfg.E), device="cuda")
    out, ids, w = k3.moe_mxfp4_layer(x[:0], z[:0], None, dev.w1, dev.w3, dev.w2, 2)
    assert out.shape == (0, cfg.D) and ids.shape == (0, 2) and w.shape == (0, 2)
    for bad in (dict(x=x.float()), dict(z=z[:1]), dict(z=z[:, :4].contiguous()), dict(w2=dev.w2[:4]), dict(k=9), dict(k=0)):
        a = {"x": x, "z": z, "w2": dev.w2, "k": 2, **bad}
        with pytest.raises((TypeError, ValueError, k3.K3MoeError)):
            k3.moe_mxfp4_layer(a["x"], a["z"], None, dev.w1, dev.w3, a["w2"], a["k"])
    with pytest.raises(k3.K3MoeError):  # 17 tokens
        k3.moe_mxfp4_layer(x[:1].repeat(17, 1), z[:1].repeat(17, 1), None, dev.w1, dev.w3, dev.w2, 2)


def test_graph_replays(k3):
    """Captured once, replayed on new inputs with eager work between."""
    cfg = BASE.with_(T=4, E=16, k=4, D=512, I=544, config_id=112)
    dev = upload_experts(cfg, expert_blocks(k3))
    x = torch.randn((cfg.T, cfg.D), device="cuda").bfloat16()
    z = torch.randn((cfg.T, cfg.E), device="cuda")
    out = torch.empty((cfg.T, cfg.D), device="cuda")
    work = torch.empty(k3.moe_mxfp4_layer_workspace_size(cfg.T, cfg.D, cfg.I, cfg.E, cfg.k), dtype=torch.uint8, device="cuda")
    call = lambda: k3.moe_mxfp4_layer(x, z, None, dev.w1, dev.w3, dev.w2, cfg.k, out=out, workspace=work)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, ids, _ = call()
    for i in range(6):
        x.copy_(torch.randn((cfg.T, cfg.D), device="cuda").bfloat16())
        z.copy_(torch.randn((cfg.T, cfg.E), device="cuda"))
        work.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        want, wids, _ = k3.moe_mxfp4_layer(x, z, None, dev.w1, dev.w3, dev.w2, cfg.k)
        assert torch.equal(out, want) and torch.equal(ids, wids), i


def test_two_streams_at_once(k3):
    """Calls that overlap, each with its own workspace, give the bits of calls alone."""
    cfg = BASE.with_(T=8, E=32, k=8, D=1024, I=1024, config_id=113)
    dev = upload_experts(cfg, expert_blocks(k3))
    xs = [torch.randn((cfg.T, cfg.D), device="cuda").bfloat16() for _ in range(2)]
    zs = [torch.randn((cfg.T, cfg.E), device="cuda") for _ in range(2)]
    want = [k3.moe_mxfp4_layer(xs[i], zs[i], None, dev.w1, dev.w3, dev.w2, cfg.k)[0] for i in range(2)]
    need = k3.moe_mxfp4_layer_workspace_size(cfg.T, cfg.D, cfg.I, cfg.E, cfg.k)
    work = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [[torch.empty((cfg.T, cfg.D), device="cuda") for _ in range(20)] for _ in range(2)]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for r in range(20):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                k3.moe_mxfp4_layer(xs[i], zs[i], None, dev.w1, dev.w3, dev.w2, cfg.k, out=outs[i][r], workspace=work[i])
    torch.cuda.synchronize()
    for i in range(2):
        for r in range(20):
            assert torch.equal(outs[i][r], want[i]), (i, r)


@pytest.mark.slow
@pytest.mark.parametrize("T", [1, 8])
def test_k3_shape(k3, k3_experts, T):
    cfg = moe_inputs.DECODE8.with_(T=T)
    check(k3, cfg, dev=k3_experts)


def test_from_float_weights(k3):
    """The calls together, as a user has them: float expert matrices quantised, repacked, tiled and used, and a
    dense projection of the layer's output by mxfp4_linear."""
    E, k, D, I, T, N = 6, 2, 256, 512, 5, 384
    g = torch.Generator().manual_seed(3)
    ws = [torch.randn((E, I, D), generator=g) * D**-0.5, torch.randn((E, I, D), generator=g) * D**-0.5,
          torch.randn((E, D, I), generator=g) * I**-0.5]
    pairs = [k3.mxfp4_quantize(t.cuda(), saturate=False) for t in ws]
    tiled = [k3.mxfp4_tile(k3.mxfp4_repack(*p)) for p in pairs]
    x = torch.randn((T, D), generator=g).bfloat16()
    z = torch.randn((T, E), generator=g)
    out, ids, w = k3.moe_mxfp4_layer(x.cuda(), z.cuda(), None, *tiled, k)
    src = [[tuple(a[e].cpu().numpy() for a in p) for p in pairs] for e in range(E)]
    bits = x.view(torch.int16).numpy().view(np.uint16)
    ref, bound = layer_ref(bits, ids.cpu().numpy(), w.cpu().numpy(), src)
    assert np.all(np.abs(out.cpu().double().numpy() - ref) <= bound)
    wp, wsc = k3.mxfp4_quantize(torch.randn((N, D), generator=g).cuda())
    p, s = k3.mxfp4_quantize(out)
    a, b = k3.mxfp4_unpack(p, s).double(), k3.mxfp4_unpack(wp, wsc).double()
    got = k3.mxfp4_linear(out, wp, wsc).double()
    assert bool(((got - a @ b.t()).abs() <= D * U * (a.abs() @ b.abs().t())).all())


@pytest.mark.parametrize("T,E,k,D,I", [(16, 64, 64, 64, 64), (16, 8192, 8, 32, 32), (16, 70, 33, 96, 64), (1, 1, 1, 65536, 32),
                                       (2, 1, 1, 32, 65536), (16, 2, 1, 8192, 4096)])
def test_largest_counts_and_sides(k3, T, E, k, D, I):
    check(k3, BASE.with_(T=T, E=E, k=k, D=D, I=I, config_id=112))


@pytest.mark.parametrize("T,E", [(1, 8), (5, 70), (3, 1100)])
def test_logits_that_are_no_numbers(k3, T, E):
    """The router's ids and weights bit for bit, whatever the logits; a token's NaN weights stay its own."""
    cfg = BASE.with_(T=T, E=E, k=4, D=64, I=64, config_id=113)
    dev = upload_experts(cfg, expert_blocks(k3))
    batch, z, b = inputs(cfg)
    clean = run(k3, dev, bf16_dev(batch.x), z, b, cfg.k)
    z[T - 1, :] = np.nan
    z[0, 1:3] = np.inf, -np.inf
    out, ids, w = run(k3, dev, bf16_dev(batch.x), z, b, cfg.k)
    rids, rw = k3.moe_route_topk(torch.from_numpy(z).cuda(), torch.from_numpy(b).cuda(), cfg.k)
    assert torch.equal(ids, rids) and torch.equal(w.view(torch.int32), rw.view(torch.int32))
    assert torch.equal(torch.isnan(out).all(dim=1), torch.isnan(w).any(dim=1))
    for t in range(1, T - 1):
        assert torch.equal(out[t], clean[0][t]) and torch.equal(ids[t], clean[1][t])
