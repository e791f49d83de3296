"""A verify step out of the calls as they are used together: residual and norm, gate logits by an 8-bit product, grouped
routing, the routed FFN, the next residual and norm, the vocabulary head by an 8-bit product, the verification of the
drafted tokens, and the width that their acceptance suggests. Every stage against its oracle on what the stage before
gave, and the whole captured in a graph and replayed on new inputs."""

import numpy as np
import pytest
import torch

import moe_inputs
from moe_inputs.device import upload_experts
from oracle import mx4, mx8
from oracle.draft import verify_ref
from oracle.ffn import ffn_ref
from oracle.groups import route_groups_ref
from oracle.verify import verify_distinct_ref
from tests.gpu_util import assert_ffn_close, expert_blocks, to_dev_u8

pytestmark = pytest.mark.gpu

S, W, V = 3, 4, 1003
CFG = moe_inputs.TINY.with_(E=32, k=4, D=512, I=512, T=S * W, config_id=95)
GROUPS, KEEP = 8, 3


class Model:
    def __init__(self, k3):
        g = np.random.default_rng(95)
        self.k3 = k3
        self.dev = upload_experts(CFG, expert_blocks(k3))
        self.batch = moe_inputs.make_batch(CFG)
        n = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.gate, self.head = k3.mxfp4_quantize(n(CFG.E, CFG.D) / 16), k3.mxfp4_quantize(n(V, CFG.D) / 8)
        self.gamma1, self.gamma2 = 1 + 0.1 * n(CFG.D), 1 + 0.1 * n(CFG.D)
        self.bias = 0.05 * n(CFG.E)

    def inputs(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        u = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
        q = torch.softmax(n(S, W - 1, V), -1)
        return [n(S * W, CFG.D).bfloat16(), n(S * W, CFG.D).bfloat16(), q, q.argmax(-1).int(), u(S, W - 1) * 0.2, u(S)]

    def step(self, x, hidden, q, draft, ua, us):
        k3 = self.k3
        c1, s1, hidden, y = k3.mxfp8_rms_norm(x, self.gamma1, residual=hidden, normed=True)
        z = k3.mxfp8_matmul(c1, s1, *self.gate)
        ids, w = k3.moe_route_groups(z, self.bias, CFG.k, GROUPS, KEEP, route_scale=1.5)
        f = k3.moe_mxfp4_ffn(y, ids, w, self.dev.w1, self.dev.w3, self.dev.w2)
        c2, s2, hidden2, _ = k3.mxfp8_rms_norm(f.bfloat16(), self.gamma2, residual=hidden)
        logits = k3.mxfp8_matmul(c2, s2, *self.head, out_dtype=torch.bfloat16).view(S, W, V)
        n, tokens, chance = k3.moe_verify_draft(logits, draft, ua, us, draft_probs=q)
        return dict(c1=c1, s1=s1, hidden=hidden, y=y, z=z, ids=ids, w=w, f=f, c2=c2, s2=s2, hidden2=hidden2, logits=logits, n=n, tokens=tokens,
                    chance=chance, distinct=k3.moe_verify_width_distinct(ids, S, W, CFG.E))


def assert_product(got, codes, scale, w, eps):
    """The bound of an fp32 sum of two parts per block (2^-23 an addition), and one rounding to the output's type."""
    a, b = mx8.values_ref(codes, scale), mx4.values_ref(*[t.cpu().numpy() for t in w])
    ref = a @ b.T
    bound = (2 * a.shape[1] // 32 + 16) * 2.0**-23 * (np.abs(a) @ np.abs(b).T)
    assert (np.abs(got.double().cpu().numpy().reshape(ref.shape) - ref) <= bound * (1 + eps) + eps / 2 * np.abs(ref)).all()


def test_step_against_the_oracles(k3):
    m = Model(k3)
    x, hidden, q, draft, ua, us = m.inputs(1)
    r = m.step(x, hidden, q, draft, ua, us)
    h = {n: t.cpu() for n, t in r.items()}
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    v, y = mx8.norm_ref(f64(x), f64(hidden), f64(m.gamma1), 1e-5)
    rc, rs = mx8.quantize_ref(y)
    assert np.array_equal(h["c1"].numpy(), rc) and np.array_equal(h["s1"].numpy(), rs)
    assert_product(h["z"], rc, rs, m.gate, 0.0)
    ids, w = route_groups_ref(h["z"].numpy(), f64(m.bias).astype(np.float32), CFG.k, GROUPS, KEEP, route_scale=1.5)
    assert np.array_equal(h["ids"].numpy(), ids) and np.allclose(h["w"].numpy(), w, rtol=2.0**-23, atol=0)
    bits = h["y"].view(torch.int16).numpy().view(np.uint16)
    assert_ffn_close(h["f"].numpy(), ffn_ref(bits, ids, w, m.batch.experts), "step")
    v, y = mx8.norm_ref(f64(r["f"].bfloat16()), f64(r["hidden"]), f64(m.gamma2), 1e-5)
    rc, rs = mx8.quantize_ref(y)
    assert np.array_equal(h["c2"].numpy(), rc) and np.array_equal(h["s2"].numpy(), rs)
    assert_product(h["logits"], rc, rs, m.head, 2.0**-7)
    n, tokens, chance = verify_ref(h["logits"].float().numpy(), draft.cpu().numpy(), ua.cpu().numpy(), us.cpu().numpy(), q.cpu().numpy())
    assert np.array_equal(h["n"].numpy(), n) and np.array_equal(h["tokens"].numpy(), tokens)
    assert np.allclose(h["chance"].numpy(), chance, rtol=2.0**-23, atol=1e-44)
    assert np.array_equal(h["distinct"].numpy(), verify_distinct_ref(ids, S, W, CFG.E))
    width, rates = k3.moe_verify_width_choose(h["distinct"].tolist(), S, accept=chance.mean(0), expert_bytes=1e6, bytes_per_s=1e12, fixed_s=1e-5)
    assert 1 <= width <= W and rates[width - 1] == max(rates)


def test_step_in_a_graph(k3):
    m = Model(k3)
    buf = m.inputs(2)
    m.step(*buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(*buf)
    for rep in range(3):
        for b, t in zip(buf, m.inputs(10 + rep)):
            b.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for name, t in m.step(*buf).items():
            assert torch.equal(out[name], t), (rep, name)
