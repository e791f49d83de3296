"""GPU parity of the verification of drafts against the long-double oracle: counts and tokens equal (fp64 sums differ from
the oracle's by about 1e-15 of the total, which no uniform of these seeds lies that near a border of), probabilities
within a step of fp32."""

import numpy as np
import pytest
import torch

from oracle.draft import verify_ref

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(g, S, W, V, dtype="f32", spread=2.0, probs=True):
    """Logits with a likely token per row, a draft near them, and proposals sampled from it (or its likeliest)."""
    l = g.standard_normal((S, W, V)) * spread
    l[np.arange(S)[:, None], np.arange(W)[None], g.integers(0, V, (S, W))] += 4 + np.log(V)
    logits = torch.from_numpy(l).float().to(TORCH[dtype])
    d = l[:, : W - 1] + 0.4 * g.standard_normal((S, W - 1, V))
    q = np.exp(d - d.max(-1, keepdims=True)) if W > 1 else d
    q = (q / q.sum(-1, keepdims=True) if W > 1 else q).astype(np.float32)
    if probs:
        pick = (np.cumsum(q.astype(np.float64), -1) <= g.random((S, W - 1, 1))).sum(-1)
    else:
        pick = q.argmax(-1) if W > 1 else np.zeros((S, 0), np.int64)
    return dict(logits=logits, draft=np.minimum(pick, V - 1).astype(np.int32), u_accept=g.random((S, W - 1)).astype(np.float32),
                u_sample=g.random(S).astype(np.float32), probs=q if probs else None)


def call(k3, c, **kw):
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return k3.moe_verify_draft(c["logits"].cuda(), dev(c["draft"]), dev(c["u_accept"]), dev(c["u_sample"]), draft_probs=dev(c["probs"]),
                               draft_len=dev(c.get("length")), temperature=dev(c.get("temperature")), **kw)


def check(k3, c, what=None):
    n, tokens, chance = [t.cpu().numpy() for t in call(k3, c)]
    rn, rt, rc = verify_ref(c["logits"].float().numpy(), c["draft"], c["u_accept"], c["u_sample"], c["probs"], c.get("length"), c.get("temperature"))
    assert np.array_equal(n, rn), what
    assert np.array_equal(tokens, rt), what
    assert np.allclose(chance, rc, rtol=2.0**-23, atol=1e-44), what
    return n, tokens


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("S,W,V", [(1, 1, 1), (3, 2, 7), (1, 8, 4096), (2, 8, 4097), (5, 3, 12345), (40, 4, 333), (7, 1, 9000), (2, 64, 501)])
def test_shapes(k3, dtype, probs, S, W, V):
    g = np.random.default_rng([S, W, V, probs])
    n, _ = check(k3, make(g, S, W, V, dtype, probs=probs), (dtype, S, W, V))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_full_vocabulary(k3, dtype):
    g = np.random.default_rng(9)
    n, _ = check(k3, make(g, 3, 8, 163840, dtype))
    assert n.max() > 0


@pytest.mark.parametrize("S,W,V", [(2, 3, 300001), (1, 2, 1200007), (40, 2, 50000), (520, 2, 20500)])
@pytest.mark.parametrize("probs", [True, False])
def test_many_chunks(k3, S, W, V, probs):
    """More chunks than a wave has lanes, and enough of them for several to a workgroup."""
    g = np.random.default_rng([S, V])
    c = make(g, S, W, V, "bf16", probs=probs)
    c["u_accept"][::2] = 0.999  # rejected, mostly
    check(k3, c)
    c["temperature"] = g.choice([0.0, 0.8], S).astype(np.float32)
    check(k3, c)


def test_draft_probabilities_of_zero(k3):
    g = np.random.default_rng(21)
    c = make(g, 12, 4, 3000)
    i = np.arange(12)[:, None], np.arange(3)[None]
    c["probs"][i[0], i[1], c["draft"]] = 0.0  # accepted wherever p is above 0
    c["logits"][3, 1, c["draft"][3, 1]] = -np.inf
    n, _ = check(k3, c)
    assert n[3] == 1 and (np.delete(n, 3) == 3).all()


def test_lengths_and_temperatures(k3):
    g = np.random.default_rng(12)
    S, W, V = 48, 6, 5003
    for probs in (True, False):
        c = make(g, S, W, V, "f16", probs=probs)
        c["length"] = g.integers(-1, W + 2, S).astype(np.int32)
        check(k3, c, "lengths")
        c["temperature"] = g.choice([0.0, 0.5, 1.0, 1.7, -1.0, 100.0, 1e-3], S).astype(np.float32)
        check(k3, c, "temperatures")
        c["temperature"][:4] = [np.nan, np.inf, 1e-38, 1e30]
        check(k3, c, "odd temperatures")


def test_greedy_ties_go_to_the_lowest_index(k3):
    g = np.random.default_rng(13)
    S, W, V = 6, 4, 9001
    c = make(g, S, W, V)
    c["logits"] = torch.from_numpy(g.integers(0, 3, (S, W, V)).astype(np.float32))
    c["temperature"] = np.zeros(S, np.float32)
    top = c["logits"].numpy().argmax(-1)
    c["draft"] = top[:, : W - 1].astype(np.int32)
    c["draft"][1, 0] += 1  # as likely, but not the lowest
    n, t = check(k3, c)
    assert n.tolist() == [3, 0, 3, 3, 3, 3] and t[1].tolist() == [top[1, 0], -1, -1, -1]


def test_masked_rows(k3):
    """-inf, NaN and +inf among the logits; rows with nothing left; a draft that sits on masked places."""
    g = np.random.default_rng(14)
    S, W, V = 10, 3, 8200
    for temperature in (None, np.zeros(S, np.float32), np.full(S, 0.7, np.float32), np.full(S, np.inf, np.float32)):
        c = make(g, S, W, V)
        l = c["logits"]
        l[0, 0] = -np.inf
        l[1, :, ::2] = -np.inf
        l[2, :, 5:] = -np.inf
        l[3, 0] = float("nan")
        l[4, :, 1::2] = float("nan")
        l[5, 0, [7, 8000]] = np.inf
        l[6, :, : V - 1] = -np.inf
        l[7, 1:, 4096:] = float(np.finfo(np.float32).min)
        l[8, 0, 0] = np.inf
        c["draft"][8, 0] = 0
        l[9] = float(np.finfo(np.float32).min)
        if temperature is not None:
            c["temperature"] = temperature
        check(k3, c, temperature)


def test_proposals_outside_the_vocabulary(k3):
    g = np.random.default_rng(15)
    for probs in (True, False):
        c = make(g, 4, 3, 700, probs=probs)
        c["draft"][:, 0] = [-1, 700, 2**31 - 1, -2**31]
        n, t = check(k3, c)
        assert n.tolist() == [0] * 4 and (t[:, 0] >= 0).all() and (t[:, 0] < 700).all()


def test_uniforms_at_their_ends(k3):
    g = np.random.default_rng(16)
    S, W, V = 8, 3, 5000
    for u in (0.0, 1.0 - 2.0**-24, 1.0, np.nan, -1.0, 5.0):
        c = make(g, S, W, V)
        c["u_sample"][:] = u
        n, t = check(k3, c, u)
        assert (t[np.arange(S), n] >= 0).all()
        c["u_accept"][:] = u
        check(k3, c, u)


def test_draft_equal_to_target(k3):
    """q = p in fp32: nearly everything is accepted; where max(p - q, 0) has nothing left, p stands in."""
    g = np.random.default_rng(17)
    S, W, V = 16, 4, 64
    c = make(g, S, W, V)
    c["logits"] = torch.zeros((S, W, V))  # p = 1/64 exactly, and so is q
    c["probs"] = np.full((S, W - 1, V), 1 / 64, np.float32)
    c["u_accept"][:] = 0.999
    n, _ = check(k3, c)
    assert (n == W - 1).all()
    c["u_accept"][:] = 1.0  # not below: rejected, with nothing left of p - q
    n, t = check(k3, c)
    assert (n == 0).all() and (t[:, 0] == (c["u_sample"] * 64).astype(int)).all()


def test_accepted_tokens_follow_the_target(k3):
    """The rule's purpose: over many uniforms the first token is distributed as p (chi-squared over 8 tokens, 20000 draws, 7 degrees
    of freedom: 40 is exceeded with probability 1.3e-6, and the seed is fixed)."""
    g = np.random.default_rng(18)
    S, V = 20000, 8
    p_logits = np.array([0.3, -1, 2, 0, 0.5, -2, 1, 1.5])
    q = np.array([0.3, 0.05, 0.1, 0.2, 0.05, 0.1, 0.1, 0.1])
    c = dict(logits=torch.from_numpy(np.tile(p_logits, (S, 2, 1))).float(), probs=np.tile(q, (S, 1, 1)).astype(np.float32),
             draft=g.choice(V, (S, 1), p=q).astype(np.int32), u_accept=g.random((S, 1)).astype(np.float32), u_sample=g.random(S).astype(np.float32))
    n, tokens, chance = [t.cpu().numpy() for t in call(k3, c)]
    p = np.exp(p_logits) / np.exp(p_logits).sum()
    count = np.bincount(tokens[:, 0], minlength=V)
    assert ((count - S * p) ** 2 / (S * p)).sum() < 40
    # accepted with probability sum min(p, q); four standard deviations
    a = np.minimum(p, q).sum()
    assert abs(n.mean() - a) < 4 * np.sqrt(a * (1 - a) / S) and abs(chance.mean() - a) < 4 * np.sqrt(0.25 / S)


def test_workspace_buffers_and_graph(k3):
    """Workspace full of ones, given outputs, two graphs on one workspace, replayed on new inputs with eager work between."""
    g = np.random.default_rng(19)
    S, W, V = 3, 4, 10007
    c = make(g, S, W, V)
    dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (c["draft"], c["u_accept"], c["u_sample"], c["probs"])]
    logits = c["logits"].cuda()
    ws = torch.full((k3.moe_verify_draft_workspace_size(S, W, V),), 255, dtype=torch.uint8, device="cuda")
    run = lambda **kw: k3.moe_verify_draft(logits, *dev[:3], draft_probs=dev[3], **kw)  # noqa: E731
    want = run()
    got = run(workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(workspace=ws)
        graphs.append((graph, out))
    for rep in range(3):
        logits.copy_(torch.from_numpy(g.standard_normal((S, W, V))).float())
        dev[2].copy_(torch.rand(S, device="cuda"))
        for graph, out in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(run(), out)), rep


def test_two_streams(k3):
    g = np.random.default_rng(20)
    cases = [make(g, 4, 8, 30011, "bf16") for _ in range(2)]
    want = [call(k3, c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append(call(k3, c))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_empty(k3):
    z = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    n, t, a = k3.moe_verify_draft(z(0, 3, 50), z(0, 2, d=torch.int32), z(0, 2), z(0))
    assert n.shape == (0,) and t.shape == (0, 3) and a.shape == (0, 2)
