"""Cases that measure four groups of operators of the library: the residual's addition with a root-mean-square norm and
an output in microscaled 8 bits, products of such rows (or of float rows rounded on the way) with microscaled 4-bit
weights, routing to experts by groups, and the verification of drafted tokens against the target's distribution.

Formats.  A microscaled 8-bit matrix holds E4M3 codes (largest magnitude 448, three mantissa bits, smallest exponent
-6) u8 [R, K] and an E8M0 byte e for each 32 neighbours of a row, u8 [R, K/32], that stands for 2^(e - 127); 4-bit
weights hold E2M1 codes, two a byte, u8 [N, K/2], with scales of the same kind.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of a decode step between two layers: residual added, normed rows in bf16 for the router too: latency
        {"name": "norm-1x7168-bf16", "op": "norm", "R": 1, "K": 7168, "x": "bf16", "gamma": "bf16", "residual": True, "y": True, "out": "bf16", "saturate": True},
        # a final norm in fp32 with ragged sizes, scales that never clamp
        {"name": "norm-1003x4128-f32", "op": "norm", "R": 1003, "K": 4128, "x": "f32", "gamma": "f32", "residual": False, "y": True, "out": "f32", "saturate": False},
        # a prompt's hidden rows between two layers: bandwidth
        {"name": "norm-16384x7168-bf16", "op": "norm", "R": 16384, "K": 7168, "x": "bf16", "gamma": "bf16", "residual": True, "y": False, "out": "bf16", "saturate": True},
        # one token through the latent projection (hidden 7168 to latent 3584), rounded on the way
        {"name": "linear-1x3584x7168-bf16", "op": "linear", "M": 1, "N": 3584, "K": 7168, "x": "bf16", "out": "f32", "saturate": True},
        # ragged sizes, half-precision rows
        {"name": "linear-77x1003x4128-f16", "op": "linear", "M": 77, "N": 1003, "K": 4128, "x": "f16", "out": "bf16", "saturate": False},
        # eight tokens of a verify step, already in 8 bits, through the dense feed-forward layer of the model (width 33792)
        {"name": "matmul-8x33792x7168", "op": "matmul", "M": 8, "N": 33792, "K": 7168, "out": "f32"},
        # a prompt through a dense projection of the hidden width
        {"name": "matmul-4096x7168x7168", "op": "matmul", "M": 4096, "N": 7168, "K": 7168, "out": "bf16"},
        # eight tokens of a verify step to 16 of 896 experts, half of eight groups: latency
        {"name": "route-8x896-sigmoid", "op": "route", "T": 8, "E": 896, "groups": 8, "keep": 4, "top": 2, "k": 16, "score": "sigmoid", "bias": True, "normalize": True, "rscale": 2.5},
        # a prompt, softmax scores, groups ranked by their best expert
        {"name": "route-16384x896-softmax", "op": "route", "T": 16384, "E": 896, "groups": 16, "keep": 5, "top": 1, "k": 16, "score": "softmax", "bias": False, "normalize": False, "rscale": 16.0},
        # one sequence with seven proposals of a draft that takes its likeliest token
        {"name": "verify-1x8x163840-bf16", "op": "verify", "S": 1, "W": 8, "V": 163840, "x": "bf16", "probs": False, "ragged": False, "temperature": "one"},
        # a batch of sequences whose draft samples, fp32 logits
        {"name": "verify-32x8x163840-f32", "op": "verify", "S": 32, "W": 8, "V": 163840, "x": "f32", "probs": True, "ragged": False, "temperature": "one"},
        # odd vocabulary, draft lengths and temperatures of their own (greedy ones among them)
        {"name": "verify-13x5x32003-f16", "op": "verify", "S": 13, "W": 5, "V": 32003, "x": "f16", "probs": True, "ragged": True, "temperature": "mixed"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "matmul", "route", "verify"])
    types = ["f32", "bf16", "f16"]
    if op == "norm":
        K = 32 * _log(rng, 1, 512)
        R = _log(rng, 1, min(100000, 16384 * 7168 // (3 * K)))
        x = rng.choice(types)
        return {"op": op, "R": R, "K": K, "x": x, "gamma": rng.choice([x, "f32"]), "residual": rng.random() < 0.7, "y": rng.random() < 0.5,
                "out": rng.choice(["f32", "bf16"]), "saturate": rng.random() < 0.5}
    if op in ("linear", "matmul"):
        M, N, K = _log(rng, 1, 4096), _log(rng, 1, 7168), 32 * _log(rng, 1, 224)
        if op == "matmul":
            return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["f32", "bf16"])}
        return {"op": op, "M": _log(rng, 1, 512), "N": N, "K": K, "x": rng.choice(types), "out": rng.choice(["f32", "bf16"]), "saturate": rng.random() < 0.5}
    if op == "route":
        groups, size = _log(rng, 1, 32), _log(rng, 1, 128)
        E = groups * size
        keep = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, min(16384, 16384 * 896 // E)), "E": E, "groups": groups, "keep": keep, "top": rng.choice([1, 2]),
                "k": _log(rng, 1, min(keep * size, 32)), "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.6,
                "normalize": rng.random() < 0.5, "rscale": rng.choice([1.0, 2.5])}
    W = rng.randint(1, 12)
    V = _log(rng, 100, 200000)
    return {"op": op, "S": _log(rng, 1, max(1, min(64, 32 * 8 * 163840 // (W * V)))), "W": W, "V": V, "x": rng.choice(types), "probs": rng.random() < 0.6,
            "ragged": rng.random() < 0.4, "temperature": rng.choice(["one", "mixed"])}


# ---------------------------------------------------------------------------
# inputs


def _rows(g, R, K, dtype):
    """Activations: normal, with the few wide channels that hidden states have."""
    x = torch.randn((R, K), generator=g, device="cuda")
    wide = torch.rand((K,), generator=g, device="cuda") < 0.005
    return (x * torch.where(wide, 16.0, 1.0)).to(dtype)


def _bytes(g, shape):
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


def _scales(g, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    m4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    m8 = [(c % 8) * 2.0**-9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)] + [math.nan]
    s = {"case": case, "table4": torch.tensor(m4 + [-v for v in m4], device="cuda"), "table8": torch.tensor(m8 + [-v for v in m8], device="cuda")}
    if op == "norm":
        R, K = case["R"], case["K"]
        s["x"] = _rows(g, R, K, DTYPES[case["x"]])
        s["residual"] = (4.0 * _rows(g, R, K, torch.float32)).to(DTYPES[case["x"]]) if case["residual"] else None
        s["gamma"] = (1.0 + 0.2 * torch.randn((K,), generator=g, device="cuda")).to(DTYPES[case["gamma"]])
    elif op in ("linear", "matmul"):
        M, N, K = case["M"], case["N"], case["K"]
        s["wp"], s["ws"] = _bytes(g, (N, K // 2)), _scales(g, (N, K // 32), 118, 122)
        if op == "linear":
            s["x"] = _rows(g, M, K, DTYPES[case["x"]])
        else:  # rows as a rounding leaves them: blocks that fill the range of E4M3
            sign = _bytes(g, (M, K)) & 128
            v = torch.randn((M, K), generator=g, device="cuda").abs() * 120.0
            ex = torch.frexp(v)[1].clamp(min=-5, max=9) - 1
            s["codes"] = (((ex + 7) * 8 + ((torch.ldexp(v, -ex) - 1.0) * 8).clamp(min=0, max=6)).clamp(max=126).to(torch.uint8) | sign).contiguous()
            s["scale"] = _scales(g, (M, K // 32), 117, 122)
    elif op == "route":
        s["logits"] = torch.randn((case["T"], case["E"]), generator=g, device="cuda")
        s["bias"] = 0.1 * torch.randn((case["E"],), generator=g, device="cuda") if case["bias"] else None
        if case["score"] == "softmax" and case["bias"]:  # a balance bias is of the scores' size
            s["bias"] = s["bias"] * (4.0 / case["E"])
    else:
        S, W, V = case["S"], case["W"], case["V"]
        t = 2.5 * torch.randn((S, W, V), generator=g, device="cuda")
        top = torch.randint(0, V, (S, W, 1), generator=g, device="cuda")
        t.scatter_add_(2, top, torch.rand((S, W, 1), generator=g, device="cuda") * 8.0 + 6.0)
        d = t[:, : W - 1] + 0.3 * torch.randn((S, W - 1, V), generator=g, device="cuda")
        s["logits"] = t.to(DTYPES[case["x"]])
        if case["probs"]:
            s["probs"] = torch.softmax(d, -1)
            pick = torch.rand((S, W - 1, 1), generator=g, device="cuda")
            s["draft"] = (torch.cumsum(s["probs"].double(), -1) <= pick).sum(-1).clamp(max=V - 1).int()
        else:
            s["probs"] = None
            s["draft"] = d.argmax(-1).int()
        s["u_accept"] = torch.rand((S, W - 1), generator=g, device="cuda")
        s["u_sample"] = torch.rand((S,), generator=g, device="cuda")
        s["length"] = torch.randint(0, W, (S,), generator=g, device="cuda", dtype=torch.int32) if case["ragged"] else None
        if case["temperature"] == "mixed":
            kinds = torch.tensor([0.0, 0.7, 1.0, 1.3], device="cuda")
            s["temperature"] = kinds[torch.randint(0, 4, (S,), generator=g, device="cuda")]
        else:
            s["temperature"] = None
    return s


# ---------------------------------------------------------------------------
# plain forms


def _power(e):
    """2^e in fp64, made of its bits: a power function may be a step off, which moves what lies midway between two codes."""
    return torch.bitwise_left_shift(e.long() + 1023, 52).view(torch.float64)


def _round8(v, saturate):
    """v [R, K] (fp64: a value next to a border between two codes has to fall on its own side) rounded to microscaled 8 bits."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top == 0, -127, torch.frexp(top)[1] - 9).clamp(min=-127)  # floor(log2(top)) - 8
    if not saturate:
        e = e + (top * _power(-e) > 448)
    q = b * _power(-e)
    step = (torch.frexp(q)[1] - 1).clamp(min=-6) - 3
    r = (torch.round(q * _power(-step)) * _power(step)).clamp(min=-448, max=448)
    return (r * _power(e)).reshape(v.shape)


def _values4(packed, scale, t):
    """fp32 values of a microscaled 4-bit matrix; t: the 16 codes' values."""
    v = torch.stack((t[(packed & 15).int()], t[(packed >> 4).int()]), -1).reshape(*scale.shape, 32)
    return (v * _power(scale.int() - 127).float()[..., None]).reshape(packed.shape[0], -1)


def _values8(codes, scale, t):
    """fp32 values of a microscaled 8-bit matrix; t: the 256 codes' values."""
    return (t[codes.int()].reshape(*scale.shape, 32) * _power(scale.int() - 127).float()[..., None]).reshape(codes.shape)


def _plain_norm(s):
    c = s["case"]
    v = s["x"].double()
    if c["residual"]:
        v = v + s["residual"].double()
    y = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * s["gamma"].double()
    out = [_round8(y, c["saturate"]).to(DTYPES[c["out"]])]
    if c["residual"]:
        out.append(v.to(DTYPES[c["x"]]))
    if c["y"]:
        out.append(y.to(DTYPES[c["x"]]))
    return out


def _plain_route(s):
    c = s["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    z = s["logits"].double()
    gate = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.exp(z - z.amax(-1, keepdim=True))
    if c["score"] == "softmax":
        gate = gate / gate.sum(-1, keepdim=True)
    score = gate if s["bias"] is None else gate + s["bias"].double()
    best = torch.sort(score.reshape(T, G, E // G), dim=-1, descending=True)[0][..., : c["top"]].sum(-1)
    kept = torch.sort(best, dim=-1, descending=True, stable=True)[1][:, : c["keep"]]
    alive = torch.zeros((T, G), device=z.device, dtype=torch.bool).scatter_(1, kept, True)
    score = torch.where(alive.repeat_interleave(E // G, 1), score, -math.inf)
    ids = torch.sort(score, dim=-1, descending=True, stable=True)[1][:, : c["k"]]
    w = torch.gather(gate, 1, ids)
    if c["normalize"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.int(), (w * c["rscale"]).float()


def _plain_verify(s):
    """In fp64: a sum over the vocabulary decides between neighbours whose probabilities are 1e-6 of it."""
    S, W, V = s["logits"].shape
    l = s["logits"].double()
    t = torch.ones((S,), device=l.device) if s["temperature"] is None else s["temperature"]
    greedy = t <= 0
    m, at = l.max(-1, keepdim=True)
    at = torch.where(l == m, torch.arange(V, device=l.device), V).amin(-1, keepdim=True)  # the lowest index of the largest
    p = torch.exp((l - m) / torch.where(greedy, 1.0, t.double())[:, None, None])
    p = p / p.sum(-1, keepdim=True)
    p = torch.where(greedy[:, None, None], torch.zeros_like(p).scatter_(2, at, 1.0), p)
    n = torch.full((S,), W - 1, device=l.device) if s["length"] is None else s["length"].long()
    d = s["draft"].long()[..., None]
    px = torch.gather(p[:, : W - 1], 2, d)[..., 0]
    q = torch.zeros_like(p[:, : W - 1]).scatter_(2, d, 1.0) if s["probs"] is None else s["probs"].double()
    q = torch.where(greedy[:, None, None], torch.zeros_like(q).scatter_(2, d, 1.0), q)
    qx = torch.gather(q, 2, d)[..., 0]
    there = torch.arange(W - 1, device=l.device) < n[:, None]
    take = (s["u_accept"].double() * qx < px) & there
    count = torch.cumprod(take.int(), 1).sum(1)
    row = torch.gather(p, 1, count[:, None, None].expand(S, 1, V))[:, 0]
    if W > 1:
        less = torch.gather(q, 1, count.clamp(max=W - 2)[:, None, None].expand(S, 1, V))[:, 0]
        left = (row - less).clamp(min=0)
        row = torch.where((count < n)[:, None] & (left.sum(-1, keepdim=True) > 0), left, row)
    total = torch.cumsum(row, -1)
    token = (total <= s["u_sample"].double()[:, None] * total[:, -1:]).sum(-1).clamp(max=V - 1)
    place = torch.arange(W, device=l.device)
    tokens = torch.where(place < count[:, None], torch.nn.functional.pad(s["draft"].long(), (0, 1)), -1)
    tokens = torch.where(place == count[:, None], token[:, None], tokens)
    chance = torch.where(there, (px / qx.clamp(min=1e-300)).clamp(max=1.0), 0.0)
    return count.int(), tokens.int(), chance.float()


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import mxfp4_mixture_experts_moe_amd as k3

        if op == "norm":
            codes, scale, total, y = k3.mxfp8_rms_norm(state["x"], state["gamma"], residual=state["residual"], eps=1e-5, saturate=c["saturate"], normed=c["y"])
            return [t for t in (k3.mxfp8_unpack(codes, scale, DTYPES[c["out"]]), total, y) if t is not None]
        if op == "linear":
            codes, scale = k3.mxfp8_quantize(state["x"], saturate=c["saturate"])
            return k3.mxfp8_matmul(codes, scale, state["wp"], state["ws"], out_dtype=DTYPES[c["out"]])
        if op == "matmul":
            return k3.mxfp8_matmul(state["codes"], state["scale"], state["wp"], state["ws"], out_dtype=DTYPES[c["out"]])
        if op == "route":
            return k3.moe_route_groups(state["logits"], state["bias"], c["k"], c["groups"], c["keep"], group_top=c["top"], score=c["score"],
                                       normalize=c["normalize"], route_scale=c["rscale"])
        return k3.moe_verify_draft(state["logits"], state["draft"], state["u_accept"], state["u_sample"], draft_probs=state["probs"],
                                   draft_len=state["length"], temperature=state["temperature"])
    if op == "norm":
        return _plain_norm(state)
    if op == "linear":
        a = _round8(state["x"].double(), c["saturate"]).float()
        return (a @ _values4(state["wp"], state["ws"], state["table4"]).t()).to(DTYPES[c["out"]])
    if op == "matmul":
        a = _values8(state["codes"], state["scale"], state["table8"])
        return (a @ _values4(state["wp"], state["ws"], state["table4"]).t()).to(DTYPES[c["out"]])
    if op == "route":
        return _plain_route(state)
    return _plain_verify(state)


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op == "norm":
        n, x = case["R"] * case["K"], size[case["x"]]
        return {"bytes": n * (x * (1 + 2 * case["residual"] + case["y"]) + size[case["out"]]) + case["K"] * size[case["gamma"]], "flops": 8 * n}
    if op in ("linear", "matmul"):
        M, N, K = case["M"], case["N"], case["K"]
        a = M * K * (size[case["x"]] if op == "linear" else 33 / 32)
        return {"bytes": a + N * K * 17 / 32 + M * N * size[case["out"]], "flops": 2 * M * N * K}
    if op == "route":
        T, E = case["T"], case["E"]
        return {"bytes": T * (E * 4 + case["k"] * 8) + (E * 4 if case["bias"] else 0), "flops": 10 * T * E}
    S, W, V = case["S"], case["W"], case["V"]
    # every row of logits once, and the one row of the draft's probabilities that is sampled from
    return {"bytes": S * W * V * size[case["x"]] + (S * V * 4 if case["probs"] and W > 1 else 0) + S * (W * 16 + 16), "flops": 10 * S * W * V}


# ---------------------------------------------------------------------------
# the same results in 64 bits, from the definitions


def _two_to(e):
    """2^e in fp64 from its bits (a power function may be off by a step, which moves ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_round8(v, saturate):
    """By a search among the 127 magnitudes of E4M3: the nearest, ties to the even code."""
    mags = torch.tensor([(c % 8) * 2.0**-9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)], device=v.device, dtype=torch.float64)
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    # exponent field of the double: floor(log2(top)); zero blocks get the smallest scale
    e = ((top.view(torch.int64) >> 52) - 1023 - 8).clamp(min=-127)
    if not saturate:
        e = torch.where(top > 448.0 * _two_to(e), e + 1, e)
    unit = _two_to(e)
    a = (b / unit).abs()
    hi = torch.searchsorted(mags, a.contiguous()).clamp(min=1, max=126)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    code = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (torch.sign(b) * mags[code] * unit).reshape(v.shape)


def _exact_code4(code):
    """E2M1 by its fields: sign, two exponent bits (bias 1), one mantissa bit."""
    code = code.long()
    ex, man = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, _two_to(ex - 1) * (1.0 + 0.5 * man))
    return torch.where(code >= 8, -mag, mag)


def _exact_values4(packed, scale):
    R, K = packed.shape[0], packed.shape[1] * 2
    out = torch.empty((R, K), device=packed.device, dtype=torch.float64)
    out[:, 0::2] = _exact_code4(packed % 16)
    out[:, 1::2] = _exact_code4(packed // 16)
    return out * _two_to(scale.long() - 127).repeat_interleave(32, dim=1)


def _exact_values8(codes, scale):
    """E4M3 by its fields: sign, four exponent bits (bias 7), three mantissa bits."""
    c = codes.long()
    ex, man = ((c >> 3) & 15).double(), (c & 7).double() / 8.0
    mag = torch.where(ex == 0, man * 2.0**-6, _two_to(ex - 7) * (1.0 + man))
    return torch.where(c >= 128, -mag, mag) * _two_to(scale.long() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = s["gamma"].double() * v * torch.rsqrt(torch.einsum("rk,rk->r", v, v)[:, None] / case["K"] + 1e-5)
        return [_exact_round8(y, case["saturate"])] + ([v] if case["residual"] else []) + ([y] if case["y"] else [])
    if op in ("linear", "matmul"):
        a = _exact_round8(s["x"].double(), case["saturate"]) if op == "linear" else _exact_values8(s["codes"], s["scale"])
        return a @ _exact_values4(s["wp"], s["ws"]).t()
    if op == "route":
        T, E, G = case["T"], case["E"], case["groups"]
        if T * E > 3000000:
            return None
        z = s["logits"].double().cpu().numpy()
        gate = 1.0 / (1.0 + np.exp(-z)) if case["score"] == "sigmoid" else np.exp(z) / np.exp(z).sum(1, keepdims=True)
        score = gate if s["bias"] is None else gate + s["bias"].double().cpu().numpy()
        weight = []
        for t in range(T):
            rank = sorted(range(G), key=lambda i: (-float(np.sort(score[t, i * (E // G): (i + 1) * (E // G)])[::-1][: case["top"]].sum()), i))
            among = [e for i in rank[: case["keep"]] for e in range(i * (E // G), (i + 1) * (E // G))]
            ids = sorted(among, key=lambda e: (-score[t, e], e))[: case["k"]]
            w = gate[t, ids]
            weight.append(w / (w.sum() if case["normalize"] else 1.0) * case["rscale"])
        return None, torch.tensor(np.stack(weight))
    S, W, V = case["S"], case["W"], case["V"]
    chance = torch.zeros((S, W - 1), dtype=torch.float64)
    for i in range(S):
        t = 1.0 if s["temperature"] is None else float(s["temperature"][i])
        for w in range(W - 1 if s["length"] is None else int(s["length"][i])):
            l = s["logits"][i, w].double()
            x = int(s["draft"][i, w])
            if t <= 0:
                chance[i, w] = float(x == int((l == l.max()).nonzero()[0]))
                continue
            p = float(torch.exp(l[x] / t - torch.logsumexp(l / t, 0)))
            q = 1.0 if s["probs"] is None else float(s["probs"][i, w, x])
            chance[i, w] = min(1.0, p / q) if q > 0 else float(p > 0)
    return None, None, chance
