"""Cases that measure four operators of the library: microscaled 4-bit rounding (quantise and read back), the linear
layer and the plain product of microscaled 4-bit matrices, and a routed mixture-of-experts layer for a few tokens.

Formats.  E2M1 codes stand for {0, 0.5, 1, 1.5, 2, 3, 4, 6} with the sign in bit 3; 32 neighbouring codes of a row
share one E8M0 byte e that stands for 2^(e - 127).  ``packed`` u8 [R, K/2] holds element 2i in the low and 2i + 1 in
the high nibble of byte i, ``scale`` u8 [R, K/32] the exponent bytes.  Expert matrices hold 17-byte blocks (exponent,
then codes j and j + 16 in the two nibbles of byte 1 + j) in the stage-tiled block order: 16-row groups, a group's
blocks in stages of 16, a stage row by row.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # the activations of a verify step (8 rows of the hidden width) before a 4-bit product: latency
        {"name": "round-8x7168-bf16", "op": "round", "R": 8, "K": 7168, "x": "bf16", "out": "bf16", "saturate": True},
        # a dense matrix in fp32 with ragged sizes, scales that never clamp
        {"name": "round-1003x4128-f32", "op": "round", "R": 1003, "K": 4128, "x": "f32", "out": "f32", "saturate": False},
        # a prompt's hidden rows, or a dense weight matrix: bandwidth
        {"name": "round-16384x7168-bf16", "op": "round", "R": 16384, "K": 7168, "x": "bf16", "out": "bf16", "saturate": True},
        # one token through the latent projection (hidden 7168 to latent 3584)
        {"name": "linear-1x3584x7168-bf16", "op": "linear", "M": 1, "N": 3584, "K": 7168, "x": "bf16", "out": "f32", "saturate": True},
        # eight tokens of a verify step through the dense feed-forward layer of the model (width 33792)
        {"name": "linear-8x33792x7168-bf16", "op": "linear", "M": 8, "N": 33792, "K": 7168, "x": "bf16", "out": "bf16", "saturate": True},
        # ragged sizes, half-precision rows
        {"name": "linear-77x1003x4128-f16", "op": "linear", "M": 77, "N": 1003, "K": 4128, "x": "f16", "out": "f32", "saturate": False},
        # a verify batch against the latent up projection, both operands already in 4 bits
        {"name": "matmul-128x7168x3584", "op": "matmul", "M": 128, "N": 7168, "K": 3584, "out": "f32"},
        # a prompt through a dense projection of the hidden width
        {"name": "matmul-4096x7168x7168", "op": "matmul", "M": 4096, "N": 7168, "K": 7168, "out": "bf16"},
        # a tiny layer: launches and hand-overs only
        {"name": "layer-1-tiny", "op": "layer", "T": 1, "E": 8, "k": 2, "D": 128, "I": 256, "normalize": True, "rscale": 1.0, "bias": True},
        # one token of a decode step through the 896-expert layer
        {"name": "layer-1-k3", "op": "layer", "T": 1, "E": 896, "k": 16, "D": 3584, "I": 3072, "normalize": True, "rscale": 1.0, "bias": True},
        # eight tokens of a decode step through it
        {"name": "layer-8-k3", "op": "layer", "T": 8, "E": 896, "k": 16, "D": 3584, "I": 3072, "normalize": True, "rscale": 1.0, "bias": True},
        # more tokens than fit one tile per expert, block counts that end inside a stage, no bias, raw gates
        {"name": "layer-13-ragged", "op": "layer", "T": 13, "E": 61, "k": 5, "D": 1056, "I": 736, "normalize": False, "rscale": 2.5, "bias": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["round", "linear", "matmul", "layer"])
    if op == "round":
        K = 32 * _log(rng, 1, 512)
        R = _log(rng, 1, min(100000, 16384 * 7168 // K))
        return {"op": op, "R": R, "K": K, "x": rng.choice(["f32", "bf16", "f16"]), "out": rng.choice(["f32", "bf16"]),
                "saturate": rng.random() < 0.5}
    if op in ("linear", "matmul"):
        M, N, K = _log(rng, 1, 4096), _log(rng, 1, 8192), 32 * _log(rng, 1, 256)
        if op == "matmul":
            return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["f32", "bf16"])}
        return {"op": op, "M": _log(rng, 1, 512), "N": N, "K": K, "x": rng.choice(["f32", "bf16", "f16"]),
                "out": rng.choice(["f32", "bf16"]), "saturate": rng.random() < 0.5}
    E = _log(rng, 1, 1500)
    T = rng.randint(1, 16)
    k = _log(rng, 1, min(E, 24))
    D, I = 32 * _log(rng, 1, 128), 32 * _log(rng, 1, 96)
    while E * D * I > 896 * 3584 * 3072 or T * k * D * I > 128 * 3584 * 3072:
        D, I = max(32, D // 64 * 32), max(32, I // 64 * 32)
    return {"op": op, "T": T, "E": E, "k": k, "D": D, "I": I, "normalize": rng.random() < 0.5,
            "rscale": rng.choice([1.0, 2.5]), "bias": rng.random() < 0.7}


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


def _experts(g, E, N, K):
    b = _bytes(g, (E, N, K // 32, 17))
    b[..., 0] = _scales(g, (E, N, K // 32), 118, 122)
    return b


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    m = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    s = {"case": case, "table": torch.tensor(m + [-v for v in m], device="cuda")}
    op = case["op"]
    if op == "round":
        s["x"] = _rows(g, case["R"], case["K"], DTYPES[case["x"]])
    elif op in ("linear", "matmul"):
        M, N, K = case["M"], case["N"], case["K"]
        s["wp"], s["ws"] = _bytes(g, (N, K // 2)), _scales(g, (N, K // 32), 118, 122)
        if op == "linear":
            s["x"] = _rows(g, M, K, DTYPES[case["x"]])
        else:
            s["ap"], s["as"] = _bytes(g, (M, K // 2)), _scales(g, (M, K // 32), 123, 128)
    else:
        T, E, D, I = case["T"], case["E"], case["D"], case["I"]
        s["w1"], s["w3"], s["w2"] = _experts(g, E, I, D), _experts(g, E, I, D), _experts(g, E, D, I)
        s["x"] = torch.randn((T, D), generator=g, device="cuda").to(torch.bfloat16)
        s["logits"] = torch.randn((T, E), generator=g, device="cuda")
        s["bias"] = 0.1 * torch.randn((E,), generator=g, device="cuda") if case["bias"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms


def _round(x, saturate):
    """fp32 values of x [R, K] rounded to microscaled 4 bits."""
    v = x.float().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(top)[1] - 3  # floor(log2(top)) - 2
    e = torch.where(top == 0, -127, e).clamp(min=-127)
    if not saturate:
        e = e + (torch.ldexp(top, -e) > 6)
    q = torch.ldexp(v, -e)
    a = q.abs()
    # nearest E2M1 magnitude, ties to the even code, as a sum of steps
    m = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5).float() + (a >= 3.5) + 2.0 * (a > 5.0)
    return torch.ldexp(torch.copysign(m, q), e).reshape(x.shape)


def _values(packed, scale, t):
    """fp32 values of a microscaled matrix (packed, scale); t: the 16 codes' values."""
    v = torch.stack((t[(packed & 15).int()], t[(packed >> 4).int()]), -1).reshape(*scale.shape, 32)
    return torch.ldexp(v, scale.int()[..., None] - 127).reshape(packed.shape[0], -1)


def _tiled_order(N, nb, device):
    """Storage index of block b of row r of a stage-tiled N x nb matrix of blocks, [N, nb]."""
    r = torch.arange(N, device=device)[:, None]
    b = torch.arange(nb, device=device)[None, :]
    G, s = r // 16, b // 16
    return 16 * G * nb + 16 * s * (N - 16 * G).clamp(max=16) + (r % 16) * (nb - 16 * s).clamp(max=16) + b % 16


def _expert_values(w, ids, t):
    """fp32 matrices [n, N, K] of the chosen experts of w u8 [E, N, K/32, 17]."""
    E, N, nb, _ = w.shape
    b = w.reshape(E, N * nb, 17)[ids][:, _tiled_order(N, nb, w.device).reshape(-1)]
    c = b[..., 1:]
    v = torch.cat((t[(c & 15).int()], t[(c >> 4).int()]), -1)
    return torch.ldexp(v, b[..., :1].int() - 127).reshape(ids.numel(), N, nb * 32)


def _plain_layer(s):
    c, x, k = s["case"], s["x"], s["case"]["k"]
    gate = torch.sigmoid(s["logits"].double())
    score = gate if s["bias"] is None else gate + s["bias"].double()
    ids = torch.sort(score, dim=-1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(gate, 1, ids)
    w = (w / w.sum(-1, keepdim=True) if c["normalize"] else w) * c["rscale"]
    w = w.float()
    flat = ids.reshape(-1)
    rows = x.float().repeat_interleave(k, 0)[:, :, None]
    a = torch.bmm(_expert_values(s["w1"], flat, s["table"]), rows)
    h = a * torch.sigmoid(a) * torch.bmm(_expert_values(s["w3"], flat, s["table"]), rows)
    y = torch.bmm(_expert_values(s["w2"], flat, s["table"]), h).reshape(c["T"], k, c["D"])
    return (y * w[:, :, None]).sum(1), ids.int(), w


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import mxfp4_mixture_experts_moe_amd as k3

        if op == "round":
            packed, scale = k3.mxfp4_quantize(state["x"], saturate=c["saturate"])
            return k3.mxfp4_unpack(packed, scale, DTYPES[c["out"]])
        if op == "linear":
            return k3.mxfp4_linear(state["x"], state["wp"], state["ws"], saturate=c["saturate"], out_dtype=DTYPES[c["out"]])
        if op == "matmul":
            return k3.mxfp4_matmul(state["ap"], state["as"], state["wp"], state["ws"], out_dtype=DTYPES[c["out"]])
        return k3.moe_mxfp4_layer(state["x"], state["logits"], state["bias"], state["w1"], state["w3"], state["w2"], c["k"],
                                  normalize=c["normalize"], route_scale=c["rscale"])
    if op == "round":
        return _round(state["x"], c["saturate"]).to(DTYPES[c["out"]])
    if op == "linear":
        return (_round(state["x"], c["saturate"]) @ _values(state["wp"], state["ws"], state["table"]).t()).to(DTYPES[c["out"]])
    if op == "matmul":
        return (_values(state["ap"], state["as"], state["table"]) @ _values(state["wp"], state["ws"], state["table"]).t()).to(DTYPES[c["out"]])
    return _plain_layer(state)


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op == "round":
        n = case["R"] * case["K"]
        return {"bytes": n * (size[case["x"]] + size[case["out"]]), "flops": 2 * n}
    if op in ("linear", "matmul"):
        M, N, K = case["M"], case["N"], case["K"]
        a = M * K * (size[case["x"]] if op == "linear" else 17 / 32)
        return {"bytes": a + N * K * 17 / 32 + M * N * size[case["out"]], "flops": 2 * M * N * K}
    T, E, k, D, I = (case[n] for n in ("T", "E", "k", "D", "I"))
    used = E * (1 - (1 - k / E) ** T)  # distinct experts of T tokens, expected
    return {"bytes": used * 3 * D * I * 17 / 32 + T * (E * 4 + D * 2 + D * 4 + k * 8) + (E * 4 if case["bias"] else 0),
            "flops": 6 * T * k * D * I}


# ---------------------------------------------------------------------------
# the same results in 64 bits, from the definitions


def _exact_round(x, saturate):
    v = x.double().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    # exponent field of the double: floor(log2(top)); zero blocks get the smallest scale
    e = ((top.view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)
    if not saturate:
        e = torch.where(top > 6.0 * torch.pow(2.0, e.double()), e + 1, e)
    unit = torch.pow(2.0, e.double())
    a = (v / unit).abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    m = (torch.round(a / step) * step).clamp(max=6.0)  # half to even: the even multiple is the even code
    return (torch.sign(v) * m * unit).reshape(x.shape)


def _exact_code(code):
    """E2M1 by its fields: sign, two exponent bits (bias 1), one mantissa bit."""
    code = code.long()
    ex, man = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, torch.pow(2.0, ex - 1.0) * (1.0 + 0.5 * man))
    return torch.where(code >= 8, -mag, mag)


def _exact_values(packed, scale):
    R, K = packed.shape[0], packed.shape[1] * 2
    out = torch.empty((R, K), device=packed.device, dtype=torch.float64)
    out[:, 0::2] = _exact_code(packed % 16)
    out[:, 1::2] = _exact_code(packed // 16)
    return out * torch.pow(2.0, scale.double() - 127.0).repeat_interleave(32, dim=1)


def _exact_matrix(w, e):
    """fp64 matrix [N, K] of expert e of w u8 [E, N, nb, 17]: group by group, stage by stage."""
    _, N, nb, _ = w.shape
    flat = w[e].reshape(N * nb, 17)
    parts = []
    full = N // 16
    for s in range(-(-nb // 16)):
        width = min(16, nb - 16 * s)
        g = flat[: 16 * full * nb].reshape(full, 16 * nb, 17)[:, 256 * s: 256 * s + 16 * width]
        parts.append(g.reshape(full * 16, width, 17))
    b = torch.cat(parts, 1)  # N is a multiple of 16
    c = b[:, :, 1:]
    v = torch.cat((_exact_code(c % 16), _exact_code(c // 16)), -1)
    return (v * torch.pow(2.0, b[:, :, :1].double() - 127.0)).reshape(N, nb * 32)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "round":
        return _exact_round(s["x"], case["saturate"])
    if op in ("linear", "matmul"):
        a = _exact_round(s["x"], case["saturate"]) if op == "linear" else _exact_values(s["ap"], s["as"])
        return a @ _exact_values(s["wp"], s["ws"]).t()
    T, E, k = case["T"], case["E"], case["k"]
    gate = 1.0 / (1.0 + torch.exp(-s["logits"].double().cpu()))
    score = gate + (s["bias"].double().cpu() if s["bias"] is not None else 0.0)
    order = [sorted(range(E), key=lambda e: (-row[e], e))[:k] for row in score.tolist()]
    weight = [[float(gate[t, e]) for e in order[t]] for t in range(T)]
    weight = [[v / sum(r) if case["normalize"] else v for v in r] for r in weight]
    weight = [[v * case["rscale"] for v in r] for r in weight]
    x = s["x"].double()
    out = torch.zeros((T, case["D"]), device=x.device, dtype=torch.float64)
    for e in sorted({e for r in order for e in r}):
        ts = [t for t in range(T) if e in order[t]]
        ws = torch.tensor([weight[t][order[t].index(e)] for t in ts], device=x.device, dtype=torch.float64)
        xe = x[ts]
        a = xe @ _exact_matrix(s["w1"], e).t()
        h = a / (1.0 + torch.exp(-a)) * (xe @ _exact_matrix(s["w3"], e).t())
        out[ts] += ws[:, None] * (h @ _exact_matrix(s["w2"], e).t())
    return out, None, torch.tensor(weight, dtype=torch.float64)
