"""moe_mxfp4_layer on values that its number formats have to cope with (a few
channels of x far above the rest, infinities, sums beyond fp32) and over
workspaces of NaN.

Bound for such x, with u = 2^-24 (half a step of fp32).  A 32-block of x enters
as five base-32 digits, the first of step 2^s with max |x| < 2^(s + 4), so the
last one's step is 2^(s - 20): a bf16 value (8 significant bits) of magnitude
2^-17 max |x| >= 2^(s - 13) or more, whose last bit is at least 2^(s - 20), is
held exactly.  The digits of a value add up to at most 3.1 |x| in magnitude (the
first that is not 0 to |x| + 1/2 of its step, at least 1/2 of which is |x|; what
it leaves is at most 1/2 a step, the later digits' own rounding 1/30 of one).
So with five columns of D products each, summed in fp32 in some order,
  |dg| <= 3.1 (D + 13) u (|W1| |x|), |du| likewise with W3,
with no term in the block's largest magnitude.  The rest is the layer's usual
bound: |silu'| <= 1.1; exp, add, divide and two products good to (8 + 4 |g|) u |h|;
h in five digits, 2^-24 of its block's largest; (k + 2) u for the weighted sum.
"""

import numpy as np
import pytest
import torch

from oracle import mx4

pytestmark = pytest.mark.gpu

U = 2.0**-24


def experts(k3, g, E, D, I, quiet):
    """Random experts whose w1 and w3 are zero in the channels `quiet`: (device matrices, fp64 matrices)."""
    dev, host = [], []
    for shape in ((E, I, D), (E, I, D), (E, D, I)):
        w = torch.randn(shape, generator=g) * shape[-1] ** -0.5
        if len(host) < 2:
            w[..., quiet] = 0.0
        p, s = k3.mxfp4_quantize(w.cuda(), saturate=False)
        dev.append(k3.mxfp4_tile(k3.mxfp4_repack(p, s)))
        host.append([mx4.values_ref(p[e].cpu().numpy(), s[e].cpu().numpy()) for e in range(E)])
    return dev, host


def exact_x_ref(x, ids, w, host):
    """fp64 result and the bound above."""
    T, D = x.shape
    out, bound, mag = np.zeros((T, D)), np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            w1, w3, w2 = (m[e] for m in host)
            I = w1.shape[0]
            g, up = w1 @ x[t], w3 @ x[t]
            silu = g / (1 + np.exp(-g))
            h = silu * up
            dg, du = (3.1 * (D + 13) * U * (np.abs(m) @ np.abs(x[t])) for m in (w1, w3))
            dh = 1.1 * dg * np.abs(up) + np.abs(silu) * du + 1.1 * dg * du + (8 + 4 * np.abs(g)) * U * np.abs(h)
            hm = np.repeat((np.abs(h) + dh).reshape(-1, 32).max(-1), 32)
            a2, wt = np.abs(w2), float(w[t, j])
            y = w2 @ h
            out[t] += wt * y
            bound[t] += abs(wt) * (a2 @ dh + (I + 8) * U * (a2 @ (np.abs(h) + hm / 16)) + 2.0**-24 * (a2 @ hm))
            mag[t] += np.abs(wt * y)
    return out, bound + (ids.shape[1] + 2) * U * mag


@pytest.mark.parametrize("T,D,I", [(1, 64, 64), (2, 64, 96), (5, 544, 64), (16, 96, 64), (3, 1056, 544)])
def test_wide_channels_leave_the_others_their_bits(k3, T, D, I):
    """Two channels 2^13 times the others, which no gate or up weight reads: the others count in full."""
    g = torch.Generator().manual_seed(T * D + I)
    quiet = [5, D - 3]
    dev, host = experts(k3, g, 4, D, I, quiet)
    x = (torch.rand((T, D), generator=g) * 1.5 + 0.5) * (torch.randint(0, 2, (T, D), generator=g) * 2 - 1)
    x[:, quiet] *= 8192.0
    if T > 1:
        x[1, quiet] = 0.25  # a row without them beside one with them
    x = x.bfloat16()
    z = torch.randn((T, 4), generator=g)
    out, ids, w = k3.moe_mxfp4_layer(x.cuda(), z.cuda(), None, *dev, 2)
    ref, bound = exact_x_ref(x.double().numpy(), ids.cpu().numpy(), w.cpu().numpy(), host)
    err = np.abs(out.cpu().double().numpy() - ref)
    print(f"[layer] wide channels T={T} D={D} I={I}: worst error / bound {np.max(err / bound):.3f}", flush=True)
    assert np.all(err <= bound)


@pytest.mark.parametrize("T,E,k,D,I", [(1, 8, 2, 2048, 64), (4, 8, 8, 64, 2048), (9, 16, 4, 1056, 736)])
def test_sums_read_finished_rows_alone(k3, T, E, k, D, I):
    """Few sums behind long down units, and many behind short ones, over workspaces whose every float is NaN: no sum
    takes a row of y that its down unit has not written yet, in any of the calls."""
    g = torch.Generator().manual_seed(T + D)
    dev, _ = experts(k3, g, E, D, I, [])
    x, z = torch.randn((T, D), generator=g).bfloat16().cuda(), torch.randn((T, E), generator=g).cuda()
    want = k3.moe_mxfp4_layer(x, z, None, *dev, k)[0]
    assert bool(torch.isfinite(want).all())
    work = torch.empty(k3.moe_mxfp4_layer_workspace_size(T, D, I, E, k), dtype=torch.uint8, device="cuda")
    for i in range(24):
        work.fill_(255)
        assert torch.equal(k3.moe_mxfp4_layer(x, z, None, *dev, k, workspace=work)[0], want), i


@pytest.mark.parametrize("what", ["inf", "-inf", "nan", "h overflows", "x at the largest bf16"])
def test_values_beyond_fp32_stay_in_their_token(k3, what):
    """NaN in every output of the token, as moe_mxfp4_ffn gives; the others keep their bits."""
    g = torch.Generator().manual_seed(11)
    T, E, k, D, I = 6, 4, 2, 96, 64
    dev, _ = experts(k3, g, E, D, I, [])
    x, z = torch.randn((T, D), generator=g).bfloat16(), torch.randn((T, E), generator=g).cuda()
    want, ids, w = k3.moe_mxfp4_layer(x.cuda(), z, None, *dev, k)
    if what == "h overflows":
        x[2] *= 2.0**80  # g and u near 2^80, h near 2^160
    elif what == "x at the largest bf16":
        x[2, 40:44] = torch.finfo(torch.bfloat16).max
    else:
        x[2, 40] = float(what)
    out = k3.moe_mxfp4_layer(x.cuda(), z, None, *dev, k)[0]
    ffn = k3.moe_mxfp4_ffn(x.cuda(), ids, w, *dev)
    others = [0, 1, 3, 4, 5]
    assert bool(torch.isnan(out[2]).all()) and torch.equal(out[others], want[others])
    assert torch.equal(torch.isnan(ffn), torch.isnan(out))
