"""Pins of the oracles of 8-bit rounding, grouped routing and draft verification against something other than themselves:
bit patterns worked by hand, torch's own E4M3 conversion, brute force, and closed forms."""

import itertools

import numpy as np
import torch

from oracle import mx8
from oracle.draft import pick, probabilities, verify_ref
from oracle.groups import route_groups_ref
from oracle.route import route_ref


def test_magnitudes_are_torchs_e4m3():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mx8.MAGNITUDES, t) and t[126] == 448 and t[1] == 2.0**-9 and t[8] == 2.0**-6


def test_quantize_by_hand():
    x = np.zeros((1, 64))
    x[0, :4] = [1.0, -0.3, 0.0625 * 1.0625, 500.0 / 256]  # block maximum 1.953: floor(log2) = 0, e = -8
    x[0, 32:35] = [448.0, -17.0, 2.0**-10]
    c, s = mx8.quantize_ref(x)
    assert s.tolist() == [[119, 127]]
    # 256 = 2^8: 1111.000; -76.8 -> -80 = -(1.25 * 2^6) or -72: step 8, 76.8 is nearer 80? no: 76.8 - 72 = 4.8, 80 - 76.8 = 3.2
    assert c[0, 0] == 0x78 and c[0, 1] == 0x80 | 0x6A
    assert c[0, 2] == 0x58  # 17 lies midway between 16 and 18: the even code
    assert c[0, 3] == 0x7E  # 500 is clamped to 448
    assert c[0, 32:35].tolist() == [0x7E, 0x80 | 0x58, 0x00]
    c, s = mx8.quantize_ref(x, saturate=False)
    assert s.tolist() == [[120, 127]] and c[0, 3] == 0x78  # 250 -> 256


def test_quantize_is_torchs_conversion_inside_the_range():
    g = np.random.default_rng(0)
    x = g.standard_normal((50, 32)).astype(np.float32) * 100
    x[:, 0] = 300  # scale 2^0
    c, s = mx8.quantize_ref(np.clip(x, -440, 440))
    assert (s == 127).all()
    assert np.array_equal(c, torch.from_numpy(np.clip(x, -440, 440)).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert np.array_equal(mx8.values_ref(c, s), torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy())


def test_norm_of_a_constant_row():
    v, y = mx8.norm_ref(np.full((1, 8), 3.0), np.full((1, 8), -1.0), np.arange(8), 0.0)
    assert np.array_equal(v, np.full((1, 8), 2)) and np.array_equal(y, np.arange(8)[None])


def test_groups_by_brute_force():
    """Among all sets of `keep` groups the kept one has the largest scores in order; one group is the plain router."""
    g = np.random.default_rng(1)
    z, b = g.standard_normal((6, 24)), 0.1 * g.standard_normal(24)
    for score in ("sigmoid", "softmax"):
        ids, w = route_groups_ref(z, b, 4, 6, 3, 2, score)
        e = np.exp(z)
        gate = e / (1 + e) if score == "sigmoid" else e / e.sum(1, keepdims=True)
        s = gate + b
        for t in range(6):
            top2 = [sum(sorted(s[t, 4 * i: 4 * i + 4])[-2:]) for i in range(6)]
            best = max(itertools.combinations(range(6), 3), key=lambda c: sum(top2[i] for i in c))
            among = sorted((e for i in best for e in range(4 * i, 4 * i + 4)), key=lambda e: -s[t, e])[:4]
            assert ids[t].tolist() == among
            assert np.allclose(w[t], gate[t, among] / gate[t, among].sum(), rtol=1e-6)
    a, c = route_ref(z, b, 5), route_groups_ref(z, b, 5, 1, 1)
    assert np.array_equal(a[0], c[0]) and np.array_equal(a[1], c[1])


def test_group_ties_by_hand():
    z = np.array([[0.0, 1, 1, 0, 1, 0, 0, 1]])  # every pair of experts has the same two scores
    ids, _ = route_groups_ref(z, None, 3, 4, 2)
    assert ids.tolist() == [[1, 2, 0]]
    z = np.full((1, 4), -np.inf)
    ids, w = route_groups_ref(z, None, 2, 2, 1, score="softmax")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


def test_verification_by_hand():
    p = np.log(np.array([0.5, 0.25, 0.25]))
    l = np.tile(p, (1, 2, 1))
    q = np.array([[[0.25, 0.5, 0.25]]], np.float32)
    # proposal 1: p / q = 0.5; accepted below it, and then p itself is sampled from: cumulative 0.5, 0.75, 1
    n, t, c = verify_ref(l, np.array([[1]]), np.array([[0.499]], np.float32), np.array([0.6], np.float32), q)
    assert n.tolist() == [1] and t.tolist() == [[1, 1]] and abs(c[0, 0] - 0.5) < 1e-7
    # rejected: only token 0 has p above q
    n, t, _ = verify_ref(l, np.array([[1]]), np.array([[0.501]], np.float32), np.array([0.99], np.float32), q)
    assert n.tolist() == [0] and t.tolist() == [[0, -1]]
    # no draft distribution: the proposal itself is excluded; the others 0.5 : 0.25
    n, t, _ = verify_ref(l, np.array([[1]]), np.array([[0.3]], np.float32), np.array([0.67], np.float32))
    assert n.tolist() == [0] and t.tolist() == [[2, -1]]
    # greedy
    n, t, c = verify_ref(l, np.array([[0]]), np.array([[0.9]], np.float32), np.array([0.9], np.float32), q, temperature=[0.0])
    assert n.tolist() == [1] and t.tolist() == [[0, 0]] and c.tolist() == [[1.0]]


def test_probabilities_and_pick():
    assert np.allclose(probabilities(np.array([0.0, np.log(3.0), -np.inf, np.nan]), 1.0).astype(float), [0.25, 0.75, 0, 0])
    assert probabilities(np.array([1.0, np.inf, np.inf]), 1.0).astype(float).tolist() == [0, 0.5, 0.5]
    assert probabilities(np.array([-np.inf, np.nan]), 1.0).astype(float).tolist() == [0, 0]
    m = np.array([0, 0.5, 0, 0.5], np.longdouble)
    assert [pick(m, u) for u in (0.0, 0.4999, 0.5, 0.9, 1.0)] == [1, 1, 3, 3, 3] and pick(m * 0, 0.3) == -1
