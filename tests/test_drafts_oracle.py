"""The oracle of the drafted-token operators (oracle/drafts.py) against values worked by hand, closed forms and
enumeration; and Rotary.make's frequencies against their definitions."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import drafts as ref


def test_turn_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = [math.pi / 2, math.pi]          # at position 1: a quarter and a half turn
    assert np.allclose(ref.turn(x, [1], quarter), [[[-3, -2, 1, -4, 5, 6, 7, 8]]])
    assert np.allclose(ref.turn(x, [1], quarter, interleaved=True), [[[-2, 1, -3, -4, 5, 6, 7, 8]]])
    assert np.allclose(ref.turn(x, [-1], quarter, magnitude=2.0), [[[6, -4, -2, -8, 5, 6, 7, 8]]])


def test_turned_products_depend_on_distances():
    rng = np.random.default_rng(0)
    q, k, f = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16)), 10000.0 ** (-np.arange(6) / 6)
    for il in (False, True):
        dot = lambda i, j: float((ref.turn(q, [i], f, 1.0, il) * ref.turn(k, [j], f, 1.0, il)).sum())
        assert math.isclose(dot(5, 2), dot(1003, 1000), rel_tol=1e-9)


def test_keys_by_hand():
    parents = [-1, 0, 0, 2, -1, 3]
    assert ref.keys_of(parents, 5, 3).tolist() == [0, 1, 2, 3, 5, 6, 8]
    assert ref.keys_of(parents, 4, 3).tolist() == [0, 1, 2, 7]
    assert ref.keys_of(parents, 5, 3, window=5).tolist() == [2, 3, 5, 6, 8]      # position 6
    assert ref.keys_of(parents, 5, 3, window=2).tolist() == [6, 8]
    assert ref.keys_of([-1, 1], 1, 3) is None and ref.keys_of([-2], 0, 3) is None and ref.keys_of([-1, 5, 1], 2, 0) is None


def test_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 0.0, 1.0]])
    q = np.array([[0.25, 0.5, 0.25], [1.0, 0.0, 0.0]])
    # token 1 is kept with probability 1/2; then 2 follows
    assert ref.verify(p, q, [0, 1], [-1, 0], [0, 0.49], 0.0) == ([0, 1], 2)
    # else what is left is token 0 alone
    assert ref.verify(p, q, [0, 1], [-1, 0], [0, 0.5], 0.999) == ([0], 0)
    # chosen drafts: 1 is kept below 1/4; else 0 and 2 are left with 1/2 and 1/4
    assert ref.verify(p, None, [0, 1], [-1, 0], [0, 0.25], 0.66) == ([0], 0)
    assert ref.verify(p, None, [0, 1], [-1, 0], [0, 0.25], 0.67) == ([0], 2)


@pytest.mark.parametrize("drawn", [True, False])
def test_verified_tokens_follow_the_target(drawn):
    """Over all drafts of two siblings (drawn independently from q) and all random numbers, the first token that comes out
    has exactly the target's probabilities: checked in fractions, the random numbers integrated by their borders."""
    p, q = [Fraction(x, 10) for x in (5, 3, 1, 1)], [Fraction(x, 10) for x in (2, 2, 5, 1)]
    out = [Fraction(0)] * 4
    drafts = list(itertools.product(range(4), repeat=2)) if drawn else [(2, 0)]
    for pair in drafts:
        chance = q[pair[0]] * q[pair[1]] if drawn else Fraction(1)
        w, z = list(p), Fraction(1)
        for x in pair:
            qq = q if drawn else [Fraction(int(i == x)) for i in range(4)]
            keep = min(Fraction(1), w[x] / (z * qq[x])) if z else Fraction(0)      # P(u z q < w)
            out[x] += chance * keep
            chance *= 1 - keep
            if chance == 0:
                break
            w = [max(a - z * b, Fraction(0)) for a, b in zip(w, qq)]
            z = sum(w)
        if chance:
            for i in range(4):
                out[i] += chance * w[i] / z
    assert out == p
    # and the oracle decides on those borders
    e = Fraction(1, 1 << 30)
    tp, tq = np.array([[float(x) for x in p]] * 3), np.array([[float(x) for x in q]] * 3) if drawn else None
    edge = p[2] / (q[2] if drawn else 1)
    for u, kept in ((edge - e, [0, 1]), (edge + e, [0])):
        assert ref.verify(tp, tq, [0, 2, 9], [-1, 0, 0], [0, float(u), 0], 0.5)[0] == kept      # 9 is no token


def test_frequencies():
    from post_int4_weight_amd import Rotary
    make = lambda **k: Rotary.make(64, device="cpu", **k)
    plain = make().inv_freq
    assert plain.dtype == torch.float64 and torch.allclose(plain, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32))
    assert torch.allclose(make(scaling="linear", factor=4.0).inv_freq, plain / 4)
    ntk = make(scaling="ntk", factor=4.0).inv_freq
    assert ntk[0] == 1 and math.isclose(ntk[-1], plain[-1] / 4, rel_tol=1e-12)
    turns = 4096 * plain / (2 * math.pi)
    for scaling, high in (("yarn", 32), ("wavelength", 4)):
        s = make(scaling=scaling, factor=8.0, original_length=4096)
        assert torch.equal(s.inv_freq[turns > high * 1.4], plain[turns > high * 1.4])
        assert torch.allclose(s.inv_freq[turns < 1 / 1.4], plain[turns < 1 / 1.4] / 8)
        assert (s.inv_freq.diff() < 0).all() and (s.inv_freq >= plain / 8 * 0.999999).all() and (s.inv_freq <= plain).all()
        assert math.isclose(s.magnitude, 1 + 0.1 * math.log(8) if scaling == "yarn" else 1.0)
    # the wavelength ramp at a pair with between 1 and 4 turns
    s, i = make(scaling="wavelength", factor=8.0, original_length=4096).inv_freq, int(((turns > 1) & (turns < 4)).nonzero()[0])
    k = (turns[i] - 1) / 3
    assert math.isclose(s[i], plain[i] * (k + (1 - k) / 8), rel_tol=1e-12)
    assert make(interleaved=True).interleaved and Rotary.make(2, device="cpu").inv_freq.tolist() == [1.0]


@pytest.mark.parametrize("bad", [dict(rotary_dim=7), dict(rotary_dim=0), dict(base=1.0), dict(factor=0.0), dict(scaling="x"),
                                 dict(scaling="yarn"), dict(scaling="wavelength", original_length=10, low=5.0, high=4.0),
                                 dict(rotary_dim=2, scaling="ntk", factor=2.0)])
def test_frequencies_refused(bad):
    from post_int4_weight_amd import Rotary
    with pytest.raises(ValueError):
        Rotary.make(**{"rotary_dim": 64, "device": "cpu", **bad})
