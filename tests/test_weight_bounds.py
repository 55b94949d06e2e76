"""The precision that the sampling kernel states for its weights, from a model of its
arithmetic in numpy (the table of 2^(j/32) and the constants are the source's own)."""
import os
import re

import numpy as np
import pytest

F = np.float32
L = np.longdouble
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "lm_head_linear_flce_gb300", "csrc", "flce_sample.cu")


def table():
    text = open(SOURCE).read()
    text = text[text.index("kPow2[32]"):]
    text = text[:text.index("};")]

    def number(x):
        x = x.rstrip("f")
        return float.fromhex(x) if "x" in x else float(x)
    t = [[number(a), number(b)] for a, b in re.findall(r"\{([^{},]+), ([^{},]+)\}", text)]
    return np.array(t).astype(F)


def fma(a, b, c):
    return (np.asarray(a, L) * np.asarray(b, L) + np.asarray(c, L)).astype(F)


def weigh(l, table):
    """Weights of logits l <= 0 at a temperature of 1, relative to 0's, in units of 2^-42."""
    c = L(1) / np.log(L(2))
    hi = F(c)
    lo, magic = F(c - L(hi)), F(1.5 * 2 ** 18)
    z = fma(l, hi, magic)
    t = table[z.view(np.uint32) & 31]
    f = (fma(l, hi, magic - z) + fma(l, lo, t[:, 1])).astype(F)
    ln2 = np.log(2.0)
    p = fma(f, F(ln2 ** 3 / 6), F(ln2 ** 2 / 2 + ln2 ** 4 / 24 * (5 / 7) / 64 ** 2))
    p = (f * fma(f, p, F(ln2))).astype(F)
    e = np.rint((z.astype(L) - L(magic)) * 32).astype(np.int64) >> 5
    th = np.ldexp(t[:, 0], e).astype(F)
    a = ((fma(th, p, th) + F(6)).astype(F) - F(6)).astype(F)
    b = ((fma(th, p, (th - a).astype(F)) + F(1.5 * 2.0 ** -19)).astype(F)
         - F(1.5 * 2.0 ** -19)).astype(F)
    units = a.astype(np.float64) * 2 ** 42 + b.astype(np.float64) * 2 ** 42
    assert (units == np.rint(units)).all()
    return units


def share_error(l, t):
    w, x = weigh(l, t), np.exp(l.astype(L))
    return float(np.abs(np.cumsum(w) / w.sum() - np.cumsum(x) / x.sum()).max())


@pytest.mark.skipif(np.finfo(L).nmant < 63, reason="needs an extended long double")
def test_weights_and_shares_are_as_precise_as_stated():
    t = table()
    assert t.shape == (32, 2)
    j = np.arange(32) / L(32)
    assert np.abs((t[:, 0].astype(L) * 2 ** t[:, 1].astype(L)) / 2 ** j - 1).max() < 2.0 ** -44
    rng = np.random.default_rng(0)
    l = (-rng.random(200000) * 30).astype(F)
    w, x = weigh(l, t), np.exp(l.astype(L))
    off = np.abs(w / 2.0 ** 42 - x)
    # two roundings to the unit's bits: 2^-43, and 2^-24 of up to 2^-22; at least half of 2^42
    # units are the largest's
    assert (off <= 2.0 ** -29 * x + 1.1 * 2.0 ** -43).all()
    some = l > -3
    assert np.sqrt(np.mean((off[some] / x[some]).astype(float) ** 2)) < 2.0 ** -31.5
    for V in (9001, 152064):  # broad rows, two tokens, and a tail below a unit
        l = (rng.standard_normal(V) * 2).astype(F)
        assert share_error(l - l.max(), t) < 2e-11
    assert max(share_error(np.array([0, -2 * rng.random()], F), t) for _ in range(2000)) < 4e-10
    l = np.full(152064, -30.2, F)
    l[0] = 0
    assert 1e-8 < share_error(l, t) < 2.0 ** -28 + 1.1 * l.size * 2.0 ** -42
