"""The layer norm's backward on rows whose mean is many times their deviation.

Tolerances, with u = 2^-24.  From the mean and rstd that the call is given, n = (h - mean)
rstd is rounded twice: 2 u |n|, whatever the mean.  Against the definition the mean is off by
its own rounding, u |mean|, and by what its sum loses (tm, as the forward's test derives it),
and rstd by tr of it.  A sum over H columns loses S of its |terms|, one over N rows
(N/32 + 80) u, and an output its type's rounding."""
import numpy as np
import pytest
import torch

from oracle import head_ops as ref
from test_gpu_layer_norm import BF, EPS, F32, U, bounds, case, f64, rnd, sum_tol

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

# one launch for small sizes; aligned, odd and unaligned rows of many; rows past 16384 columns
SHAPES = [(3, 64), (64, 4096), (1021, 264), (2048, 1024), (2500, 1001), (700, 8192), (70, 20000)]


def close(got, want, tol, dt):
    return (np.abs(f64(got) - want) <= tol + 1.01 * rnd(dt) * (np.abs(want) + tol)).all()


def check(got, dy, h, w, mean, rstd, en, er, dt):
    """en: the error of n that is not relative to n; er: that of rstd, relative."""
    N, H = h.shape
    d, W, r = f64(dy), f64(w), rstd[:, None]
    n, S = (f64(h) - mean[:, None]) * r, sum_tol(H)
    en = en + (2.01 * U + er) * np.abs(n)
    g = d * W
    c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
    a3 = (np.abs(g) * en).mean(1, keepdims=True)
    dx, dw, db = got
    size = np.abs(g) + a1 + np.abs(n) * a2
    assert close(dx, r * (g - c1 - n * c2),
                 r * ((S + 8 * U + er) * size + np.abs(n) * a3 + en * np.abs(c2) + en * a3), dt)
    for out, t, e in ((dw, d * n, np.abs(d) * en), (db, d, 0 * d)):
        assert close(out, t.sum(0), (N / 32 + 80) * U * np.abs(t).sum(0) + e.sum(0), dt)


@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("mean", [50.0, -1000.0, 10000.0])
def test_n_keeps_its_digits_at_the_mean_that_is_given(mean, N, H):
    for dt in (F32, BF):
        x, _, w, b, dy, _ = case(N, H, dt, dt, seed=1, mean=mean)
        views = [x]
        if H % 8 == 0:  # rows that are not aligned to 16 bytes
            wide = torch.empty(N, H + 1, dtype=dt, device="cuda")
            wide[:, 1:] = x
            views.append(wide[:, 1:])
        _, _, m, r = flce.flce_layer_norm(x, w, b, eps=EPS)
        for h in views:
            got = flce.flce_layer_norm_backward(dy, h, w, m, r)
            check(got, dy, h, w, f64(m), f64(r), 0.0, 0.0, dt)


@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("mean", [50.0, 1000.0])
def test_gradients_of_the_definition(mean, N, H):
    x, _, w, b, dy, _ = case(N, H, F32, F32, seed=2, mean=mean)
    leaves = [t.requires_grad_() for t in (x, w, b)]
    flce.layer_norm(*leaves, eps=EPS).backward(dy)
    _, mean_, rstd, _, tm, tr = bounds(x, None, w, b)
    check([t.grad for t in leaves], dy, x, w, mean_, rstd,
          ((tm + U * np.abs(mean_)) * rstd)[:, None], tr[:, None], F32)
    want = ref.layer_norm_backward(f64(dy), f64(x), f64(w), EPS)
    # the same against the oracle's own gradient, as a whole: n is off by this much at most
    en = ((tm + 1.1 * U * np.abs(mean_)) * rstd).max() + tr.max() * 6
    for t, v in zip(leaves, want):
        size = np.linalg.norm(v)
        assert np.linalg.norm(f64(t.grad) - v) <= (4 * en + 1e-5) * size
