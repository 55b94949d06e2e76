"""The layer norm's backward on both sides of the size up to which it is one launch: as many
launches as the rule says, and the same gradients from either (to FP32's rounding of their
sums: N/32 + 80 and H/512 + 16 units of the terms, as the forward's test derives it)."""
import numpy as np
import pytest
import torch

from test_gpu_layer_norm import BF, EPS, F32, U, case, f64, rnd, sum_tol

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")


def launches(call):
    before = flce.flce_kernel_launch_count()
    out = call()
    return flce.flce_kernel_launch_count() - before, out


@pytest.mark.parametrize("N,H,want", [
    (64, 4096, 1), (192, 4096, 1), (193, 4096, 2), (256, 4096, 2), (219, 3584, 1), (220, 3584, 2),
    (409, 2560, 1), (410, 2560, 2), (1021, 1001, 1), (1047, 1001, 1), (1048, 1001, 2),
    (96, 8192, 1), (97, 8192, 2), (2, 8200, 2), (2048, 512, 1), (2049, 64, 2)])
def test_one_launch_or_two(N, H, want):
    for dt in (BF, F32):
        x, res, w, b, dy, dh = case(N, H, dt, dt, seed=3)
        _, h, mean, rstd = flce.flce_layer_norm(x, w, b, eps=EPS, residual=res)
        n, (dx, dw, db) = launches(
            lambda: flce.flce_layer_norm_backward(dy, h, w, mean, rstd, dh=dh))
        assert n == want
        r, d = f64(rstd)[:, None], f64(dy)
        v = (f64(h) - f64(mean)[:, None]) * r
        g = d * f64(w)
        c1, c2 = g.mean(1, keepdims=True), (g * v).mean(1, keepdims=True)
        size = r * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                    + np.abs(v) * np.abs(g * v).mean(1, keepdims=True))
        tol = (sum_tol(H) + 16 * U) * size + 2 * U * np.abs(f64(dh))
        ref = r * (g - c1 - v * c2) + f64(dh)
        assert (np.abs(f64(dx) - ref) <= tol + 1.01 * rnd(dt) * (np.abs(ref) + tol)).all()
        for out, t in ((dw, d * v), (db, d)):
            tol = (N / 32 + 84) * U * np.abs(t).sum(0)
            assert (np.abs(f64(out) - t.sum(0)) <= tol + 1.01 * rnd(dt)
                    * (np.abs(t.sum(0)) + tol)).all()
