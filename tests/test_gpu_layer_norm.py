"""Layer norm (forward, 8-bit output, backward) against the float64 definition.

Tolerances.  u = 2^-24 is the float32 rounding unit, e the rounding of the output type
(2^-8 for bf16, u for float32), S = (H/512 + 16) u what a sum over H columns loses of the
sum of its |terms|, sd the deviation of a row, A the root mean square of |x| + |residual|.

The sum h = x + residual is rounded to u of it.  The mean is taken of differences from a
warp's own mean, which lies within 6 sd + S A of the row's (of 32 warps): it is off by
tm = S (8 sd + S A) + 2 u A.  A deviation h - mean is off by tm, by the rounding of h
and by a few u of the differences' size: rstd (tm + u (|x| + |res|) + 16 u sd + 4 u |d|)
in units of rstd.  rstd itself: S of the squares, u A rstd twice for the rounding of
h, and (S A rstd)^2.  A gradient's error is relative to the sizes of its terms, which may
cancel, with 3 u rstd (|h| + |mean|) for n = (h - mean) rstd, which the backward takes
from the stored values."""
import numpy as np
import pytest
import torch

from oracle import head_ops as ref

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def rnd(dt):
    return 2.0 ** -8 if dt == BF else U


def f64(t):
    return t.detach().double().cpu().numpy()


def sum_tol(H):
    return (H / 512 + 16) * U


def case(N, H, dt, wdt, seed=0, mean=0.0):
    g = torch.Generator().manual_seed(seed)

    def t(std, at=0.0):
        return (torch.randn(N, H, generator=g) * std + at).to(dt).cuda()
    x, res = t(1.0, mean), t(3.0)
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(wdt).cuda()
    b = torch.randn(H, generator=g).to(wdt).cuda()
    return x, res, w, b, t(0.1), t(0.2)


def bounds(x, res, w, b):
    """(y, mean, rstd) and the errors that they may have before y is rounded."""
    size = np.abs(f64(x)) + (0 if res is None else np.abs(f64(res)))
    H = size.shape[1]
    W, Bi = (None if t is None else f64(t) for t in (w, b))
    y, h, mean, rstd = ref.layer_norm(f64(x), W, Bi, EPS, None if res is None else f64(res))
    d, r = np.abs(h - mean[:, None]), rstd[:, None]
    sd, A = np.sqrt((d * d).mean(1, keepdims=True)), np.sqrt((size ** 2).mean(1, keepdims=True))
    S = sum_tol(H)
    tm = S * (8 * sd + S * A) + 2 * U * A
    tr = S + 4 * U + 2 * U * A * r + (S * A * r) ** 2
    w1, b1 = 1.0 if W is None else np.abs(W), 0.0 if Bi is None else np.abs(Bi)
    ty = w1 * r * (tm + U * size + 16 * U * sd + 4 * U * d + tr * d) + 4 * U * (w1 * r * d + b1)
    return y, mean, rstd, ty, tm[:, 0], tr[:, 0]


SHAPES = [(1, 1), (1, 3584), (3, 127), (5, 128), (4, 129), (33, 1001), (257, 512), (7, 2056),
          (2, 8192), (2, 16384), (3, 65536), (300, 8), (1021, 264), (2, 16388)]
PARTS = [(True, True, True), (False, True, True), (True, False, True), (True, True, False),
         (False, False, False)]  # residual, weight, bias


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("N,H", SHAPES)
def test_forward(N, H, dt, wdt):
    for mean in (0.0, 50.0):
        x, res, w, b, _, _ = case(N, H, dt, wdt, mean=mean)
        for has in PARTS:
            r, w_, b_ = (t if k else None for k, t in zip(has, (res, w, b)))
            y, h, m, rstd = flce.flce_layer_norm(x, w_, b_, eps=EPS, residual=r)
            if r is None:
                assert h is x
            else:
                assert torch.equal(h, (x.float() + r.float()).to(dt))  # rounded once
            ry, rm, rr, ty, tm, tr = bounds(x, r, w_, b_)
            assert (np.abs(f64(m) - rm) <= tm + 1.01 * U * np.abs(rm)).all()
            assert (np.abs(f64(rstd) / rr - 1) <= tr).all()
            assert (np.abs(f64(y) - ry) <= ty + 1.01 * rnd(dt) * (np.abs(ry) + ty)).all()


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("N,H", SHAPES)
def test_fp8_output(N, H, dt, wdt):
    x, res, w, b, _, _ = case(N, H, dt, wdt, seed=1, mean=2.0)
    for has in PARTS:
        r, w_, b_ = (t if k else None for k, t in zip(has, (res, w, b)))
        q, s, *h = flce.layer_norm_fp8(x, w_, b_, eps=EPS, residual=r)
        assert q.shape == x.shape and s.shape == (N, -(-H // 128)) and len(h) == (r is not None)
        if h:
            assert torch.equal(h[0], (x.float() + r.float()).to(dt))
        ry, _, _, off, _, _ = bounds(x, r, w_, b_)
        amax = np.maximum(ref.block_amax(ry, 1), 0)
        tol = ref.block_amax(off, 1) + 2 * U * amax + 1e-11  # (a scale is never zero)
        assert (np.abs(f64(s) * 448 - amax) <= tol).all()
        # half an e4m3 step of the value (2^-4 of it, 2^-10 of the scale near zero)
        sx = ref.expand_scale(f64(s), N, H, 1)
        err = np.abs(f64(q) * sx - ry)
        assert (err <= (2.0 ** -4 * np.abs(ry) + 2.0 ** -10 * sx) * 1.001 + off
                + ref.expand_scale(tol, N, H, 1)).all()
        assert f64(q).__abs__().max() <= 448


def check_backward(got, dy, h, w, mean, rstd, dh, dt, wdt, bdt):
    N, H = h.shape
    r, m, hh, d = f64(rstd)[:, None], f64(mean)[:, None], f64(h), f64(dy)
    n, en = (hh - m) * r, 3 * U * r * (np.abs(hh) + np.abs(m))
    g = d if w is None else d * f64(w)
    S = sum_tol(H)
    c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
    a3 = (np.abs(g) * en).mean(1, keepdims=True)
    dx, dw, db = got
    if dx is not None:
        rdx = r * (g - c1 - n * c2) + (0 if dh is None else f64(dh))
        tol = r * ((S + 8 * U) * (np.abs(g) + a1 + np.abs(n) * a2) + np.abs(n) * a3
                   + en * np.abs(c2)) + (0 if dh is None else 2 * U * np.abs(f64(dh)))
        assert (np.abs(f64(dx) - rdx) <= tol + 1.01 * rnd(dt) * (np.abs(rdx) + tol)).all()
    for out, t, e, o in ((dw, d * n, np.abs(d) * en, wdt), (db, d, 0 * d, bdt)):
        if out is not None:
            assert out.dtype == o
            tol = (N / 32 + 80) * U * np.abs(t).sum(0) + e.sum(0)
            assert (np.abs(f64(out) - t.sum(0)) <= tol + 1.01 * rnd(o)
                    * (np.abs(t.sum(0)) + tol)).all()


# (beside the forward's: with rows enough for every way to split them)
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("N,H", SHAPES + [(2048, 1001), (2049, 1001), (2500, 1000), (700, 8192),
                                          (9000, 64), (400, 16384), (130, 16388), (2048, 1024),
                                          (300001, 24)])
def test_backward(N, H, dt, wdt):
    x, res, w, b, dy, dh = case(N, H, dt, wdt, seed=2, mean=1.0)
    y, h, mean, rstd = flce.flce_layer_norm(x, w, b, eps=EPS, residual=res)
    for w_, extra in ((w, dh), (w, None), (None, dh)):
        got = flce.flce_layer_norm_backward(dy, h, w_, mean, rstd, dh=extra)
        assert all(t is not None for t in got[::2]) and (got[1] is None) == (w_ is None)
        check_backward(got, dy, h, w_, mean, rstd, extra, dt, wdt, dt if w_ is None else wdt)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)):
        got = flce.flce_layer_norm_backward(dy, h, w, mean, rstd, dh=dh, need_dx=need[0],
                                            need_dweight=need[1], need_dbias=need[2])
        assert [t is not None for t in got] == [bool(k) for k in need]
        check_backward(got, dy, h, w, mean, rstd, dh, dt, wdt, wdt)
    got = flce.flce_layer_norm_backward(dy, h, None, mean, rstd, need_dx=False, bias_dtype=F32)
    assert got[0] is None and got[1] is None
    check_backward(got, dy, h, None, mean, rstd, None, dt, wdt, F32)


@pytest.mark.parametrize("N,H", [(3000, 520), (300, 520), (100, 20000), (5000, 1001)])
def test_backward_is_the_same_every_time(N, H):
    x, res, w, b, dy, dh = case(N, H, BF, F32, seed=3)
    y, h, mean, rstd = flce.flce_layer_norm(x, w, b, residual=res)
    a = flce.flce_layer_norm_backward(dy, h, w, mean, rstd, dh=dh)
    for _ in range(3):
        c = flce.flce_layer_norm_backward(dy, h, w, mean, rstd, dh=dh)
        assert all(torch.equal(p, q) for p, q in zip(a, c))


@pytest.mark.parametrize("parts", PARTS)
def test_autograd_matches_differences_of_the_definition(parts):
    """<grad, d> against central differences of the float64 definition: the step 1e-4
    leaves a truncation error of about 1e-8 of the third derivative's size and the
    float32 gradient an error of about 1e-6 of the terms."""
    N, H = 6, 200
    x, res, w, b, a, c = case(N, H, F32, F32, seed=4)
    leaves = [x] + [t if k else None for k, t in zip(parts, (res, w, b))]
    leaves = [t if t is None else t.requires_grad_() for t in leaves]
    x, res, w, b = leaves
    out = flce.layer_norm(x, w, b, eps=EPS, residual=res)
    y, h = out if res is not None else (out, None)
    ((y * a).sum() + (0 if h is None else (h * c).sum())).backward()
    rng = np.random.default_rng(5)

    def loss(p):
        yy, hh, _, _ = ref.layer_norm(p[0], p[2], p[3], EPS, p[1])
        return (yy * f64(a)).sum() + (0 if h is None else (hh * f64(c)).sum())
    for _ in range(4):
        d = [None if t is None else rng.standard_normal(tuple(t.shape)) for t in leaves]
        p = [None if t is None else f64(t) for t in leaves]
        up, down = ([None if u is None else u + s * v for u, v in zip(p, d)]
                    for s in (1e-4, -1e-4))
        num = (loss(up) - loss(down)) / 2e-4
        terms = [f64(t.grad) * v for t, v in zip(leaves, d) if t is not None]
        assert abs(sum(t.sum() for t in terms) - num) <= 1e-5 * sum(np.abs(t).sum() for t in terms)


def test_autograd_parts():
    x, res, w, b, a, _ = case(5, 64, F32, F32, seed=6)
    x.requires_grad_()
    y = flce.layer_norm(x, w, b)
    (y * 1.0).sum().backward()  # an expanded, strided gradient
    assert x.grad is not None and w.grad is None
    for who in range(4):  # one gradient alone
        leaves = [t.detach().clone().requires_grad_(i == who) for i, t in enumerate((x, res, w, b))]
        y, h = flce.layer_norm(leaves[0], leaves[2], leaves[3], residual=leaves[1])
        (y * a).sum().backward()
        assert [t.grad is not None for t in leaves] == [i == who for i in range(4)]
        mean, rstd = flce.flce_layer_norm(h.detach())[2:]
        want = flce.flce_layer_norm_backward(a, h.detach(), w, mean, rstd)
        want = (want[0], want[0], want[1], want[2])[who]
        assert torch.allclose(leaves[who].grad, want, rtol=1e-5, atol=1e-5)
    x2 = x.detach().clone().requires_grad_()
    y, h = flce.layer_norm(x2, w, b, residual=res)
    h.sum().backward()          # only the sum is used
    assert torch.equal(x2.grad, torch.ones_like(x2))
    x3 = x.detach().view(1, 5, 1, 64).requires_grad_()
    assert flce.layer_norm(x3, w).shape == (1, 5, 1, 64)
    b2 = b.to(BF).requires_grad_()  # a bias alone, of another type than x
    flce.layer_norm(x3, None, b2).sum().backward()
    assert b2.grad.dtype == BF and (b2.grad == 5).all()


def test_strided_rows_and_unaligned_views():
    g = torch.Generator().manual_seed(7)
    for dt in (BF, F32):
        big = torch.randn(6, 4, 400, generator=g).to(dt).cuda()
        w = torch.randn(384, generator=g).to(dt).cuda()
        b = torch.randn(384, generator=g).to(dt).cuda()
        for lo in (0, 1, 3, 8):
            x = big[:, -1, lo:lo + 384]         # the last token of each sequence
            r = big[:, 0, lo:lo + 384]
            p = flce.layer_norm_fp8(x, w, b, residual=r)
            c = flce.layer_norm_fp8(x.contiguous(), w.clone(), b.clone(), residual=r.contiguous())
            assert all(torch.equal(u.float(), v.float()) for u, v in zip(p, c))
            y, h, mean, rstd = flce.flce_layer_norm(x, w, b)
            y2, h2, mean2, rstd2 = flce.flce_layer_norm(x.contiguous(), w, b)
            assert torch.equal(y, y2) and torch.equal(rstd, rstd2) and torch.equal(mean, mean2)
            got = flce.flce_layer_norm_backward(r, h, w, mean, rstd)
            want = flce.flce_layer_norm_backward(r.contiguous(), h2, w, mean2, rstd2)
            # (the small backward adds in another order where rows are not aligned)
            for u, v in zip(got, want):
                assert torch.allclose(u.float(), v.float(), rtol=2 * rnd(dt), atol=1e-5)
        wu = torch.randn(385, generator=g).to(dt).cuda()[1:]  # unaligned parameters
        bu = torch.randn(385, generator=g).to(dt).cuda()[1:]
        x = big[:, 0, :384]
        assert torch.equal(flce.layer_norm(x, wu, bu), flce.layer_norm(x, wu.clone(), bu.clone()))
        assert torch.equal(flce.layer_norm(x, w, bu), flce.layer_norm(x, w, bu.clone()))
    x = torch.randn(64, 6, generator=g).cuda().t()  # columns instead of rows
    w = torch.ones(64, device="cuda")
    assert torch.equal(flce.layer_norm(x, w), flce.layer_norm(x.contiguous(), w))


@pytest.mark.parametrize("H", [64, 1000, 1001, 16384, 16388, 40000])
def test_the_sum_in_the_place_of_an_input(H):
    for dt in (BF, F32):
        x, res, w, b, _, _ = case(6, H, dt, dt, seed=8)
        for residual in (res, None):
            want = flce.flce_layer_norm(x, w, b, residual=residual, residual_out=torch.empty_like(x))
            want8 = flce.layer_norm_fp8(x, w, b, residual=residual,
                                        residual_out=torch.empty_like(x))
            for place in (0, 1):
                p, r = x.clone(), None if residual is None else residual.clone()
                if place and r is None:
                    continue
                got = flce.flce_layer_norm(p, w, b, residual=r, residual_out=(p, r)[place])
                p, r = x.clone(), None if residual is None else residual.clone()
                got8 = flce.layer_norm_fp8(p, w, b, residual=r, residual_out=(p, r)[place])
                assert got8[2] is (p, r)[place]
                for u, v in zip(want + want8, got + got8):
                    assert torch.equal(u.float(), v.float())


def test_writes_stay_inside():
    for H in (40, 1001, 3584, 16388):
        for dt in (BF, F32):
            x, res, w, b, _, _ = case(5, H, dt, dt, seed=9)
            buf = torch.full((7, H), 7.0, dtype=dt, device="cuda")
            flce.layer_norm_fp8(x, w, b, residual=res, residual_out=buf[1:6])
            assert (buf[0] == 7).all() and (buf[6] == 7).all()


def test_gradients_stay_inside_their_buffers():
    """The C call into the middle of larger buffers, workspace included."""
    from lm_head_linear_flce_gb300 import head_ops
    for N, H in ((5, 40), (70, 1001), (2500, 1000), (4, 16384), (70, 16400)):
        x, _, w, b, dy, _ = case(N, H, BF, BF, seed=10)
        y, h, mean, rstd = flce.flce_layer_norm(x, w, b)
        want = flce.flce_layer_norm_backward(dy, h, w, mean, rstd)
        size = head_ops._fn("flce_layer_norm_workspace_size")(N, H)
        ws = torch.full((size + 512,), 91, dtype=torch.uint8, device="cuda")
        dx = torch.full((N + 2, H), 7.0, dtype=BF, device="cuda")
        par = torch.full((2, H + 16), 7.0, dtype=BF, device="cuda")
        head_ops._call("flce_layer_norm_backward", 0, dy.data_ptr(), None, h.data_ptr(), H,
                       w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), N, H, 0, 0,
                       dx[1:].data_ptr(), par[0, 8:].data_ptr(), par[1, 8:].data_ptr(),
                       ws[256:].data_ptr(), size)
        assert (dx[0] == 7).all() and (dx[-1] == 7).all()
        assert (par[:, :8] == 7).all() and (par[:, -8:] == 7).all()
        assert (ws[:256] == 91).all() and (ws[-256:] == 91).all()
        for p, q in zip((dx[1:-1], par[0, 8:-8], par[1, 8:-8]), want):
            assert torch.equal(p, q)


def test_zero_rows_equal_values_and_non_finite_values():
    w, b = torch.ones(256, device="cuda", dtype=BF), torch.ones(256, device="cuda", dtype=BF)
    for shape in ((0, 256), (2, 0, 256)):
        x = torch.empty(shape, device="cuda", dtype=BF, requires_grad=True)
        wg, bg = w.clone().requires_grad_(), b.clone().requires_grad_()
        y = flce.layer_norm(x, wg, bg)
        y.sum().backward()
        assert y.shape == shape and (wg.grad == 0).all() and (bg.grad == 0).all()
        q, s = flce.layer_norm_fp8(x.detach(), w, b)
        assert q.shape == shape and s.shape == (*shape[:-1], 2)
    for H in (256, 1001, 16400):
        w, b = (torch.ones(H, device="cuda", dtype=BF) for _ in range(2))
        z = torch.full((2, H), 5.0, device="cuda", dtype=BF)  # no variance: the bias
        assert (flce.layer_norm(z, w, b) == 1).all()
        q, s = flce.layer_norm_fp8(z, w)
        assert (q.float() == 0).all() and torch.isfinite(s).all() and (s > 0).all()
        x = torch.randn(4, H, device="cuda").to(BF)
        x[1, 5] = float("nan")
        x[2, 200] = float("inf")
        y, _, mean, rstd = flce.flce_layer_norm(x, w, b)
        assert torch.isfinite(y[[0, 3]]).all() and torch.isnan(y[1:3]).all()
        assert torch.isnan(rstd[1:3]).all() and torch.isfinite(rstd[[0, 3]]).all()
        q, s = flce.layer_norm_fp8(x, w, b)
        assert torch.isfinite(q[[0, 3]].float()).all() and torch.isnan(q[1:3].float()).all()
        dy = torch.randn(4, H, device="cuda").to(BF)
        y, h, mean, rstd = flce.flce_layer_norm(x, w, b)
        dx, dw, db = flce.flce_layer_norm_backward(dy, h, w, mean, rstd)
        assert torch.isfinite(dx[[0, 3]]).all() and torch.isnan(dx[1:3]).all()
        assert torch.isfinite(db).all()  # (dbias does not see x)


def test_on_another_stream_and_in_a_graph():
    for N, H in ((64, 1024), (4000, 520)):
        x, res, w, b, dy, dh = case(N, H, BF, BF, seed=12)
        want = flce.layer_norm_fp8(x, w, b, residual=res)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            xx = x * 1
            got = flce.layer_norm_fp8(xx, w, b, residual=res)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(u.float(), v.float()) for u, v in zip(want, got))
        y, h, mean, rstd = flce.flce_layer_norm(x, w, b, residual=res)
        grads = flce.flce_layer_norm_backward(dy, h, w, mean, rstd, dh=dh)
        graph = torch.cuda.CUDAGraph()
        zx = torch.zeros_like(x)
        with torch.cuda.graph(graph):
            gy, gh, gm, gr = flce.flce_layer_norm(zx, w, b, residual=res)
            ggrads = flce.flce_layer_norm_backward(dy, gh, w, gm, gr, dh=dh)
        zx.copy_(x)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, y) and all(torch.equal(p, q) for p, q in zip(ggrads, grads))


def test_refusals():
    x, res, w, b, dy, _ = case(4, 64, BF, BF)
    s = torch.ones(4, device="cuda")
    for call in (lambda: flce.layer_norm(x, w[:63]), lambda: flce.layer_norm(x.half(), w),
                 lambda: flce.layer_norm(x, w, b[:63]), lambda: flce.layer_norm(x, w, b.float()),
                 lambda: flce.layer_norm(x, None, b.half()),
                 lambda: flce.layer_norm(x, w, residual=res[:3]),
                 lambda: flce.layer_norm(x, w, residual=res.float()),
                 lambda: flce.layer_norm_fp8(x, w, residual=res, residual_out=res[:, :32]),
                 lambda: flce.layer_norm(x, w.cpu()), lambda: flce.layer_norm(x, w, b.cpu()),
                 lambda: flce.flce_layer_norm_backward(dy[:2], x, w, s, s),
                 lambda: flce.flce_layer_norm_backward(dy, x, w, s[:3], s),
                 lambda: flce.flce_layer_norm_backward(dy, x, w, s, s[:3]),
                 lambda: flce.flce_layer_norm_backward(dy, x, w, s.to(BF), s),
                 lambda: flce.flce_layer_norm_backward(dy, x, None, s, s, bias_dtype=torch.half),
                 lambda: flce.flce_layer_norm_backward(dy.float(), x, w, s, s)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(flce.FlceError):  # the sum would overwrite a neighbour of x
        flce.layer_norm_fp8(x[1:3], w, residual_out=x[:2])
    with pytest.raises(flce.FlceError):
        flce.layer_norm(torch.zeros(1, 65537, device="cuda"))


def test_second_derivatives_are_refused():
    """The backward is not differentiable: a loss that holds a gradient raises, by
    whichever input it is differentiated, and does not lose the terms through it."""
    x, res, w, b, a, _ = case(4, 64, F32, F32, seed=13)
    for residual in (None, res):
        p, q, c = (t.clone().requires_grad_() for t in (x, w, b))
        out = flce.layer_norm(p, q, c, residual=residual)
        y, s = (out, None) if residual is None else out
        loss = (y * a).sum()
        got = torch.autograd.grad(loss + (0 if s is None else s.sum()), (p, q, c),
                                  create_graph=True)
        for g, by in ((got[0], p), (got[0], q), (got[1], p)):
            with pytest.raises(RuntimeError, match="cannot be differentiated again"):
                torch.autograd.grad(g.square().sum() + y.sum(), by, retain_graph=True)
        # dbias depends on dy alone, here through y
        loss = y.square().sum()
        (g,) = torch.autograd.grad(loss, c, create_graph=True)
        with pytest.raises(RuntimeError, match="cannot be differentiated again"):
            torch.autograd.grad(g.sum(), p, retain_graph=True)
    # a gradient that is used as a number, and a graph that is not differentiated again
    p = x.clone().requires_grad_()
    y = flce.layer_norm(p, w, b)
    (g,) = torch.autograd.grad(y.sum(), p, create_graph=True)
    (y.sum() * g.detach().sum()).backward()
    assert torch.isfinite(p.grad).all()


def test_a_written_tensor_counts_as_modified_and_one_that_wants_a_gradient_is_refused():
    x, res, w, b, _, _ = case(5, 64, BF, BF, seed=14)
    y, h = flce.layer_norm(x.requires_grad_(), w, b, residual=res)  # h is kept for the backward
    for call in (flce.layer_norm_fp8, flce.flce_layer_norm):
        buf = torch.empty_like(x)
        call(x.detach(), w, b, residual=res, residual_out=buf)
        assert buf._version == 1
    flce.layer_norm_fp8(res, w, b, residual=h.detach(), residual_out=h.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    leaf = torch.zeros_like(x).requires_grad_()
    for out in (leaf, leaf * 1):
        for call in (flce.layer_norm_fp8, flce.flce_layer_norm):
            with pytest.raises(ValueError, match="gradient"):
                call(x.detach(), w, b, residual=res, residual_out=out)
    with torch.no_grad():
        assert flce.layer_norm_fp8(x, w, b, residual=res, residual_out=leaf)[2] is leaf


def test_the_captured_backward_beside_a_living_eager_graph():
    """The explicit backward is what a graph captures; an eager graph of the same leaves
    lives on and gives the same gradients."""
    x, res, w, b, dy, _ = case(40, 256, BF, BF, seed=15)
    p, q = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = flce.layer_norm(p, q, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, h, mean, rstd = flce.flce_layer_norm(p.detach(), q.detach(), b)
        dx, dw, _ = flce.flce_layer_norm_backward(dy, h, q.detach(), mean, rstd)
    graph.replay()
    y.backward(dy)
    torch.cuda.synchronize()
    assert torch.equal(p.grad, dx)
    assert torch.allclose(q.grad.float(), dw.float(), rtol=2.0 ** -7, atol=1e-4)


@pytest.mark.parametrize("N,H", [(33000, 65536), (140000, 16384)])
def test_matrices_past_2_31_elements(N, H):
    """The last rows of a matrix are as they are by themselves (dx up to the rounding of
    sums in another order)."""
    g = torch.Generator(device="cuda").manual_seed(21)
    x = torch.randn(N, H, dtype=BF, device="cuda", generator=g)
    w, b = (torch.randn(H, dtype=BF, device="cuda", generator=g) for _ in range(2))
    y, h, mean, rstd = flce.flce_layer_norm(x, w, b)
    for part in (slice(N - 3, N), slice(0, 3)):
        y3, h3, m3, r3 = flce.flce_layer_norm(x[part].clone(), w, b)
        assert torch.equal(y[part], y3) and torch.equal(mean[part], m3)
    dx, dw, db = flce.flce_layer_norm_backward(y, h, w, mean, rstd)
    for part in (slice(N - 3, N), slice(0, 3)):
        d3 = flce.flce_layer_norm_backward(y[part].clone(), h[part].clone(), w, mean[part].clone(),
                                           rstd[part].clone())[0]
        assert torch.allclose(dx[part].float(), d3.float(), rtol=2.0 ** -7, atol=1e-4)
    # columns' sums: of the first one in 64 bits
    col = y[:, 0].double()
    n = (x[:, 0].double() - mean.double()) * rstd.double()
    for got, t in ((dw[0], col * n), (db[0], col)):
        tol = (N / 32 + 80) * U * t.abs().sum().item()
        assert abs(got.item() - t.sum().item()) <= tol + 1.01 * rnd(BF) * abs(t.sum().item())


def test_a_captured_training_step():
    """Forward and autograd's backward in a graph, after a warm-up on a side stream whose
    graph is gone; a replay follows new values."""
    x, res, w, b, a, _ = case(50, 384, F32, F32, seed=18)
    leaves = [t.clone().requires_grad_() for t in (x, res, w, b)]

    def step():
        y, h = flce.layer_norm(leaves[0], leaves[2], leaves[3], residual=leaves[1])
        return torch.autograd.grad((y * a).sum() + h.sum(), leaves)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (19, 20):
        with torch.no_grad():
            for t, v in zip(leaves, case(50, 384, F32, F32, seed=seed)):
                t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


@pytest.mark.parametrize("N,H", [(5, 200), (64, 3584), (700, 4096), (9, 1001)])
def test_bf16_gradient_against_the_forward_as_it_is(N, H):
    """The forward norms the sum as it is, the backward takes the sum as it was stored,
    rounded by up to e = 2^-8 of it.  Against the gradient of the forward, that is
    en = e rstd |h| on each n: |n| mean(|g| en) + en (|mean(g n)| + mean(|g| en)) of dx and
    |dy| en of each term of dweight; beside the errors that the backward has on the
    stored sum (see check_backward)."""
    x, res, w, b, dy, dh = case(N, H, BF, BF, seed=16, mean=1.0)
    y, h, mean, rstd = flce.flce_layer_norm(x, w, b, eps=EPS, residual=res)
    dx, dw, db = flce.flce_layer_norm_backward(dy, h, w, mean, rstd, dh=dh)
    s = f64(x) + f64(res)
    rdx, rdw, rdb = ref.layer_norm_backward(f64(dy), s, f64(w), EPS, f64(dh))
    n, _, m, r = ref.layer_norm(s, None, None, EPS)
    r, g, e, S = r[:, None], np.abs(f64(dy) * f64(w)), 1.01 * rnd(BF), sum_tol(H)
    en = e * r * np.abs(s) + 4 * U * r * (np.abs(s) + np.abs(m[:, None]))
    c2 = np.abs((f64(dy) * f64(w) * n).mean(1, keepdims=True))
    a3 = (g * en).mean(1, keepdims=True)
    big = g + g.mean(1, keepdims=True) + np.abs(n) * (g * np.abs(n)).mean(1, keepdims=True)
    # (rstd and mean are the forward's, off by tr and tm: within 16 S of n here)
    tol = r * (np.abs(n) * a3 + en * (c2 + a3) + (32 * S + 12 * U) * big) + 2 * U * np.abs(f64(dh))
    assert (np.abs(f64(dx) - rdx) <= tol + e * (np.abs(rdx) + tol)).all()
    d = np.abs(f64(dy))
    tol = (d * en).sum(0) + (N / 32 + 80) * U * (d * np.abs(n)).sum(0) + 32 * S * d.sum(0)
    assert (np.abs(f64(dw) - rdw) <= tol + e * (np.abs(rdw) + tol)).all()
    tol = (N / 32 + 80) * U * d.sum(0)
    assert (np.abs(f64(db) - rdb) <= tol + e * (np.abs(rdb) + tol)).all()
