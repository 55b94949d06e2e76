"""RMS norm (forward, 8-bit output, backward) and the block quantiser against
the float64 definitions.

Tolerances.  u = 2^-24 is the float32 rounding unit, e the rounding of the
output type (2^-8 for bf16, u for float32).  A sum of squares over H columns
goes through at most H/256 + 16 additions, so rstd is within (H/512 + 12) u and y
within that plus 4 u and e, relative to |y|.  A gradient's error is relative to
the row's largest term, since g and h * rstd^2 * mean(g h) may cancel; dweight's to
the column's sum of |terms|."""
import numpy as np
import pytest
import torch

from oracle import head_ops as ref

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def rnd(dt):
    return 2.0 ** -8 if dt == BF else U


def f64(t):
    return t.detach().double().cpu().numpy()


def sum_tol(H):
    return (H / 512 + 16) * U


def case(N, H, dt, wdt, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed)

    def t(std):
        return (torch.randn(N, H, generator=g) * std).to(dt).cuda()
    x, res = t(1.0), t(3.0) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(wdt).cuda()
    return x, res, w, t(0.1), t(0.2)


SHAPES = [(1, 1), (1, 3584), (3, 127), (5, 128), (4, 129), (33, 1001), (257, 512), (7, 2056),
          (2, 8192), (3, 65536), (300, 8), (1021, 264), (2, 16388)]


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("N,H", SHAPES)
def test_forward(N, H, dt, wdt):
    x, res, w, _, _ = case(N, H, dt, wdt)
    y, h, rstd = flce.flce_rms_norm(x, w, eps=EPS, residual=res)
    assert torch.equal(h, (x.float() + res.float()).to(dt))  # rounded once
    ry, _, rr = ref.rms_norm(f64(x), f64(w), EPS, f64(res))
    assert (np.abs(f64(rstd) / rr - 1) <= sum_tol(H)).all()
    # h itself is rounded to float32 before it is squared: 2 u on y
    assert (np.abs(f64(y) - ry) <= (sum_tol(H) + 6 * U + 1.01 * rnd(dt)) * np.abs(ry)
            + 2 * U * np.abs(f64(x))  # x + residual may cancel
            * rr[:, None] * np.abs(f64(w))).all()
    y2, h2, rstd2 = flce.flce_rms_norm(x, w, eps=EPS)
    assert h2 is x
    ry, _, rr = ref.rms_norm(f64(x), f64(w), EPS)
    assert (np.abs(f64(y2) - ry) <= (sum_tol(H) + 6 * U + 1.01 * rnd(dt)) * np.abs(ry)).all()


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("N,H", SHAPES)
def test_fp8_output(N, H, dt, wdt):
    x, res, w, _, _ = case(N, H, dt, wdt, seed=1)
    q, s, h = flce.rms_norm_fp8(x, w, eps=EPS, residual=res)
    assert q.shape == x.shape and s.shape == (N, -(-H // 128)) and h.shape == x.shape
    assert torch.equal(h, (x.float() + res.float()).to(dt))
    ry, _, rr = ref.rms_norm(f64(x), f64(w), EPS, f64(res))
    off = (sum_tol(H) + 6 * U) * np.abs(ry) + 2 * U * np.abs(f64(x)) * rr[:, None] * np.abs(f64(w))
    amax = ref.block_amax(ry, 1)
    tol = ref.block_amax(off, 1) + 2 * U * amax
    assert (np.abs(f64(s) * 448 - amax) <= tol).all()
    # half an e4m3 step of the value (2^-4 of it, 2^-10 of the scale near zero)
    sx = ref.expand_scale(f64(s), N, H, 1)
    err = np.abs(f64(q) * sx - ry)
    assert (err <= (2.0 ** -4 * np.abs(ry) + 2.0 ** -10 * sx) * 1.001 + off
            + ref.expand_scale(tol, N, H, 1)).all()
    assert f64(q).__abs__().max() <= 448


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("N,H", SHAPES)
def test_backward(N, H, dt, wdt):
    x, res, w, dy, dh = case(N, H, dt, wdt, seed=2)
    y, h, rstd = flce.flce_rms_norm(x, w, eps=EPS, residual=res)
    for extra in (dh, None):
        dx, dw = flce.flce_rms_norm_backward(dy, h, w, rstd, dh=extra)
        # the gradient of the norm of the stored h: rstd is given, so the
        # formula is taken with it
        r, g, hh = f64(rstd)[:, None], f64(dy) * f64(w), f64(h)
        m = (g * hh).mean(1, keepdims=True)
        rdx = r * (g - hh * r ** 2 * m) + (0 if extra is None else f64(extra))
        big = r * np.abs(g) + r ** 3 * np.abs(hh) * np.abs(g * hh).mean(1, keepdims=True) \
            + (0 if extra is None else np.abs(f64(extra)))
        assert (np.abs(f64(dx) - rdx) <= (sum_tol(H) + 8 * U) * big
                + 1.01 * rnd(dt) * np.abs(rdx)).all()
        t = f64(dy) * hh * r
        tol = (N / 32 + 80) * U * np.abs(t).sum(0) + 1.01 * rnd(wdt) * np.abs(t.sum(0))
        assert (np.abs(f64(dw) - t.sum(0)) <= tol).all()
    only_dx, none = flce.flce_rms_norm_backward(dy, h, w, rstd, need_dweight=False)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = flce.flce_rms_norm_backward(dy, h, w, rstd, need_dx=False)
    assert none is None and torch.equal(only_dw, dw)


def test_backward_is_the_same_every_time():
    x, res, w, dy, dh = case(3000, 520, BF, F32, seed=3)
    y, h, rstd = flce.flce_rms_norm(x, w, residual=res)
    a = flce.flce_rms_norm_backward(dy, h, w, rstd, dh=dh)
    for _ in range(3):
        b = flce.flce_rms_norm_backward(dy, h, w, rstd, dh=dh)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_autograd_matches_differences_of_the_definition():
    """<grad, d> against central differences of the float64 definition: the
    step 1e-4 leaves a truncation error of about 1e-8 of the third derivative's
    size and the float32 gradient an error of about 1e-6 of the terms."""
    N, H = 6, 200
    x, res, w, a, b = case(N, H, F32, F32, seed=4)
    x, res, w = x.requires_grad_(), res.requires_grad_(), w.requires_grad_()
    y, h = flce.rms_norm(x, w, eps=EPS, residual=res)
    ((y * a).sum() + (h * b).sum()).backward()
    assert torch.equal(x.grad, res.grad)
    rng = np.random.default_rng(5)

    def loss(x_, r_, w_):
        yy, hh, _ = ref.rms_norm(x_, w_, EPS, r_)
        return (yy * f64(a)).sum() + (hh * f64(b)).sum()
    for _ in range(4):
        d = [rng.standard_normal(s) for s in ((N, H), (N, H), (H,))]
        e = 1e-4
        p = [f64(t) for t in (x, res, w)]
        num = (loss(*[u + e * v for u, v in zip(p, d)]) -
               loss(*[u - e * v for u, v in zip(p, d)])) / (2 * e)
        got = sum((f64(t.grad) * v).sum() for t, v in zip((x, res, w), d))
        size = sum((np.abs(f64(t.grad) * v)).sum() for t, v in zip((x, res, w), d))
        assert abs(got - num) <= 1e-5 * size


def test_autograd_parts():
    x, res, w, a, _ = case(5, 64, F32, F32, seed=6)
    x.requires_grad_()
    y = flce.rms_norm(x, w)
    (y * 1.0).sum().backward()  # an expanded, strided gradient
    assert x.grad is not None and w.grad is None
    x2 = x.detach().clone().requires_grad_()
    y, h = flce.rms_norm(x2, w, residual=res)
    h.sum().backward()          # only the sum is used
    assert torch.equal(x2.grad, torch.ones_like(x2))
    x3 = x.detach().view(1, 5, 1, 64).requires_grad_()
    assert flce.rms_norm(x3, w).shape == (1, 5, 1, 64)


def test_strided_rows_and_unaligned_views():
    g = torch.Generator().manual_seed(7)
    for dt in (BF, F32):
        big = torch.randn(6, 4, 400, generator=g).to(dt).cuda()
        w = torch.randn(384, generator=g).to(dt).cuda()
        for lo in (0, 1, 3, 8):
            x = big[:, -1, lo:lo + 384]         # the last token of each sequence
            r = big[:, 0, lo:lo + 384]
            a = flce.rms_norm_fp8(x, w, residual=r)
            b = flce.rms_norm_fp8(x.contiguous(), w.clone(), residual=r.contiguous())
            for u, v in zip(a, b):
                assert torch.equal(u.float(), v.float())
            y, h, rstd = flce.flce_rms_norm(x, w)
            y2, h2, rstd2 = flce.flce_rms_norm(x.contiguous(), w)
            assert torch.equal(y, y2) and torch.equal(rstd, rstd2)
            dx, dw = flce.flce_rms_norm_backward(r, h, w, rstd)
            dx2, dw2 = flce.flce_rms_norm_backward(r.contiguous(), h2, w, rstd2)
            assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        wu = torch.randn(385, generator=g).to(dt).cuda()[1:]  # an unaligned weight
        x = big[:, 0, :384]
        assert torch.equal(flce.rms_norm(x, wu), flce.rms_norm(x, wu.clone()))
    x = torch.randn(64, 6, generator=g).cuda().t()  # columns instead of rows
    w = torch.ones(64, device="cuda")
    assert torch.equal(flce.rms_norm(x, w), flce.rms_norm(x.contiguous(), w))


@pytest.mark.parametrize("H", [128, 1000, 1001, 40000])
def test_residual_in_place(H):
    x, res, w, _, _ = case(9, H, BF, BF, seed=8)
    want = flce.rms_norm_fp8(x, w, residual=res)
    mine = res.clone()
    got = flce.rms_norm_fp8(x, w, residual=mine, residual_out=mine)
    assert got[2] is mine
    for u, v in zip(want, got):
        assert torch.equal(u.float(), v.float())


def test_writes_stay_inside():
    for H in (40, 1001, 3584):
        for dt in (BF, F32):
            x, res, w, _, _ = case(5, H, dt, dt, seed=9)
            buf = torch.full((7, H), 7.0, dtype=dt, device="cuda")
            flce.rms_norm_fp8(x, w, residual=res, residual_out=buf[1:6])
            assert (buf[0] == 7).all() and (buf[6] == 7).all()


def test_zero_rows_zero_values_and_non_finite_values():
    w = torch.ones(256, device="cuda", dtype=BF)
    for shape in ((0, 256), (2, 0, 256)):
        x = torch.empty(shape, device="cuda", dtype=BF, requires_grad=True)
        wg = w.clone().requires_grad_()
        y = flce.rms_norm(x, wg)
        y.sum().backward()
        assert y.shape == shape and (wg.grad == 0).all()
        q, s = flce.rms_norm_fp8(x.detach(), w)
        assert q.shape == shape and s.shape == (*shape[:-1], 2)
    z = torch.zeros(2, 256, device="cuda", dtype=BF)
    q, s = flce.rms_norm_fp8(z, w)
    assert (q.float() == 0).all() and torch.isfinite(s).all() and (s > 0).all()
    assert (flce.rms_norm(z, w) == 0).all()
    x = torch.ones(4, 256, device="cuda", dtype=BF)
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    y = flce.rms_norm(x, w)
    assert torch.isfinite(y[[0, 3]]).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 200]) and (y[2, :128] == 0).all()
    q, s = flce.rms_norm_fp8(x, w)
    assert torch.isfinite(q[[0, 3]].float()).all() and torch.isnan(q[1].float()).all()
    assert torch.isnan(q[2, 200].float())


# ------------------------------------------------------------ quantiser
def np_quantize(x, block_rows):
    """Exactly the documented float32 steps."""
    R, K = x.shape
    amax = ref.block_amax(x.astype(np.float64), block_rows).astype(np.float32)
    inv = np.float32(448) / amax
    scaled = (x.astype(np.float32) * ref.expand_scale(inv, R, K, block_rows).astype(np.float32))
    return ref.round_e4m3(scaled.astype(np.float64)), amax / np.float32(448)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 128), (127, 129), (128, 128), (129, 256), (300, 1000),
                                 (5, 2056), (1000, 64), (257, 4096)])
def test_quantize_bit_for_bit(R, K, block_rows, dt):
    g = torch.Generator().manual_seed(R + K)
    x = (torch.randn(R, K, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))).to(dt)
    x[R // 2] = 0
    q, s = flce.quantize_fp8(x.cuda(), block_rows=block_rows)
    rq, rs = np_quantize(x.float().numpy(), block_rows)
    assert q.shape == (R, K) and s.shape == rs.shape
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(f64(q), rq)


def test_quantize_strides_values_and_shapes():
    g = torch.Generator().manual_seed(11)
    big = torch.randn(300, 520, generator=g).cuda()
    for lo in (0, 1, 4):
        v = big[:, lo:lo + 512]
        for br in (1, 128):
            a, b = flce.quantize_fp8(v, br), flce.quantize_fp8(v.contiguous(), br)
            assert torch.equal(a[0].float(), b[0].float()) and torch.equal(a[1], b[1])
    q, s = flce.quantize_fp8(big.view(3, 100, 520), block_rows=1)
    assert q.shape == (3, 100, 520) and s.shape == (3, 100, 5)
    q, s = flce.quantize_fp8(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 1)
    x = torch.zeros(2, 256, device="cuda")
    x[0, 3], x[1, 130] = float("nan"), 1e-38
    q, s = flce.quantize_fp8(x, block_rows=1)
    assert torch.isnan(q[0, 3].float()) and torch.isfinite(s).all() and (s > 0).all()
    assert (q[0, 4:].float() == 0).all()
    x[0, 3] = float("inf")
    q, s = flce.quantize_fp8(x, block_rows=1)
    assert torch.isinf(s[0, 0]) and torch.isfinite(s[0, 1])


def test_on_another_stream_and_in_a_graph():
    x, res, w, dy, dh = case(64, 1024, BF, BF, seed=12)
    want = flce.rms_norm_fp8(x, w, residual=res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        xx = x * 1
        got = flce.rms_norm_fp8(xx, w, residual=res)
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip(want, got):
        assert torch.equal(u.float(), v.float())
    y, h, rstd = flce.flce_rms_norm(x, w, residual=res)
    dx, dw = flce.flce_rms_norm_backward(dy, h, w, rstd, dh=dh)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gh, gr = flce.flce_rms_norm(x, w, residual=res)
        gdx, gdw = flce.flce_rms_norm_backward(dy, gh, w, gr, dh=dh)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gy, y) and torch.equal(gdx, dx) and torch.equal(gdw, dw)


def test_refusals():
    x, res, w, dy, _ = case(4, 64, BF, BF)
    for call in (lambda: flce.rms_norm(x, w[:63]), lambda: flce.rms_norm(x.half(), w),
                 lambda: flce.rms_norm(x, w, residual=res[:3]),
                 lambda: flce.rms_norm(x, w, residual=res.float()),
                 lambda: flce.rms_norm_fp8(x, w, residual=res, residual_out=res[:, :32]),
                 lambda: flce.rms_norm(x, w.cpu()),
                 lambda: flce.flce_rms_norm_backward(dy[:2], x, w, torch.ones(4, device="cuda")),
                 lambda: flce.flce_rms_norm_backward(dy, x, w, torch.ones(3, device="cuda")),
                 lambda: flce.quantize_fp8(x, block_rows=32),
                 lambda: flce.quantize_fp8(x.view(2, 2, 64))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(flce.FlceError):  # the sum would overwrite the weight's neighbour x
        flce.rms_norm_fp8(x[1:3], w, residual_out=x[:2])


@pytest.mark.parametrize("H", [64, 1001, 16384, 16388, 40000])
def test_sum_in_the_place_of_x(H):
    for dt in (BF, F32):
        x, res, w, _, _ = case(6, H, dt, dt, seed=17)
        for residual in (res, None):
            want = flce.flce_rms_norm(x, w, residual=residual, residual_out=torch.empty_like(x))
            want8 = flce.rms_norm_fp8(x, w, residual=residual, residual_out=torch.empty_like(x))
            mine = x.clone()
            got = flce.flce_rms_norm(mine, w, residual=residual, residual_out=mine)
            mine = x.clone()
            got8 = flce.rms_norm_fp8(mine, w, residual=residual, residual_out=mine)
            for a, b in zip(want + want8, got + got8):
                assert torch.equal(a.float(), b.float())


def test_second_derivatives_are_refused():
    """The backward is not differentiable: a loss that holds a gradient raises,
    by whichever input it is differentiated, and does not lose the terms that go
    through it."""
    x, res, w, a, _ = case(4, 64, F32, F32, seed=13)
    ones = torch.ones_like(a)
    for residual in (None, res):
        rstd = flce.flce_rms_norm(x, w, residual=residual)[2]
        h = x if residual is None else x + residual
        want = flce.flce_rms_norm_backward(a, h, w, rstd, dh=None if residual is None else ones)
        for power in (1, 2):  # a gradient dy that is given, and one that depends on y
            p, q = x.clone().requires_grad_(), w.clone().requires_grad_()
            out = flce.rms_norm(p, q, residual=residual)
            y, s = (out, None) if residual is None else out
            loss = (y.pow(power) * (a if power == 1 else a / (2 * y.detach()))).sum()
            got = torch.autograd.grad(loss + (0 if s is None else s.sum()), (p, q),
                                      create_graph=True)
            for g, t in zip(got, want):  # the gradient itself is as ever
                assert torch.allclose(g, t, rtol=1e-5, atol=1e-5)
            for g, by in ((got[0], p), (got[0], q), (got[1], p)):
                with pytest.raises(RuntimeError, match="cannot be differentiated again"):
                    torch.autograd.grad(g.square().sum() + y.sum(), by, retain_graph=True)
        # dweight does not depend on the weight, where dy is given
        q = w.clone().requires_grad_()
        out = flce.rms_norm(x, q, residual=residual)
        y = out if residual is None else out[0]
        (g,) = torch.autograd.grad((y * a).sum(), q, create_graph=True)
        assert torch.equal(torch.autograd.grad(g.sum() + (y * a).sum(), q)[0], g)
    # a gradient that is used as a number, and a graph that is not differentiated again
    p = x.clone().requires_grad_()
    y = flce.rms_norm(p, w)
    (g,) = torch.autograd.grad(y.sum(), p, create_graph=True)
    (y.sum() * g.detach().sum()).backward()
    assert torch.isfinite(p.grad).all()


def test_a_written_tensor_counts_as_modified():
    """Autograd sees what residual_out overwrites."""
    x, res, w, _, _ = case(5, 64, BF, BF, seed=14)
    y, h = flce.rms_norm(x.requires_grad_(), w, residual=res)  # h is kept for the backward
    for call in (flce.rms_norm_fp8, flce.flce_rms_norm):
        buf = torch.empty_like(x)
        call(x.detach(), w, residual=res, residual_out=buf)
        assert buf._version == 1
    flce.rms_norm_fp8(res, w, residual=h.detach(), residual_out=h.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    with torch.inference_mode():  # tensors without a version
        buf = torch.empty_like(x)
        assert flce.rms_norm_fp8(x, w, residual=res, residual_out=buf)[2] is buf


def test_an_output_that_wants_a_gradient_is_refused():
    x, res, w, _, _ = case(4, 64, BF, BF, seed=15)
    leaf = torch.zeros_like(x).requires_grad_()
    for out in (leaf, leaf * 1):
        for call in (flce.rms_norm_fp8, flce.flce_rms_norm):
            with pytest.raises(ValueError, match="gradient"):
                call(x, w, residual=res, residual_out=out)
    with torch.no_grad():
        assert flce.rms_norm_fp8(x, w, residual=res, residual_out=leaf)[2] is leaf
    assert torch.equal(leaf.detach(), (x.float() + res.float()).to(BF))


@pytest.mark.parametrize("N,H", [(5, 200), (64, 3584), (700, 4096), (9, 1001)])
def test_bf16_gradient_against_the_forward_as_it_is(N, H):
    """The forward norms the sum as it is, the backward takes the sum as it was
    stored, rounded by up to e = 2^-8.  Against the gradient of the forward, that
    is e of each place where the sum stands: r^3 |h| (|m| + mean |g h|) of dx, with
    m = mean(g h), and r |dy h| of each term of dweight; beside the errors that the
    backward has on the stored sum (see test_backward)."""
    x, res, w, dy, dh = case(N, H, BF, BF, seed=16)
    y, h, rstd = flce.flce_rms_norm(x, w, eps=EPS, residual=res)
    dx, dw = flce.flce_rms_norm_backward(dy, h, w, rstd, dh=dh)
    s = f64(x) + f64(res)
    rdx, rdw = ref.rms_norm_backward(f64(dy), s, f64(w), EPS, f64(dh))
    r = 1 / np.sqrt((s * s).mean(1, keepdims=True) + EPS)
    g, e = f64(dy) * f64(w), 1.01 * rnd(BF)
    m, am = (g * s).mean(1, keepdims=True), np.abs(g * s).mean(1, keepdims=True)
    big = r * np.abs(g) + r ** 3 * np.abs(s) * am + np.abs(f64(dh))
    tol = e * r ** 3 * np.abs(s) * (np.abs(m) + (1 + e) * am) + (sum_tol(H) + 12 * U) * big
    assert (np.abs(f64(dx) - rdx) <= tol + e * (np.abs(rdx) + tol)).all()
    t = np.abs(f64(dy) * s * r).sum(0)
    tol = (e + (N / 32 + 80 + H / 256) * U) * t
    assert (np.abs(f64(dw) - rdw) <= tol + e * (np.abs(rdw) + tol)).all()
