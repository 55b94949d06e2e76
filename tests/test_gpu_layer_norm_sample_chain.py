"""Layer norm, LM head and sampling together, as a model with a layer norm uses them: a
training step and decode steps against the float64 definitions, captured, without
synchronisation, and the example's variants."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import head_ops as ref
from tests._parity import assert_grad, assert_loss

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def f64(t):
    return t.detach().double().cpu().numpy()


def test_training_step_through_layer_norm_and_loss():
    """The loss of the norm's bf16 output and its gradients, chained by the float64
    definitions (the tolerances are those of the loss and gradients by themselves: the
    norm's backward takes a row's parts along two directions away and rescales it).  h as
    it is stored is what the backward norms, and its statistics are those of x + r
    before it was rounded: 2^-9 of h at most on average over a row."""
    N, H, V = 300, 256, 1000
    g = torch.Generator().manual_seed(0)
    x, r = torch.randn(N, H, generator=g).to(BF), torch.randn(N, H, generator=g).to(BF)
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(BF)
    b = (0.2 * torch.randn(H, generator=g)).to(BF)
    W = (0.05 * torch.randn(V, H, generator=g)).to(BF)
    labels = torch.randint(0, V, (N,), generator=g)
    labels[::7] = -100
    leaves = [t.cuda().requires_grad_() for t in (x, r, w, b, W)]
    y, h = flce.layer_norm(leaves[0], leaves[2], leaves[3], residual=leaves[1])
    loss = flce.linear_cross_entropy(y, leaves[4], labels.cuda())
    loss.backward()
    yb = y.detach().cpu()
    want = oracle.forward(yb, W, labels)
    dy, dW = oracle.backward(yb, W, labels)
    assert_loss(loss.item(), want["loss"])
    dx, dw, db = ref.layer_norm_backward(dy, f64(h), f64(w), 1e-5)
    for name, t, d in (("x", leaves[0], dx), ("residual", leaves[1], dx), ("weight", leaves[2], dw),
                       ("bias", leaves[3], db), ("head", leaves[4], dW)):
        assert_grad(name, f64(t.grad), d)


def parts(B, H, V, seed):
    g = torch.Generator().manual_seed(seed)

    def t(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(BF).cuda()
    x, r, w, b, W = t(B, H), t(B, H), 1 + t(H, std=0.2), t(H, std=0.2), t(V, H, std=0.05)
    tokens = torch.randint(0, V, (B, 64), generator=g).cuda()
    allowed = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g).int().cuda()
    lim = dict(temperature=torch.rand(B, generator=g).cuda() + 0.3,
               top_k=torch.randint(0, 200, (B,), generator=g).int().cuda(),
               top_p=torch.rand(B, generator=g).cuda(),
               min_p=0.1 * torch.rand(B, generator=g).cuda())
    return x, r, w, b, flce.quantize_fp8(W), tokens, allowed, torch.rand(B, generator=g).cuda(), lim


@pytest.mark.parametrize("B", [1, 5, 100])
def test_decode_step(B):
    """Each stage's output feeds the next stage's float64 definition."""
    H, V = 512, 3001
    x, r, w, b, (Wq, Ws), tokens, allowed, u, lim = parts(B, H, V, B)
    stream = r.clone()
    q, s, h = flce.layer_norm_fp8(x, w, b, residual=stream, residual_out=stream)
    assert h is stream and torch.equal(stream, (x.float() + r.float()).to(BF))
    y = ref.layer_norm(f64(x), f64(w), f64(b), 1e-5, f64(r))[0]
    sx = ref.expand_scale(f64(s), B, H, 1)
    assert (np.abs(f64(q) * sx - y) <= 2.0 ** -4 * 1.01 * np.abs(y) + 2.0 ** -9 * sx).all()
    z = flce.matmul_fp8(q, s, Wq, Ws)
    l = flce.process_logits(z, tokens=tokens, allowed=allowed,
                            frequency_penalty=torch.full((B,), 0.3, device="cuda"),
                            out_dtype=torch.float32)
    got = flce.sample_logits(l, u, **lim).tolist()
    rows, bits = f64(l), allowed.cpu().numpy().view(np.uint32)
    e = 2.0 ** -28 + V * 2.0 ** -42
    for i, token in enumerate(got):
        assert bits[i, token // 32] >> np.uint32(token % 32) & 1  # the grammar allows it
        T, k, p, m = (lim[n][i].item() for n in ("temperature", "top_k", "top_p", "min_p"))
        assert any(ref.sample(rows[i], u[i].item() + du, T, k, p + dp, m) == token
                   for du in (0, -e, e) for dp in (0, -e, e))


def step(x, r, w, b, W8, tokens, allowed, u, lim):
    q, s, h = flce.layer_norm_fp8(x, w, b, residual=r)
    z = flce.matmul_fp8(q, s, *W8)
    z = flce.process_logits(z, tokens=tokens, allowed=allowed, out_dtype=torch.float32)
    return h, flce.sample_logits(z, u, **lim)


def test_decode_steps_in_two_graphs():
    """Captured steps follow what is written into their buffers, two graphs in turn and
    at once on two streams."""
    x, r, w, b, W8, tokens, allowed, u, lim = parts(6, 256, 20000, 9)
    x2, u2 = x.clone(), u.clone()
    step(x, r, w, b, W8, tokens, allowed, u, lim)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = step(x, r, w, b, W8, tokens, allowed, u, lim)
    with torch.cuda.graph(g2):
        o2 = step(x2, r, w, b, W8, tokens, allowed, u2, lim)
    side = torch.cuda.Stream()
    for k in range(4):
        x.normal_(), x2.normal_(), u.uniform_(), u2.uniform_()
        lim["temperature"].uniform_(0.2, 1.0)
        torch.cuda.synchronize()
        g1.replay()
        with torch.cuda.stream(side):
            g2.replay()
        torch.cuda.synchronize()
        for o, a, v in ((o1, x, u), (o2, x2, u2)):
            want = step(a, r, w, b, W8, tokens, allowed, v, lim)
            assert all(torch.equal(p, q) for p, q in zip(o, want))


@pytest.mark.parametrize("B", [1, 40, 300])
def test_calls_in_a_row_wait_for_one_another(B):
    """Each call reads what the one before wrote, in memory used again and again, with no
    synchronisation between them: the same bits as with one after every call."""
    H, V, steps = 640, 4016, 25
    x, r, w, b, W8, tokens, allowed, u, lim = parts(B, H, V, B)
    g = torch.Generator().manual_seed(B)
    embedding = torch.randn(V, H, generator=g).to(BF).cuda()

    def chain(wait):
        a, stream, out = x, r.clone(), []
        for _ in range(steps):
            q, s, _ = flce.layer_norm_fp8(a, w, b, residual=stream, residual_out=stream)
            wait()
            z = flce.matmul_fp8(q, s, *W8, out_dtype=torch.float32)
            wait()
            flce.process_logits(z, tokens=tokens, allowed=allowed, out=z)
            wait()
            token = flce.sample_logits(z, u, **lim)
            wait()
            out.append(token)
            y, h, mean, rstd = flce.flce_layer_norm(embedding[token], w, b, residual=stream)
            wait()
            dx, dw, db = flce.flce_layer_norm_backward(y, h, w, mean, rstd)
            wait()
            a = flce.flce_layer_norm(dx, dw, db)[0]
            wait()
            stream = flce.flce_layer_norm(stream, w)[0]
        torch.cuda.synchronize()
        return torch.stack(out), a, stream
    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(chain(lambda: None), want))
    assert (want[0] >= 0).all() and torch.isfinite(want[1].float()).all()


@pytest.mark.parametrize("more", [["--layer-norm"], ["--layer-norm", "--batch", "1"],
                                  ["--batch", "9", "--temperature", "0.5"]])
def test_example_runs(more):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "lm_head_step.py"),
                        "--hidden", "256", "--vocab", "4000", "--tokens", "64", "--steps", "4"]
                       + more, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "training: loss" in r.stdout and "decoded:" in r.stdout
