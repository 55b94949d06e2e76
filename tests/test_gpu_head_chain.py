"""The operators around the LM head together: a training step through the norm
and the fused cross-entropy against the float64 definitions, a decode step
through the 8-bit head against the same chain in float64, and the example."""
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


def test_training_step_through_norm_and_loss():
    """The loss of the norm's bf16 output and its gradients, chained by the
    float64 definitions (the tolerances are those of the loss and gradients by
    themselves: the norm's backward only rescales rows)."""
    N, H, V = 300, 256, 1000
    g = torch.Generator().manual_seed(0)
    x, r = torch.randn(N, H, generator=g).to(BF), torch.randn(N, H, generator=g).to(BF)
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(BF)
    W = (0.05 * torch.randn(V, H, generator=g)).to(BF)
    labels = torch.randint(0, V, (N,), generator=g)
    labels[::7] = -100
    leaves = [t.cuda().requires_grad_() for t in (x, r, w, W)]
    y, h = flce.rms_norm(leaves[0], leaves[2], residual=leaves[1])
    loss = flce.linear_cross_entropy(y, leaves[3], labels.cuda())
    loss.backward()
    yb = y.detach().cpu()
    want = oracle.forward(yb, W, labels)
    dy, dW = oracle.backward(yb, W, labels)
    assert_loss(loss.item(), want["loss"])
    dx, dw = ref.rms_norm_backward(dy, f64(h), f64(w), 1e-6)
    for name, t, d in (("x", leaves[0], dx), ("residual", leaves[1], dx), ("norm", leaves[2], dw),
                       ("head", leaves[3], dW)):
        assert_grad(name, f64(t.grad), d)


@pytest.mark.parametrize("B", [1, 5, 100])
def test_decode_step(B):
    """Each stage's output feeds the next stage's float64 definition."""
    H, V, L = 512, 3001, 40
    g = torch.Generator().manual_seed(B)
    x, r = torch.randn(B, H, generator=g).to(BF).cuda(), torch.randn(B, H, generator=g).to(BF).cuda()
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(BF).cuda()
    W = (0.05 * torch.randn(V, H, generator=g)).to(BF).cuda()
    Wq, Ws = flce.quantize_fp8(W)
    stream = r.clone()
    q, s, h = flce.rms_norm_fp8(x, w, residual=stream, residual_out=stream)
    assert h is stream and torch.equal(stream, (x.float() + r.float()).to(BF))
    z = flce.matmul_fp8(q, s, Wq, Ws)
    zr, mag = ref.matmul_fp8(f64(q), f64(s), f64(Wq), f64(Ws))
    assert (np.abs(f64(z) - zr) <= 2.0 ** -15 * mag + 1.01 * 2.0 ** -8 * np.abs(zr)).all()
    # against the bf16 head: two roundings to 8 bits, each 2^-4 at most of a
    # value, add up like independent errors over the row
    y, _, _ = ref.rms_norm(f64(x), f64(w), 1e-6, f64(r))
    full = y @ f64(W).T
    assert np.linalg.norm(f64(z) - full) <= 0.06 * np.linalg.norm(full)
    tokens = torch.randint(0, V, (B, L), generator=g)
    pen = torch.full((B,), 1.3)
    allowed = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g).int()
    out = flce.process_logits(z, tokens=tokens.cuda(), repetition_penalty=pen.cuda(),
                              allowed=allowed.cuda(), out_dtype=torch.float32)
    want = ref.process_logits(f64(z), tokens=tokens.numpy(), repetition=pen.numpy(),
                              allowed=allowed.numpy())
    fin = np.isfinite(want)
    got = f64(out)
    assert np.array_equal(fin, np.isfinite(got))
    assert (np.abs(got[fin] - want[fin]) <= 2.0 ** -22 * np.abs(want[fin])).all()


def test_decode_step_in_a_graph():
    """A captured step follows new inputs and lengths written into its buffers."""
    B, H, V = 3, 256, 2000
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, H, generator=g).to(BF).cuda()
    w = torch.ones(H, dtype=BF, device="cuda")
    Wq, Ws = flce.quantize_fp8((0.05 * torch.randn(V, H, generator=g)).to(BF).cuda())
    tokens = torch.randint(0, V, (B, 64), generator=g).cuda()
    lengths = torch.tensor([1, 5, 9], dtype=torch.int32, device="cuda")
    freq = torch.ones(B, device="cuda")

    def step():
        q, s = flce.rms_norm_fp8(x, w)
        return flce.process_logits(flce.matmul_fp8(q, s, Wq, Ws), tokens=tokens, lengths=lengths,
                                   frequency_penalty=freq, out_dtype=torch.float32)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(torch.randn(B, H, generator=g).to(BF))
        lengths += 7
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "lm_head_step.py"),
                        "--hidden", "256", "--vocab", "4000", "--tokens", "64", "--steps", "4"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "training: loss" in r.stdout and "decoded:" in r.stdout


@pytest.mark.parametrize("B", [1, 40, 200])
def test_calls_in_a_row_wait_for_one_another(B):
    """Each call reads what the one before wrote, in memory used again and again,
    with no synchronisation between them: the same bits as with one after every
    call."""
    H, V, L, steps = 640, 4016, 9, 30
    g = torch.Generator().manual_seed(B)
    x = torch.randn(B, H, generator=g).to(BF).cuda()
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(BF).cuda()
    Wq, Ws = flce.quantize_fp8((0.05 * torch.randn(V, H, generator=g)).to(BF).cuda())
    back, bs = flce.quantize_fp8((0.05 * torch.randn(H, V, generator=g)).to(BF).cuda())
    tok = torch.randint(0, V, (B, L), generator=g).cuda()
    fp = torch.full((B,), 0.5).cuda()

    def chain(wait):
        stream = x.clone()
        for _ in range(steps):
            q, s = flce.rms_norm_fp8(stream, w)
            wait()
            z = flce.matmul_fp8(q, s, Wq, Ws, out_dtype=torch.float32)
            wait()
            flce.process_logits(z, tokens=tok, frequency_penalty=fp, out=z)
            wait()
            zq, zs = flce.quantize_fp8(z, block_rows=1)
            wait()
            y = flce.matmul_fp8(zq, zs, back, bs)
            wait()
            y, h, rstd = flce.flce_rms_norm(y, w, residual=stream)
            wait()
            stream, dw = flce.flce_rms_norm_backward(y, h, w, rstd)
            wait()
            stream = flce.flce_rms_norm(stream, dw)[0]
        torch.cuda.synchronize()
        return stream, z

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        got = chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.isfinite(want[0].float()).all() and want[0].float().abs().max() > 0


def test_threads_with_streams_of_their_own():
    """Four threads run decode steps at once, each on its own stream and, every
    other one, on sizes that no thread has used before: the same bits as alone."""
    import threading

    def setup(i):
        g = torch.Generator().manual_seed(i)
        B, H, V = (1, 40, 100, 3)[i], 256 + 128 * i, 3001 + 1000 * i
        x = torch.randn(B, H, generator=g).to(BF).cuda()
        w = (1 + 0.2 * torch.randn(H, generator=g)).to(BF).cuda()
        W = (0.05 * torch.randn(V, H, generator=g)).to(BF).cuda()
        tok = torch.randint(0, V, (B, 30), generator=g).cuda()
        return x, w, W, tok, torch.full((B,), 0.5, device="cuda")

    def step(x, w, W, tok, fp):
        b, bs = flce.quantize_fp8(W)
        q, s = flce.rms_norm_fp8(x, w)
        z = flce.matmul_fp8(q, s, b, bs)
        y, h, rstd = flce.flce_rms_norm(x, w)
        dx, dw = flce.flce_rms_norm_backward(y, h, w, rstd)
        return flce.process_logits(z, tokens=tok, frequency_penalty=fp), dx, dw
    data = [setup(i) for i in range(4)]
    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)

    def work(i):
        s = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(s):
            outs = [step(*data[i]) for _ in range(20)]
        s.synchronize()
        wrong.extend(i for o in outs for a, b in zip(o, want[i]) if not torch.equal(a, b))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
