"""Operators around the LM head: the norm in front of it, 8-bit operands with
block scales and the head's product on them, and the processing of its logits.

Training:  y, h = rms_norm(x, weight, residual=res); linear_cross_entropy(y, W, labels)
Serving:   q, s, h = rms_norm_fp8(x, weight, residual=res)
           z = matmul_fp8(q, s, Wq, Ws)          # Wq, Ws = quantize_fp8(W), once
           l = process_logits(z, tokens=..., allowed=...)

As in the rest of the binding, tensors become device pointers on torch's
current stream, every step runs in the library's kernels (``include/flce.h``
says what each computes), and wrong arguments raise before anything is
enqueued.  A tensor that another stream wrote or will free follows torch's own
rules (wait for that stream, ``record_stream``).
"""
from __future__ import annotations

import ctypes

import torch

from . import _I64, _INT, _P, _SZ, FlceError, library

__all__ = ["flce_rms_norm", "flce_rms_norm_backward", "rms_norm", "rms_norm_fp8", "quantize_fp8",
           "matmul_fp8", "process_logits"]

_F32 = ctypes.c_float
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
_FP8 = torch.float8_e4m3fn
_GROUP = 128

_ARGS = {
    "flce_rms_norm_forward": [_P, _I64, _P, _I64, _P, _I64, _I64, _F32, _INT, _INT, _P, _P, _P,
                              _P],
    "flce_rms_norm_fp8": [_P, _I64, _P, _I64, _P, _I64, _I64, _F32, _INT, _INT, _P, _P, _P, _P],
    "flce_rms_norm_backward": [_P, _P, _P, _I64, _P, _P, _I64, _I64, _INT, _INT, _P, _P, _P, _SZ,
                               _P],
    "flce_rms_norm_workspace_size": [_I64, _I64],
    "flce_quantize_fp8": [_P, _I64, _I64, _I64, _INT, _INT, _P, _P, _P],
    "flce_matmul_fp8": [_P, _I64, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _INT, _P],
    "flce_process_logits": [_P, _I64, _INT, _I64, _I64, _P, _I64, _INT, _I64, _P, _P, _P, _P, _P,
                            _P, _INT, _P, _I64, _P, _I64, _P, _I64, _INT, _P],
}
_fns: dict = {}


def _fn(name):
    """The entry point with its argument types set, looked up once per library."""
    lib = library()
    hit = _fns.get(name)
    if hit is None or hit[0] is not lib:
        fn = getattr(lib, name)
        fn.argtypes = _ARGS[name]
        fn.restype = _SZ if name.endswith("workspace_size") else _INT
        _fns[name] = hit = (lib, fn)
    return hit[1]


def _call(name, device, *args):
    """Calls an entry point on torch's current stream of `device`."""
    index = device.index
    if index == torch.cuda.current_device():
        st = _fn(name)(*args, torch.cuda.current_stream(index).cuda_stream)
    else:
        with torch.cuda.device(device):
            st = _fn(name)(*args, torch.cuda.current_stream(index).cuda_stream)
    if st != 0:
        raise FlceError(st, name)


def _cuda(name, t, dtypes, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _rows(t):
    """t as a matrix of its last dimension's rows with a constant row distance
    (a view wherever the strides allow it): (matrix, row distance)."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    n, w = t.shape
    if n == 0 or w == 0:
        return t, w
    if w > 1 and t.stride(1) != 1 or n > 1 and t.stride(0) < w:
        t = t.contiguous()
    return t, t.stride(0) if n > 1 else w


def _optr(t):
    return None if t is None else t.data_ptr()


def _check_norm(x, weight, residual):
    _cuda("x", x, _DTYPE)
    _cuda("weight", weight, _DTYPE, x.device)
    if x.dim() < 1 or weight.dim() != 1 or weight.shape[0] != x.shape[-1] or x.shape[-1] == 0:
        raise ValueError("expected x [..., H] and weight [H]")
    if residual is not None:
        _cuda("residual", residual, (x.dtype,), x.device)
        if residual.shape != x.shape:
            raise ValueError("residual must have the shape of x")


def _norm_call(name, x, weight, eps, residual, residual_out, outs):
    """The shared front of both norms: the row views, the sum's buffer, the call."""
    xm, ldx = _rows(x)
    rm, ldr = _rows(residual) if residual is not None else (None, 0)
    h = residual_out
    if h is not None:
        _cuda("residual_out", h, (x.dtype,), x.device)
        if h.shape != x.shape or not h.is_contiguous():
            raise ValueError("residual_out must be contiguous, with the shape of x")
    elif residual is not None:
        h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    N, H = xm.shape
    weight = weight.contiguous()
    _call(name, x.device, xm.data_ptr(), ldx, _optr(rm), ldr, weight.data_ptr(), N, H, eps,
          _DTYPE[x.dtype], _DTYPE[weight.dtype], *outs(h))
    return h


def flce_rms_norm(x, weight, *, eps=1e-6, residual=None, residual_out=None):
    """Calls flce_rms_norm_forward; returns (y, h, rstd): the norm of
    h = x + residual (x itself without a residual) times weight, the sum, and
    the per-row 1 / sqrt(mean(h^2) + eps) the backward needs."""
    _check_norm(x, weight, residual)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    h = _norm_call("flce_rms_norm_forward", x, weight, eps, residual, residual_out,
                   lambda h: (y.data_ptr(), _optr(h), rstd.data_ptr()))
    return y, (x if h is None else h), rstd


def flce_rms_norm_backward(dy, h, weight, rstd, *, dh=None, need_dx=True, need_dweight=True):
    """Calls flce_rms_norm_backward; returns (dx or None, dweight or None).

    dx is the gradient of x and of the residual alike; dh (or None) is the
    gradient that reaches h by its other uses."""
    _check_norm(h, weight, None)
    for name, t in (("dy", dy), ("dh", dh)):
        if t is not None:
            _cuda(name, t, (h.dtype,), h.device)
            if t.shape != h.shape:
                raise ValueError(f"{name} must have the shape of h")
    _cuda("rstd", rstd, (torch.float32,), h.device)
    if rstd.shape != h.shape[:-1] or not rstd.is_contiguous():
        raise ValueError("rstd must be as flce_rms_norm returned it")
    hm, ldh = _rows(h)
    N, H = hm.shape
    dy = dy.contiguous()
    dh = None if dh is None else dh.contiguous()
    dx = torch.empty(h.shape, dtype=h.dtype, device=h.device) if need_dx else None
    dw = ws = None
    if need_dweight:
        dw = torch.empty(H, dtype=weight.dtype, device=h.device)
        ws = torch.empty(_fn("flce_rms_norm_workspace_size")(N, H), dtype=torch.uint8,
                         device=h.device)
    weight = weight.contiguous()
    _call("flce_rms_norm_backward", h.device, dy.data_ptr(), _optr(dh), hm.data_ptr(), ldh,
          weight.data_ptr(), rstd.data_ptr(), N, H, _DTYPE[h.dtype], _DTYPE[weight.dtype],
          _optr(dx), _optr(dw), _optr(ws), 0 if ws is None else ws.numel())
    return dx, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = flce_rms_norm(x, weight, eps=eps, residual=residual)
        ctx.save_for_backward(h, weight, rstd)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return (y, h) if ctx.has_residual else y

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None:  # only the sum was used
            dx = dh
            dw = None
        else:
            dx, dw = flce_rms_norm_backward(dy, h, weight, rstd, dh=dh,
                                            need_dx=need[0] or need[2], need_dweight=need[1])
        return (dx if need[0] else None, dw,
                dx if ctx.has_residual and need[2] else None, None)


def rms_norm(x, weight, eps=1e-6, residual=None):
    """Root-mean-square norm over the last dimension, differentiable.

    x: bf16 or float32 [..., H]; weight: bf16 or float32 [H].  Without a residual
    returns y = x * weight / sqrt(mean(x^2) + eps).  With one (as x) returns
    (y, h): the norm of h = x + residual, and h, the new residual stream.  Sums
    are FP32; y and h are rounded once."""
    return _RmsNorm.apply(x, weight, residual, eps)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, residual_out=None):
    """The norm with its output in 8 bits: (q, scale), or (q, scale, h) with a
    residual.  q: float8_e4m3fn [..., H]; scale: float32 [..., ceil(H / 128)],
    one per row and 128 columns; q * scale stands for y.  residual_out: where
    to write h (may be residual itself).  No gradient."""
    _check_norm(x, weight, residual)
    H = x.shape[-1]
    q = torch.empty(x.shape, dtype=_FP8, device=x.device)
    scale = torch.empty(*x.shape[:-1], -(-H // _GROUP), dtype=torch.float32, device=x.device)
    h = _norm_call("flce_rms_norm_fp8", x, weight, eps, residual, residual_out,
                   lambda h: (q.data_ptr(), scale.data_ptr(), _optr(h)))
    return (q, scale) if h is None else (q, scale, h)


def quantize_fp8(x, block_rows=128):
    """x [R, K] (bf16 or float32) in 8 bits: (q, scale) with q float8_e4m3fn
    [R, K] and scale float32 [ceil(R / block_rows), ceil(K / 128)].  block_rows
    is 128 for a weight, 1 for activations (x may then be [..., K])."""
    _cuda("x", x, _DTYPE)
    if block_rows not in (1, _GROUP):
        raise ValueError(f"block_rows must be 1 or {_GROUP}, got {block_rows}")
    if x.dim() < 1 or (block_rows != 1 and x.dim() != 2) or x.shape[-1] == 0:
        raise ValueError("expected x [R, K]")
    K = x.shape[-1]
    lead = x.shape[:-1] if block_rows == 1 else (-(-x.shape[0] // block_rows),)
    xm, ldx = _rows(x)
    q = torch.empty(x.shape, dtype=_FP8, device=x.device)
    scale = torch.empty(*lead, -(-K // _GROUP), dtype=torch.float32, device=x.device)
    _call("flce_quantize_fp8", x.device, xm.data_ptr(), ldx, xm.shape[0], K, _DTYPE[x.dtype],
          block_rows, q.data_ptr(), scale.data_ptr())
    return q, scale


def matmul_fp8(a, a_scale, b, b_scale, out_dtype=torch.bfloat16):
    """a @ b.T on 8-bit operands: [..., V] of out_dtype (bf16 or float32).

    a: float8_e4m3fn [..., K] with a_scale float32 [..., ceil(K / 128)], as
    rms_norm_fp8 or quantize_fp8(block_rows=1) give them; b: float8_e4m3fn
    [V, K] with b_scale float32 [ceil(V / 128), ceil(K / 128)], as
    quantize_fp8(W) gives them.  K must be a multiple of 16.  As with
    flce_logits, where V is no multiple of 8 the result is a view of rows padded
    to one (16-byte rows).  No gradient."""
    _cuda("a", a, (_FP8,))
    dev = a.device
    _cuda("b", b, (_FP8,), dev)
    _cuda("a_scale", a_scale, (torch.float32,), dev)
    _cuda("b_scale", b_scale, (torch.float32,), dev)
    if out_dtype not in _DTYPE:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if a.dim() < 1 or b.dim() != 2 or a.shape[-1] != b.shape[1] or b.shape[0] == 0:
        raise ValueError("expected a [..., K] and b [V, K]")
    V, K = b.shape
    groups = -(-K // _GROUP)
    if a_scale.shape != (*a.shape[:-1], groups):
        raise ValueError("a_scale must be [..., ceil(K / 128)], one row per row of a")
    if b_scale.shape != (-(-V // _GROUP), groups):
        raise ValueError("b_scale must be [ceil(V / 128), ceil(K / 128)]")
    am, lda = _rows(a)
    bm, ldb = _rows(b)
    M = am.shape[0]
    a_scale, b_scale = a_scale.contiguous(), b_scale.contiguous()
    if K % 16 == 0:  # the kernels' 16-byte rows; a view that lacks them is copied
        if (lda | am.data_ptr()) % 16:
            am, lda = am.clone(memory_format=torch.contiguous_format), K
        if (ldb | bm.data_ptr()) % 16:
            bm, ldb = bm.clone(memory_format=torch.contiguous_format), K
    ld = (V + 7) // 8 * 8
    y = torch.empty(*a.shape[:-1], ld, dtype=out_dtype, device=dev)
    _call("flce_matmul_fp8", dev, am.data_ptr(), lda, a_scale.data_ptr(), bm.data_ptr(), ldb,
          b_scale.data_ptr(), M, V, K, y.data_ptr(), ld, _DTYPE[out_dtype])
    return y if ld == V else y[..., :V]


_IDS = (torch.int32, torch.int64)


def _per_row(name, t, B, dtype, device):
    if t is None:
        return None
    _cuda(name, t, (dtype,), device)
    if t.shape != (B,):
        raise ValueError(f"{name} must be [B]")
    return t.contiguous()


def process_logits(logits, *, tokens=None, lengths=None, prompt_lengths=None,
                   repetition_penalty=None, frequency_penalty=None, presence_penalty=None,
                   bias_ids=None, bias_values=None, allowed=None, out=None, out_dtype=None):
    """Penalties for repeated tokens, biases and grammar masks on logits [B, V].

    tokens: int32 or int64 [B, L], each row's history, of which the first
    lengths[b] entries count (all without lengths) and the first
    prompt_lengths[b] of those are the prompt (none without it); ids outside
    [0, V) do not count.  A token of the history has its logit divided by
    repetition_penalty[b] where positive and multiplied by it elsewhere; one that
    was generated c times loses frequency_penalty[b] * c + presence_penalty[b].
    Then bias_values[b, i] is added at bias_ids[b, i] (the last of equal ids; ids
    outside [0, V) are skipped), and a column v whose bit v % 32 of
    allowed[b, v // 32] (int32) is 0 becomes -inf.  Any part may be left out.

    logits: bf16 or float32.  Returns out (given, or new: out_dtype, default
    that of logits); out may be logits itself."""
    _cuda("logits", logits, _DTYPE)
    if logits.dim() != 2 or logits.shape[1] == 0:
        raise ValueError("expected logits [B, V]")
    B, V = logits.shape
    dev = logits.device
    if out is None:
        out = torch.empty(B, V, dtype=out_dtype or logits.dtype, device=dev)
    elif out_dtype is not None and out_dtype != out.dtype:
        raise ValueError("out and out_dtype disagree")
    _cuda("out", out, _DTYPE, dev)
    if out.shape != (B, V) or V > 1 and out.stride(1) != 1 or B > 1 and out.stride(0) < V:
        raise ValueError("out must be [B, V] with contiguous rows")
    if out is logits:
        zm, ldz = out, out.stride(0) if B > 1 else V
    else:
        zm, ldz = _rows(logits)
    L = ldt = 0
    if tokens is not None:
        _cuda("tokens", tokens, _IDS, dev)
        if tokens.dim() != 2 or tokens.shape[0] != B:
            raise ValueError("tokens must be [B, L]")
        tokens, ldt = _rows(tokens)
        L = tokens.shape[1]
    elif lengths is not None or prompt_lengths is not None:
        raise ValueError("lengths and prompt_lengths need tokens")
    nb = 0
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values go together")
    if bias_ids is not None:
        _cuda("bias_ids", bias_ids, _IDS, dev)
        _cuda("bias_values", bias_values, (torch.float32,), dev)
        if bias_ids.dim() != 2 or bias_ids.shape[0] != B or bias_values.shape != bias_ids.shape:
            raise ValueError("bias_ids and bias_values must be [B, n]")
        bias_ids, bias_values = bias_ids.contiguous(), bias_values.contiguous()
        nb = bias_ids.shape[1]
    lda = 0
    if allowed is not None:
        _cuda("allowed", allowed, (torch.int32,), dev)
        if allowed.dim() != 2 or allowed.shape[0] != B or allowed.shape[1] < -(-V // 32):
            raise ValueError("allowed must be [B, ceil(V / 32)]")
        allowed, lda = _rows(allowed)
    lengths = _per_row("lengths", lengths, B, torch.int32, dev)
    prompt_lengths = _per_row("prompt_lengths", prompt_lengths, B, torch.int32, dev)
    rep = _per_row("repetition_penalty", repetition_penalty, B, torch.float32, dev)
    freq = _per_row("frequency_penalty", frequency_penalty, B, torch.float32, dev)
    pres = _per_row("presence_penalty", presence_penalty, B, torch.float32, dev)
    _call("flce_process_logits", dev, zm.data_ptr(), ldz, _DTYPE[logits.dtype], B, V,
          _optr(tokens) if L else None, ldt, int(L > 0 and tokens.dtype == torch.int64), L,
          _optr(lengths), _optr(prompt_lengths), _optr(rep), _optr(freq), _optr(pres),
          _optr(bias_ids) if nb else None, int(nb > 0 and bias_ids.dtype == torch.int64),
          _optr(bias_values) if nb else None, nb, _optr(allowed), lda, out.data_ptr(),
          out.stride(0) if B > 1 else V, _DTYPE[out.dtype])
    return out
