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

import lm_head_linear_flce_gb300 as _pkg

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
_bound = None


def _fn(name):
    """The entry point with its argument types set, looked up once per library."""
    global _bound
    if _bound is None or _bound is not _pkg._lib:
        lib = library()
        for n, args in _ARGS.items():
            fn = getattr(lib, n)
            fn.argtypes = args
            fn.restype = _SZ if n.endswith("workspace_size") else _INT
            _fns[n] = fn
        _bound = lib
    return _fns[name]


# A decode step's calls are bound by the host, so the stream is taken without
# building a Stream object where this torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name, index, *args):
    """Calls an entry point on torch's current stream of device `index`."""
    if index == torch.cuda.current_device():
        st = _fn(name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = _fn(name)(*args, _raw_stream(index))
    if st != 0:
        raise FlceError(st, name)


def _cuda(name, t, dtypes, index=None):
    """Refuses t unless it is a CUDA tensor of one of the dtypes, on device `index`."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _rows(t, w):
    """t as rows of its last dimension (w elements) a constant distance apart, a
    view wherever the strides allow it: (tensor to keep, address, distance)."""
    if t.is_contiguous():
        return t, t.data_ptr(), w
    if t.dim() != 2:
        t = t.reshape(-1, w)
    n = t.shape[0]
    if w > 1 and t.stride(1) != 1 or n > 1 and t.stride(0) < w:
        t = t.contiguous()
    return t, t.data_ptr(), t.stride(0) if n > 1 else w


def _optr(t):
    return None if t is None else t.data_ptr()


_FP8_ONLY, _F32_ONLY, _I32_ONLY = (_FP8,), (torch.float32,), (torch.int32,)


def _check_norm(x, weight, residual):
    """(device index, row length) of a norm's arguments."""
    _cuda("x", x, _DTYPE)
    index = x.get_device()
    _cuda("weight", weight, _DTYPE, index)
    H = x.shape[-1] if x.dim() else 0
    if H == 0 or weight.dim() != 1 or weight.shape[0] != H:
        raise ValueError("expected x [..., H] and weight [H]")
    if residual is not None:
        _cuda("residual", residual, (x.dtype,), index)
        if residual.shape != x.shape:
            raise ValueError("residual must have the shape of x")
    return index, H


def _sum_buffer(x, residual, residual_out):
    """Where the norm writes h: residual_out, or a new tensor if there is a residual."""
    if residual_out is not None:
        _cuda("residual_out", residual_out, (x.dtype,), x.get_device())
        if residual_out.shape != x.shape or not residual_out.is_contiguous():
            raise ValueError("residual_out must be contiguous, with the shape of x")
        return residual_out
    if residual is None:
        return None
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def flce_rms_norm(x, weight, *, eps=1e-6, residual=None, residual_out=None):
    """Calls flce_rms_norm_forward; returns (y, h, rstd): the norm of
    h = x + residual (x itself without a residual) times weight, the sum, and
    the per-row 1 / sqrt(mean(h^2) + eps) the backward needs."""
    index, H = _check_norm(x, weight, residual)
    h = _sum_buffer(x, residual, residual_out)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    xm, xp, ldx = _rows(x, H)
    rm, rp, ldr = _rows(residual, H) if residual is not None else (None, None, 0)
    weight = weight.contiguous()
    _call("flce_rms_norm_forward", index, xp, ldx, rp, ldr, weight.data_ptr(), rstd.numel(), H,
          eps, _DTYPE[x.dtype], _DTYPE[weight.dtype], y.data_ptr(), _optr(h), rstd.data_ptr())
    return y, (x if h is None else h), rstd


def flce_rms_norm_backward(dy, h, weight, rstd, *, dh=None, need_dx=True, need_dweight=True):
    """Calls flce_rms_norm_backward; returns (dx or None, dweight or None).

    dx is the gradient of x and of the residual alike; dh (or None) is the
    gradient that reaches h by its other uses."""
    index, H = _check_norm(h, weight, None)
    for name, t in (("dy", dy), ("dh", dh)):
        if t is not None:
            _cuda(name, t, (h.dtype,), index)
            if t.shape != h.shape:
                raise ValueError(f"{name} must have the shape of h")
    _cuda("rstd", rstd, _F32_ONLY, index)
    if rstd.shape != h.shape[:-1] or not rstd.is_contiguous():
        raise ValueError("rstd must be as flce_rms_norm returned it")
    hm, hp, ldh = _rows(h, H)
    N = rstd.numel()
    dy = dy.contiguous()
    dh = None if dh is None else dh.contiguous()
    dx = torch.empty_like(h, memory_format=torch.contiguous_format) if need_dx else None
    dw = ws = None
    nws = 0
    weight = weight.contiguous()
    if need_dweight:
        dw = torch.empty_like(weight)
        nws = _fn("flce_rms_norm_workspace_size")(N, H)
        ws = torch.empty(nws, dtype=torch.uint8, device=h.device)
    _call("flce_rms_norm_backward", index, dy.data_ptr(), _optr(dh), hp, ldh, weight.data_ptr(),
          rstd.data_ptr(), N, H, _DTYPE[h.dtype], _DTYPE[weight.dtype], _optr(dx), _optr(dw),
          _optr(ws), nws)
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
    index, H = _check_norm(x, weight, residual)
    h = _sum_buffer(x, residual, residual_out)
    groups = -(-H // _GROUP)
    q = torch.empty_like(x, dtype=_FP8, memory_format=torch.contiguous_format)
    scale = torch.empty((*x.shape[:-1], groups), dtype=torch.float32, device=x.device)
    xm, xp, ldx = _rows(x, H)
    rm, rp, ldr = _rows(residual, H) if residual is not None else (None, None, 0)
    weight = weight.contiguous()
    _call("flce_rms_norm_fp8", index, xp, ldx, rp, ldr, weight.data_ptr(),
          scale.numel() // groups, H, eps, _DTYPE[x.dtype], _DTYPE[weight.dtype], q.data_ptr(),
          scale.data_ptr(), _optr(h))
    return (q, scale) if h is None else (q, scale, h)


def quantize_fp8(x, block_rows=128):
    """x [R, K] (bf16 or float32) in 8 bits: (q, scale) with q float8_e4m3fn
    [R, K] and scale float32 [ceil(R / block_rows), ceil(K / 128)].  block_rows
    is 128 for a weight, 1 for activations (x may then be [..., K])."""
    _cuda("x", x, _DTYPE)
    if block_rows not in (1, _GROUP):
        raise ValueError(f"block_rows must be 1 or {_GROUP}, got {block_rows}")
    shape = x.shape
    if len(shape) < 1 or (block_rows != 1 and len(shape) != 2) or shape[-1] == 0:
        raise ValueError("expected x [R, K]")
    K = shape[-1]
    lead = shape[:-1] if block_rows == 1 else (-(-shape[0] // block_rows),)
    xm, xp, ldx = _rows(x, K)
    q = torch.empty_like(x, dtype=_FP8, memory_format=torch.contiguous_format)
    scale = torch.empty((*lead, -(-K // _GROUP)), dtype=torch.float32, device=x.device)
    _call("flce_quantize_fp8", x.get_device(), xp, ldx, x.numel() // K, K, _DTYPE[x.dtype],
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
    _cuda("a", a, _FP8_ONLY)
    index = a.get_device()
    _cuda("b", b, _FP8_ONLY, index)
    _cuda("a_scale", a_scale, _F32_ONLY, index)
    _cuda("b_scale", b_scale, _F32_ONLY, index)
    out = _DTYPE.get(out_dtype)
    if out is None:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    shape = a.shape
    if len(shape) < 1 or b.dim() != 2 or shape[-1] != b.shape[1] or b.shape[0] == 0 \
            or shape[-1] == 0:
        raise ValueError("expected a [..., K] and b [V, K]")
    V, K = b.shape
    lead = shape[:-1]
    groups = -(-K // _GROUP)
    if a_scale.shape != (*lead, groups):
        raise ValueError("a_scale must be [..., ceil(K / 128)], one row per row of a")
    if b_scale.shape != (-(-V // _GROUP), groups):
        raise ValueError("b_scale must be [ceil(V / 128), ceil(K / 128)]")
    am, ap, lda = _rows(a, K)
    bm, bp, ldb = _rows(b, K)
    a_scale, b_scale = a_scale.contiguous(), b_scale.contiguous()
    if K % 16 == 0:  # the kernels' 16-byte rows; a view that lacks them is copied
        if (lda | ap) % 16:
            am = am.clone(memory_format=torch.contiguous_format)
            ap, lda = am.data_ptr(), K
        if (ldb | bp) % 16:
            bm = bm.clone(memory_format=torch.contiguous_format)
            bp, ldb = bm.data_ptr(), K
    ld = (V + 7) // 8 * 8
    y = torch.empty((*lead, ld), dtype=out_dtype, device=a.device)
    _call("flce_matmul_fp8", index, ap, lda, a_scale.data_ptr(), bp, ldb, b_scale.data_ptr(),
          a.numel() // K, V, K, y.data_ptr(), ld, out)
    return y if ld == V else y[..., :V]


_IDS = (torch.int32, torch.int64)


def _per_row(name, t, B, dtypes, index):
    """The address of an optional [B] argument, and the tensor that holds it."""
    if t is None:
        return None, None
    _cuda(name, t, dtypes, index)
    if t.dim() != 1 or t.shape[0] != B:
        raise ValueError(f"{name} must be [B]")
    t = t.contiguous()
    return t, t.data_ptr()


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
    index = logits.get_device()
    if out is None:
        out = torch.empty((B, V), dtype=out_dtype or logits.dtype, device=logits.device)
        _cuda("out", out, _DTYPE)
        op, ldo = out.data_ptr(), V
    else:
        if out_dtype is not None and out_dtype != out.dtype:
            raise ValueError("out and out_dtype disagree")
        _cuda("out", out, _DTYPE, index)
        if out.shape != (B, V) or V > 1 and out.stride(1) != 1 or B > 1 and out.stride(0) < V:
            raise ValueError("out must be [B, V] with contiguous rows")
        op, ldo = out.data_ptr(), out.stride(0) if B > 1 else V
    zm, zp, ldz = (out, op, ldo) if out is logits else _rows(logits, V)
    L = ldt = t64 = 0
    tp = None
    if tokens is not None:
        _cuda("tokens", tokens, _IDS, index)
        if tokens.dim() != 2 or tokens.shape[0] != B:
            raise ValueError("tokens must be [B, L]")
        L = tokens.shape[1]
        if L:
            tokens, tp, ldt = _rows(tokens, L)
            t64 = int(tokens.dtype == torch.int64)
    elif lengths is not None or prompt_lengths is not None:
        raise ValueError("lengths and prompt_lengths need tokens")
    nb = b64 = 0
    ip = vp = None
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values go together")
    if bias_ids is not None:
        _cuda("bias_ids", bias_ids, _IDS, index)
        _cuda("bias_values", bias_values, _F32_ONLY, index)
        if bias_ids.dim() != 2 or bias_ids.shape[0] != B or bias_values.shape != bias_ids.shape:
            raise ValueError("bias_ids and bias_values must be [B, n]")
        nb = bias_ids.shape[1]
        if nb:
            bias_ids, bias_values = bias_ids.contiguous(), bias_values.contiguous()
            ip, vp = bias_ids.data_ptr(), bias_values.data_ptr()
            b64 = int(bias_ids.dtype == torch.int64)
    mp, ldm = None, 0
    if allowed is not None:
        _cuda("allowed", allowed, _I32_ONLY, index)
        if allowed.dim() != 2 or allowed.shape[0] != B or allowed.shape[1] < -(-V // 32):
            raise ValueError("allowed must be [B, ceil(V / 32)]")
        allowed, mp, ldm = _rows(allowed, allowed.shape[1])
    lengths, lp = _per_row("lengths", lengths, B, _I32_ONLY, index)
    prompt_lengths, pp = _per_row("prompt_lengths", prompt_lengths, B, _I32_ONLY, index)
    rep, rpp = _per_row("repetition_penalty", repetition_penalty, B, _F32_ONLY, index)
    freq, fpp = _per_row("frequency_penalty", frequency_penalty, B, _F32_ONLY, index)
    pres, ppp = _per_row("presence_penalty", presence_penalty, B, _F32_ONLY, index)
    _call("flce_process_logits", index, zp, ldz, _DTYPE[logits.dtype], B, V, tp, ldt, t64, L, lp,
          pp, rpp, fpp, ppp, ip, b64, vp, nb, mp, ldm, op, ldo, _DTYPE[out.dtype])
    return out
