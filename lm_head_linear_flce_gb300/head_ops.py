"""Operators around the LM head: the norm in front of it (RMS or layer norm), 8-bit
operands with block scales and the head's product on them, the processing of its
logits, and the sampling of a token.

Training:  y, h = rms_norm(x, weight, residual=res)      # or layer_norm(x, weight, bias, ...)
           linear_cross_entropy(y, W, labels)
Serving:   q, s, h = rms_norm_fp8(x, weight, residual=res)      # or layer_norm_fp8
           z = matmul_fp8(q, s, Wq, Ws)          # Wq, Ws = quantize_fp8(W), once
           l = process_logits(z, tokens=..., allowed=...)
           token = sample_logits(l, u, temperature=..., top_k=..., top_p=..., min_p=...)

Every step runs in the library's kernels on torch's current stream
(``include/flce.h`` says what each computes); the calls go through a small native
module (``csrc/flce_torch.cpp``), and wrong arguments raise before anything is
enqueued.  A tensor that another stream wrote or will free follows torch's own
rules (wait for that stream, ``record_stream``).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

import lm_head_linear_flce_gb300 as _pkg

from . import _I64, _INT, _P, _SZ, FlceError, library

__all__ = ["flce_rms_norm", "flce_rms_norm_backward", "rms_norm", "rms_norm_fp8",
           "flce_layer_norm", "flce_layer_norm_backward", "layer_norm", "layer_norm_fp8",
           "quantize_fp8", "matmul_fp8", "process_logits", "sample_logits"]

_F32 = ctypes.c_float
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}

_ARGS = {
    "flce_rms_norm_forward": [_P, _I64, _P, _I64, _P, _I64, _I64, _F32, _INT, _INT, _P, _P, _P,
                              _P],
    "flce_rms_norm_fp8": [_P, _I64, _P, _I64, _P, _I64, _I64, _F32, _INT, _INT, _P, _P, _P, _P],
    "flce_rms_norm_backward": [_P, _P, _P, _I64, _P, _P, _I64, _I64, _INT, _INT, _P, _P, _P, _SZ,
                               _P],
    "flce_rms_norm_workspace_size": [_I64, _I64],
    "flce_layer_norm_forward": [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _F32, _INT, _INT, _P, _P,
                                _P, _P, _P],
    "flce_layer_norm_fp8": [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _F32, _INT, _INT, _P, _P, _P,
                            _P],
    "flce_layer_norm_backward": [_P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P, _P,
                                 _P, _SZ, _P],
    "flce_layer_norm_workspace_size": [_I64, _I64],
    "flce_quantize_fp8": [_P, _I64, _I64, _I64, _INT, _INT, _P, _P, _P],
    "flce_matmul_fp8": [_P, _I64, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _INT, _P],
    "flce_selftest_matmul_fp8_timeout": [_I64, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _I64,
                                         _P, _I64, _INT, _P],
    "flce_process_logits": [_P, _I64, _INT, _I64, _I64, _P, _I64, _INT, _I64, _P, _P, _P, _P, _P,
                            _P, _INT, _P, _I64, _P, _I64, _P, _I64, _INT, _P],
    "flce_sample_logits": [_P, _I64, _INT, _I64, _I64, _P, _P, _P, _P, _P, _P, _P],
}
_fns: dict = {}
_bound = None
_module = None


def _native():
    """The native module (raises if it has not been built)."""
    global _module
    if _module is None:
        path = os.path.join(os.path.dirname(_pkg.library_path), "_flce_torch.so")
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with lm_head_linear_flce_gb300._build.build() "
                "(nvcc, sm_103a); there is no fallback implementation")
        library()
        loader = importlib.machinery.ExtensionFileLoader("_flce_torch", path)
        spec = importlib.util.spec_from_file_location("_flce_torch", path, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _module = module
    return _module


def _ok(out, name):
    """What a native call returned, or its status raised."""
    if type(out) is int:
        raise FlceError(out, name)
    return out


def _fn(name):
    """A C entry point with its argument types set: for callers that bring
    their own buffers."""
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


def _call(name, index, *args):
    """Calls a C entry point on torch's current stream of device `index`."""
    with torch.cuda.device(index):
        st = _fn(name)(*args, torch.cuda.current_stream(index).cuda_stream)
    if st != 0:
        raise FlceError(st, name)


def flce_rms_norm(x, weight, *, eps=1e-6, residual=None, residual_out=None):
    """Calls flce_rms_norm_forward; returns (y, h, rstd): the norm of
    h = x + residual (x itself without a residual) times weight, the sum, and
    the per-row 1 / sqrt(mean(h^2) + eps) the backward needs."""
    y, h, rstd = _ok(_native().rms_norm_forward(x, weight, eps, residual, residual_out),
                     "flce_rms_norm_forward")
    return y, (x if h is None else h), rstd


def flce_rms_norm_backward(dy, h, weight, rstd, *, dh=None, need_dx=True, need_dweight=True):
    """Calls flce_rms_norm_backward; returns (dx or None, dweight or None).

    dx is the gradient of x and of the residual alike; dh (or None) is the
    gradient that reaches h by its other uses."""
    return _ok(_native().rms_norm_backward(dy, h, weight, rstd, dh, need_dx, need_dweight),
               "flce_rms_norm_backward")


class _NotTwice(torch.autograd.Function):
    """A gradient as it is; differentiating it by what it depends on raises."""

    @staticmethod
    def forward(ctx, name, grad, *depends_on):
        ctx.name = name
        return grad

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name}'s gradient cannot be differentiated again")


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
            if torch.is_grad_enabled():
                # create_graph=True: constants would lose what the gradients depend on
                # without a word.  (torch's once_differentiable looks at dy and dh alone.)
                h = h if need[0] or need[2] else None  # (else it is given)
                dx = dx if dx is None else _NotTwice.apply("rms_norm", dx, dy, dh, h, weight)
                dw = dw if dw is None else _NotTwice.apply("rms_norm", dw, dy, h)
        return (dx if need[0] else None, dw,
                dx if ctx.has_residual and need[2] else None, None)


def rms_norm(x, weight, eps=1e-6, residual=None):
    """Root-mean-square norm over the last dimension, differentiable (once: a
    gradient taken with create_graph=True raises when it is differentiated).

    x: bf16 or float32 [..., H]; weight: bf16 or float32 [H].  Without a residual
    returns y = x * weight / sqrt(mean(x^2) + eps).  With one (as x) returns
    (y, h): the norm of h = x + residual, and h, the new residual stream.  Sums
    are FP32; y and h are rounded once.  The backward takes h as rounded."""
    return _RmsNorm.apply(x, weight, residual, eps)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, residual_out=None):
    """The norm with its output in 8 bits: (q, scale), or (q, scale, h) with a
    residual.  q: float8_e4m3fn [..., H]; scale: float32 [..., ceil(H / 128)],
    one per row and 128 columns; q * scale stands for y.  residual_out: where
    to write h (may be residual itself; it may not require a gradient).  No
    gradient."""
    q, scale, h = _ok(_native().rms_norm_fp8(x, weight, eps, residual, residual_out),
                      "flce_rms_norm_fp8")
    return (q, scale) if h is None else (q, scale, h)


def flce_layer_norm(x, weight=None, bias=None, *, eps=1e-5, residual=None, residual_out=None):
    """Calls flce_layer_norm_forward; returns (y, h, mean, rstd): the norm of
    h = x + residual (x itself without a residual), the sum, and the per-row mean and
    1 / sqrt(variance + eps) the backward needs."""
    y, h, mean, rstd = _ok(_native().layer_norm_forward(x, weight, bias, eps, residual,
                                                        residual_out), "flce_layer_norm_forward")
    return y, (x if h is None else h), mean, rstd


def flce_layer_norm_backward(dy, h, weight, mean, rstd, *, dh=None, need_dx=True,
                             need_dweight=True, need_dbias=True, bias_dtype=None):
    """Calls flce_layer_norm_backward; returns (dx or None, dweight or None, dbias or
    None).

    weight may be None (then there is no dweight).  dx is the gradient of x and of the
    residual alike; dh (or None) is the gradient that reaches h by its other uses.
    bias_dtype: the bias's type where there is no weight (default: that of h)."""
    code = -1
    if need_dbias:
        code = _DTYPE.get(bias_dtype or (weight if weight is not None else h).dtype, 2)
    return _ok(_native().layer_norm_backward(dy, h, weight, mean, rstd, dh, need_dx,
                                             need_dweight and weight is not None, code),
               "flce_layer_norm_backward")


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps):
        y, h, mean, rstd = flce_layer_norm(x, weight, bias, eps=eps, residual=residual)
        ctx.save_for_backward(h, weight, mean, rstd)
        ctx.has_residual = residual is not None
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.set_materialize_grads(False)
        return (y, h) if ctx.has_residual else y

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None:  # only the sum was used
            dx = dh
            dw = db = None
        else:
            dx, dw, db = flce_layer_norm_backward(
                dy, h, weight, mean, rstd, dh=dh, need_dx=need[0] or need[3],
                need_dweight=need[1], need_dbias=need[2], bias_dtype=ctx.bias_dtype)
            if torch.is_grad_enabled():
                # create_graph=True: as in _RmsNorm
                h = h if need[0] or need[3] else None
                dx = dx if dx is None else _NotTwice.apply("layer_norm", dx, dy, dh, h, weight)
                dw = dw if dw is None else _NotTwice.apply("layer_norm", dw, dy, h)
                db = db if db is None else _NotTwice.apply("layer_norm", db, dy)
        return (dx if need[0] else None, dw, db,
                dx if ctx.has_residual and need[3] else None, None)


def layer_norm(x, weight=None, bias=None, eps=1e-5, residual=None):
    """Layer norm over the last dimension, differentiable (once: a gradient taken with
    create_graph=True raises when it is differentiated).

    x: bf16 or float32 [..., H]; weight and bias: bf16 or float32 [H], of one type, each
    may be None.  Without a residual returns y = (x - mean) / sqrt(variance + eps) *
    weight + bias.  With one (as x) returns (y, h): the norm of h = x + residual, and h,
    the new residual stream.  Sums are FP32; y and h are rounded once.  The backward
    takes h as rounded.  A backward pass that is captured into a CUDA graph while an eager
    graph of the same leaves lives is flce_layer_norm_backward's: autograd's own waiting for
    the leaves' stream cannot be captured."""
    return _LayerNorm.apply(x, weight, bias, residual, eps)


def layer_norm_fp8(x, weight=None, bias=None, eps=1e-5, residual=None, residual_out=None):
    """The layer norm with its output in 8 bits: (q, scale), or (q, scale, h) with a
    residual; q, scale and residual_out as in rms_norm_fp8.  No gradient."""
    q, scale, h = _ok(_native().layer_norm_fp8(x, weight, bias, eps, residual, residual_out),
                      "flce_layer_norm_fp8")
    return (q, scale) if h is None else (q, scale, h)


def quantize_fp8(x, block_rows=128):
    """x [R, K] (bf16 or float32) in 8 bits: (q, scale) with q float8_e4m3fn
    [R, K] and scale float32 [ceil(R / block_rows), ceil(K / 128)].  block_rows
    is 128 for a weight, 1 for activations (x may then be [..., K]).  No
    gradient."""
    return _ok(_native().quantize_fp8(x, block_rows), "flce_quantize_fp8")


def matmul_fp8(a, a_scale, b, b_scale, out_dtype=torch.bfloat16):
    """a @ b.T on 8-bit operands: [..., V] of out_dtype (bf16 or float32).

    a: float8_e4m3fn [..., K] with a_scale float32 [..., ceil(K / 128)], as
    rms_norm_fp8 or quantize_fp8(block_rows=1) give them; b: float8_e4m3fn
    [V, K] with b_scale float32 [ceil(V / 128), ceil(K / 128)], as
    quantize_fp8(W) gives them.  K must be a multiple of 16; an operand whose rows
    are not 16-byte aligned is copied, on every call.  As with
    flce_logits, where V is no multiple of 8 the result is a view of rows padded
    to one (16-byte rows).  No gradient.  If a wait inside the kernel runs out
    (flce_set_wait_limit_ns), what it had not finished is NaN."""
    out = _DTYPE.get(out_dtype)
    if out is None:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    return _ok(_native().matmul_fp8(a, a_scale, b, b_scale, out), "flce_matmul_fp8")[0]


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
    that of logits); out may be logits itself, and may not require a gradient.
    No gradient."""
    code = -1 if out_dtype is None else _DTYPE.get(out_dtype)
    if code is None:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    return _ok(_native().process_logits(
        logits, tokens, lengths, prompt_lengths, repetition_penalty, frequency_penalty,
        presence_penalty, bias_ids, bias_values, allowed, out, code), "flce_process_logits")[0]


def sample_logits(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None):
    """A token a row: int64 [B] of ids, -1 where a row of logits [B, V] (bf16 or float32)
    has nothing above -inf.

    u: float32 [B], random numbers in [0, 1).  Tokens are weighed exp(l / temperature[b])
    and put in order, larger logits first, equal ones by id.  Kept are the first top_k[b]
    (int32; 0: all), of these the ones before which less than top_p[b] of their mass lies
    (the first always; 1: all), of these the ones that weigh at least min_p[b] of what the
    first does (0: all).  The result is the first token by id at which the kept ones' mass
    exceeds u[b] of its total.  temperature, top_p and min_p: float32 [B]; any of them may
    be left out.  A temperature of 0 (below 2^-64) takes the largest logit.  A repeated call
    gives the same tokens; in a row that neither its top_k nor min_p alone limits, one within
    about 1e-9 of a border may be another in a batch of another size.  No gradient."""
    return _ok(_native().sample_logits(logits, u, temperature, top_k, top_p, min_p),
               "flce_sample_logits")[0]
