"""Float64 definitions of the operators around the LM head (numpy, tests only).

Each function is the formula of include/flce.h written out plainly; nothing is
shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

GROUP = 128
FP8_MAX = 448.0
AMAX_MIN = 2.0 ** -100


def rms_norm(x, weight, eps, residual=None):
    """(y, h, rstd) in float64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * np.asarray(weight, np.float64), h, rstd


def rms_norm_backward(dy, h, weight, eps, dh=None):
    """(dx, dweight) for y = h * rstd(h) * weight, plus dh on dx."""
    dy, h, w = (np.asarray(t, np.float64) for t in (dy, h, weight))
    rstd = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = dy * w
    dx = rstd * (g - h * rstd ** 2 * (g * h).mean(-1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * h * rstd).sum(0)


def round_e4m3(v):
    """The nearest e4m3 value, ties to even, saturating at 448 (NaN stays NaN)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    e = np.maximum(np.frexp(np.where((a > 0) & np.isfinite(a), a, 1.0))[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, FP8_MAX), v)


def block_amax(x, block_rows):
    """max |x| over each block_rows x 128 block, at least 2^-100."""
    R, K = x.shape
    out = np.empty((-(-R // block_rows), -(-K // GROUP)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            blk = x[i * block_rows:(i + 1) * block_rows, j * GROUP:(j + 1) * GROUP]
            out[i, j] = max(np.abs(blk).max(), AMAX_MIN)
    return out


def expand_scale(scale, R, K, block_rows):
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), block_rows, 0), GROUP, 1)
    return s[:R, :K]


def matmul_fp8(a, a_scale, b, b_scale):
    """(y, sum of |terms|): the products of the values the operands stand for."""
    a = np.asarray(a, np.float64) * expand_scale(a_scale, *a.shape, 1)
    b = np.asarray(b, np.float64) * expand_scale(b_scale, *b.shape, GROUP)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def process_logits(logits, tokens=None, lengths=None, prompt_lengths=None, repetition=None,
                   frequency=None, presence=None, bias_ids=None, bias_values=None, allowed=None):
    """Row by row and entry by entry."""
    out = np.array(logits, np.float64)
    B, V = out.shape
    for b in range(B):
        n = 0 if tokens is None else tokens.shape[1]
        if lengths is not None:
            n = min(max(int(lengths[b]), 0), n)
        prompt = 0 if prompt_lengths is None else int(prompt_lengths[b])
        seen, count = set(), {}
        for i in range(n):
            t = int(tokens[b, i])
            if 0 <= t < V:
                seen.add(t)
                if i >= prompt:
                    count[t] = count.get(t, 0) + 1
        for t in seen:
            l = out[b, t]
            if repetition is not None:
                l = l / float(repetition[b]) if l > 0 else l * float(repetition[b])
            c = count.get(t, 0)
            if frequency is not None:
                l -= float(frequency[b]) * c
            if presence is not None and c > 0:
                l -= float(presence[b])
            out[b, t] = l
        if bias_ids is not None:
            chosen = {int(v): i for i, v in enumerate(bias_ids[b]) if 0 <= int(v) < V}
            for v, i in chosen.items():
                out[b, v] += float(bias_values[b, i])
        if allowed is not None:
            words = np.asarray(allowed[b]).astype(np.int64) & 0xFFFFFFFF
            for v in range(V):
                if not (int(words[v // 32]) >> (v % 32)) & 1:
                    out[b, v] = -np.inf
    return out
