"""The operators around the LM head, as cases that can be timed and checked.

* ``rms_norm``: the norm in front of the head, with the residual's addition;
  forward and backward (training) or with an 8-bit output and scales (serving).
* ``quantize_fp8``: a matrix in e4m3 with one scale per block of 128 columns.
* ``matmul_fp8``: the LM head (or any linear layer) on such operands.
* ``process_logits``: penalties, biases and grammar masks before sampling.

``run`` computes a case in its plain form, from elementary torch operations in
32 bits, or, where ``own`` is set, by the calls a user makes of the package.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
GROUP = 128          # columns (and, for weights, rows) that share a scale
FP8_MAX = 448.0
AMAX_MIN = 2.0 ** -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence decodes one token: latency of the final norm of a 7B model
        {"name": "norm fp8, one token", "op": "norm_fp8", "N": 1, "H": 3584, "dtype": "bf16",
         "residual": True},
        # a training step's final norm, forward and backward
        {"name": "norm train 8192 x 3584", "op": "norm_train", "N": 8192, "H": 3584,
         "dtype": "bf16", "residual": True},
        # an odd width in float32, no residual: a norm over a small model's features
        {"name": "norm train odd, float32", "op": "norm_train", "N": 1021, "H": 1001,
         "dtype": "f32", "residual": False},
        # laying out the 8-bit LM head of a 152064-token vocabulary, once per load
        {"name": "quantize LM head", "op": "quantize", "R": 152064, "K": 3584, "dtype": "bf16",
         "block_rows": 128},
        # activations that no norm has quantised, a ragged prefill batch
        {"name": "quantize activations", "op": "quantize", "R": 777, "K": 2056, "dtype": "f32",
         "block_rows": 1},
        # the LM head for one token: all of the weight is read for one row
        {"name": "head, one token", "op": "matmul", "M": 1, "V": 152064, "K": 3584,
         "out": "bf16"},
        # a decode batch on a shard of the vocabulary, no size a multiple of a tile
        {"name": "head, ragged batch", "op": "matmul", "M": 37, "V": 32003, "K": 2064,
         "out": "f32"},
        # a large decode batch
        {"name": "head, 256 tokens", "op": "matmul", "M": 256, "V": 151936, "K": 4096,
         "out": "bf16"},
        # scoring a chunk of a prompt: logits of every token
        {"name": "head, 4096 tokens", "op": "matmul", "M": 4096, "V": 152064, "K": 3584,
         "out": "bf16"},
        # one sequence, short history, no grammar
        {"name": "logits, one row", "op": "logits", "B": 1, "V": 152064, "L": 500, "nb": 8,
         "dtype": "bf16", "mask": False, "ids": "i64"},
        # a serving batch with long histories and grammars
        {"name": "logits, long histories", "op": "logits", "B": 64, "V": 151936, "L": 32768,
         "nb": 300, "dtype": "bf16", "mask": True, "ids": "i32"},
        # a large batch in float32, a vocabulary that is no multiple of anything
        {"name": "logits, 256 odd rows", "op": "logits", "B": 256, "V": 128255, "L": 2000,
         "nb": 0, "dtype": "f32", "mask": True, "ids": "i64"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fp8", "norm_train", "quantize", "matmul", "matmul", "logits"])
    if op in ("norm_fp8", "norm_train"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        N = min(_log_int(rng, 1, 16384), 8192 * 3584 // H)
        return {"op": op, "N": N, "H": H, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.7}
    if op == "quantize":
        K = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            K = max(64, K // 64 * 64)
        R = min(_log_int(rng, 1, 152064), 152064 * 3584 // K)
        return {"op": op, "R": R, "K": K, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "block_rows": rng.choice([1, 128])}
    if op == "matmul":
        K = max(128, _log_int(rng, 128, 8192) // 16 * 16)
        M = _log_int(rng, 1, 4096)
        V = min(_log_int(rng, 1000, 152064), 152064 * 3584 // K)
        return {"op": op, "M": M, "V": V, "K": K, "out": rng.choice(["bf16", "bf16", "f32"])}
    return {"op": op, "B": _log_int(rng, 1, 256), "V": _log_int(rng, 1000, 152064),
            "L": rng.choice([0, _log_int(rng, 1, 32768), _log_int(rng, 1, 32768)]),
            "nb": rng.choice([0, _log_int(rng, 1, 300)]), "dtype": rng.choice(["bf16", "f32"]),
            "mask": rng.random() < 0.6, "ids": rng.choice(["i32", "i64"])}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _groups(n):
    return -(-n // GROUP)


def _e4m3_input(g, rows, cols, std, block_rows):
    """A random matrix quantised block by block: e4m3 values and float32 scales."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * std
    return _plain_quantize(x, block_rows)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = {"op": op}
    if op in ("norm_fp8", "norm_train"):
        N, H, dt = case["N"], case["H"], DTYPES[case["dtype"]]

        def t(std):
            return (torch.randn(N, H, generator=g, device="cuda") * std).to(dt)
        st["x"] = t(1.0)
        # the residual stream is larger than a layer's output, with a few large channels
        st["residual"] = t(3.0) if case["residual"] else None
        if st["residual"] is not None:
            st["residual"][:, ::97] *= 8
        st["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)
        if op == "norm_train":
            st["dy"] = t(0.02)
            st["dres"] = t(0.01) if case["residual"] else None
    elif op == "quantize":
        R, K = case["R"], case["K"]
        st["x"] = (torch.randn(R, K, generator=g, device="cuda") * 0.02).to(DTYPES[case["dtype"]])
        st["block_rows"] = case["block_rows"]
    elif op == "matmul":
        st["a"], st["a_scale"] = _e4m3_input(g, case["M"], case["K"], 1.0, 1)
        st["b"], st["b_scale"] = _e4m3_input(g, case["V"], case["K"], 0.02, 128)
        st["out"] = DTYPES[case["out"]]
    else:
        B, V, L, nb = case["B"], case["V"], case["L"], case["nb"]
        idt = torch.int32 if case["ids"] == "i32" else torch.int64
        st["logits"] = (torch.randn(B, V, generator=g, device="cuda") * 3).to(DTYPES[case["dtype"]])
        # token frequencies fall off as in text: many repeats of a few ids
        u = torch.rand(B, L, generator=g, device="cuda")
        st["tokens"] = (torch.exp(u * math.log(V)).to(torch.int64) - 1).clamp_(0, V - 1).to(idt)
        ln = (torch.rand(B, generator=g, device="cuda") * (L + 1)).to(torch.int32).clamp_(max=L)
        ln[0] = L
        if B > 2:
            ln[1] = 0  # a request that has just begun
        st["lengths"] = ln
        st["prompt_lengths"] = (ln * torch.rand(B, generator=g, device="cuda")).to(torch.int32)
        st["repetition"] = 1 + 0.3 * torch.rand(B, generator=g, device="cuda")
        st["frequency"] = 0.5 * torch.rand(B, generator=g, device="cuda")
        st["presence"] = 0.5 * torch.rand(B, generator=g, device="cuda")
        st["bias_ids"] = st["bias_values"] = st["allowed"] = None
        if nb:
            # distinct ids per row (a stride that shares no factor with V walks all of them)
            start = torch.randint(0, V, (B, 1), generator=g, device="cuda")
            step = next(s for s in range(max(1, V // (nb + 1)), 2 * V + 2) if math.gcd(s, V) == 1)
            st["bias_ids"] = ((start + torch.arange(nb, device="cuda") * step) % V).to(idt)
            st["bias_values"] = torch.randn(B, nb, generator=g, device="cuda") * 4
        if case["mask"]:
            words = (V + 31) // 32
            m = torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=g, device="cuda",
                              dtype=torch.int64)
            m &= torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=g, device="cuda",
                               dtype=torch.int64)
            m[::3] = -1                  # requests without a grammar allow everything
            if B > 4:
                m[4] = 0                 # a grammar that has run into a dead end
            st["allowed"] = m.to(torch.int32)
    return st


# ------------------------------------------------------------- plain forms
def _expand(scale, rows, cols, block_rows):
    return scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]


def _plain_quantize(y, block_rows):
    """Blocks of block_rows x 128: a = max |y|, scale = a / 448, q = e4m3(y * (448 / a))."""
    R, K = y.shape
    gr, gk = -(-R // block_rows), _groups(K)
    pad = torch.zeros(gr * block_rows, gk * GROUP, device=y.device)
    pad[:R, :K] = y
    amax = pad.view(gr, block_rows, gk, GROUP).abs().amax((1, 3)).clamp(min=AMAX_MIN)
    q = (pad.view(gr, block_rows, gk, GROUP) * (FP8_MAX / amax)[:, None, :, None])
    q = q.view(gr * block_rows, gk * GROUP)[:R, :K].to(torch.float8_e4m3fn)
    return q.contiguous(), amax / FP8_MAX


def _plain_norm(st):
    x, w = st["x"].float(), st["weight"].float()
    h = x if st["residual"] is None else x + st["residual"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    return h, r, h * r * w


def _plain(st):
    op = st["op"]
    if op == "norm_fp8":
        h, _, y = _plain_norm(st)
        q, s = _plain_quantize(y, 1)
        return [q, s] if st["residual"] is None else [q, s, h.to(st["x"].dtype)]
    if op == "norm_train":
        dt = st["x"].dtype
        h, r, y = _plain_norm(st)
        dy = st["dy"].float()
        g = dy * st["weight"].float()
        dh = r * (g - h * r.square() * (g * h).mean(1, keepdim=True))
        dw = (dy * h * r).sum(0)
        if st["residual"] is None:
            return [y.to(dt), dh.to(dt), dw.to(dt)]
        return [y.to(dt), h.to(dt), (dh + st["dres"].float()).to(dt), dw.to(dt)]
    if op == "quantize":
        return list(_plain_quantize(st["x"].float(), st["block_rows"]))
    if op == "matmul":
        a, b = st["a"], st["b"]
        af = a.float() * _expand(st["a_scale"], *a.shape, 1)
        bf = b.float() * _expand(st["b_scale"], *b.shape, 128)
        return (af @ bf.t()).to(st["out"])
    l = st["logits"].float()
    B, V = l.shape
    tok = st["tokens"].long()
    pos = torch.arange(tok.shape[1], device=tok.device)
    live = pos < st["lengths"][:, None]
    gen = live & (pos >= st["prompt_lengths"][:, None])
    count = torch.zeros(B, V, device=l.device).scatter_add_(1, tok, gen.float())
    seen = torch.zeros(B, V, device=l.device).scatter_add_(1, tok, live.float()) > 0
    rp = st["repetition"][:, None]
    l = torch.where(seen, torch.where(l > 0, l / rp, l * rp), l)
    l = l - st["frequency"][:, None] * count - st["presence"][:, None] * (count > 0)
    if st["bias_ids"] is not None:
        l = l.scatter_add(1, st["bias_ids"].long(), st["bias_values"])
    if st["allowed"] is not None:
        v = torch.arange(V, device=l.device)
        bit = (st["allowed"][:, v // 32] >> (v % 32).int()) & 1
        l = torch.where(bit == 1, l, -math.inf)
    return l


def run(st):
    if not own:
        return _plain(st)
    import lm_head_linear_flce_gb300 as flce
    op = st["op"]
    if op == "norm_fp8":
        return list(flce.rms_norm_fp8(st["x"], st["weight"], eps=EPS, residual=st["residual"]))
    if op == "norm_train":
        y, h, rstd = flce.flce_rms_norm(st["x"], st["weight"], eps=EPS, residual=st["residual"])
        dx, dw = flce.flce_rms_norm_backward(st["dy"], h, st["weight"], rstd, dh=st["dres"])
        return [y, dx, dw] if st["residual"] is None else [y, h, dx, dw]
    if op == "quantize":
        return list(flce.quantize_fp8(st["x"], block_rows=st["block_rows"]))
    if op == "matmul":
        return flce.matmul_fp8(st["a"], st["a_scale"], st["b"], st["b_scale"],
                               out_dtype=st["out"])
    return flce.process_logits(
        st["logits"], tokens=st["tokens"], lengths=st["lengths"],
        prompt_lengths=st["prompt_lengths"], repetition_penalty=st["repetition"],
        frequency_penalty=st["frequency"], presence_penalty=st["presence"],
        bias_ids=st["bias_ids"], bias_values=st["bias_values"], allowed=st["allowed"],
        out_dtype=torch.float32)


# ---------------------------------------------------------- work and truth
def work(case):
    op = case["op"]
    if op in ("norm_fp8", "norm_train"):
        N, H, e = case["N"], case["H"], 2 if case["dtype"] == "bf16" else 4
        res = 1 if case["residual"] else 0
        if op == "norm_fp8":
            return {"bytes": N * H * (e * (1 + 2 * res) + 1) + 4 * N * _groups(H) + e * H,
                    "flops": 8 * N * H}
        # x, dy in, y, dx out; with a residual: it and its gradient in, the sum out
        return {"bytes": N * H * e * (4 + 3 * res) + 2 * e * H, "flops": 16 * N * H}
    if op == "quantize":
        R, K, e = case["R"], case["K"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": R * K * (e + 1) + 4 * -(-R // case["block_rows"]) * _groups(K),
                "flops": 3 * R * K}
    if op == "matmul":
        M, V, K = case["M"], case["V"], case["K"]
        scales = 4 * _groups(K) * (M + _groups(V))
        return {"bytes": (M + V) * K + scales + M * V * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * V * K}
    B, V = case["B"], case["V"]
    e, i = 2 if case["dtype"] == "bf16" else 4, 4 if case["ids"] == "i32" else 8
    mask = B * 4 * ((V + 31) // 32) if case["mask"] else 0
    # lengths are spread evenly up to L: half of the history is live
    return {"bytes": B * V * (e + 4) + mask + B * (case["L"] // 2 * i + case["nb"] * (i + 4)),
            "flops": 4 * B * V}


def _round_e4m3(v):
    """float64 values rounded to the nearest e4m3 value, ties to even."""
    a = np.abs(v)
    e = np.maximum(np.frexp(np.where(a > 0, a, 1.0))[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, FP8_MAX), v)


def _exact_quantize(y, block_rows):
    R, K = y.shape
    q, s = np.empty_like(y), np.empty((-(-R // block_rows), _groups(K)))
    for j in range(s.shape[1]):
        c = slice(j * GROUP, (j + 1) * GROUP)
        col = np.abs(y[:, c]).max(1)
        s[:, j] = np.maximum.reduceat(col, np.arange(0, R, block_rows))
        np.maximum(s[:, j], AMAX_MIN, out=s[:, j])
        s[:, j] /= FP8_MAX
        q[:, c] = _round_e4m3(y[:, c] / np.repeat(s[:, j], block_rows)[:R, None])
    return q, s


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]

    def f64(t):
        return None if t is None else t.double().cpu().numpy()
    if op in ("norm_fp8", "norm_train"):
        x, res, w = f64(st["x"]), f64(st["residual"]), f64(st["weight"])
        h = x if res is None else x + res
        ms = np.einsum("nh,nh->n", h, h) / h.shape[1]
        u = h / np.sqrt(ms + EPS)[:, None]
        if op == "norm_fp8":
            out = list(_exact_quantize(u * w, 1))
            return out if res is None else out + [h]
        dy, dres = f64(st["dy"]), f64(st["dres"])
        du = dy * w
        dh = (du - u * (np.einsum("nh,nh->n", du, u) / h.shape[1])[:, None])
        dh /= np.sqrt(ms + EPS)[:, None]
        dw = np.einsum("nh,nh->h", dy, u)
        return [u * w, dh, dw] if res is None else [u * w, h, dh + dres, dw]
    if op == "quantize":
        if case["R"] * case["K"] > 1 << 26:
            return None
        return list(_exact_quantize(f64(st["x"]), case["block_rows"]))
    if op == "matmul":
        if case["M"] * case["V"] * case["K"] > 1 << 42:
            return None
        a, b = st["a"].double(), st["b"].double()
        out = torch.zeros(case["M"], case["V"], dtype=torch.float64, device="cuda")
        rows = torch.arange(case["V"], device="cuda") // 128
        for j in range(_groups(case["K"])):  # block by block, scaled after each product
            c = slice(j * GROUP, (j + 1) * GROUP)
            part = a[:, c] @ b[:, c].t()
            out += part * st["a_scale"][:, j, None].double() * st["b_scale"][rows, j].double()
        return out
    l = f64(st["logits"])
    V = l.shape[1]
    tok, ln, pl = (st[k].cpu().numpy() for k in ("tokens", "lengths", "prompt_lengths"))
    rp, fp, pp = f64(st["repetition"]), f64(st["frequency"]), f64(st["presence"])
    ids, vals = (None, None) if st["bias_ids"] is None else (st["bias_ids"].cpu().numpy(),
                                                            f64(st["bias_values"]))
    words = None if st["allowed"] is None else st["allowed"].cpu().numpy().view(np.uint32)
    for b in range(l.shape[0]):
        live = tok[b, :ln[b]].astype(np.int64)
        seen = np.unique(live)
        row = l[b]
        row[seen] = np.where(row[seen] > 0, row[seen] / rp[b], row[seen] * rp[b])
        gen, times = np.unique(live[pl[b]:], return_counts=True)
        row[gen] -= fp[b] * times + pp[b]
        if ids is not None:
            row[ids[b]] += vals[b]
        if words is not None:
            bits = np.unpackbits(words[b].astype("<u4").view(np.uint8), bitorder="little")[:V]
            row[bits == 0] = -np.inf
    return l
