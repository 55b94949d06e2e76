"""Layer norm in front of the LM head and sampling behind it, as cases that can be
timed and checked.

* ``layer_norm``: the norm with mean, weight and bias, with the residual's
  addition; forward and backward (training) or with an 8-bit output and scales
  (serving).
* ``sample_logits``: a token a row by temperature, top-k, top-p and min-p, from a
  given random number.

``run`` computes a case in its plain form, from elementary torch operations, or,
where ``own`` is set, by the calls a user makes of the package.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
GROUP = 128          # columns that share a scale
FP8_MAX = 448.0
AMAX_MIN = 2.0 ** -100
GREEDY = 2.0 ** -64  # temperatures below it take the largest logit
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence decodes one token: latency of the final norm
        {"name": "layer norm fp8, one token", "op": "norm_fp8", "N": 1, "H": 4096,
         "dtype": "bf16", "residual": True},
        # a ragged prefill batch into an 8-bit linear layer
        {"name": "layer norm fp8, ragged batch", "op": "norm_fp8", "N": 777, "H": 2056,
         "dtype": "f32", "residual": False},
        # a training step's final norm, forward and backward
        {"name": "layer norm train 8192 x 3584", "op": "norm_train", "N": 8192, "H": 3584,
         "dtype": "bf16", "residual": True},
        # an odd width, no residual: a norm over a small model's features
        {"name": "layer norm train odd, float32", "op": "norm_train", "N": 1021, "H": 1001,
         "dtype": "f32", "residual": False},
        # a long context in float32
        {"name": "layer norm train 16384 x 2048, float32", "op": "norm_train", "N": 16384,
         "H": 2048, "dtype": "f32", "residual": True},
        # one sequence: latency of picking a token
        {"name": "sample, one row", "op": "sample", "B": 1, "V": 152064, "dtype": "bf16",
         "limits": "kp", "masked": False},
        # a serving batch, every limit in use, some requests with grammars
        {"name": "sample, 64 rows", "op": "sample", "B": 64, "V": 151936, "dtype": "bf16",
         "limits": "kpm", "masked": True},
        # a large batch of processed (float32) logits
        {"name": "sample, 256 rows", "op": "sample", "B": 256, "V": 152064, "dtype": "f32",
         "limits": "kp", "masked": True},
        # nucleus sampling alone: all of the vocabulary counts in the mass
        {"name": "sample, top-p alone", "op": "sample", "B": 64, "V": 152064, "dtype": "f32",
         "limits": "p", "masked": False},
        # a small vocabulary of no round size, min-p alone
        {"name": "sample, min-p alone, odd", "op": "sample", "B": 37, "V": 32003, "dtype": "f32",
         "limits": "m", "masked": False},
        # rollouts for reinforcement learning: the distribution as it is
        {"name": "sample, temperature alone", "op": "sample", "B": 256, "V": 128255,
         "dtype": "bf16", "limits": "", "masked": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fp8", "norm_train", "sample", "sample"])
    if op != "sample":
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        N = min(_log_int(rng, 1, 16384), 8192 * 3584 // H)
        return {"op": op, "N": N, "H": H, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.7}
    return {"op": op, "B": _log_int(rng, 1, 256), "V": _log_int(rng, 1000, 152064),
            "dtype": rng.choice(["bf16", "f32"]),
            "limits": rng.choice(["", "k", "p", "m", "kp", "kp", "pm", "kpm"]),
            "masked": rng.random() < 0.4}


def _groups(n):
    return -(-n // GROUP)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")
    st = {"op": case["op"]}
    if case["op"] != "sample":
        N, H, dt = case["N"], case["H"], DTYPES[case["dtype"]]
        # the residual stream is larger than a layer's output, has a few large channels
        # and a mean
        st["x"] = normal(N, H).to(dt)
        st["residual"] = None
        if case["residual"]:
            res = normal(N, H) * 3 + 0.5
            res[:, ::97] *= 8
            st["residual"] = res.to(dt)
        st["weight"] = (1 + 0.2 * normal(H)).to(dt)
        st["bias"] = (0.1 * normal(H)).to(dt)
        if case["op"] == "norm_train":
            st["dy"] = (0.02 * normal(N, H)).to(dt)
            st["dres"] = (0.01 * normal(N, H)).to(dt) if case["residual"] else None
        return st
    B, V = case["B"], case["V"]
    # a broad bulk, and a few dozen continuations that are likely
    l = normal(B, V) * 2
    likely = torch.randint(0, V, (B, 40), generator=g, device="cuda")
    l.scatter_add_(1, likely, 4 + 8 * uniform(B, 40))
    if case["masked"]:
        allowed = uniform(B, V) < 0.3
        allowed[::3] = True              # requests without a grammar allow everything
        if B > 4:
            allowed[4] = False           # a grammar that has run into a dead end
        l = torch.where(allowed, l, -math.inf)
    st["logits"] = l.to(DTYPES[case["dtype"]])
    st["u"] = uniform(B)
    # each request has its own settings; about one in eight leaves a limit off
    st["temperature"] = 0.5 + uniform(B)
    st["top_k"] = st["top_p"] = st["min_p"] = None
    if "k" in case["limits"]:
        st["top_k"] = torch.exp(uniform(B) * math.log(1000)).to(torch.int32).clamp_(min=1)
        st["top_k"][0] = 50
        st["top_k"][7::8] = 0
    if "p" in case["limits"]:
        st["top_p"] = 0.5 + 0.49 * uniform(B)
        st["top_p"][6::8] = 1.0
    if "m" in case["limits"]:
        st["min_p"] = 0.2 * uniform(B)
        st["min_p"][5::8] = 0.0
    if B > 2:
        st["temperature"][2] = 0.0       # a request that decodes greedily
    return st


# ------------------------------------------------------------- plain forms
def _plain_quantize(y):
    """Groups of 128 columns: a = max |y|, scale = a / 448, q = e4m3(y * (448 / a))."""
    N, H = y.shape
    pad = torch.zeros(N, _groups(H) * GROUP, device=y.device)
    pad[:, :H] = y
    pad = pad.view(N, _groups(H), GROUP)
    amax = pad.abs().amax(2).clamp(min=AMAX_MIN)
    q = (pad * (FP8_MAX / amax)[:, :, None]).view(N, -1)[:, :H].to(torch.float8_e4m3fn)
    return [q.contiguous(), amax / FP8_MAX]


def _plain_norm(st):
    x, w, dt = st["x"].float(), st["weight"].float(), st["x"].dtype
    h = x if st["residual"] is None else x + st["residual"].float()
    d = h - h.mean(1, keepdim=True)
    r = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    n = d * r
    y = n * w + st["bias"].float()
    sums = [] if st["residual"] is None else [h.to(dt)]
    if st["op"] == "norm_fp8":
        return _plain_quantize(y) + sums
    dy = st["dy"].float()
    g = dy * w
    dx = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return [y.to(dt)] + sums + [dx.to(dt), (dy * n).sum(0).to(dt), dy.sum(0).to(dt)]


def _plain_sample(st):
    """In 64 bits: next to a border of the cumulative mass 32 pick another token."""
    l = st["logits"].double()
    B, V = l.shape
    top = l.amax(1, keepdim=True)
    alive = top > -math.inf
    T = st["temperature"].double()[:, None]
    greedy = T < GREEDY
    w = torch.exp((l - torch.where(alive, top, 0.0)) / torch.where(greedy, 1.0, T))
    ordered, order = torch.sort(l, dim=1, descending=True, stable=True)
    mass = w.gather(1, order)
    rank = torch.arange(V, device=l.device)
    first = rank == 0
    keep = ordered > -math.inf
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        keep = keep & ((rank < k) | (k <= 0))
    mass = torch.where(keep, mass, 0.0)
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        before = mass.cumsum(1) - mass
        keep = keep & ((p >= 1) | (before < p * mass.sum(1, keepdim=True)) | first)
    if st["min_p"] is not None:
        keep = keep & ((mass >= st["min_p"].double()[:, None]) | first)
    keep = torch.where(greedy, first, keep)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    mass = torch.where(kept, w, 0.0).cumsum(1)
    token = (mass <= st["u"].double()[:, None] * mass[:, -1:]).sum(1)
    return torch.where(alive[:, 0], token, -1)


def run(st):
    if not own:
        return _plain_sample(st) if st["op"] == "sample" else _plain_norm(st)
    import lm_head_linear_flce_gb300 as flce
    if st["op"] == "sample":
        return flce.sample_logits(st["logits"], st["u"], temperature=st["temperature"],
                                  top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
    if st["op"] == "norm_fp8":
        return list(flce.layer_norm_fp8(st["x"], st["weight"], st["bias"], eps=EPS,
                                        residual=st["residual"]))
    y, h, mean, rstd = flce.flce_layer_norm(st["x"], st["weight"], st["bias"], eps=EPS,
                                            residual=st["residual"])
    grads = flce.flce_layer_norm_backward(st["dy"], h, st["weight"], mean, rstd, dh=st["dres"])
    return [y] + ([] if st["residual"] is None else [h]) + list(grads)


# ---------------------------------------------------------- work and truth
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        return {"bytes": B * V * e + B * (16 + 4 * len(case["limits"])), "flops": 4 * B * V}
    N, H, res = case["N"], case["H"], 1 if case["residual"] else 0
    if case["op"] == "norm_fp8":
        return {"bytes": N * H * (e * (1 + 2 * res) + 1) + 4 * N * _groups(H) + 2 * e * H,
                "flops": 10 * N * H}
    # x, dy in, y, dx out; with a residual: it and its gradient in, the sum out
    return {"bytes": N * H * e * (4 + 3 * res) + 4 * e * H, "flops": 20 * N * H}


def _round_e4m3(v):
    """float64 values rounded to the nearest e4m3 value, ties to even."""
    a = np.abs(v)
    e = np.maximum(np.frexp(np.where(a > 0, a, 1.0))[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, FP8_MAX), v)


def _exact_norm(case, st):
    x, res, w, b, dy, dres = (None if st.get(k) is None else st[k].double().cpu().numpy()
                              for k in ("x", "residual", "weight", "bias", "dy", "dres"))
    h = x if res is None else x + res
    H = h.shape[1]
    mean = np.einsum("nh->n", h) / H
    var = np.einsum("nh,nh->n", h, h) / H - mean ** 2  # (64 bits: the difference is harmless)
    sd = np.sqrt(var + EPS)
    u = (h - mean[:, None]) / sd[:, None]
    y = u * w + b
    sums = [] if res is None else [h]
    if case["op"] == "norm_fp8":
        q, s = np.empty_like(y), np.empty((y.shape[0], _groups(H)))
        for j in range(s.shape[1]):
            c = slice(j * GROUP, (j + 1) * GROUP)
            s[:, j] = np.maximum(np.abs(y[:, c]).max(1), AMAX_MIN) / FP8_MAX
            q[:, c] = _round_e4m3(y[:, c] / s[:, j, None])
        return [q, s] + sums
    du = dy * w
    # what the mean and the standard deviation take out of du: its parts along 1 and u
    along = np.einsum("nh,nh->n", du, u) / H
    dx = (du - (np.einsum("nh->n", du) / H)[:, None] - u * along[:, None]) / sd[:, None]
    if dres is not None:
        dx += dres
    return [y] + sums + [dx, np.einsum("nh,nh->h", dy, u), dy.sum(0)]


def _exact_sample(st):
    """Row by row, on the tokens that are left after each limit."""
    settings = {k: None if st[k] is None else st[k].double().cpu().numpy()
                for k in ("u", "temperature", "top_k", "top_p", "min_p")}
    logits = st["logits"].double().cpu().numpy()
    out = np.empty(logits.shape[0], np.int64)
    for b, l in enumerate(logits):
        u, T, k, p, m = (None if v is None else v[b] for v in settings.values())
        ids = np.flatnonzero(l > -np.inf)
        if not ids.size:
            out[b] = -1
            continue
        if T < GREEDY:
            out[b] = l.argmax()
            continue
        ids = ids[np.argsort(-l[ids], kind="stable")]
        if k is not None and k > 0:
            ids = ids[:int(k)]
        w = np.exp((l[ids] - l[ids[0]]) / T)
        if p is not None and p < 1:
            n = 1 + np.searchsorted(np.cumsum(w)[:-1], p * w.sum(), side="left")
            ids, w = ids[:n], w[:n]
        if m is not None:
            n = max(1, np.count_nonzero(w >= m))
            ids, w = ids[:n], w[:n]
        by_id = np.argsort(ids)
        mass = np.cumsum(w[by_id])
        out[b] = ids[by_id[np.searchsorted(mass, u * mass[-1], side="right")]]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_sample(st) if case["op"] == "sample" else _exact_norm(case, st)
