"""Sampling against the float64 definition.

Tolerance.  A weight is right to 2^-29 of it and 2^-43 of the largest (at least one weight
is 1), so a share of the mass is to E = 2^-28 + V 2^-42.  The token has to be one
that the definition takes for a u, a top_p and a min_p that are each off by up to E:
where none of them is that close to a border, it is the definition's own."""
import threading

import numpy as np
import pytest
import torch

from oracle import head_ops as ref

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def accepted(l, u, T, k, p, m, token):
    e = 2.0 ** -28 + l.size * 2.0 ** -42
    u = min(max(0.0 if np.isnan(u) else u, 0.0), 1 - 2.0 ** -24)
    if ref.sample(l, u, T, k, p, m) == token:
        return True
    for q in (p,) if p >= 1 else (p - e, p, p + e):
        for n in (m * (1 - e), m, m * (1 + e)):
            lo, hi = (ref.sample(l, v, T, k, q, n) for v in (u - e, u + e))
            if lo <= token <= hi and l[token] > -INF:
                return True
    return False


def check(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    got = flce.sample_logits(logits, u, temperature=temperature, top_k=top_k, top_p=top_p,
                             min_p=min_p)
    assert got.dtype == torch.int64 and got.shape == logits.shape[:1]
    l, got_, u_ = logits.double().cpu().numpy(), got.tolist(), u.tolist()
    T, k, p, m = ([d] * len(got_) if t is None else t.tolist() for t, d in
                  ((temperature, 1.0), (top_k, 0), (top_p, 1.0), (min_p, 0.0)))
    p = [1.0 if np.isnan(v) or v > 1 else v for v in p]
    m = [0.0 if np.isnan(v) else v for v in m]
    for b, token in enumerate(got_):
        assert accepted(l[b], u_[b], T[b], k[b], p[b], m[b], token), \
            (b, token, u_[b], T[b], k[b], p[b], m[b])
    return got


def rand(g, *s):
    return torch.rand(*s, generator=g).cuda()


def ints(g, n, hi):
    return torch.randint(0, hi, (n,), generator=g).int().cuda()


def rows(kind, B, V, g):
    r = torch.randn(B, V, generator=g)
    return {"normal": lambda: r * 3, "equal": lambda: r * 0, "two": lambda: (r > 0).float(),
            "wide": lambda: r * 300, "close": lambda: r * 1e-4, "sorted": lambda: r.sort(1)[0],
            "masked": lambda: torch.where(torch.rand(B, V, generator=g) < 0.02, r, -INF),
            "lowest": lambda: torch.where(torch.rand(B, V, generator=g) < 0.1, r,
                                          torch.finfo(BF).min)}[kind]()


SIZES = [1, 2, 7, 8, 31, 33, 257, 1000, 2049, 4099, 50257]
KINDS = ["normal", "equal", "two", "wide", "close", "sorted", "masked", "lowest"]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", SIZES)
def test_each_limit_and_all_of_them(V, kind, dt):
    g = torch.Generator().manual_seed(V)
    B = 4 if V > 9000 else 8
    l = rows(kind, B, V, g).to(dt).cuda()
    u, T, k = rand(g, B), rand(g, B) * 2 + 0.05, ints(g, B, min(V, 2000) + 2)
    p, m = rand(g, B), rand(g, B) * 0.5
    check(l, u)
    check(l, u, T)
    check(l, u, T, top_k=k)
    check(l, u, T, top_p=p)
    check(l, u, T, min_p=m * 0.2)
    check(l, u, T, k, p, m)
    check(l, u, T, k, 1 - p * 1e-3)
    check(l, u, None, None, p, m * 0.01)


@pytest.mark.parametrize("B,V,dt", [(1, 152064, BF), (3, 152064, F32), (2, 128255, BF),
                                    (1, 1 << 21, BF), (2, (1 << 21) - 1, F32)])
def test_long_rows(B, V, dt):
    g = torch.Generator().manual_seed(V)
    for scale in (1.0, 4.0):
        l = (torch.randn(B, V, generator=g) * scale).to(dt).cuda()
        u, T = rand(g, B), rand(g, B) + 0.3
        check(l, u, T)
        check(l, u, T, top_k=ints(g, B, 100) + 1, top_p=rand(g, B))
        check(l, u, T, top_k=ints(g, B, V))
        check(l, u, T, top_p=rand(g, B))
        check(l, u, T, top_p=1 - rand(g, B) * 1e-4, min_p=rand(g, B) * 1e-3)


@pytest.mark.parametrize("B", [1, 37, 44, 53, 66, 76, 77, 88, 133, 152, 153, 400])
def test_rows_by_one_cta_or_several(B):
    """However many rows there are, each gives what it gives alone."""
    g = torch.Generator().manual_seed(B)
    l = (torch.randn(B, 9001, generator=g) * 2).cuda()
    u, T, k, p = rand(g, B), rand(g, B) + 0.2, ints(g, B, 3000), rand(g, B)
    some = list(range(0, B, max(1, B // 5)))
    for lim in (dict(), dict(temperature=T, top_k=k), dict(temperature=T, top_p=p),
                dict(temperature=T, top_k=k, top_p=p), dict(min_p=p * 0.1)):
        got = flce.sample_logits(l, u, **lim)
        sub = check(l[some], u[some], *(lim[n][some] if n in lim else None for n in
                                        ("temperature", "top_k", "top_p", "min_p")))
        for b, token in zip(some, sub.tolist()):
            assert got[b].item() == token or accepted(
                l[b].double().cpu().numpy(), u[b].item(),
                *((lim[n][b].item() if n in lim else d) for n, d in
                  (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))),
                got[b].item())
        assert (got >= 0).all() and (got < 9001).all()


def test_edges_of_the_arguments():
    g = torch.Generator().manual_seed(5)
    V = 300
    l = torch.randn(1, V, generator=g).cuda() * 2
    for name, values in (("u", [0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, NAN, INF, -INF, 2.0 ** -149]),
                         ("temperature", [0.0, -1.0, NAN, 2.0 ** -65, 2.0 ** -63, 1e-6, 1e-3, 1e3,
                                          1e30, 3e38, INF]),
                         ("top_p", [0.0, -1.0, 1e-30, 1e-7, 0.5, 0.9999, 1 - 2.0 ** -24, 1.0, 2.0,
                                    NAN, INF, -INF]),
                         ("min_p", [0.0, -1.0, 1e-30, 1e-7, 0.5, 1 - 2.0 ** -24, 1.0, 1.5, NAN, INF,
                                    -INF])):
        n = len(values)
        t = torch.tensor(values, device="cuda")
        z = l.expand(n, V).contiguous()
        u = rand(g, n)
        if name == "u":
            for kw in (dict(), dict(top_k=ints(g, n, V)), dict(top_p=rand(g, n))):
                check(z, t, **kw)
        else:
            for v in (u, u * 0, u * 0 + 1):
                check(z, v, **{name: t})
    k = torch.tensor([0, -1, -2 ** 31, 1, 2, V - 1, V, V + 1, 2 ** 31 - 1], dtype=torch.int32)
    check(l.expand(9, V).contiguous(), rand(g, 9), top_k=k.cuda())
    # the largest weighs alone below a temperature of 2^-64, whatever the limits
    u = rand(g, 3)
    z = l.expand(3, V).contiguous()
    z[:, 7] = z[:, 100] = 50.0  # equals: the lowest id
    got = flce.sample_logits(z, u, temperature=torch.tensor([0.0, 1e-30, NAN], device="cuda"),
                             top_k=ints(g, 3, 5) + 2, top_p=rand(g, 3))
    assert got.tolist() == [7, 7, 7]


@pytest.mark.parametrize("V", [40, 3000, 40000])
def test_zeros_of_both_signs_are_equal(V):
    g = torch.Generator().manual_seed(11)
    for dt in (BF, F32):
        l = torch.where(torch.rand(6, V, generator=g) < 0.5, 0.0, -0.0)
        l[3:] -= (torch.rand(3, V, generator=g) < 0.3).float() * 1e-3
        l = l.to(dt).cuda()
        u, k, p = rand(g, 6), ints(g, 6, V), rand(g, 6)
        for kw in (dict(), dict(top_k=k), dict(top_k=k % 20 + 1), dict(top_p=p),
                   dict(top_k=k, top_p=p), dict(min_p=p)):
            check(l, u, **kw)


def test_values_that_are_no_numbers():
    V = 700
    g = torch.Generator().manual_seed(6)
    for dt in (BF, F32):
        l = torch.randn(9, V, generator=g)
        l[0] = -INF
        l[1] = NAN
        l[2, ::3] = NAN
        l[3, [5, 600]] = INF
        l[4, 1:] = -INF
        l[5, :-1] = NAN
        l[6] = INF
        l[7, 3], l[7, 4] = torch.finfo(BF).max, torch.finfo(BF).min
        l[8] = torch.finfo(BF).min
        l = l.to(dt).cuda()
        u, k = rand(g, 9), ints(g, 9, 9)
        for kw in (dict(), dict(top_k=k), dict(top_p=u.flip(0)), dict(min_p=u * 0.1),
                   dict(temperature=u * 0), dict(temperature=u * 1e-3),
                   dict(temperature=u + 0.5, top_k=k, top_p=u.flip(0), min_p=u * 0.1)):
            got = check(l, u, **kw).tolist()
            assert got[:2] == [-1, -1] and got[4] == 0 and got[5] == V - 1 and got[3] in (5, 600)


@pytest.mark.parametrize("dt", [BF, F32])
def test_strides_and_alignment(dt):
    g = torch.Generator().manual_seed(7)
    for V in (1003, 20000):
        big = torch.randn(6, V + 40, generator=g).to(dt).cuda()
        u, k, p = rand(g, 6), ints(g, 6, 80) + 1, rand(g, 6)
        for lo in (0, 1, 2, 3, 5, 8, 31):
            z = big[:, lo:lo + V]
            for kw in (dict(), dict(top_k=k), dict(top_p=p), dict(top_k=k, min_p=p * 0.1)):
                got = check(z, u, **kw)
                # the same tokens but where a u lies on a border
                same = flce.sample_logits(z.contiguous(), u, **kw)
                assert (got == same).sum() >= 5
    # the row in front and the one behind are not read as part of it
    z = torch.full((3, 1001), 99.0, dtype=dt).cuda()
    z[1] = torch.randn(1001, generator=g).to(dt).cuda()
    check(z[1:2], rand(g, 1))
    wide = torch.full((4, 2000), 99.0, dtype=dt).cuda()
    wide[:, 500:1501] = torch.randn(4, 1001, generator=g).to(dt).cuda()
    check(wide[:, 500:1501], rand(g, 4), top_k=ints(g, 4, 50))
    # parameters with strides, rows in reverse order of memory, an expanded row
    z = torch.randn(8, 512, generator=g).to(dt).cuda()
    par = rand(g, 8, 4)
    check(z[::2], par[::2, 0], par[::2, 1] + 0.1, top_p=par[::2, 2], min_p=par[::2, 3])
    check(z[:1].expand(5, 512), par[:5, 0])
    check(torch.randn(512, 4, generator=g).to(dt).cuda().t(), par[:4, 1])


def test_a_matrix_past_2_31_elements():
    V, B = 1 << 16, 40000  # 5.2 GB of bf16
    l = torch.zeros(B, V, dtype=BF, device="cuda")
    at = torch.randint(0, V, (B,), device="cuda")
    l.scatter_(1, at[:, None], 100.0)
    u = torch.rand(B, device="cuda")
    k = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    assert torch.equal(flce.sample_logits(l, u), at)
    assert torch.equal(flce.sample_logits(l, u, top_k=k, top_p=u), at)


@pytest.mark.parametrize("dt", [BF, F32])
def test_borders_among_more_tokens_than_a_list_holds(dt):
    g = torch.Generator().manual_seed(13)
    V = 60000
    for l in (torch.randn(5, V, generator=g) * 0.02, torch.randn(5, V, generator=g).round(),
              -4 + torch.randn(5, V, generator=g).round() / 64, torch.full((5, V), -3.0),
              torch.randn(5, V, generator=g).sign() * 1e-3):
        l = l.to(dt).cuda()
        u, p, T = rand(g, 5), rand(g, 5), rand(g, 5) + 0.5
        k = torch.tensor([3, 1024, 1025, 5000, V - 1], dtype=torch.int32, device="cuda")
        for kw in (dict(top_p=p), dict(top_p=1 - p * 1e-3), dict(top_k=k), dict(top_k=k, top_p=p),
                   dict(top_k=k, top_p=p, min_p=p * 0.9)):
            check(l, u, T, **kw)


@pytest.mark.parametrize("dt", [BF, F32])
def test_temperatures_from_end_to_end(dt):
    g = torch.Generator().manual_seed(12)
    T = torch.tensor([2.0 ** -63, 1e-15, 1e-9, 1e-7, 1e-6, 1e-5, 1e-4, 1e-3, 1e-2, 0.1, 10.0, 1e3,
                      1e6, 1e20, 2.0 ** 99, 2.0 ** 101], device="cuda")
    n = T.numel()
    for V, scale, shift in ((5000, 3.0, 0.0), (5000, 1e-3, 100.0), (70000, 1e4, -3e4),
                            (5000, 1e36, 0.0), (5000, 1e-30, 0.0)):
        l = (torch.randn(1, V, generator=g) * scale + shift).to(dt).cuda().expand(n, V).contiguous()
        u, k, p = rand(g, n), ints(g, n, 900) + 1, rand(g, n)
        for kw in (dict(), dict(top_k=k), dict(top_p=p), dict(top_p=1 - p * 1e-5),
                   dict(top_k=k, top_p=p), dict(min_p=p)):
            check(l, u, T, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=6), dict(top_p=0.8), dict(min_p=0.2)])
def test_each_token_takes_its_share_of_u(kw):
    n, V = 4096, 11
    g = torch.Generator().manual_seed(8)
    l = (torch.randn(1, V, generator=g) * 1.5).cuda()
    u = ((torch.arange(n) + 0.5) / n).cuda()
    par = {a: torch.full((n,), v, device="cuda", dtype=torch.int32 if a == "top_k" else F32)
           for a, v in kw.items()}
    got = flce.sample_logits(l.expand(n, V).contiguous(), u, **par)
    assert (got[1:] >= got[:-1]).all()  # in the order of u
    w = np.exp(l[0].double().cpu().numpy())
    order = np.argsort(-w)
    if "top_k" in kw:
        w[order[6:]] = 0
    if "top_p" in kw:
        before = np.cumsum(w[order]) - w[order]
        w[order[before >= np.float64(np.float32(0.8)) * w.sum()]] = 0
    if "min_p" in kw:
        w[w < np.float64(np.float32(0.2)) * w.max()] = 0
    share = np.bincount(got.cpu().numpy(), minlength=V) / n
    assert np.abs(share - w / w.sum()).max() <= 1.0 / n
    assert (share[w == 0] == 0).all()


def test_the_same_every_time_in_a_graph_and_on_other_streams():
    g = torch.Generator().manual_seed(9)
    B, V = 20, 50257
    l = (torch.randn(B, V, generator=g) * 2).to(BF).cuda()
    u, T, k, p = rand(g, B), rand(g, B) + 0.5, ints(g, B, 3000), rand(g, B)
    kws = [dict(temperature=T), dict(temperature=T, top_k=k), dict(temperature=T, top_p=p),
           dict(temperature=T, top_k=k, top_p=p, min_p=p * 0.01)]
    want = [flce.sample_logits(l, u, **kw) for kw in kws]
    for _ in range(3):
        assert all(torch.equal(flce.sample_logits(l, u, **kw), w) for kw, w in zip(kws, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ll = l * 1
        got = [flce.sample_logits(ll, u, **kw) for kw in kws]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    z, v = torch.zeros_like(l), torch.zeros_like(u)
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([flce.sample_logits(z, v, **kw) for kw in kws])
        graphs.append(graph)
    z.copy_(l), v.copy_(u)  # a replay reads what is there then
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(side):  # both at once
        graphs[1].replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_calls_from_two_threads():
    g = torch.Generator().manual_seed(10)
    l = (torch.randn(6, 9000, generator=g) * 2).cuda()
    u, k = rand(g, 6), ints(g, 6, 40) + 1
    want = flce.sample_logits(l, u, top_k=k)
    torch.cuda.synchronize()
    wrong = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                if not torch.equal(flce.sample_logits(l, u, top_k=k), want):
                    wrong.append(1)
    threads = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in threads], [t.join() for t in threads]
    assert not wrong


def test_no_rows_and_writes_stay_inside():
    z = torch.empty(0, 1000, device="cuda")
    assert flce.sample_logits(z, torch.empty(0, device="cuda")).shape == (0,)
    # the C call, into the middle of a buffer
    from lm_head_linear_flce_gb300 import head_ops
    out = torch.full((9,), 77, dtype=torch.int64, device="cuda")
    l, u = torch.randn(5, 4099, device="cuda"), torch.rand(5, device="cuda")
    head_ops._call("flce_sample_logits", l.device.index, l.data_ptr(), 4099, 1, 5, 4099,
                   u.data_ptr(), None, None, None, None, out[2:].data_ptr())
    assert out[[0, 1, 7, 8]].tolist() == [77] * 4
    assert torch.equal(out[2:7], flce.sample_logits(l, u))


def test_refusals():
    l, u = torch.randn(4, 100, device="cuda"), torch.rand(4, device="cuda")
    k = torch.ones(4, dtype=torch.int32, device="cuda")
    for call in (lambda: flce.sample_logits(l[0], u), lambda: flce.sample_logits(l.half(), u),
                 lambda: flce.sample_logits(l, u[:3]), lambda: flce.sample_logits(l, u.double()),
                 lambda: flce.sample_logits(l, u.cpu()), lambda: flce.sample_logits(l, u, top_k=u),
                 lambda: flce.sample_logits(l, u, top_k=k.long()),
                 lambda: flce.sample_logits(l, u, temperature=k),
                 lambda: flce.sample_logits(l, u, top_p=u[:2]),
                 lambda: flce.sample_logits(l, u, min_p=u[:, None]),
                 lambda: flce.sample_logits(l, u, temperature=u.to(BF))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(flce.FlceError):
        flce.sample_logits(torch.empty(2, (1 << 21) + 1, device="cuda"), u[:2])
    with pytest.raises(ValueError):
        flce.sample_logits(torch.empty(2, 0, device="cuda"), u[:2])
    x = l.clone().requires_grad_()
    assert not flce.sample_logits(x, u).requires_grad
