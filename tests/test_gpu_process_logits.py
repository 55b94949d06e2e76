"""Penalties, biases and masks on logits against the float64 definition.

Tolerance per element: at most five float32 roundings of intermediate values no
larger than |l| * r + |f| c + |p| + |bias| (r the repetition's factor), and one
rounding to the output type."""
import numpy as np
import pytest
import torch

from oracle import head_ops as ref

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

BF, F32 = torch.bfloat16, torch.float32


def case(B, V, L, nb, dt=F32, ids=torch.int64, seed=0):
    g = torch.Generator().manual_seed(seed)
    k = dict(tokens=torch.randint(-3, V + 5, (B, L), generator=g).clamp(max=V + 2).to(ids),
             lengths=torch.randint(0, L + 1, (B,), generator=g).int(),
             repetition_penalty=torch.rand(B, generator=g) + 0.6,
             frequency_penalty=torch.randn(B, generator=g) * 0.5,
             presence_penalty=torch.randn(B, generator=g) * 0.5)
    if L:  # many repeats of a few ids
        k["tokens"][:, ::2] = torch.randint(0, min(V, 7), k["tokens"][:, ::2].shape,
                                            generator=g).to(ids)
        k["lengths"][0] = L
    k["prompt_lengths"] = (k["lengths"].float() * torch.rand(B, generator=g)).int()
    if nb:
        k["bias_ids"] = torch.randint(-1, V + 1, (B, nb), generator=g).to(ids)
        k["bias_values"] = torch.randn(B, nb, generator=g) * 5
    words = (V + 31) // 32
    k["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=g).int()
    k["allowed"][0] = -1
    if B > 2:
        k["allowed"][2] = 0
    z = (torch.randn(B, V, generator=g) * 4).to(dt)
    return z, k


def oracle(z, k):
    names = dict(repetition_penalty="repetition", frequency_penalty="frequency",
                 presence_penalty="presence")
    kk = {names.get(n, n): (t.double().numpy() if t.is_floating_point() else t.numpy())
          for n, t in k.items() if t is not None}
    return ref.process_logits(z.double().numpy(), **kk)


def run(z, k, **kw):
    return flce.process_logits(z.cuda(), **{n: None if t is None else t.cuda()
                                            for n, t in k.items()}, **kw)


def check(got, z, k):
    want = oracle(z, k)
    B, V = z.shape
    size = np.abs(z.double().numpy()) * 2
    if k.get("tokens") is not None:
        L = k["tokens"].shape[1]
        for n in ("frequency_penalty", "presence_penalty"):
            if k.get(n) is not None:
                size = size + np.abs(k[n].double().numpy())[:, None] * (L if n[0] == "f" else 1)
    if k.get("bias_values") is not None:
        size = size + np.abs(k["bias_values"].double().numpy()).max(1)[:, None]
    g = got.detach().double().cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(g)) and np.array_equal(np.isneginf(want), np.isneginf(g))
    tol = 5 * 2.0 ** -24 * size
    if got.dtype == BF:
        tol = tol + 1.01 * 2.0 ** -8 * np.abs(np.where(fin, want, 0))
    assert (np.abs(np.where(fin, g - np.where(fin, want, 0), 0)) <= tol).all()


SHAPES = [(1, 1, 1, 1), (1, 31, 0, 0), (2, 32, 5, 2), (3, 33, 100, 0), (5, 1000, 17, 300),
          (4, 8191, 300, 3), (2, 8193, 2000, 1), (3, 20000, 5000, 20), (1, 70001, 3000, 9),
          (6, 152064, 700, 5), (2, 300000, 40, 2), (130, 257, 64, 4)]


@pytest.mark.parametrize("dt,odt", [(BF, F32), (F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("B,V,L,nb", SHAPES)
def test_matches_the_definition(B, V, L, nb, dt, odt):
    z, k = case(B, V, L, nb, dt, torch.int32 if B % 2 else torch.int64, seed=V)
    check(run(z, k, out_dtype=odt), z, k)


@pytest.mark.parametrize("drop", ["tokens", "lengths", "prompt_lengths", "repetition_penalty",
                                  "frequency_penalty", "presence_penalty", "bias", "allowed",
                                  "all"])
def test_any_part_may_be_left_out(drop):
    z, k = case(4, 3000, 200, 6, BF, seed=1)
    if drop == "all":
        assert torch.equal(run(z, {}).cpu(), z)
        return
    gone = {"tokens": ["tokens", "lengths", "prompt_lengths"],
            "bias": ["bias_ids", "bias_values"]}.get(drop, [drop])
    for n in gone:
        k[n] = None
    check(run(z, k, out_dtype=F32), z, k)


@pytest.mark.parametrize("L", [20, 20000])
@pytest.mark.parametrize("V", [1001, 50000, 152064])
def test_long_histories_count_exactly(V, L):
    """Frequencies that are small integers and zero logits: the result is
    exactly -count."""
    g = torch.Generator().manual_seed(V)
    B = 3
    tok = torch.randint(0, V, (B, L), generator=g)
    tok[:, : L // 2] = torch.randint(0, 3, (B, L // 2), generator=g) * (V // 3)
    out = run(torch.zeros(B, V), dict(tokens=tok, frequency_penalty=torch.ones(B)))
    want = torch.zeros(B, V).scatter_add_(1, tok, -torch.ones(B, L))
    assert torch.equal(out.cpu(), want)


def test_lengths_are_clamped():
    z, k = case(3, 100, 10, 0, seed=2)
    k["lengths"] = torch.tensor([-5, 1000, 4], dtype=torch.int32)
    k["prompt_lengths"] = torch.tensor([3, 2000, -7], dtype=torch.int32)
    got = run(z, k)
    k["lengths"] = torch.tensor([0, 10, 4], dtype=torch.int32)
    check(got, z, k)


@pytest.mark.parametrize("dt", [BF, F32])
def test_in_place_and_strided(dt):
    for V in (1000, 1003, 40001):
        z, k = case(4, V, 50, 5, dt, seed=3)
        want = run(z, k)
        mine = z.cuda()
        assert flce.process_logits(mine, out=mine, **{n: t.cuda() for n, t in k.items()}) is mine
        assert torch.equal(mine, want)
        # rows of a wider buffer; its other columns stay as they are
        wide = torch.full((4, V + 13), 5.0, dtype=dt, device="cuda")
        wide[:, 3:V + 3] = z.cuda()
        view = wide[:, 3:V + 3]
        flce.process_logits(view, out=view, **{n: t.cuda() for n, t in k.items()})
        assert torch.equal(view, want)
        assert (wide[:, :3] == 5).all() and (wide[:, V + 3:] == 5).all()
        out = torch.full((4, V + 5), 9.0, device="cuda")
        flce.process_logits(z.cuda(), out=out[:, :V], **{n: t.cuda() for n, t in k.items()})
        assert (out[:, V:] == 9).all()
        # history and mask as views of longer buffers
        kk = {n: t.cuda() for n, t in k.items()}
        kk["tokens"] = torch.cat([kk["tokens"], torch.zeros_like(kk["tokens"])], 1)[:, :50]
        kk["allowed"] = torch.cat([kk["allowed"], kk["allowed"] * 0], 1)
        assert torch.equal(flce.process_logits(z.cuda(), **kk), want)


def test_non_finite_logits_and_empty_rows():
    z = torch.zeros(2, 64)
    z[0, 0], z[0, 1], z[0, 2], z[0, 3] = float("inf"), -float("inf"), float("nan"), -3e38
    k = dict(tokens=torch.tensor([[0, 1, 2, 3], [5, 5, 5, 5]]),
             repetition_penalty=torch.tensor([1.2, 1.0]))
    got = run(z, k).cpu()
    assert got[0, 0] == float("inf") and got[0, 1] == -float("inf") and torch.isnan(got[0, 2])
    assert got[0, 3] == -float("inf")  # beyond float32
    k["allowed"] = torch.zeros(2, 2, dtype=torch.int32)
    assert (run(z, k) == -float("inf")).all()
    e = flce.process_logits(torch.empty(0, 64, device="cuda"))
    assert e.shape == (0, 64)


def fast_oracle(z, k):
    """The definition, vectorised over a row (checked against the entry by entry
    one below): for batches of millions of columns."""
    out = z.double().numpy().copy()
    B, V = out.shape
    for b in range(B):
        tok = k["tokens"][b, :int(k["lengths"][b])].numpy().astype(np.int64)
        ok = (tok >= 0) & (tok < V)
        gen = ok & (np.arange(len(tok)) >= int(k["prompt_lengths"][b]))
        seen = np.unique(tok[ok])
        r = float(k["repetition_penalty"][b])
        out[b, seen] = np.where(out[b, seen] > 0, out[b, seen] / r, out[b, seen] * r)
        ids, times = np.unique(tok[gen], return_counts=True)
        out[b, ids] -= float(k["frequency_penalty"][b]) * times + float(k["presence_penalty"][b])
        if k.get("bias_ids") is not None:
            last = {int(v): i for i, v in enumerate(k["bias_ids"][b].tolist()) if 0 <= v < V}
            for v, i in last.items():
                out[b, v] += float(k["bias_values"][b, i])
        if k.get("allowed") is not None:
            w = k["allowed"][b].numpy().astype("<i4").view(np.uint8)
            out[b, np.unpackbits(w, bitorder="little")[:V] == 0] = -np.inf
    return out


def test_fast_oracle_is_the_definition():
    z, k = case(5, 3001, 200, 7, BF, seed=11)
    a, b = oracle(z, k), fast_oracle(z, k)
    assert np.array_equal(np.isfinite(a), np.isfinite(b))
    fin = np.isfinite(a)
    assert np.allclose(a[fin], b[fin], rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("dt,odt", [(BF, F32), (F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("B,V,L,nb,mask", [(30, 152064, 300, 300, True), (33, 128255, 3000, 0, True),
                                           (70, 60001, 20, 5, False), (9, 500000, 33000, 20, True),
                                           (40, 110000, 700, 600, True), (500, 8500, 32768, 3, True),
                                           (32, 131072, 0, 0, True), (5, 1000003, 100, 1, False)])
def test_large_batches(B, V, L, nb, mask, dt, odt):
    """Millions of columns: aligned and unaligned rows, histories around 2^15,
    more biases than a list holds, in place too where the types allow."""
    z, k = case(B, V, L, nb, dt, torch.int64 if nb % 2 else torch.int32, seed=B)
    if not mask:
        k["allowed"] = None
    want = fast_oracle(z, k)
    kk = {n: None if t is None else t.cuda() for n, t in k.items()}
    zz = z.cuda()
    got = flce.process_logits(zz, out_dtype=odt, **kk)
    size = np.abs(z.double().numpy()).max() * 2 + L * 2 + 40
    g = got.double().cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(g))
    tol = 5 * 2.0 ** -24 * size + (1.01 * 2.0 ** -8 * np.abs(want[fin]) if odt == BF else 0)
    assert (np.abs(g[fin] - want[fin]) <= tol).all()
    if dt == odt:
        assert flce.process_logits(zz, out=zz, **kk) is zz
        assert torch.equal(zz, got)
        wide = torch.full((B, V + 7), 3.0, dtype=dt, device="cuda")
        wide[:, 2:V + 2] = z.cuda()
        view = wide[:, 2:V + 2]
        flce.process_logits(view, out=view, **kk)
        assert torch.equal(view, got)
        assert (wide[:, :2] == 3).all() and (wide[:, V + 2:] == 3).all()
    del kk, zz, got


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_histories_of_every_start_and_length(offset, ids):
    # rows that begin anywhere in their 16 bytes and end anywhere in the next ones
    z, k = case(40, 300, 37, 0, ids=ids, seed=offset)
    wide = torch.full((40, 41 + offset), 5, dtype=ids)
    wide[:, offset:offset + 37] = k["tokens"]
    k["lengths"] = torch.arange(40).clamp(max=37).int()
    k["prompt_lengths"] = k["lengths"] // 2
    on_gpu = {n: None if t is None else t.cuda() for n, t in k.items()}
    on_gpu["tokens"] = wide.cuda()[:, offset:offset + 37]
    check(flce.process_logits(z.cuda(), **on_gpu), z, k)


def test_side_stream_and_graph():
    z, k = case(4, 40000, 3000, 5, BF, seed=4)
    want = run(z, k)
    zz, kk = z.cuda(), {n: t.cuda() for n, t in k.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = flce.process_logits(zz * 1, **kk)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = flce.process_logits(zz, **kk)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    z, k = case(3, 100, 10, 2)
    z, k = z.cuda(), {n: t.cuda() for n, t in k.items()}
    bad = [dict(k, tokens=k["tokens"][:2]), dict(k, tokens=k["tokens"].float()),
           dict(k, lengths=k["lengths"].long()), dict(k, lengths=k["lengths"][:2]),
           dict(k, bias_values=None), dict(k, bias_values=k["bias_values"][:, :1]),
           dict(k, allowed=k["allowed"][:, :3]), dict(k, allowed=k["allowed"].bool()),
           dict(k, repetition_penalty=k["repetition_penalty"].double()),
           dict(k, tokens=None), dict(k, out=z[:2]), dict(k, out=z, out_dtype=BF),
           dict(k, out=torch.empty(3, 100, device="cuda").half())]
    for kw in bad:
        with pytest.raises(ValueError):
            flce.process_logits(z, **kw)
    with pytest.raises(ValueError):
        flce.process_logits(z.half())
    buf = torch.zeros(6, 100, device="cuda")
    with pytest.raises(flce.FlceError):  # a shifted overlap
        flce.process_logits(buf[0:3], out=buf[1:4])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 1025, 2050, 4097, 8194, 40001])
def test_narrow_blocks_in_place(V, offset, dt):
    """Rows, or a row's last block, of fewer columns than a window, starting
    anywhere in one: each column is penalised once."""
    B, L = 5, 12
    z, k = case(B, V, L, 2, dt, seed=V + offset)
    k["allowed"] = None
    k["tokens"][:, ::3] = V - 1  # the last columns among them
    k["lengths"] = torch.full((B,), L, dtype=torch.int32)
    k["prompt_lengths"] = torch.arange(B, dtype=torch.int32)
    wide = torch.full((B, (V + offset + 11) // 4 * 4), 5.0, dtype=dt, device="cuda")
    view = wide[:, offset:offset + V]
    view.copy_(z)
    flce.process_logits(view, out=view, **{n: None if t is None else t.cuda()
                                           for n, t in k.items()})
    check(view, z, k)
    assert (wide[:, :offset] == 5).all() and (wide[:, offset + V:] == 5).all()


def test_a_written_tensor_counts_as_modified():
    z = torch.randn(3, 64, device="cuda")
    flce.process_logits(z, out=z)
    assert z._version == 1
    a = torch.randn(3, 64, device="cuda").requires_grad_()
    b = a * 2
    c = b.square()  # keeps b
    flce.process_logits(b.detach(), out=b.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        c.sum().backward()
    with torch.inference_mode():  # tensors without a version
        z = torch.zeros(3, 64, device="cuda")
        assert flce.process_logits(z, out=z) is z


def test_an_output_that_wants_a_gradient_is_refused():
    z = torch.randn(3, 64, device="cuda").requires_grad_()
    for out in (z, z * 1):
        with pytest.raises(ValueError, match="gradient"):
            flce.process_logits(z, out=out)
    with torch.no_grad():
        assert flce.process_logits(z, out=z) is z


@pytest.mark.parametrize("prompt", [None, 0, 1, "all"])
@pytest.mark.parametrize("L", [32767, 32768, 32769])
def test_one_id_throughout_a_history_around_2_to_15(L, prompt):
    """The largest counts that 16 bits hold, and the first that take 32: logits of
    one, halved where seen, less the count, and their neighbours untouched."""
    V = 1000
    ids = torch.tensor([0, 1, 500, 501, 998, 999])
    B = len(ids)
    k = dict(tokens=ids[:, None].expand(B, L).contiguous(),
             repetition_penalty=torch.full((B,), 2.0), frequency_penalty=torch.ones(B))
    n = {None: 0, "all": L}.get(prompt, prompt)
    if prompt is not None:
        k["prompt_lengths"] = torch.full((B,), n, dtype=torch.int32)
    want = torch.ones(B, V)
    want[torch.arange(B), ids] = 0.5 - (L - n)
    assert torch.equal(run(torch.ones(B, V), k).cpu(), want)
    k["tokens"] = k["tokens"].int()
    assert torch.equal(run(torch.ones(B, V), k).cpu(), want)


@pytest.mark.parametrize("V", [3001, 30000])
def test_long_histories_with_many_biases(V):
    z, k = case(3, V, 33000, 700, F32, torch.int32, seed=V)
    k["bias_ids"][:, ::5] = k["bias_ids"][:, 1:2]  # one id again and again
    check(run(z, k), z, k)


@pytest.mark.parametrize("B,V", [(2, 9001), (64, 9000)])
def test_a_history_buffer_longer_than_its_histories(B, V):
    """Rows of a buffer of 131072 ids of which up to 500 are live: the same as in
    a buffer of 500 (other counters, other blocks)."""
    z, k = case(B, V, 500, 4, BF, torch.int64, seed=V)
    want = run(z, k, out_dtype=F32)
    wide = torch.full((B, 131072), 7, dtype=torch.int64, device="cuda")
    wide[:, :500] = k["tokens"].cuda()
    got = flce.process_logits(z.cuda(), out_dtype=F32, **dict(
        {n: t.cuda() for n, t in k.items()}, tokens=wide))
    assert torch.equal(got, want)
