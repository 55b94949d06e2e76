"""Sampling next to a border, for batches of different sizes and rows of different alignment,
which a row's tokens are spread over CTAs, warps and lanes by.

A float32 u can lie within 1e-11 of a border of the cumulative mass, so what decides there is
how masses are added.  Against a known largest logit every weight is an integer of its own,
and sums of them are the same in any order: with top-k, or min-p alone, a row gives one token
however it is split.  Where the mass of all tokens is taken while the largest logit is still
looked for, a lane's sum is rounded as that goes up: there the token may be the one on the
border's other side, if the border is as close to u as the weights are right (2^-28 of the mass
and 2^-42 a token, as include/flce.h has it)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

BF, F32 = torch.bfloat16, torch.float32


def close_calls(l, kept, n):
    """n values u, float32, as near to borders of the kept tokens' cumulative mass as they can
    be, and for each the first and the last token that the definition takes for a u that is off
    by as much as a share of the mass may be."""
    w = np.where(kept, np.exp(l - l.max()), 0.0)
    share = np.cumsum(w) / w.sum()
    u = share.astype(np.float32)
    ids = np.flatnonzero(kept & (u > 0) & (u < 1 - 2.0 ** -20))
    u = u[ids[np.argsort(np.abs(u - share)[ids], kind="stable")[:n]]]
    e = 2.0 ** -28 + l.size * 2.0 ** -42
    return u, *(np.searchsorted(share, np.float64(u) + off, side="right") for off in (-e, e))


def splits(row, u, dt, **limits):
    """Tokens of the same row for each u, in batches of several sizes and at several offsets."""
    V, n = row.size, u.size
    out = []
    for lead in (0, 1, 3, 6):
        wide = torch.zeros(n, V + 8, dtype=dt, device="cuda")
        wide[:, lead:lead + V] = torch.from_numpy(row).cuda().to(dt)
        l, v = wide[:, lead:lead + V], torch.from_numpy(u).cuda()
        for size in (n, 152, 64, 37, 5, 1):
            got = []
            for b in range(0, n if size > 1 else min(n, 40), size):
                k = min(size, n - b)
                got += flce.sample_logits(
                    l[b:b + k], v[b:b + k],
                    **{name: torch.full((k,), x, device="cuda", dtype=torch.int32 if
                                        name == "top_k" else F32)
                       for name, x in limits.items()}).tolist()
            out.append((lead, size, np.array(got)))
    return out


def logits(kind, V, dt):
    l = torch.randn(V, generator=torch.Generator().manual_seed(V)) * 2
    l = {"random": l, "rising": l.sort()[0], "falling": l.sort(descending=True)[0]}[kind]
    return l.to(dt).double().numpy()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", ["random", "rising", "falling"])
@pytest.mark.parametrize("V,limits", [
    (9001, dict(top_k=60)), (9001, dict(top_k=1000)), (9001, dict(top_k=5000)),
    (9001, dict(min_p=1e-3)), (60000, dict(min_p=1e-6)), (60000, dict(top_k=59000))])
def test_one_token_however_a_row_is_split(V, limits, kind, dt):
    l = logits(kind, V, dt)
    order = np.argsort(-l, kind="stable")
    kept = np.zeros(V, bool)
    kept[order[:limits.get("top_k", V)]] = True
    if "min_p" in limits:
        kept &= np.exp(l - l.max()) >= np.float64(np.float32(limits["min_p"]))
    u, first, last = close_calls(l, kept, 160)
    runs = splits(l, u, dt, **limits)
    for lead, size, got in runs:
        assert (got == runs[0][2][:got.size]).all() and kept[got].all(), (lead, size)
        assert ((got >= first[:got.size]) & (got <= last[:got.size])).all(), (lead, size)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", ["random", "rising", "falling"])
@pytest.mark.parametrize("V", [9001, 60000])
def test_either_side_of_a_border_where_all_tokens_are_weighed(V, kind, dt):
    l = logits(kind, V, dt)
    u, first, last = close_calls(l, np.ones(V, bool), 160)
    runs = splits(l, u, dt)
    for lead, size, got in runs:
        assert ((got >= first[:got.size]) & (got <= last[:got.size])).all(), (lead, size)


@pytest.mark.parametrize("B", [150, 229, 400])
@pytest.mark.parametrize("V", [79999, 80001, 131072])
def test_large_batches_of_long_rows(B, V):
    """By one CTA a row or two, as the limits, the batch and the length have it: the tokens
    of the same rows alone, and of the definition."""
    from oracle import head_ops as ref
    g = torch.Generator(device="cuda").manual_seed(B)
    l = (torch.randn(B, V, generator=g, device="cuda") * 3).to(BF)
    u, p = (torch.rand(B, generator=g, device="cuda") for _ in range(2))
    k = torch.randint(1, 3000, (B,), generator=g, device="cuda").int()
    some = [0, B // 2, B - 1]
    for name, limits in (("all", {}), ("k", dict(top_k=k)), ("p", dict(top_p=p)),
                         ("m", dict(min_p=p * 0.01)), ("kp", dict(top_k=k, top_p=p))):
        got = flce.sample_logits(l, u, **limits)
        assert ((got >= 0) & (got < V)).all()
        for b in some:
            one = {n: t[b:b + 1] for n, t in limits.items()}
            alone = flce.sample_logits(l[b:b + 1], u[b:b + 1], **one).item()
            row, e = l[b].double().cpu().numpy(), 2.0 ** -28 + V * 2.0 ** -41
            takes = {ref.sample(row, u[b].item() + d, 1.0, int(one["top_k"]) if "top_k" in one
                                else 0, one["top_p"].item() + q if "top_p" in one else 1.0,
                                one["min_p"].item() if "min_p" in one else 0.0)
                     for d in (-e, 0.0, e) for q in (-e, 0.0, e)}
            assert min(takes) <= got[b].item() <= max(takes), (name, b)
            if "top_k" in limits or name == "m":
                assert got[b].item() == alone, (name, b)
