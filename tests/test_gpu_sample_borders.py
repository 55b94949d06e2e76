"""Sampling next to the borders that its limits set, against the float64 definition."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")


@pytest.mark.parametrize("V,top_k", [(3, None), (3, 2), (400, None), (400, 399)])
@pytest.mark.parametrize("T", [0.37, 1.0, 1.7])
@pytest.mark.parametrize("min_p", [1e-12, 1e-10, 9.43e-10, 1e-9, 3.3e-9, 1e-8, 1e-7, 1e-6, 1e-4,
                                   0.02, 0.1, 0.5, 0.9])
def test_min_p_keeps_what_lies_above_its_border(min_p, T, V, top_k):
    """A token's weight against min_p's, as (l - max) / T against ln(min_p): right where they
    are 2^-28 apart.  (The border's logarithm is as far off as a weight is, 2^-29 of it, and by
    2^-36 for its multiple of ln 2.)  With the largest logit at -T ln(min_p) the border is
    near zero, where float32 logits lie as close as need be."""
    T, min_p = np.float32(T), np.float32(min_p)
    ln_m = np.log(np.float64(min_p))
    step = 2.0 ** -27 * np.array([1, 1.5, 4, 20, 100, 1000, 30000])
    rows = []
    for off in (0.0, 1e-7, -3e-6, 2e-4, 0.03):
        top = np.float32(-T * ln_m + off)
        border = np.float64(top) + np.float64(T) * ln_m
        for d in np.concatenate([step, -step]):
            near = np.float32(border + T * d)
            if near < top:
                rows.append((near, top))  # the first one, by id, that is kept
    l = np.full((len(rows), V), -40.0 * T, np.float32)
    l[:, :2] = rows
    apart = (l[:, 0].astype(np.float64) - l[:, 1]) / np.float64(T) - ln_m
    sure = np.abs(apart) > 2.0 ** -28
    assert sure.sum() >= 20
    n = len(rows)

    def full(v, dt=torch.float32):
        return torch.full((n,), v, dtype=dt, device="cuda")
    got = flce.sample_logits(torch.from_numpy(l).cuda(), full(0.0), temperature=full(float(T)),
                             min_p=full(float(min_p)),
                             top_k=None if top_k is None else full(top_k, torch.int32))
    want = np.where(apart >= 0, 0, 1)
    assert (got.cpu().numpy() == want)[sure].all(), (apart[sure], got.cpu().numpy()[sure])


def test_the_largest_logit_reaches_any_min_p():
    """min_p of 1 keeps what equals the largest logit, and nothing else; the least min_p keeps
    the largest too."""
    values = [1.0, 2.0, float("inf"), 1 - 2.0 ** -24, 0.5, 2.0 ** -30, 2.0 ** -126, 2.0 ** -149]
    n = len(values)
    for top in (0.0, 1.0, -1e-30, 100.0, 3e38, -3e38):
        l = torch.full((n, 5), float("-inf"), device="cuda")
        l[:, 2] = l[:, 4] = top
        got = flce.sample_logits(l, torch.tensor([0.4] * n, device="cuda"),
                                 min_p=torch.tensor(values, device="cuda"))
        assert got.tolist() == [2] * n
        got = flce.sample_logits(l, torch.tensor([0.6] * n, device="cuda"),
                                 min_p=torch.tensor(values, device="cuda"))
        assert got.tolist() == [4] * n
