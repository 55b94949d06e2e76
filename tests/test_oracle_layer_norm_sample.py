"""Pins of the float64 definitions of the layer norm and of sampling (CPU): closed
forms, differences, torch's own layer norm in float64, frequencies."""
import numpy as np
import pytest
import torch

from oracle import head_ops as ref


def test_layer_norm_matches_torch_in_float64():
    g = np.random.default_rng(0)
    x, res, w, b = (g.standard_normal(s) for s in ((5, 33), (5, 33), 33, 33))
    y, h, mean, rstd = ref.layer_norm(x, w, b, 1e-5, res)
    want = torch.nn.functional.layer_norm(torch.from_numpy(x + res), (33,), torch.from_numpy(w),
                                          torch.from_numpy(b), 1e-5)
    assert np.allclose(y, want.numpy(), rtol=1e-12, atol=1e-13)
    assert np.array_equal(h, x + res) and np.allclose(mean, h.mean(1))
    assert np.allclose(rstd, 1 / np.sqrt(h.var(1) + 1e-5))
    y, *_ = ref.layer_norm(x, None, None, 0.0)
    assert np.allclose(y.mean(1), 0, atol=1e-14) and np.allclose(y.var(1), 1)


def test_layer_norm_backward_matches_differences():
    g = np.random.default_rng(1)
    x, w, b, dy, dh = (g.standard_normal(s) for s in ((3, 7), 7, 7, (3, 7), (3, 7)))

    def loss(x_, w_, b_):
        y, h, _, _ = ref.layer_norm(x_, w_, b_, 1e-2)
        return (y * dy).sum() + (h * dh).sum()
    grads = ref.layer_norm_backward(dy, x, w, 1e-2, dh)
    for k, (p, got) in enumerate(zip((x, w, b), grads)):
        for i in np.ndindex(p.shape):
            d = np.zeros(p.shape)
            d[i] = 1e-6
            up, down = [[q + s * d if j == k else q for j, q in enumerate((x, w, b))]
                        for s in (1, -1)]
            assert np.isclose((loss(*up) - loss(*down)) / 2e-6, got[i], rtol=1e-6, atol=1e-8)


def test_sample_by_hand():
    l = np.log([1.0, 4.0, 2.0, 1.0, 2.0])  # masses of 10 in all; ties 2, 4 and 0, 3
    assert [ref.sample(l, u) for u in (0, 0.0999, 0.1001, 0.4999, 0.5001, 0.6999, 0.7001, 0.8001)] \
        == [0, 0, 1, 1, 2, 2, 3, 4]
    assert {ref.sample(l, u, top_k=2) for u in np.linspace(0, 0.999, 50)} == {1, 2}
    assert {ref.sample(l, u, top_k=4) for u in np.linspace(0, 0.999, 50)} == {0, 1, 2, 4}
    # the mass before 1, 2, 4, 0 is 0, 4, 6, 8
    assert {ref.sample(l, u, top_p=0.41) for u in np.linspace(0, 0.999, 50)} == {1, 2}
    assert {ref.sample(l, u, top_p=0.39) for u in np.linspace(0, 0.999, 50)} == {1}
    assert {ref.sample(l, u, top_p=0.0) for u in (0, 0.9)} == {1}
    # top_p of what top_k left: 4 + 2 + 2 of 8
    assert {ref.sample(l, u, top_k=3, top_p=0.74) for u in np.linspace(0, 0.999, 50)} == {1, 2}
    assert {ref.sample(l, u, min_p=0.49) for u in np.linspace(0, 0.999, 50)} == {1, 2, 4}
    assert ref.sample(l, 0.99, temperature=0) == 1 and ref.sample(l, 0.99, temperature=1e-30) == 1
    assert ref.sample([1.0, 1.0], 0.6, temperature=0) == 0
    assert ref.sample([-np.inf, np.nan], 0.5) == -1
    assert ref.sample([np.inf, 0.0, np.inf], 0.6) == 2
    assert ref.sample(l, 1.5) == 4 and ref.sample(l, -1) == 0 and ref.sample(l, np.nan) == 0


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_sample_takes_each_token_its_share_of_u(T):
    l = np.random.default_rng(2).standard_normal(9) * 2
    w = np.exp(l / T)
    n = 4000
    got = np.bincount([ref.sample(l, (i + 0.5) / n, temperature=T) for i in range(n)], minlength=9)
    assert np.abs(got / n - w / w.sum()).max() <= 1.0 / n
