"""Pins of the float64 definitions of the operators around the LM head (CPU):
closed forms, differences, torch's own formulas in float64."""
import numpy as np
import pytest
import torch

from oracle import head_ops as ref


def test_norm_of_a_constant_row_is_the_weight():
    w = np.linspace(-2, 3, 10)
    y, h, rstd = ref.rms_norm(np.full((1, 10), 5.0), w, 0.0)
    assert np.allclose(y[0], w, rtol=1e-14) and np.isclose(rstd[0], 0.2)
    y, h, _ = ref.rms_norm(np.zeros((1, 10)), w, 1e-6, np.ones((1, 10)))
    assert (h == 1).all() and np.allclose(y[0], w / np.sqrt(1 + 1e-6))


def test_norm_backward_matches_differences():
    g = np.random.default_rng(0)
    x, res, w, dy, dh = (g.standard_normal(s) for s in ((3, 7), (3, 7), 7, (3, 7), (3, 7)))

    def loss(x_, w_):
        y, h, _ = ref.rms_norm(x_, w_, 1e-2, res)
        return (y * dy).sum() + (h * dh).sum()
    dx, dw = ref.rms_norm_backward(dy, x + res, w, 1e-2, dh)
    e = 1e-6
    for i in np.ndindex(3, 7):
        d = np.zeros((3, 7))
        d[i] = e
        assert np.isclose((loss(x + d, w) - loss(x - d, w)) / (2 * e), dx[i], rtol=1e-6, atol=1e-8)
    for i in range(7):
        d = np.zeros(7)
        d[i] = e
        assert np.isclose((loss(x, w + d) - loss(x, w - d)) / (2 * e), dw[i], rtol=1e-6, atol=1e-8)


def test_round_e4m3_matches_the_storage_type():
    v = np.random.default_rng(1).standard_normal(20000).astype(np.float32) * 40
    v = np.concatenate([v, v * 1e-3, np.float32([0, -0.0, 448, 460, 2.0 ** -9, 2.0 ** -10, 17, 19,
                                                 0.4375 * 2 ** -6])])
    v = np.clip(v, -448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.round_e4m3(v), want)


def test_block_amax_and_matmul_against_loops():
    g = np.random.default_rng(2)
    a, b = g.standard_normal((3, 200)), g.standard_normal((130, 200))
    sa, sb = g.random((3, 2)) + 0.5, g.random((2, 2)) + 0.5
    y, mag = ref.matmul_fp8(a, sa, b, sb)
    for m, v in ((0, 0), (2, 127), (1, 129)):
        t = [a[m, k] * sa[m, k // 128] * b[v, k] * sb[v // 128, k // 128] for k in range(200)]
        assert np.isclose(y[m, v], sum(t)) and np.isclose(mag[m, v], sum(map(abs, t)))
    am = ref.block_amax(b, 128)
    assert am.shape == (2, 2) and am[1, 1] == np.abs(b[128:, 128:]).max()
    assert (ref.block_amax(np.zeros((1, 5)), 1) == 2.0 ** -100).all()


def test_process_logits_by_hand():
    z = np.array([[2.0, -2.0, 1.0, 0.0, 3.0]])
    out = ref.process_logits(z, tokens=np.array([[0, 1, 1, 9, -1, 4]]), lengths=[5],
                             prompt_lengths=[1], repetition=[2.0], frequency=[0.5],
                             presence=[0.25], bias_ids=np.array([[2, 2, 7]]),
                             bias_values=np.array([[5.0, 1.0, 9.0]]),
                             allowed=np.array([[0b10111]]))
    # 0: in the prompt only; 1: generated twice; 2: last bias entry; 3: masked; 4: past the length
    assert np.array_equal(out, [[1.0, -4.0 - 1.0 - 0.25, 2.0, -np.inf, 3.0]])
    assert np.isneginf(ref.process_logits(z, allowed=np.zeros((1, 1), int))).all()
    assert np.array_equal(ref.process_logits(z), z)


@pytest.mark.parametrize("n", [1, 2, 128, 129])
def test_expand_scale_shapes(n):
    s = ref.expand_scale(np.ones((-(-n // 128), 2)), n, 130, 128)
    assert s.shape == (n, 130)
