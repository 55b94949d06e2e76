"""What a norm's backward is asked for, where the answer to that raises: the error that it
raises, and nothing enqueued."""
import pytest
import torch

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")


class Neither:
    def __bool__(self):
        raise KeyError("neither")


def test_a_flag_that_is_neither_true_nor_false():
    x = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    _, h, rstd = flce.flce_rms_norm(x, w)
    _, h2, mean, rstd2 = flce.flce_layer_norm(x, w)
    before = flce.flce_kernel_launch_count()
    for flag, error in ((torch.ones(2), RuntimeError), (Neither(), KeyError)):
        for name in ("need_dx", "need_dweight"):
            with pytest.raises(error):
                flce.flce_rms_norm_backward(x, h, w, rstd, **{name: flag})
            with pytest.raises(error):
                flce.flce_layer_norm_backward(x, h2, w, mean, rstd2, **{name: flag})
    assert flce.flce_kernel_launch_count() == before
    # what is merely true or false counts as that
    dx, dw, db = flce.flce_layer_norm_backward(x, h2, w, mean, rstd2, need_dx=1, need_dweight=[],
                                               need_dbias=torch.ones(1))
    assert dx is not None and dw is None and db is not None
