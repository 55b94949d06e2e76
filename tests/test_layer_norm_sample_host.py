"""The layer norm and sampling without a GPU: refusals on the host, before anything is
enqueued (made-up device addresses), and of the Python layer."""
import os

import pytest
import torch

flce = pytest.importorskip("lm_head_linear_flce_gb300")
from lm_head_linear_flce_gb300 import head_ops  # noqa: E402

INVALID, SHAPE, SMALL = 1, 2, 3
BASE = 1 << 40
G = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(flce.library_path):
        from lm_head_linear_flce_gb300 import _build
        _build.build()


def fn(name):
    return head_ops._fn(name)


# Calls that are refused never reach the device; those that pass every check
# would, so they are made only where no kernel can run.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses")


def norm(name="flce_layer_norm_forward", **kw):
    a = dict(x=BASE, ldx=64, res=BASE + G, ldr=64, w=BASE + 2 * G, b=BASE + 3 * G, N=4, H=64,
             eps=1e-5, dt=0, wdt=0, y=BASE + 4 * G, h=BASE + 5 * G, mean=BASE + 6 * G,
             rstd=BASE + 7 * G)
    a.update(kw)
    tail = [a["y"], a["mean"], a["h"]] if name == "flce_layer_norm_fp8" else \
        [a["y"], a["h"], a["mean"], a["rstd"]]
    return fn(name)(a["x"], a["ldx"], a["res"], a["ldr"], a["w"], a["b"], a["N"], a["H"], a["eps"],
                    a["dt"], a["wdt"], *tail, None)


@pytest.mark.parametrize("name", ["flce_layer_norm_forward", "flce_layer_norm_fp8"])
def test_norm_refusals(name):
    for kw in (dict(x=None), dict(y=None), dict(N=-1), dict(H=0), dict(dt=2), dict(wdt=-1),
               dict(ldx=63), dict(ldr=10), dict(x=BASE + 1), dict(w=BASE + 2 * G + 1),
               dict(b=BASE + 3 * G + 1), dict(h=BASE + 5 * G + 1), dict(mean=BASE + 6 * G + 2),
               dict(y=BASE), dict(y=BASE + G + 2), dict(y=BASE + 2 * G), dict(y=BASE + 3 * G),
               dict(h=BASE + 64), dict(h=BASE, ldx=80), dict(h=BASE + 4 * G), dict(h=BASE + 3 * G),
               dict(mean=BASE + 3 * G), dict(mean=BASE + 4 * G), dict(mean=BASE + 5 * G)):
        assert norm(name, **kw) == INVALID, kw
    assert norm(name, H=65537, ldx=65537, ldr=65537) == SHAPE
    assert norm(name, N=1 << 31) == SHAPE
    assert norm(name, N=0, x=None, y=None) == 0
    if name == "flce_layer_norm_fp8":
        assert norm(name, mean=None) == INVALID  # no scales
    else:
        for kw in (dict(mean=None), dict(rstd=None), dict(rstd=BASE + 6 * G),
                   dict(rstd=BASE + 7 * G + 3)):
            assert norm(name, **kw) == INVALID, kw


@no_gpu
def test_norm_optional_arguments_pass_the_checks():
    # refused neither as an overlap nor as an argument: it gets as far as the device query
    for kw in (dict(h=BASE), dict(h=BASE + G), dict(res=None, ldr=0), dict(h=None), dict(w=None),
               dict(b=None), dict(w=None, b=None), dict(mean=None, rstd=None)):
        assert norm(**kw) not in (0, INVALID, SHAPE), kw


def test_norm_backward_refusals():
    size = fn("flce_layer_norm_workspace_size")
    need = size(100, 64)
    assert need >= 64 * 8 and size(0, 64) >= 256
    assert size(4, 0) == size(-1, 64) == size(4, 65537) == size(1 << 31, 64) == 0

    def call(**kw):
        a = dict(dy=BASE, dh=BASE + G, h=BASE + 2 * G, ldh=64, w=BASE + 3 * G, mean=BASE + 4 * G,
                 rstd=BASE + 5 * G, N=100, H=64, dt=0, wdt=0, dx=BASE + 6 * G, dw=BASE + 7 * G,
                 db=BASE + 8 * G, ws=BASE + 9 * G, wsb=need)
        a.update(kw)
        return fn("flce_layer_norm_backward")(*a.values(), None)
    for kw in (dict(dy=None), dict(h=None), dict(mean=None), dict(rstd=None), dict(ldh=3),
               dict(dt=7), dict(wdt=7), dict(ws=None), dict(ws=BASE + 9 * G + 16), dict(dx=BASE),
               dict(dx=BASE + G), dict(dx=BASE + 2 * G + 2), dict(dw=BASE + 6 * G),
               dict(db=BASE + 7 * G), dict(db=BASE + 9 * G), dict(dw=BASE + 4 * G),
               dict(dx=BASE + 6 * G + 1), dict(db=BASE + 8 * G + 1), dict(mean=BASE + 4 * G + 2),
               dict(N=-1), dict(H=0), dict(ws=BASE), dict(ws=BASE + G), dict(ws=BASE + 2 * G),
               dict(ws=BASE + 3 * G), dict(ws=BASE + 6 * G), dict(ws=BASE + 4 * G - 256)):
        assert call(**kw) == INVALID, kw
    assert call(wsb=need - 1) == SMALL and call(dw=None, wsb=need - 1) == SMALL
    assert call(H=1 << 17, ldh=1 << 17) == SHAPE


def test_workspaces_grow_with_nothing_but_the_sizes():
    """A plan's partial sums are bounded by what 152 SMs hold, however many rows."""
    size = fn("flce_layer_norm_workspace_size")
    for H in (1, 64, 127, 512, 1001, 3584, 8192, 16384):
        assert size(10 ** 6, H) == size(10 ** 7, H) <= 304 * 8 * H + 256
    assert size(10 ** 6, 40000) == (10 ** 6 + 63) // 64 * 40000 * 8


def test_sample_refusals():
    def call(**kw):
        a = dict(z=BASE, ld=1000, dt=0, B=4, V=1000, u=BASE + G, t=BASE + 2 * G, k=BASE + 3 * G,
                 p=BASE + 4 * G, m=BASE + 5 * G, out=BASE + 6 * G)
        a.update(kw)
        return fn("flce_sample_logits")(*a.values(), None)
    for kw in (dict(z=None), dict(u=None), dict(out=None), dict(B=-1), dict(V=0), dict(dt=2),
               dict(ld=999), dict(z=BASE + 1), dict(dt=1, z=BASE + 2), dict(u=BASE + G + 2),
               dict(t=BASE + 1 + 2 * G), dict(k=BASE + 2 + 3 * G), dict(p=BASE + 3 + 4 * G),
               dict(m=BASE + 1 + 5 * G), dict(out=BASE + 6 * G + 4), dict(out=BASE),
               dict(out=BASE + G), dict(out=BASE + 3 * G), dict(out=BASE + 5 * G + 8)):
        assert call(**kw) == INVALID, kw
    assert call(B=65536) == SHAPE
    assert call(V=(1 << 21) + 1, ld=1 << 22) == SHAPE
    assert call(B=0, z=None, u=None, out=None) == 0


def test_python_layer_refuses_wrong_tensors():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
    for call in (lambda: flce.layer_norm(x, w), lambda: flce.layer_norm(x),
                 lambda: flce.layer_norm_fp8(x, w), lambda: flce.sample_logits(x, torch.zeros(2)),
                 lambda: flce.flce_layer_norm_backward(x, x, w, torch.ones(2), torch.ones(2))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="^h must be a CUDA tensor"):
        flce.flce_layer_norm_backward(x, x, w, torch.ones(2), torch.ones(2))


def test_calls_raise_without_the_native_module(monkeypatch, tmp_path):
    monkeypatch.setattr(flce, "library_path", str(tmp_path / "libflce.so"))
    monkeypatch.setattr(head_ops, "_module", None)
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
    for call in (lambda: flce.layer_norm(x, w), lambda: flce.layer_norm_fp8(x, w),
                 lambda: flce.sample_logits(x, torch.zeros(2))):
        with pytest.raises(RuntimeError, match="no fallback"):
            call()
