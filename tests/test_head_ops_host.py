"""The operators around the LM head without a GPU: refusals on the host, before
anything is enqueued (made-up device addresses), and of the Python layer."""
import ctypes
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


def norm(name="flce_rms_norm_forward", **kw):
    a = dict(x=BASE, ldx=64, res=BASE + G, ldr=64, w=BASE + 2 * G, N=4, H=64, eps=1e-6, dt=0, wdt=0,
             y=BASE + 3 * G, h=BASE + 4 * G, rstd=BASE + 5 * G)
    a.update(kw)
    if name == "flce_rms_norm_fp8":
        tail = [a["y"], a["rstd"], a["h"]]
    else:
        tail = [a["y"], a["h"], a["rstd"]]
    return fn(name)(a["x"], a["ldx"], a["res"], a["ldr"], a["w"], a["N"], a["H"], a["eps"],
                    a["dt"], a["wdt"], *tail, None)


@pytest.mark.parametrize("name", ["flce_rms_norm_forward", "flce_rms_norm_fp8"])
def test_norm_refusals(name):
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(N=-1), dict(H=0), dict(dt=2),
               dict(wdt=-1), dict(ldx=63), dict(ldr=10), dict(x=BASE + 1), dict(w=BASE + 2 * G + 1),
               dict(h=BASE + 4 * G + 1),
               dict(y=BASE), dict(y=BASE + G + 2), dict(y=BASE + 2 * G),     # over an input
               dict(h=BASE + 64), dict(h=BASE, ldx=80), dict(h=BASE + 3 * G),
               dict(h=BASE + 2 * G)):
        assert norm(name, **kw) == INVALID, kw
    assert norm(name, H=65537, ldx=65537, ldr=65537) == SHAPE
    assert norm(name, N=1 << 31) == SHAPE
    assert norm(name, N=0, x=None, y=None) == 0
    if name == "flce_rms_norm_fp8":
        assert norm(name, rstd=None) == INVALID  # no scales


@no_gpu
def test_norm_in_place_residual_passes_the_checks():
    # refused neither as an overlap nor as an argument: it gets as far as the device query
    for kw in (dict(h=BASE), dict(h=BASE + G), dict(res=None, ldr=0), dict(h=None)):
        assert norm(**kw) not in (0, INVALID, SHAPE)


def test_norm_backward_refusals():
    need = fn("flce_rms_norm_workspace_size")(100, 64)
    assert need >= 64 * 4 and fn("flce_rms_norm_workspace_size")(0, 64) >= 256
    assert fn("flce_rms_norm_workspace_size")(4, 0) == 0
    assert fn("flce_rms_norm_workspace_size")(-1, 64) == 0
    assert fn("flce_rms_norm_workspace_size")(4, 65537) == 0

    def call(**kw):
        a = dict(dy=BASE, dh=BASE + G, h=BASE + 2 * G, ldh=64, w=BASE + 3 * G, rstd=BASE + 4 * G,
                 N=100, H=64, dt=0, wdt=0, dx=BASE + 5 * G, dw=BASE + 6 * G, ws=BASE + 7 * G,
                 wsb=need)
        a.update(kw)
        return fn("flce_rms_norm_backward")(*[a[k] for k in (
            "dy", "dh", "h", "ldh", "w", "rstd", "N", "H", "dt", "wdt", "dx", "dw", "ws", "wsb")],
            None)
    for kw in (dict(dy=None), dict(h=None), dict(rstd=None), dict(w=None), dict(ldh=3), dict(dt=7),
               dict(ws=None), dict(ws=BASE + 7 * G + 16), dict(dx=BASE), dict(dx=BASE + G),
               dict(dx=BASE + 2 * G + 2), dict(dw=BASE + 5 * G), dict(dw=BASE + 7 * G),
               dict(dx=BASE + 5 * G + 1), dict(N=-1)):
        assert call(**kw) == INVALID, kw
    assert call(wsb=need - 1) == SMALL
    assert call(H=1 << 17, ldh=1 << 17) == SHAPE


def test_quantize_refusals():
    def call(**kw):
        a = dict(x=BASE, ldx=64, R=10, K=64, dt=1, br=128, q=BASE + G, s=BASE + 2 * G)
        a.update(kw)
        return fn("flce_quantize_fp8")(*a.values(), None)
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(R=-1), dict(K=0), dict(br=64),
               dict(br=0), dict(ldx=63), dict(dt=3), dict(x=BASE + 2), dict(q=BASE),
               dict(s=BASE + 4), dict(s=BASE + G)):
        assert call(**kw) == INVALID, kw
    assert call(K=65537, ldx=65537) == SHAPE
    assert call(R=0, x=None) == 0


def test_matmul_refusals():
    def call(**kw):
        a = dict(A=BASE, lda=256, sa=BASE + G, B=BASE + 2 * G, ldb=256, sb=BASE + 3 * G, M=4, V=100,
                 K=256, y=BASE + 4 * G, ldy=100, dt=0)
        a.update(kw)
        return fn("flce_matmul_fp8")(*a.values(), None)
    for kw in (dict(A=None), dict(B=None), dict(sa=None), dict(sb=None), dict(y=None), dict(M=-1),
               dict(V=0), dict(K=0), dict(dt=2), dict(lda=240), dict(ldb=264), dict(ldy=99),
               dict(A=BASE + 8), dict(B=BASE + 2 * G + 1), dict(y=BASE + 4 * G + 1),
               dict(y=BASE + 16), dict(y=BASE + 2 * G), dict(y=BASE + G), dict(y=BASE + 3 * G)):
        assert call(**kw) == INVALID, kw
    assert call(K=200, lda=208, ldb=208) == SHAPE      # not a multiple of 16
    assert call(K=65552, lda=65552, ldb=65552) == SHAPE
    assert call(M=0, A=None) == 0


def test_process_logits_refusals():
    def call(**kw):
        a = dict(z=BASE, ldz=1000, dt=0, B=4, V=1000, tok=BASE + G, ldt=50, t64=1, L=50,
                 ln=BASE + 2 * G, pl=BASE + 3 * G, rep=BASE + 4 * G, fr=BASE + 5 * G,
                 pr=BASE + 6 * G, bi=BASE + 7 * G, b64=0, bv=BASE + 8 * G, nb=3, al=BASE + 9 * G,
                 lda=32, out=BASE + 10 * G, ldo=1000, odt=1)
        a.update(kw)
        return fn("flce_process_logits")(*a.values(), None)
    for kw in (dict(z=None), dict(out=None), dict(B=-1), dict(V=0), dict(L=-1), dict(nb=-1),
               dict(dt=5), dict(odt=5), dict(ldz=999), dict(ldo=10), dict(tok=None), dict(ldt=49),
               dict(bi=None), dict(bv=None), dict(lda=31), dict(tok=BASE + G + 4),
               dict(out=BASE + 10 * G + 2), dict(z=BASE + 1), dict(al=BASE + 9 * G + 2),
               dict(out=BASE), dict(out=BASE + G), dict(out=BASE + 9 * G),
               dict(out=BASE + 2, odt=0)):
        assert call(**kw) == INVALID, kw
    assert call(nb=65536) == SHAPE
    assert call(V=(1 << 30) + 1, ldz=1 << 31, ldo=1 << 31, lda=1 << 27) == SHAPE
    assert call(B=0, z=None) == 0


def test_python_layer_refuses_wrong_tensors():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
    for call in (lambda: flce.rms_norm(x, w), lambda: flce.rms_norm_fp8(x, w),
                 lambda: flce.quantize_fp8(x), lambda: flce.process_logits(x),
                 lambda: flce.matmul_fp8(x, w, x, w),
                 lambda: flce.flce_rms_norm_backward(x, x, w, torch.ones(2))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_calls_raise_without_the_native_module(monkeypatch, tmp_path):
    monkeypatch.setattr(flce, "library_path", str(tmp_path / "libflce.so"))
    monkeypatch.setattr(head_ops, "_module", None)
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
    for call in (lambda: flce.rms_norm(x, w), lambda: flce.rms_norm_fp8(x, w),
                 lambda: flce.quantize_fp8(x), lambda: flce.process_logits(x),
                 lambda: flce.matmul_fp8(x, w, x, w)):
        with pytest.raises(RuntimeError, match="no fallback"):
            call()


# Made-up addresses that a check does not refuse would reach the device, so these
# too are made only where no kernel can run.
@no_gpu
@pytest.mark.parametrize("off", [1, 2, 3])
def test_float_outputs_and_statistics_that_are_not_aligned(off):
    for name in ("flce_rms_norm_forward", "flce_rms_norm_fp8"):  # rstd, and the scales
        assert norm(name, rstd=BASE + 5 * G + off) == INVALID
    need = fn("flce_rms_norm_workspace_size")(100, 64)
    assert fn("flce_rms_norm_backward")(BASE, None, BASE + 2 * G, 64, BASE + 3 * G,
                                        BASE + 4 * G + off, 100, 64, 0, 0, BASE + 5 * G,
                                        BASE + 6 * G, BASE + 7 * G, need, None) == INVALID
    for rows in (1, 128):
        assert fn("flce_quantize_fp8")(BASE, 64, 10, 64, 1, rows, BASE + G, BASE + 2 * G + off,
                                       None) == INVALID


def test_the_backward_names_its_own_arguments():
    h, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="^h must be a CUDA tensor"):
        flce.flce_rms_norm_backward(h, h, w, torch.ones(2))
    with pytest.raises(ValueError, match="^x must be a CUDA tensor"):
        flce.rms_norm(h, w)


def test_matmul_selftest_refusals():
    def call(stop_after=0, limit=1000, **kw):
        a = dict(A=BASE, lda=256, sa=BASE + G, B=BASE + 2 * G, ldb=256, sb=BASE + 3 * G, M=4, V=100,
                 K=256, y=BASE + 4 * G, ldy=100, dt=0)
        a.update(kw)
        return fn("flce_selftest_matmul_fp8_timeout")(stop_after, limit, *a.values(), None)
    assert call(stop_after=-1) == INVALID and call(limit=0) == INVALID
    assert call(A=None) == INVALID and call(ldy=99) == INVALID  # as the product itself
    assert call(K=200, lda=208, ldb=208) == SHAPE
    assert call(M=0, A=None) == 0
