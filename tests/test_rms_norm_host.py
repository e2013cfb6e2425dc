"""CPU tests of root-mean-square norm's C ABI: the refusals that precede any CUDA call (the addresses are never
followed)."""
import ctypes

import pytest

BASE = 0x7000_0000_0000          # 16-byte aligned, not memory of this process


@pytest.fixture(scope="module")
def prnn():
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn as m
    return m


def test_forward_refusals(prnn):
    def fwd(dtype=0, rows=4, cols=8, x=BASE, xs=8, res=BASE + 4096, rs=8, w=None, eps=1e-6, y=BASE + 8192, ys=8,
            h=BASE + 12288, hs=8, rstd=None):
        return prnn._lib.prnn_rms_norm_forward(dtype, rows, cols, x, xs, res, rs, w, eps, y, ys, h, hs, rstd, None)
    E = prnn.PRNN_ERR_INVALID_ARG
    assert fwd(rows=0) == prnn.PRNN_OK
    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=0), dict(x=None), dict(y=None), dict(h=None),
               dict(xs=7), dict(ys=7), dict(rs=7), dict(hs=7), dict(x=BASE + 2), dict(res=BASE + 4097),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=BASE + 16),
               dict(y=BASE, ys=9), dict(h=BASE + 16), dict(h=BASE + 4096, hs=9), dict(h=BASE + 8192),
               dict(rstd=BASE + 2), dict(rstd=BASE + 8192), dict(rstd=BASE + 12288), dict(rstd=BASE),
               dict(rstd=BASE + 4096), dict(w=BASE + 8192), dict(w=BASE + 12288 + 64), dict(w=BASE + 1),
               dict(w=BASE + 65536, rstd=BASE + 65536 + 16), dict(rows=2 ** 62, xs=2 ** 40)):
        assert fwd(**kw) == E, kw


def test_forward_e4m3_refusals(prnn):
    def fwd(dtype=2, rows=4, cols=300, x=BASE, xs=300, res=None, rs=0, w=None, eps=1e-6, group=128, q=BASE + 8192,
            qs=300, scale=BASE + 16384, h=None, hs=0, rstd=None):
        return prnn._lib.prnn_rms_norm_quantized(dtype, rows, cols, x, xs, res, rs, w, eps, group, q, qs, scale, h,
                                                    hs, rstd, None)
    E = prnn.PRNN_ERR_INVALID_ARG
    assert fwd(rows=0) == prnn.PRNN_OK
    for kw in (dict(group=64), dict(group=-1), dict(group=256), dict(q=None), dict(scale=None), dict(qs=299),
               dict(scale=BASE + 16386), dict(q=BASE), dict(q=BASE + 2399), dict(scale=BASE + 8192 + 1196),
               dict(scale=BASE + 8192 - 44), dict(scale=BASE + 8192 - 4, group=0), dict(rstd=BASE + 16384),
               dict(res=BASE + 4096, rs=300), dict(res=BASE + 32768, rs=300, h=BASE + 8192, hs=300)):
        assert fwd(**kw) == E, kw


def test_backward_refusals(prnn):
    n = ctypes.c_size_t()
    E = prnn.PRNN_ERR_INVALID_ARG
    assert prnn._lib.prnn_rms_norm_workspace(4, 8, ctypes.byref(n)) == prnn.PRNN_OK
    need = n.value
    assert 0 < need <= 4096 and need % 16 == 0
    assert prnn._lib.prnn_rms_norm_workspace(4, 0, ctypes.byref(n)) == E
    assert prnn._lib.prnn_rms_norm_workspace(-1, 8, ctypes.byref(n)) == E
    assert prnn._lib.prnn_rms_norm_workspace(4, 8, None) == E

    def bwd(dtype=0, rows=4, cols=8, dy=BASE, dys=8, h=BASE + 4096, hs=8, w=None, rstd=BASE + 8192, dh=BASE + 12288,
            dhs=8, dx=BASE + 16384, dxs=8, dw=BASE + 20480, ws=BASE + 65536, wsn=need):
        return prnn._lib.prnn_rms_norm_backward(dtype, rows, cols, dy, dys, h, hs, w, rstd, dh, dhs, dx, dxs, dw, ws,
                                                wsn, None)
    for kw in (dict(dtype=3), dict(rows=-1), dict(cols=0), dict(dy=None), dict(h=None), dict(rstd=None),
               dict(dys=7), dict(hs=7), dict(dhs=7), dict(dxs=7), dict(dx=BASE + 4096), dict(dx=BASE + 16),
               dict(dx=BASE, dxs=9), dict(dx=BASE + 12288, dxs=9), dict(dw=BASE), dict(dw=BASE + 12288),
               dict(dw=BASE + 16384), dict(ws=None), dict(wsn=need - 1), dict(ws=BASE + 65544), dict(ws=BASE),
               dict(w=BASE + 20480), dict(dw=BASE + 65536), dict(dx=BASE + 8192), dict(rstd=BASE + 8194)):
        assert bwd(**kw) == E, kw
    assert bwd(dx=None, dw=None) == prnn.PRNN_OK        # nothing is wanted


def test_tensor_wrappers_refuse_host_tensors(prnn):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    for call in (lambda: prnn.rms_norm(x), lambda: prnn.rms_norm_e4m3(x),
                 lambda: prnn.rms_norm_backward(x, x, None, x[:, 0])):
        with pytest.raises(ValueError):
            call()
