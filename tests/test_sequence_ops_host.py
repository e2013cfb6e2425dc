"""CPU tests of the sequence operators' C ABI: struct layout, workspace sizes and the
refusals that precede any CUDA call (the addresses are never followed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7000_0000_0000          # 16-byte aligned, not memory of this process


@pytest.fixture(scope="module")
def prnn():
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn as m
    return m


def test_attention_struct_layout_matches_the_header(prnn, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "prnn.h"', 'int main(void) {']
    for cname in ("prnn_seq_t", "prnn_linear_attention_t"):
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        for f, _ in getattr(prnn, cname)._fields_:
            lines.append(f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));')
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        cname, field, n = line.split()
        cls = getattr(prnn, cname)
        assert int(n) == (ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset), line


def test_attention_pack_fills_the_struct(prnn):
    """The packed form used per call puts every value where the struct has it."""
    values = list(range(1, 8)) + [0.5] + list(range(100, 140))
    a = prnn.prnn_linear_attention_t.from_buffer_copy(prnn._LA_PACK(*values))
    assert (a.dtype, a.T, a.B, a.heads, a.qk_heads, a.dk, a.dv, a.scale) == (1, 2, 3, 4, 5, 6, 7, 0.5)
    flat = [a.log_decay, a.lens]
    for n in ("q", "k", "v"):
        s = getattr(a, n)
        flat += [s.data, s.stride_t, s.stride_b, s.stride_h]
    flat += [a.state, a.o.data, a.o.stride_t, a.o.stride_b, a.o.stride_h, a.state_out]
    flat += [a.d_o.data, a.d_o.stride_t, a.d_o.stride_b, a.d_o.stride_h, a.d_state_out]
    for n in ("d_q", "d_k", "d_v"):
        s = getattr(a, n)
        flat += [s.data, s.stride_t, s.stride_b, s.stride_h]
    flat += [a.d_state, a.workspace, a.workspace_bytes]
    assert flat == list(range(100, 140))


def test_layer_norm_refusals(prnn):
    def fwd(dtype=0, rows=4, cols=8, x=BASE, xs=8, gamma=None, beta=None, eps=1e-5,
            y=BASE + 4096, ys=8, mean=None, rstd=None):
        return prnn._lib.prnn_layer_norm_forward(dtype, rows, cols, x, xs, gamma, beta, eps, y, ys,
                                                 mean, rstd, None)
    E = prnn.PRNN_ERR_INVALID_ARG
    assert fwd(rows=0) == prnn.PRNN_OK                   # nothing to do
    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=0), dict(x=None),
               dict(y=None), dict(xs=7), dict(ys=7), dict(x=BASE + 2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(y=BASE + 16), dict(y=BASE, ys=9),
               dict(mean=BASE + 4096), dict(mean=BASE + 2), dict(rstd=BASE + 32),
               dict(gamma=BASE + 4096 + 16), dict(mean=BASE + 8192, rstd=BASE + 8192 + 8),
               dict(rows=2 ** 62, xs=2 ** 40)):
        assert fwd(**kw) == E, kw

    n = ctypes.c_size_t()
    assert prnn._lib.prnn_layer_norm_workspace(4, 8, ctypes.byref(n)) == prnn.PRNN_OK
    need = n.value
    assert prnn._lib.prnn_layer_norm_workspace(4, 0, ctypes.byref(n)) == E
    assert prnn._lib.prnn_layer_norm_workspace(4, 8, None) == E

    def bwd(dtype=0, rows=4, cols=8, dy=BASE, dys=8, x=BASE + 4096, xs=8, gamma=None,
            mean=BASE + 8192, rstd=BASE + 12288, dx=BASE + 16384, dxs=8, dg=BASE + 20480,
            db=BASE + 24576, ws=BASE + 65536, wsn=need):
        return prnn._lib.prnn_layer_norm_backward(dtype, rows, cols, dy, dys, x, xs, gamma, mean,
                                                  rstd, dx, dxs, dg, db, ws, wsn, None)
    for kw in (dict(dtype=3), dict(rows=-1), dict(cols=0), dict(dy=None), dict(x=None),
               dict(mean=None), dict(rstd=None), dict(dys=7), dict(xs=7), dict(dxs=7),
               dict(dx=BASE), dict(dx=BASE + 4096), dict(dg=BASE + 16384), dict(dg=BASE + 24576),
               dict(ws=None), dict(wsn=need - 1), dict(ws=BASE + 65544), dict(ws=BASE),
               dict(gamma=BASE + 20480)):
        assert bwd(**kw) == E, kw


def test_dropout_refusals(prnn):
    def fwd(dtype=1, n=100, x=BASE, r=None, y=BASE + 4096, p=0.1):
        return prnn._lib.prnn_dropout_forward(dtype, n, x, r, y, p, 1, 2, None)
    E = prnn.PRNN_ERR_INVALID_ARG
    assert fwd(n=0, x=None, y=None) == prnn.PRNN_OK
    for kw in (dict(dtype=5), dict(n=-1), dict(x=None), dict(y=None), dict(p=-0.1), dict(p=1.0),
               dict(p=float("nan")), dict(p=1 - 2 ** -40), dict(x=BASE + 1), dict(r=BASE + 4097),
               dict(y=BASE + 2), dict(r=BASE + 4098), dict(n=2 ** 61)):
        assert fwd(**kw) == E, kw
    assert prnn._lib.prnn_dropout_backward(1, 100, BASE, BASE + 2, 0.1, 1, 2, None) == E


def _attention(prnn, **kw):
    """A valid [T, B, heads, d] call of packed tensors 1 MiB apart, with changes."""
    a = prnn.prnn_linear_attention_t(dtype=2, T=10, B=2, heads=4, qk_heads=2, dk=16, dv=24,
                                     scale=0.25, log_decay=BASE)
    at = 1
    for n, h, d in (("q", 2, 16), ("k", 2, 16), ("v", 4, 24), ("o", 4, 24), ("d_o", 4, 24),
                    ("d_q", 2, 16), ("d_k", 2, 16), ("d_v", 4, 24)):
        setattr(a, n, prnn.prnn_seq_t(BASE + (at << 20), 2 * h * d, h * d, d))
        at += 1
    a.workspace, a.workspace_bytes = BASE + (64 << 20), 1 << 20
    for k, v in kw.items():
        if "." in k:
            setattr(getattr(a, k.split(".")[0]), k.split(".")[1], v)
        else:
            setattr(a, k, v)
    return bytes(a)


BAD_SHARED = [dict(dtype=3), {"T": -1}, {"B": -1}, {"heads": 0}, {"qk_heads": 0}, {"qk_heads": 3},
              {"dk": 0}, {"dv": 0}, {"scale": float("inf")}, {"log_decay": None},
              {"log_decay": BASE + 2}, {"lens": BASE + 2}, {"q.data": None}, {"k.data": None},
              {"v.data": None}, {"q.data": BASE + (1 << 20) + 1}, {"q.stride_t": -1},
              {"state": BASE + 2}, {"v.stride_t": 2 ** 61}]


def test_linear_attention_refusals(prnn):
    E, U = prnn.PRNN_ERR_INVALID_ARG, prnn.PRNN_ERR_UNSUPPORTED
    f = prnn._lib.prnn_linear_attention_forward
    assert f(None, None) == E
    for kw in BAD_SHARED + [{"o.data": None}, {"o.stride_h": 23}, {"o.stride_b": 24},
                            {"o.data": BASE + (3 << 20)}, {"o.data": BASE + (1 << 20) + 64},
                            {"state_out": BASE + (3 << 20)}, {"state": BASE + (4 << 20)},
                            {"state": BASE + (32 << 20), "state_out": BASE + (32 << 20) + 64},
                            {"lens": BASE + (4 << 20)}]:
        assert f(_attention(prnn, **kw), None) == E, kw
    for kw in ({"dk": 257}, {"dv": 257}, {"B": 1 << 24}, {"T": (1 << 29) + 1}):
        assert f(_attention(prnn, **kw), None) == U, kw
    assert f(_attention(prnn, B=0), None) == prnn.PRNN_OK
    assert f(_attention(prnn, T=0), None) == prnn.PRNN_OK     # no state wanted: nothing to do


def test_linear_attention_backward_refusals(prnn):
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_linear_attention_backward
    n = ctypes.c_size_t()
    assert prnn._lib.prnn_linear_attention_workspace(_attention(prnn), 1, ctypes.byref(n)) == 0
    assert 0 < n.value <= 1 << 20
    for kw in BAD_SHARED + [{"d_o.data": None}, {"workspace": None}, {"workspace_bytes": n.value - 1},
                            {"workspace": BASE + (64 << 20) + 8}, {"d_q.data": BASE + (7 << 20)},
                            {"d_v.data": BASE + (3 << 20)}, {"d_k.stride_h": 8},
                            {"d_state": BASE + (8 << 20)}, {"d_state_out": BASE + 2},
                            {"state": BASE + (32 << 20), "d_state": BASE + (32 << 20)},
                            {"workspace": BASE + (8 << 20)}]:
        assert f(_attention(prnn, **kw), None) == E, kw


def test_linear_attention_step_refusals(prnn):
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_linear_attention_step
    pool = BASE + (128 << 20)
    for kw in ({"heads": 0}, {"dk": 0}, {"q.data": None}, {"o.data": None}, {"log_decay": None},
               {"o.data": BASE + (3 << 20)}, {"o.stride_h": 23}, {"o.data": pool}):
        assert f(_attention(prnn, **kw), pool, 2, None, None) == E, kw
    assert f(_attention(prnn), None, 2, None, None) == E
    assert f(_attention(prnn), pool, 1, None, None) == E      # two sequences, one state
    assert f(_attention(prnn), pool, -1, None, None) == E
    assert f(_attention(prnn), pool + 2, 2, None, None) == E
    assert f(_attention(prnn), pool, 2, BASE + 2, None) == E
    assert f(_attention(prnn, B=0), pool, 0, None, None) == prnn.PRNN_OK


def test_recurrent_layers_refuse_bf16(prnn):
    h = ctypes.c_void_p()
    assert prnn._lib.prnn_create(ctypes.byref(h), 8, 8, 1, prnn.PRNN_BF16, 0) == \
        prnn.PRNN_ERR_INVALID_ARG
    assert prnn._lib.prnn_stack_create(ctypes.byref(h), 2, 8, 8, 1, prnn.PRNN_BF16, 0) == \
        prnn.PRNN_ERR_INVALID_ARG


def test_tensor_wrappers_refuse_host_tensors(prnn):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    s = torch.zeros(2, 3, 2, 4)
    ld = torch.zeros(2)
    for call in (lambda: prnn.layer_norm(x), lambda: prnn.dropout(x, 0.1, 1),
                 lambda: prnn.layer_norm_backward(x, x, None, x[:, 0], x[:, 0]),
                 lambda: prnn.linear_attention(s, s, s, ld),
                 lambda: prnn.linear_attention_backward(s, s, s, s, ld),
                 lambda: prnn.linear_attention_step(s[0], s[0], s[0], ld, torch.zeros(3, 2, 4, 4))):
        with pytest.raises(ValueError):
            call()
