"""CPU tests of the gated delta rule's C ABI: struct layout, workspace sizes and the refusals that precede any CUDA
call (the addresses are never followed)."""
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


def test_struct_layout_matches_the_header(prnn, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    cls = prnn.prnn_gated_delta_t
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "prnn.h"', 'int main(void) {',
             'printf("size %zu\\n", sizeof(prnn_gated_delta_t));']
    lines += [f'printf("{f} %zu\\n", offsetof(prnn_gated_delta_t, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        field, n = line.split()
        assert int(n) == (ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset), line


def test_packs_fill_the_struct(prnn):
    values = list(range(1, 8)) + [0.5] + list(range(100, 155))
    a = prnn.prnn_gated_delta_t.from_buffer_copy(prnn._GD_PACK(*values))
    flat = []
    for name, kind in prnn.prnn_gated_delta_t._fields_[8:]:
        x = getattr(a, name)
        flat += [x.data, x.stride_t, x.stride_b, x.stride_h] if kind is prnn.prnn_seq_t else [x]
    assert flat == list(range(100, 155))
    short = prnn.prnn_gated_delta_t.from_buffer_copy(prnn._GD_STEP_PACK(*values[:34]))
    assert short.o.stride_h == 125 and short.state_out is None and short.workspace_bytes == 0


def call(prnn, **kw):
    """A valid [T, B, heads, d] call of packed tensors 1 MiB apart, with changes."""
    a = prnn.prnn_gated_delta_t(dtype=2, T=10, B=2, heads=4, qk_heads=2, dk=16, dv=24, scale=0.25)
    at = 1
    for n, h, d in (("q", 2, 16), ("k", 2, 16), ("v", 4, 24), ("o", 4, 24), ("d_o", 4, 24), ("d_q", 2, 16),
                    ("d_k", 2, 16), ("d_v", 4, 24), ("log_decay", 4, 1), ("beta", 4, 1), ("d_log_decay", 4, 1),
                    ("d_beta", 4, 1)):
        setattr(a, n, prnn.prnn_seq_t(BASE + (at << 20), 2 * h * d, h * d, d))
        at += 1
    a.workspace, a.workspace_bytes = BASE + (64 << 20), 16 << 20
    for k, v in kw.items():
        if "." in k:
            setattr(getattr(a, k.split(".")[0]), k.split(".")[1], v)
        else:
            setattr(a, k, v)
    return bytes(a)


SHARED = [dict(dtype=3), {"T": -1}, {"B": -1}, {"heads": 0}, {"qk_heads": 0}, {"qk_heads": 3}, {"dk": 0}, {"dv": 0},
          {"scale": float("inf")}, {"log_decay.data": None}, {"beta.data": None}, {"beta.data": BASE + 2},
          {"beta.stride_t": -1}, {"lens": BASE + 2}, {"q.data": None}, {"k.data": None}, {"v.data": None},
          {"q.data": BASE + (1 << 20) + 1}, {"q.stride_t": -1}, {"state": BASE + 2}, {"v.stride_t": 2 ** 61}]


def test_forward_refusals(prnn):
    E, Un = prnn.PRNN_ERR_INVALID_ARG, prnn.PRNN_ERR_UNSUPPORTED
    f = prnn._lib.prnn_gated_delta_forward
    assert f(None, None) == E
    for kw in SHARED + [{"o.data": None}, {"o.stride_h": 23}, {"o.stride_b": 24}, {"o.data": BASE + (3 << 20)},
                        {"o.data": BASE + (1 << 20) + 64}, {"o.data": BASE + (9 << 20)}, {"beta.data": BASE + (4 << 20)},
                        {"state_out": BASE + (3 << 20)}, {"state": BASE + (4 << 20)}, {"state_out": BASE + (10 << 20)},
                        {"state": BASE + (32 << 20), "state_out": BASE + (32 << 20) + 64}, {"lens": BASE + (4 << 20)},
                        {"lens": BASE + (32 << 20), "state_out": BASE + (32 << 20)}]:
        assert f(call(prnn, **kw), None) == E, kw
    for kw in ({"dk": 257}, {"dv": 257}, {"B": 1 << 24}, {"T": (1 << 29) + 1}):
        assert f(call(prnn, **kw), None) == Un, kw
    assert f(call(prnn, B=0), None) == prnn.PRNN_OK
    assert f(call(prnn, T=0), None) == prnn.PRNN_OK           # no state wanted: nothing to do


def test_backward_refusals(prnn):
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_gated_delta_backward
    n = ctypes.c_size_t()
    assert prnn._lib.prnn_gated_delta_workspace(call(prnn), 1, ctypes.byref(n)) == 0
    assert 0 < n.value <= 16 << 20
    assert prnn._lib.prnn_gated_delta_workspace(call(prnn, dk=0), 1, ctypes.byref(ctypes.c_size_t())) == E
    assert prnn._lib.prnn_gated_delta_workspace(call(prnn), 1, None) == E
    for kw in SHARED + [{"d_o.data": None}, {"workspace": None}, {"workspace_bytes": n.value - 1},
                        {"workspace": BASE + (64 << 20) + 8}, {"d_q.data": BASE + (7 << 20)},
                        {"d_v.data": BASE + (3 << 20)}, {"d_k.stride_h": 8}, {"d_state": BASE + (8 << 20)},
                        {"d_state_out": BASE + 2}, {"state": BASE + (32 << 20), "d_state": BASE + (32 << 20)},
                        {"workspace": BASE + (8 << 20)}, {"d_beta.data": BASE + (11 << 20)},
                        {"d_beta.data": BASE + (8 << 20)}, {"d_log_decay.data": BASE + (9 << 20)},
                        {"d_beta.stride_h": 0}, {"lens": BASE + (12 << 20)}]:
        assert f(call(prnn, **kw), None) == E, kw
    assert f(call(prnn, B=0), None) == prnn.PRNN_OK
    assert f(call(prnn, T=0), None) == prnn.PRNN_OK


def test_step_refusals(prnn):
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_gated_delta_step
    pool = BASE + (128 << 20)
    for kw in ({"heads": 0}, {"dk": 0}, {"q.data": None}, {"o.data": None}, {"log_decay.data": None},
               {"beta.data": None}, {"o.data": BASE + (3 << 20)}, {"o.stride_h": 23}, {"o.data": pool},
               {"beta.data": BASE + (4 << 20)}):
        assert f(call(prnn, **kw), pool, 2, None, None) == E, kw
    for args in ((None, 2, None), (pool, 1, None), (pool, -1, None), (pool + 2, 2, None), (pool, 2, BASE + 2),
                 (BASE + (9 << 20), 2, None), (pool, 2, pool)):
        assert f(call(prnn), *args, None) == E, args
    assert f(call(prnn, dv=257), pool, 2, None, None) == prnn.PRNN_ERR_UNSUPPORTED
    assert f(call(prnn, B=0), pool, 0, None, None) == prnn.PRNN_OK


def test_gates_in_one_buffer(prnn):
    """fp32 gates and their gradients as slices of joint buffers are tensors of their own."""
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_gated_delta_backward
    at = BASE + (20 << 20)
    joint = {"d_log_decay.data": at, "d_log_decay.stride_t": 18, "d_log_decay.stride_b": 9, "d_log_decay.stride_h": 1,
             "d_beta.stride_t": 18, "d_beta.stride_b": 9, "d_beta.stride_h": 1}
    assert f(call(prnn, **joint, **{"d_beta.data": at + 4 * 3}), None) == E      # they share a column
    assert f(call(prnn, **joint, **{"d_beta.data": at + 4 * 5, "workspace": None}), None) == E


def test_tensor_wrappers_refuse_host_tensors(prnn):
    torch = pytest.importorskip("torch")
    s, g = torch.zeros(2, 3, 2, 4), torch.zeros(2, 3, 2)
    for call_ in (lambda: prnn.gated_delta_rule(s, s, s, g, g),
                  lambda: prnn.gated_delta_rule_backward(s, s, s, s, g, g),
                  lambda: prnn.gated_delta_rule_step(s[0], s[0], s[0], g[0], g[0], torch.zeros(3, 2, 4, 4))):
        with pytest.raises(ValueError):
            call_()
