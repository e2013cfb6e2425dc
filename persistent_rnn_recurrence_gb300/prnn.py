"""Thin ctypes binding of libprnn.so (declarations in include/prnn.h).

Every function here marshals arguments and calls the C ABI function of the same
name; every step of the computation runs in the library's CUDA kernels.
PyTorch only supplies device memory and streams.  Importing this module loads
the library and raises ImportError if it has not been built -- there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libprnn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m persistent_rnn_recurrence_gb300.build`")
_lib = ctypes.CDLL(LIB_PATH)

# ---- enums (mirror include/prnn.h) ------------------------------------------
PRNN_OK, PRNN_ERR_INVALID_ARG, PRNN_ERR_UNSUPPORTED, PRNN_ERR_NOT_READY, \
    PRNN_ERR_CUDA, PRNN_ERR_OOM, PRNN_ERR_TIMEOUT = range(7)
PRNN_F32, PRNN_F16, PRNN_BF16 = 0, 1, 2
PRNN_ALGO_PERSISTENT, PRNN_ALGO_PER_STEP = 0, 1
(PRNN_OPT_WAIT_TIMEOUT_US, PRNN_OPT_SYNC_MODE, PRNN_OPT_DEBUG_DROP_CTA,
 PRNN_OPT_DEBUG_DROP_STEP, PRNN_OPT_TIMING, PRNN_OPT_PROJECTION, PRNN_OPT_CTA_GROUPS,
 PRNN_OPT_WIDE_LOADS, PRNN_OPT_BANK_AWARE, PRNN_OPT_POLL_DELAY_NS,
 PRNN_OPT_POLL_BACKOFF_NS, PRNN_OPT_RECURRENT_TC, PRNN_OPT_STAGED_ORDER,
 PRNN_OPT_SPARSE_REG_WEIGHTS, PRNN_OPT_SPARSE_STAGING_DEPTH, PRNN_OPT_DENSE_WIDE,
 PRNN_OPT_DENSE_KSPLIT, PRNN_OPT_SPARSE_KSPLIT) = range(18)

PRNN_STACK_WAVEFRONT, PRNN_STACK_LAYERWISE = 0, 1

EXPORTS = ["prnn_create", "prnn_set_weights_dense", "prnn_set_weights_sparse",
           "prnn_forward", "prnn_forward_host", "prnn_destroy", "prnn_get_status", "prnn_status_string",
           "prnn_set_option", "prnn_get_info", "prnn_get_timing", "prnn_probe_sync_floor",
           "prnn_probe_cluster_exchange",
           "prnn_set_trace_buffer",
           "prnn_pack_sparse_host", "prnn_pack_sparse_host_placed", "prnn_pack_dense_ksplit_host",
           "prnn_forward_dense_noalloc",
           "prnn_set_weights_csr",
           "prnn_stack_create", "prnn_stack_set_layer", "prnn_stack_forward",
           "prnn_stack_get_status", "prnn_stack_set_option", "prnn_stack_get_timing",
           "prnn_stack_get_info", "prnn_stack_destroy", "prnn_backward",
           "prnn_sequence_status", "prnn_layer_norm_forward", "prnn_layer_norm_workspace", "prnn_layer_norm_backward",
           "prnn_dropout_forward", "prnn_dropout_backward",
           "prnn_linear_attention_workspace", "prnn_linear_attention_forward",
           "prnn_linear_attention_backward", "prnn_linear_attention_step"]


class prnn_info_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "hidden", "input", "max_batch", "wdtype", "algo", "sparse", "weights_set", "k",
        "k_padded", "sm_count", "n_cta", "rows_per_cta", "threads_per_cta",
        "threads_per_row", "projection_tensor_cores", "sparse_bank_cap", "cta_groups")] + [
        ("smem_bytes", ctypes.c_size_t), ("onchip_weight_bytes", ctypes.c_size_t),
        ("nnz", ctypes.c_size_t), ("recurrent_tensor_cores", ctypes.c_int),
        ("sparse_staged_order", ctypes.c_int), ("sparse_reg_weights", ctypes.c_int),
        ("dense_wide_batch", ctypes.c_int), ("dense_ksplit", ctypes.c_int)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class prnn_stack_info_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "layers", "hidden", "input", "max_batch", "wdtype", "algo", "layers_set",
        "n_cta_per_layer", "rows_per_cta", "threads_per_cta", "cta_groups", "batch_per_pass",
        "chunks_per_thread")] + [
        ("smem_bytes", ctypes.c_longlong), ("onchip_weight_bytes", ctypes.c_longlong)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class prnn_seq_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_longlong) for n in (
        "stride_t", "stride_b", "stride_h")]


class prnn_linear_attention_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "dtype", "T", "B", "heads", "qk_heads", "dk", "dv")] + [
        ("scale", ctypes.c_float), ("log_decay", ctypes.c_void_p), ("lens", ctypes.c_void_p),
        ("q", prnn_seq_t), ("k", prnn_seq_t), ("v", prnn_seq_t), ("state", ctypes.c_void_p),
        ("o", prnn_seq_t), ("state_out", ctypes.c_void_p), ("d_o", prnn_seq_t),
        ("d_state_out", ctypes.c_void_p), ("d_q", prnn_seq_t), ("d_k", prnn_seq_t),
        ("d_v", prnn_seq_t), ("d_state", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t)]


# The same layout for struct.pack, which fills it in one call (a decoding step
# is short enough for the difference to show).
_LA_PACK = struct.Struct("=7if40q").pack
_STEP_PACK = struct.Struct("=7if19q168x").pack   # up to o; the step uses no field behind it

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_A = ctypes.c_char_p     # prnn_linear_attention_t as packed bytes
_sig = {
    "prnn_create": ([ctypes.POINTER(_P), _I, _I, _I, _I, _I], _I),
    "prnn_set_weights_dense": ([_P, _P, _P, _P, _P], _I),
    "prnn_set_weights_sparse": ([_P, _P, _I, _P, _P, _P, _P], _I),
    "prnn_forward": ([_P, _I, _I, _P, _P, _P, _P], _I),
    "prnn_forward_host": ([_P, _I, _I, _P, _P, _P, _P], _I),
    "prnn_destroy": ([_P], _I),
    "prnn_get_status": ([_P, _P], _I),
    "prnn_status_string": ([_I], ctypes.c_char_p),
    "prnn_set_option": ([_P, _I, ctypes.c_longlong], _I),
    "prnn_get_info": ([_P, ctypes.POINTER(prnn_info_t)], _I),
    "prnn_get_timing": ([_P, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float)], _I),
    "prnn_probe_sync_floor": ([_P, _I, _I, _P, _P], _I),
    "prnn_probe_cluster_exchange": ([_I, _I, _I, _I, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_longlong)], _I),
    "prnn_set_trace_buffer": ([_P, _P, ctypes.c_size_t], _I),
    "prnn_pack_sparse_host": ([_I, _I, _I, _I, _I, _P, _P, _P, ctypes.c_size_t,
                               ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "prnn_pack_sparse_host_placed": ([_I, _I, _I, _I, _I, _P, _P, _P, ctypes.c_size_t, _P,
                                      ctypes.c_size_t, ctypes.POINTER(_I), ctypes.POINTER(_I),
                                      ctypes.POINTER(_I)], _I),
    "prnn_pack_dense_ksplit_host": ([_I, _I, _P, _I, _P, ctypes.c_size_t,
                                     ctypes.POINTER(ctypes.c_size_t)], _I),
    "prnn_forward_dense_noalloc": ([_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P], _I),
    "prnn_set_weights_csr": ([_P, _P, _I, _P, _P, _P, _P, _P], _I),
    "prnn_stack_create": ([ctypes.POINTER(_P), _I, _I, _I, _I, _I, _I], _I),
    "prnn_stack_set_layer": ([_P, _I, _P, _P, _P, _P], _I),
    "prnn_stack_forward": ([_P, _I, _I, _P, _P, _P, _P], _I),
    "prnn_stack_get_status": ([_P, _P], _I),
    "prnn_stack_set_option": ([_P, _I, ctypes.c_longlong], _I),
    "prnn_stack_get_timing": ([_P, ctypes.POINTER(ctypes.c_float)], _I),
    "prnn_stack_get_info": ([_P, ctypes.POINTER(prnn_stack_info_t)], _I),
    "prnn_stack_destroy": ([_P], _I),
    "prnn_backward": ([_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "prnn_sequence_status": ([_P], _I),
    "prnn_layer_norm_forward": ([_I, _L, _I, _P, _L, _P, _P, ctypes.c_float, _P, _L, _P, _P, _P],
                                _I),
    "prnn_layer_norm_workspace": ([_L, _I, ctypes.POINTER(ctypes.c_size_t)], _I),
    "prnn_layer_norm_backward": ([_I, _L, _I, _P, _L, _P, _L, _P, _P, _P, _P, _L, _P, _P, _P,
                                  ctypes.c_size_t, _P], _I),
    "prnn_dropout_forward": ([_I, _L, _P, _P, _P, ctypes.c_double, ctypes.c_uint64,
                              ctypes.c_uint64, _P], _I),
    "prnn_dropout_backward": ([_I, _L, _P, _P, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64,
                               _P], _I),
    "prnn_linear_attention_workspace": ([_A, _I, ctypes.POINTER(ctypes.c_size_t)], _I),
    "prnn_linear_attention_forward": ([_A, _P], _I),
    "prnn_linear_attention_backward": ([_A, _P], _I),
    "prnn_linear_attention_step": ([_A, _P, _I, _P, _P], _I),
}
for _name, (_args, _res) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class PrnnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {prnn_status_string(status)}")


def prnn_status_string(status: int) -> str:
    return _lib.prnn_status_string(int(status)).decode()


def _check(status: int, where: str) -> int:
    if status != PRNN_OK:
        raise PrnnError(status, where)
    return status


def _ptr(t) -> Optional[int]:
    """Device/host address of a tensor (or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---- the C ABI, one Python function per C function ---------------------------
def prnn_create(hidden: int, input: int, max_batch: int, wdtype: int, algo: int) -> int:
    h = _P()
    _check(_lib.prnn_create(ctypes.byref(h), hidden, input, max_batch, wdtype, algo),
           "prnn_create")
    return h.value


def prnn_set_weights_dense(h: int, Wx, Wh, bias, stream=None) -> None:
    _check(_lib.prnn_set_weights_dense(h, _ptr(Wx), _ptr(Wh), _ptr(bias), _stream(stream)),
           "prnn_set_weights_dense")


def prnn_set_weights_sparse(h: int, Wx, k: int, vals, cols, bias, stream=None) -> None:
    _check(_lib.prnn_set_weights_sparse(h, _ptr(Wx), int(k), _ptr(vals), _ptr(cols),
                                        _ptr(bias), _stream(stream)),
           "prnn_set_weights_sparse")


def prnn_set_weights_csr(h: int, Wx, nnz: int, row_ptr, cols, vals, bias, stream=None) -> None:
    _check(_lib.prnn_set_weights_csr(h, _ptr(Wx), int(nnz), _ptr(row_ptr), _ptr(cols),
                                     _ptr(vals), _ptr(bias), _stream(stream)),
           "prnn_set_weights_csr")


def prnn_forward(h: int, T: int, B: int, x, h0, y, stream=None) -> None:
    _check(_lib.prnn_forward(h, T, B, _ptr(x), _ptr(h0), _ptr(y), _stream(stream)),
           "prnn_forward")


def prnn_forward_host(h: int, T: int, B: int, x, h0, y, stream=None) -> None:
    """x, h0 (or None) and y are page-locked host buffers (e.g. pinned CPU
    tensors)."""
    _check(_lib.prnn_forward_host(h, T, B, _ptr(x), _ptr(h0), _ptr(y), _stream(stream)),
           "prnn_forward_host")


def prnn_destroy(h: int) -> None:
    _check(_lib.prnn_destroy(h), "prnn_destroy")


def prnn_get_status(h: int, stream=None) -> int:
    """Returns the status code (PRNN_OK or PRNN_ERR_TIMEOUT); does not raise
    for a timeout, so callers can test for it."""
    return _lib.prnn_get_status(h, _stream(stream))


def prnn_set_option(h: int, opt: int, value: int) -> None:
    _check(_lib.prnn_set_option(h, opt, int(value)), "prnn_set_option")


def prnn_get_info(h: int) -> dict:
    info = prnn_info_t()
    _check(_lib.prnn_get_info(h, ctypes.byref(info)), "prnn_get_info")
    return info.as_dict()


def prnn_get_timing(h: int):
    a, b = ctypes.c_float(), ctypes.c_float()
    _check(_lib.prnn_get_timing(h, ctypes.byref(a), ctypes.byref(b)), "prnn_get_timing")
    return a.value, b.value


def prnn_pack_sparse_host_placed(hidden, k, n_cta, rows_per_cta, threads_per_row, vals, cols):
    """Host-only packing with the per-CTA staging order of h: returns
    (packed[n_cta, R, ept/4, tpr, 4] uint32, place[n_cta, hidden/4] uint32 or
    None when columns stay in order, ept, bank_cap)."""
    import numpy as np
    vals = np.ascontiguousarray(vals).view(np.uint16)
    cols = np.ascontiguousarray(cols, dtype=np.uint16)
    ept, cap, placed = _I(), _I(), _I()
    st = _lib.prnn_pack_sparse_host_placed(hidden, k, n_cta, rows_per_cta, threads_per_row,
                                           vals.ctypes.data, cols.ctypes.data, None, 0, None, 0,
                                           ctypes.byref(ept), ctypes.byref(cap),
                                           ctypes.byref(placed))
    if st != PRNN_ERR_INVALID_ARG or ept.value <= 0:
        _check(st if st != PRNN_OK else PRNN_ERR_INVALID_ARG, "prnn_pack_sparse_host_placed")
    out = np.zeros((n_cta, rows_per_cta, ept.value // 4, threads_per_row, 4), dtype=np.uint32)
    place = np.zeros((n_cta, hidden // 4), dtype=np.uint32) if placed.value else None
    _check(_lib.prnn_pack_sparse_host_placed(
        hidden, k, n_cta, rows_per_cta, threads_per_row, vals.ctypes.data, cols.ctypes.data,
        out.ctypes.data, out.size, None if place is None else place.ctypes.data,
        0 if place is None else place.size, ctypes.byref(ept), ctypes.byref(cap),
        ctypes.byref(placed)), "prnn_pack_sparse_host_placed")
    return out, place, ept.value, cap.value


def prnn_probe_sync_floor(h: int, T: int, B: int, y, stream=None) -> None:
    _check(_lib.prnn_probe_sync_floor(h, T, B, _ptr(y), _stream(stream)),
           "prnn_probe_sync_floor")


def prnn_probe_cluster_exchange(hidden: int, cluster_size: int, clusters: int,
                                steps: int) -> tuple:
    """(ns per step, wrong words received) of the cluster exchange probe."""
    ns = ctypes.c_double(0.0)
    bad = ctypes.c_longlong(0)
    _check(_lib.prnn_probe_cluster_exchange(hidden, cluster_size, clusters, steps,
                                            ctypes.byref(ns), ctypes.byref(bad)),
           "prnn_probe_cluster_exchange")
    return ns.value, bad.value


def prnn_set_trace_buffer(h: int, buf, nbytes: int) -> None:
    """Set (or, with buf None, clear) the device buffer of the sparse
    kernel's phase trace: [T][n_cta][12] uint32 records per forward."""
    _check(_lib.prnn_set_trace_buffer(h, _ptr(buf), int(nbytes)), "prnn_set_trace_buffer")


def prnn_pack_dense_ksplit_host(hidden, cluster_size, wh16, transpose=False):
    """Host-only image of the K-split kernel's weights (numpy fp16 [H, H] in,
    numpy uint16 [H/128, cluster_size, nat, 128, 64] out)."""
    import numpy as np
    w = np.ascontiguousarray(wh16).view(np.uint16)
    if w.shape != (hidden, hidden):
        raise ValueError("wh16 must be [hidden, hidden]")
    need = ctypes.c_size_t()
    st = _lib.prnn_pack_dense_ksplit_host(hidden, cluster_size, w.ctypes.data, int(transpose),
                                          None, 0, ctypes.byref(need))
    if st != PRNN_ERR_INVALID_ARG or need.value == 0:
        _check(st if st != PRNN_OK else PRNN_ERR_INVALID_ARG, "prnn_pack_dense_ksplit_host")
    nat = need.value // ((hidden // 128) * cluster_size * 8192)
    out = np.zeros((hidden // 128, cluster_size, nat, 128, 64), dtype=np.uint16)
    _check(_lib.prnn_pack_dense_ksplit_host(hidden, cluster_size, w.ctypes.data, int(transpose),
                                            out.ctypes.data, out.size, ctypes.byref(need)),
           "prnn_pack_dense_ksplit_host")
    return out


def prnn_pack_sparse_host(hidden, k, n_cta, rows_per_cta, threads_per_row, vals, cols):
    """Host-only packing (numpy in, numpy out): returns (packed[n_cta, R, ept/4,
    tpr, 4] uint32, ept, bank_cap)."""
    import numpy as np
    vals = np.ascontiguousarray(vals).view(np.uint16)
    cols = np.ascontiguousarray(cols, dtype=np.uint16)
    ept, cap = _I(), _I()
    st = _lib.prnn_pack_sparse_host(hidden, k, n_cta, rows_per_cta, threads_per_row,
                                    vals.ctypes.data, cols.ctypes.data, None, 0,
                                    ctypes.byref(ept), ctypes.byref(cap))
    if st != PRNN_ERR_INVALID_ARG or ept.value <= 0:
        _check(st if st != PRNN_OK else PRNN_ERR_INVALID_ARG, "prnn_pack_sparse_host")
    out = np.zeros((n_cta, rows_per_cta, ept.value // 4, threads_per_row, 4), dtype=np.uint32)
    _check(_lib.prnn_pack_sparse_host(hidden, k, n_cta, rows_per_cta, threads_per_row,
                                      vals.ctypes.data, cols.ctypes.data, out.ctypes.data,
                                      out.size, ctypes.byref(ept), ctypes.byref(cap)),
           "prnn_pack_sparse_host")
    return out, ept.value, cap.value


def prnn_forward_dense_noalloc(T, B, H, I, wdtype, x, Wx, Wh, bias, h0, y, stream=None) -> None:
    """Dense forward from the caller's own device buffers, allocating nothing
    (see include/prnn.h for the scratch limits and the sharing rules)."""
    _check(_lib.prnn_forward_dense_noalloc(T, B, H, I, wdtype, _ptr(x), _ptr(Wx), _ptr(Wh),
                                           _ptr(bias), _ptr(h0), _ptr(y), _stream(stream)),
           "prnn_forward_dense_noalloc")


def prnn_backward(h: int, T: int, B: int, x, h0, y, dy, delta=None, dx=None, dh0=None, dWx=None,
                  dWh=None, db=None, stream=None) -> None:
    _check(_lib.prnn_backward(h, T, B, _ptr(x), _ptr(h0), _ptr(y), _ptr(dy), _ptr(delta), _ptr(dx),
                              _ptr(dh0), _ptr(dWx), _ptr(dWh), _ptr(db), _stream(stream)),
           "prnn_backward")


def prnn_stack_create(layers: int, hidden: int, input: int, max_batch: int, wdtype: int,
                      algo: int) -> int:
    out = _P()
    _check(_lib.prnn_stack_create(ctypes.byref(out), layers, hidden, input, max_batch, wdtype,
                                  algo), "prnn_stack_create")
    return out.value


def prnn_stack_set_layer(s: int, layer: int, Wx, Wh, bias, stream=None) -> None:
    _check(_lib.prnn_stack_set_layer(s, layer, _ptr(Wx), _ptr(Wh), _ptr(bias), _stream(stream)),
           "prnn_stack_set_layer")


def prnn_stack_forward(s: int, T: int, B: int, x, h0, y, stream=None) -> None:
    _check(_lib.prnn_stack_forward(s, T, B, _ptr(x), _ptr(h0), _ptr(y), _stream(stream)),
           "prnn_stack_forward")


def prnn_stack_get_status(s: int, stream=None) -> int:
    return _lib.prnn_stack_get_status(s, _stream(stream))


def prnn_stack_set_option(s: int, opt: int, value: int) -> None:
    _check(_lib.prnn_stack_set_option(s, opt, int(value)), "prnn_stack_set_option")


def prnn_stack_get_timing(s: int) -> float:
    ms = ctypes.c_float()
    _check(_lib.prnn_stack_get_timing(s, ctypes.byref(ms)), "prnn_stack_get_timing")
    return ms.value


def prnn_stack_get_info(s: int) -> dict:
    info = prnn_stack_info_t()
    _check(_lib.prnn_stack_get_info(s, ctypes.byref(info)), "prnn_stack_get_info")
    return info.as_dict()


def prnn_stack_destroy(s: int) -> None:
    _check(_lib.prnn_stack_destroy(s), "prnn_stack_destroy")


# ---- sequence operators ----------------------------------------------------------
def prnn_sequence_status(stream=None) -> int:
    """PRNN_OK, or PRNN_ERR_TIMEOUT once a kernel of the sequence operators has given up a wait."""
    return _lib.prnn_sequence_status(_stream(stream))


def prnn_layer_norm_forward(dtype, rows, cols, x, x_stride, gamma, beta, eps, y, y_stride,
                            mean=None, rstd=None, stream=None) -> None:
    _check(_lib.prnn_layer_norm_forward(dtype, rows, cols, _ptr(x), x_stride, _ptr(gamma),
                                        _ptr(beta), eps, _ptr(y), y_stride, _ptr(mean), _ptr(rstd),
                                        _stream(stream)), "prnn_layer_norm_forward")


def prnn_layer_norm_workspace(rows, cols) -> int:
    n = ctypes.c_size_t()
    _check(_lib.prnn_layer_norm_workspace(rows, cols, ctypes.byref(n)),
           "prnn_layer_norm_workspace")
    return n.value


def prnn_layer_norm_backward(dtype, rows, cols, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx,
                             dx_stride, dgamma, dbeta, workspace, workspace_bytes,
                             stream=None) -> None:
    _check(_lib.prnn_layer_norm_backward(dtype, rows, cols, _ptr(dy), dy_stride, _ptr(x), x_stride,
                                         _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx), dx_stride,
                                         _ptr(dgamma), _ptr(dbeta), _ptr(workspace),
                                         workspace_bytes, _stream(stream)),
           "prnn_layer_norm_backward")


def prnn_dropout_forward(dtype, n, x, residual, y, p, seed, offset, stream=None) -> None:
    _check(_lib.prnn_dropout_forward(dtype, n, _ptr(x), _ptr(residual), _ptr(y), p, seed, offset,
                                     _stream(stream)), "prnn_dropout_forward")


def prnn_dropout_backward(dtype, n, dy, dx, p, seed, offset, stream=None) -> None:
    _check(_lib.prnn_dropout_backward(dtype, n, _ptr(dy), _ptr(dx), p, seed, offset,
                                      _stream(stream)), "prnn_dropout_backward")


def prnn_linear_attention_workspace(a: bytes, backward: bool) -> int:
    """`a`: bytes of a prnn_linear_attention_t (``bytes(struct)``)."""
    n = ctypes.c_size_t()
    _check(_lib.prnn_linear_attention_workspace(a, int(backward), ctypes.byref(n)),
           "prnn_linear_attention_workspace")
    return n.value


def prnn_linear_attention_forward(a: bytes, stream=None) -> None:
    _check(_lib.prnn_linear_attention_forward(a, _stream(stream)), "prnn_linear_attention_forward")


def prnn_linear_attention_backward(a: bytes, stream=None) -> None:
    _check(_lib.prnn_linear_attention_backward(a, _stream(stream)),
           "prnn_linear_attention_backward")


def prnn_linear_attention_step(a: bytes, state_pool, n_slots, slots=None, stream=None) -> None:
    _check(_lib.prnn_linear_attention_step(a, _ptr(state_pool), n_slots, _ptr(slots),
                                           _stream(stream)), "prnn_linear_attention_step")


# ---- sequence operators on tensors -------------------------------------------------
# Tensors in, tensors out, on the current stream.  `stream` (a torch stream) runs the call, and
# allocates its outputs, on that stream instead; the caller orders it after the inputs' producers.  The
# tensors given to such a call may be dropped at once: their memory is not used again before the
# call has run.  (Its outputs belong to `stream`, as anything allocated there does.)
# The kernels of a decoding step take a few microseconds, so these wrappers touch each tensor's
# properties as little as the checks allow.
_torch = None
_codes = {}          # torch dtype -> prnn_dtype_t
_raw_stream = None   # device index -> the current stream's handle


def _load_torch():
    global _torch, _raw_stream
    import torch
    _codes.update({torch.float32: PRNN_F32, torch.float16: PRNN_F16, torch.bfloat16: PRNN_BF16})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    _torch = torch


def _used_on(stream, *tensors) -> None:
    """Keeps the memory of tensors that other streams allocated until `stream` has done what it has to do so far."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _dtype(t) -> int:
    code = _codes.get(t.dtype)
    if code is None:
        raise ValueError(f"dtype {t.dtype}: float32, float16 or bfloat16 is needed")
    return code


def _start(t, what):
    """t is a CUDA tensor of the current device; (its type's code, its device's index, the current
    stream's handle)."""
    if _torch is None:
        _load_torch()
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{what}: a CUDA tensor is needed")
    if i != _torch.cuda.current_device():
        raise ValueError(f"{what}: on cuda:{i}, but the current device is "
                         f"{_torch.cuda.current_device()}")
    return _dtype(t), i, _raw_stream(i)


def _like(t, shape, dtype, device, what) -> None:
    """t has this shape, dtype and device index, and its last axis is contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} on device {t.get_device()}, expected "
                         f"{tuple(shape)} {dtype} on device {device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what}: the last axis must be contiguous")


def _vector(t, n, dtype, device, what):
    """Address of a contiguous vector of n values (None: 0)."""
    if t is None:
        return 0
    if t.shape != (n,) or t.dtype is not dtype or t.get_device() != device or \
            (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} on device {t.get_device()}, expected "
                         f"{n} contiguous {dtype} on device {device}")
    return t.data_ptr()


def _rows(t, what):
    """(rows, cols, row stride) of t seen as rows of its last axis; copies nothing."""
    if t.ndim < 1 or t.shape[-1] < 1:
        raise ValueError(f"{what}: at least one value per row is needed")
    cols = t.shape[-1]
    rows = t.numel() // cols
    if t.is_contiguous():
        return rows, cols, cols
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the last axis must be contiguous")
    # the leading axes must step through memory like one axis
    stride, want = None, None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != want:
            raise ValueError(f"{what}: the leading axes must be evenly spaced rows")
        want = st * n
    return rows, cols, cols if stride is None else stride


_sizes = {}          # workspace bytes by what they depend on: sizes, layouts, device


def _norm_workspace(rows, cols):
    need = _sizes.get((rows, cols))
    if need is None:
        if len(_sizes) > 4096:
            _sizes.clear()
        need = _sizes[rows, cols] = prnn_layer_norm_workspace(rows, cols)
    return need


def layer_norm(x, gamma=None, beta=None, eps=1e-5, y=None, stream=None):
    """Layer norm over x's last axis (prnn_layer_norm_forward): (y, mean, rstd), the
    statistics fp32 with x's leading shape.  gamma, beta: fp32 [cols] or None.  y may be x."""
    if stream is not None:
        import torch
        with torch.cuda.stream(stream):
            out = layer_norm(x, gamma, beta, eps, y)
        _used_on(stream, x, gamma, beta, y)
        return out
    code, dev, st = _start(x, "layer_norm: x")
    rows, cols, xs = _rows(x, "layer_norm: x")
    if y is None:
        y, ys = _torch.empty_like(x, memory_format=_torch.contiguous_format), cols
    else:
        _like(y, x.shape, x.dtype, dev, "layer_norm: y")
        ys = _rows(y, "layer_norm: y")[2]
    f32 = _torch.float32
    lead, on = x.shape[:-1], x.device
    mean, rstd = _torch.empty(lead, dtype=f32, device=on), _torch.empty(lead, dtype=f32, device=on)
    _check(_lib.prnn_layer_norm_forward(code, rows, cols, x.data_ptr(), xs,
                                        _vector(gamma, cols, f32, dev, "layer_norm: gamma"),
                                        _vector(beta, cols, f32, dev, "layer_norm: beta"), eps,
                                        y.data_ptr(), ys, mean.data_ptr(), rstd.data_ptr(), st),
           "prnn_layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd, stream=None):
    """Gradients of layer_norm: (dx, dgamma, dbeta), the last two fp32 [cols]."""
    if stream is not None:
        import torch
        with torch.cuda.stream(stream):
            out = layer_norm_backward(dy, x, gamma, mean, rstd)
        _used_on(stream, dy, x, gamma, mean, rstd)
        return out
    code, dev, st = _start(x, "layer_norm_backward: x")
    rows, cols, xs = _rows(x, "layer_norm_backward: x")
    _like(dy, x.shape, x.dtype, dev, "layer_norm_backward: dy")
    dys = _rows(dy, "layer_norm_backward: dy")[2]
    f32, lead = _torch.float32, x.shape[:-1]
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        if t.shape != lead or t.dtype is not f32 or t.get_device() != dev or \
                not t.is_contiguous():
            raise ValueError(f"layer_norm_backward: {what} {tuple(t.shape)} {t.dtype}: expected "
                             f"{tuple(lead)} contiguous {f32} on device {dev}")
    dx = _torch.empty_like(x, memory_format=_torch.contiguous_format)
    need = _norm_workspace(rows, cols)
    on = x.device
    dgamma, dbeta = _torch.empty(cols, dtype=f32, device=on), _torch.empty(cols, dtype=f32, device=on)
    ws = _torch.empty(need, dtype=_torch.uint8, device=on)
    _check(_lib.prnn_layer_norm_backward(code, rows, cols, dy.data_ptr(), dys, x.data_ptr(), xs,
                                         _vector(gamma, cols, f32, dev, "layer_norm_backward: gamma"),
                                         mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), cols,
                                         dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), need, st),
           "prnn_layer_norm_backward")
    return dx, dgamma, dbeta


def dropout(x, p, seed, offset=0, residual=None, y=None, stream=None):
    """Dropout of x plus the residual (prnn_dropout_forward); contiguous tensors of one
    shape.  Give every use in a training step its own offset."""
    if stream is not None:
        import torch
        with torch.cuda.stream(stream):
            out = dropout(x, p, seed, offset, residual, y)
        _used_on(stream, x, residual, y)
        return out
    code, dev, st = _start(x, "dropout: x")
    if not x.is_contiguous():
        raise ValueError("dropout: x must be contiguous")
    for t, what in ((residual, "residual"), (y, "y")):
        if t is not None and t is not x:
            if t.shape != x.shape or t.dtype is not x.dtype or t.get_device() != dev or \
                    not t.is_contiguous():
                raise ValueError(f"dropout: {what} {tuple(t.shape)} {t.dtype}: expected contiguous "
                                 f"{tuple(x.shape)} {x.dtype} on device {dev}")
    if y is None:
        y = _torch.empty_like(x)
    _check(_lib.prnn_dropout_forward(code, x.numel(), x.data_ptr(),
                                     0 if residual is None else residual.data_ptr(),
                                     y.data_ptr(), p, seed, offset, st), "prnn_dropout_forward")
    return y


def dropout_backward(dy, p, seed, offset=0, dx=None, stream=None):
    """Gradient of dropout with respect to x for the same seed and offset (the residual's
    gradient is dy)."""
    return dropout(dy, p, seed, offset, None, dx, stream)


_NO_SEQ = (0, 0, 0, 0)


def _seq4(t, shape, dtype, device, what):
    """(address, strides) of a [T, B, heads, d] tensor, for prnn_seq_t."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} on device {t.get_device()}, expected "
                         f"{tuple(shape)} {dtype} on device {device}")
    st, sb, sh, s1 = t.stride()
    if s1 != 1 and shape[3] > 1:
        raise ValueError(f"{what}: the last axis must be contiguous")
    return t.data_ptr(), st, sb, sh


def _attention_shape(q, v):
    if q.ndim != 4 or v.ndim != 4 or q.shape[:2] != v.shape[:2]:
        raise ValueError(f"q {tuple(q.shape)} and v {tuple(v.shape)}: expected [T, B, qk_heads, dk] "
                         "and [T, B, heads, dv]")


def _state(t, shape, device, what):
    """Address of a contiguous fp32 state (None: 0)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not _torch.float32 or t.get_device() != device or \
            not t.is_contiguous():
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype}, expected contiguous {tuple(shape)} "
                         f"float32 on device {device}")
    return t.data_ptr()


def _decays(t, n, device, what):
    if t is None:
        raise ValueError(f"{what}: log_decay is needed")
    return _vector(t, n, _torch.float32, device, what)


def linear_attention(q, k, v, log_decay, scale=1.0, state=None, lens=None, o=None, stream=None):
    """Linear attention with a decay per head over whole sequences
    (prnn_linear_attention_forward).  q, k [T, B, qk_heads, dk], v [T, B, heads, dv], any strides
    with the last axis contiguous; log_decay fp32 [heads]; state fp32 [B, heads, dk, dv] or
    None (zeros); lens int32 [B] on the device or None.  Returns (o [T, B, heads, dv], the state
    after the last token)."""
    if stream is not None:
        import torch
        with torch.cuda.stream(stream):
            out = linear_attention(q, k, v, log_decay, scale, state, lens, o)
        _used_on(stream, q, k, v, log_decay, state, lens, o)
        return out
    what = "linear_attention: "
    code, dev, st = _start(q, what + "q")
    _attention_shape(q, v)
    qs, vs, dt = q.shape, v.shape, q.dtype
    T, B, H, dv = vs
    Hq, dk = qs[2:]
    on, shape = q.device, (B, H, dk, dv)
    if o is None:
        o = _torch.empty(vs, dtype=dt, device=on)
        o4 = (o.data_ptr(), B * H * dv, H * dv, dv)
    else:
        o4 = _seq4(o, vs, dt, dev, what + "o")
    end = _torch.empty(shape, dtype=_torch.float32, device=on)
    head = (code, T, B, H, Hq, dk, dv, scale, _decays(log_decay, H, dev, what + "log_decay"),
            _vector(lens, B, _torch.int32, dev, what + "lens"),
            *_seq4(q, qs, dt, dev, what + "q"), *_seq4(k, qs, dt, dev, what + "k"),
            *_seq4(v, vs, dt, dev, what + "v"), _state(state, shape, dev, what + "state"),
            *o4, end.data_ptr(),
            *_NO_SEQ, 0, *_NO_SEQ, *_NO_SEQ, *_NO_SEQ, 0)
    ws, p, need = _attention_workspace(head, 0, dev, on)
    _check(_lib.prnn_linear_attention_forward(_LA_PACK(*head, p, need), st),
           "prnn_linear_attention_forward")
    return o, end


def _attention_workspace(head, backward, dev, on):
    """(tensor, its address, its bytes); it must outlive the call.  The size depends on the sizes,
    the strides and the alignment of the inputs, not on where they are."""
    key = (dev, backward, *head[:7], *head[11:14], *head[15:18], *head[19:22], *head[29:32],
           (head[10] | head[14] | head[18] | head[28]) & 15)
    need = _sizes.get(key)
    if need is None:
        if len(_sizes) > 4096:
            _sizes.clear()
        n = ctypes.c_size_t()
        _check(_lib.prnn_linear_attention_workspace(_LA_PACK(*head, 0, 0), backward,
                                                    ctypes.byref(n)),
               "prnn_linear_attention_workspace")
        need = n.value
        # with an input off 16 bytes the size says nothing of the others' alignment
        if key[-1] == 0:
            _sizes[key] = need
    if need == 0:
        return None, 0, 0
    ws = _torch.empty(need, dtype=_torch.uint8, device=on)
    return ws, ws.data_ptr(), need


def linear_attention_backward(do, q, k, v, log_decay, scale=1.0, state=None, lens=None,
                              dstate=None, stream=None) -> dict:
    """Gradients of linear_attention for the loss whose gradient is `do` with respect to o and
    `dstate` (or None) with respect to the returned state: dict of dq, dk, dv and, when a state was
    given, dstate."""
    if stream is not None:
        import torch
        with torch.cuda.stream(stream):
            out = linear_attention_backward(do, q, k, v, log_decay, scale, state, lens, dstate)
        _used_on(stream, do, q, k, v, log_decay, state, lens, dstate)
        return out
    what = "linear_attention_backward: "
    code, dev, st = _start(q, what + "q")
    _attention_shape(q, v)
    qs, vs, dt = q.shape, v.shape, q.dtype
    T, B, H, dv = vs
    Hq, dk = qs[2:]
    on, shape = q.device, (B, H, dk, dv)
    dq, dkk = (_torch.empty(qs, dtype=dt, device=on) for _ in range(2))
    dvv = _torch.empty(vs, dtype=dt, device=on)
    g = {"dq": dq, "dk": dkk, "dv": dvv}
    if state is not None:
        g["dstate"] = _torch.empty(shape, dtype=_torch.float32, device=on)
    qd = (B * Hq * dk, Hq * dk, dk)
    head = (code, T, B, H, Hq, dk, dv, scale, _decays(log_decay, H, dev, what + "log_decay"),
            _vector(lens, B, _torch.int32, dev, what + "lens"),
            *_seq4(q, qs, dt, dev, what + "q"), *_seq4(k, qs, dt, dev, what + "k"),
            *_seq4(v, vs, dt, dev, what + "v"), _state(state, shape, dev, what + "state"),
            *_NO_SEQ, 0, *_seq4(do, vs, dt, dev, what + "do"),
            _state(dstate, shape, dev, what + "dstate"), dq.data_ptr(), *qd, dkk.data_ptr(), *qd,
            dvv.data_ptr(), B * H * dv, H * dv, dv,
            g["dstate"].data_ptr() if state is not None else 0)
    ws, p, need = _attention_workspace(head, 1, dev, on)
    _check(_lib.prnn_linear_attention_backward(_LA_PACK(*head, p, need), st),
           "prnn_linear_attention_backward")
    return g


def _step_strides(t, shape, dtype, device, what):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} on device {t.get_device()}, expected "
                         f"{tuple(shape)} {dtype} on device {device}")
    b, h, last = t.stride()
    if last != 1 and shape[2] > 1:
        raise ValueError(f"{what}: the last axis must be contiguous")
    return b, h


def linear_attention_step(q, k, v, log_decay, state, scale=1.0, slots=None, o=None, stream=None):
    """One token for each sequence (prnn_linear_attention_step): q, k [B, qk_heads, dk],
    v [B, heads, dv]; state fp32 [n, heads, dk, dv], updated in place: sequence b's is
    state[slots[b]] (int32 on the device; outside 0 .. n-1 marks a padding row), or state[b].
    Returns o [B, heads, dv]."""
    if stream is not None:
        import torch
        with torch.cuda.stream(stream):
            out = linear_attention_step(q, k, v, log_decay, state, scale, slots, o)
        _used_on(stream, q, k, v, log_decay, state, slots, o)
        return out
    what = "linear_attention_step: "
    code, dev, st = _start(q, what + "q")
    if q.ndim != 3 or v.ndim != 3 or q.shape[0] != v.shape[0]:
        raise ValueError(f"q {tuple(q.shape)} and v {tuple(v.shape)}: expected [B, qk_heads, dk] and "
                         "[B, heads, dv]")
    qs, vs, dt = q.shape, v.shape, q.dtype
    B, H, dv = vs
    Hq, dk = qs[1:]
    qb, qh, q1 = q.stride()
    if q1 != 1 and dk > 1:
        raise ValueError(what + "q: the last axis must be contiguous")
    kb, kh = _step_strides(k, qs, dt, dev, what + "k")
    vb, vh = _step_strides(v, vs, dt, dev, what + "v")
    if o is None:
        o, ob, oh = _torch.empty(vs, dtype=dt, device=q.device), H * dv, dv
    else:
        ob, oh = _step_strides(o, vs, dt, dev, what + "o")
    n_slots = state.shape[0]
    pool = _state(state, (n_slots, H, dk, dv), dev, what + "state")
    a = _STEP_PACK(code, 1, B, H, Hq, dk, dv, scale,
                   _decays(log_decay, H, dev, what + "log_decay"), 0, q.data_ptr(), 0, qb, qh,
                   k.data_ptr(), 0, kb, kh, v.data_ptr(), 0, vb, vh, 0, o.data_ptr(), 0, ob, oh)
    _check(_lib.prnn_linear_attention_step(
        a, pool, n_slots, _vector(slots, B, _torch.int32, dev, what + "slots"), st),
        "prnn_linear_attention_step")
    return o


# ---- convenience wrapper used by the tests and the benchmark ------------------
class Layer:
    """One RNN layer handle.  ``Layer.from_problem(p)`` uploads a
    ``synth.Problem``'s weights (as device tensors) and returns the layer."""

    def __init__(self, hidden, input, max_batch, wdtype="f16", algo="persistent"):
        self.hidden, self.input, self.max_batch = hidden, input, max_batch
        wd = {"f32": PRNN_F32, "f16": PRNN_F16}[wdtype]
        al = {"persistent": PRNN_ALGO_PERSISTENT, "per_step": PRNN_ALGO_PER_STEP}[algo]
        self.h = prnn_create(hidden, input, max_batch, wd, al)

    @classmethod
    def from_problem(cls, p, algo="persistent", max_batch=None, device="cuda"):
        import torch
        lay = cls(p.H, p.I, max_batch or max(1, p.B), p.wdtype, algo)
        try:
            lay.set_problem_weights(p, device)
        except Exception:
            lay.close()
            raise
        return lay

    def set_problem_weights(self, p, device="cuda"):
        import numpy as np
        import torch
        wt = torch.float16 if p.wdtype == "f16" else torch.float32
        Wx = torch.from_numpy(np.ascontiguousarray(p.Wx)).to(device=device, dtype=wt)
        b = torch.from_numpy(np.ascontiguousarray(p.b)).to(device)
        if getattr(p, "row_ptr", None) is not None:
            rp = torch.from_numpy(np.ascontiguousarray(p.row_ptr, dtype=np.int32)).to(device)
            vals = torch.from_numpy(np.ascontiguousarray(p.vals).view(np.int16)).to(device)
            cols = torch.from_numpy(np.ascontiguousarray(p.cols).view(np.int16)).to(device)
            prnn_set_weights_csr(self.h, Wx, int(p.vals.size), rp, cols, vals, b)
            self.n_values = int(p.vals.size)
        elif p.sparse:
            vals = torch.from_numpy(np.ascontiguousarray(p.vals).view(np.int16)).to(device)
            cols = torch.from_numpy(np.ascontiguousarray(p.cols).view(np.int16)).to(device)
            prnn_set_weights_sparse(self.h, Wx, p.k, vals, cols, b)
        else:
            Wh = torch.from_numpy(np.ascontiguousarray(p.Wh)).to(device=device, dtype=wt)
            prnn_set_weights_dense(self.h, Wx, Wh, b)
        torch.cuda.synchronize()

    def forward(self, x, h0=None, y=None, stream=None):
        """x: [T,B,I] fp32 CUDA tensor; returns y [T,B,H] fp32."""
        import torch
        T, B, _ = x.shape
        if y is None:
            y = torch.empty((T, B, self.hidden), dtype=torch.float32, device=x.device)
        prnn_forward(self.h, T, B, x, h0, y, stream)
        return y

    def backward(self, x, y, dy, h0=None, stream=None) -> dict:
        """Gradients of the loss with dL/dy = dy for the forward (x, h0) -> y:
        dict of fp32 CUDA tensors delta, dx, dh0, dWx, dWh, db."""
        import torch
        T, B, _ = x.shape
        dev = x.device
        info = self.info()
        if info["sparse"]:
            nv = self.n_values if getattr(self, "n_values", None) else info["hidden"] * info["k"]
            dwh = torch.empty(nv, device=dev)
        else:
            dwh = torch.empty(self.hidden, self.hidden, device=dev)
        g = {"delta": torch.empty_like(y),
             "dx": torch.empty_like(x), "dh0": torch.empty(B, self.hidden, device=dev),
             "dWx": torch.empty(self.hidden, self.input, device=dev), "dWh": dwh,
             "db": torch.empty(self.hidden, device=dev)}
        prnn_backward(self.h, T, B, x, h0, y, dy, g["delta"], g["dx"], g["dh0"], g["dWx"], g["dWh"],
                      g["db"], stream)
        return g

    def status(self, stream=None) -> int:
        return prnn_get_status(self.h, stream)

    def info(self) -> dict:
        return prnn_get_info(self.h)

    def set_option(self, opt, value):
        prnn_set_option(self.h, opt, value)

    def close(self):
        if getattr(self, "h", None):
            prnn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Stack:
    """A stack of dense layers (``prnn_stack_*``).  ``Stack.from_problem(p)``
    uploads a ``synth.StackProblem``'s weights and returns the stack."""

    def __init__(self, layers, hidden, input, max_batch, wdtype="f16", algo="wavefront"):
        self.layers, self.hidden, self.input = layers, hidden, input
        wd = {"f32": PRNN_F32, "f16": PRNN_F16}[wdtype]
        al = {"wavefront": PRNN_STACK_WAVEFRONT, "layerwise": PRNN_STACK_LAYERWISE}[algo]
        self.h = prnn_stack_create(layers, hidden, input, max_batch, wd, al)

    @classmethod
    def from_problem(cls, p, algo="wavefront", max_batch=None, device="cuda"):
        st = cls(p.L, p.H, p.I, max_batch or max(1, p.B), p.wdtype, algo)
        try:
            st.set_problem_weights(p, device)
        except Exception:
            st.close()
            raise
        return st

    def set_problem_weights(self, p, device="cuda"):
        import numpy as np
        import torch
        wt = torch.float16 if p.wdtype == "f16" else torch.float32
        for l, (Wx, Wh, b) in enumerate(p.layers):
            prnn_stack_set_layer(
                self.h, l, torch.from_numpy(np.ascontiguousarray(Wx)).to(device=device, dtype=wt),
                torch.from_numpy(np.ascontiguousarray(Wh)).to(device=device, dtype=wt),
                torch.from_numpy(np.ascontiguousarray(b)).to(device))
        torch.cuda.synchronize()

    def forward(self, x, h0=None, y=None, stream=None):
        """x: [T,B,I] fp32 CUDA tensor; returns y [L,T,B,H] (every layer's output)."""
        import torch
        T, B, _ = x.shape
        if y is None:
            y = torch.empty((self.layers, T, B, self.hidden), dtype=torch.float32, device=x.device)
        prnn_stack_forward(self.h, T, B, x, h0, y, stream)
        return y

    def status(self, stream=None) -> int:
        return prnn_stack_get_status(self.h, stream)

    def info(self) -> dict:
        return prnn_stack_get_info(self.h)

    def set_option(self, opt, value):
        prnn_stack_set_option(self.h, opt, value)

    def close(self):
        if getattr(self, "h", None):
            prnn_stack_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
