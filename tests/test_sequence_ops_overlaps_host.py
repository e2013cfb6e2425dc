"""CPU tests of linear attention's refusals: what a call writes beside its outputs (the state, its gradient, the pool,
the workspace) must not overlap the decays, lengths or slots that its blocks read meanwhile."""
import ctypes

import pytest

from tests.test_sequence_ops_host import BASE, _attention, prnn  # noqa: F401

FAR = BASE + (256 << 20)
STATE = 4 * 2 * 4 * 16 * 24          # bytes of [B, heads, dk, dv]


def test_forward(prnn):  # noqa: F811
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_linear_attention_forward
    for shift in (0, 4, STATE - 4):
        assert f(_attention(prnn, state_out=FAR, log_decay=FAR + shift), None) == E, shift
        assert f(_attention(prnn, state_out=FAR, lens=FAR + shift), None) == E, shift
    assert f(_attention(prnn, state_out=FAR, log_decay=FAR - 12), None) == E       # its last value
    assert f(_attention(prnn, state_out=FAR, lens=FAR - 4), None) == E


def test_backward(prnn):  # noqa: F811
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_linear_attention_backward
    n = ctypes.c_size_t()
    assert prnn._lib.prnn_linear_attention_workspace(_attention(prnn), 1, ctypes.byref(n)) == 0
    ws = BASE + (64 << 20)
    for name in ("log_decay", "lens"):
        for at in (FAR, FAR + STATE - 4):
            assert f(_attention(prnn, d_state=FAR, **{name: at}), None) == E, (name, at)
        for at in (ws, ws + n.value - 4):
            assert f(_attention(prnn, **{name: at}), None) == E, (name, at)


def test_step(prnn):  # noqa: F811
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_linear_attention_step
    pool = BASE + (128 << 20)
    for at in (pool, pool + 4, pool + STATE - 4):
        assert f(_attention(prnn, log_decay=at), pool, 2, None, None) == E
        assert f(_attention(prnn), pool, 2, at, None) == E
    assert f(_attention(prnn), pool, 2, pool - 4, None) == E


@pytest.mark.gpu
def test_forward_workspace(prnn):  # noqa: F811
    """Many steps of few sequences: the cut of time leaves states in the workspace, where there are SMs to cut for."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    E = prnn.PRNN_ERR_INVALID_ARG
    f = prnn._lib.prnn_linear_attention_forward
    n = ctypes.c_size_t()
    long = {"T": 4000, "q.stride_t": 64, "k.stride_t": 64, "v.stride_t": 192, "o.stride_t": 192}
    packed = {"q.data": FAR, "k.data": FAR + (32 << 20), "v.data": FAR + (64 << 20), "o.data": FAR + (96 << 20),
              "workspace_bytes": 1 << 26}
    assert prnn._lib.prnn_linear_attention_workspace(_attention(prnn, **long, **packed), 0, ctypes.byref(n)) == 0
    assert n.value > 4096
    ws = FAR + (512 << 20)
    for at in (ws, ws + 1024, ws + n.value - 4):
        assert f(_attention(prnn, **long, **packed, workspace=ws, log_decay=at), None) == E
        assert f(_attention(prnn, **long, **packed, workspace=ws, lens=at), None) == E
