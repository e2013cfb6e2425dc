"""Linear attention over 2^29 - 77 tokens of one head with the state in place, which is never cut over blocks:
one block is at work for several seconds, longer than any of its waits may last by itself.

With log_decay = -0.125 what lies more than 256 tokens back weighs e^-32, far under any bound here, so windows
of 768 tokens started from zero 512 tokens early are the 64-bit reference.  Bounds as for every call of the
16-bit kernel (2^-15 of the sum over absolute values for factors held in two parts, one rounding to bf16,
(d + 768 + 64) fp32 additions)."""
import pytest

pytestmark = pytest.mark.gpu
T, D, WARM, CHECKED, LOG_DECAY, SCALE = 2 ** 29 - 77, 16, 512, 256, -0.125, 0.25
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of free device memory")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    yield torch, prnn
    torch.cuda.empty_cache()


def windows(torch, k, v):
    """(outputs, state) of every window [768, W, D], token by token in 64 bits; q is k."""
    decay = torch.tensor(LOG_DECAY, dtype=torch.float32).double().exp().item()
    S = torch.zeros(k.shape[1], D, D, dtype=torch.float64, device=k.device)
    o = torch.empty_like(v)
    for t in range(k.shape[0]):
        S = decay * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = SCALE * torch.einsum("wde,wd->we", S, k[t])
    return o[WARM:], S


def test_one_block_at_work_for_seconds(env):
    torch, prnn = env
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    k, v = (torch.empty(T, 1, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k.normal_(0.0, 0.25, generator=gen)
    v.normal_(0.0, 1.0, generator=gen)
    o = torch.full_like(v, 9.0)
    state = torch.zeros(1, 1, D, D, device="cuda")
    ld = torch.tensor([LOG_DECAY], device="cuda")
    a = prnn.prnn_linear_attention_t(dtype=prnn.PRNN_BF16, T=T, B=1, heads=1, qk_heads=1, dk=D, dv=D, scale=SCALE,
                                     log_decay=ld.data_ptr(), state=state.data_ptr(), state_out=state.data_ptr())
    for n, t in (("q", k), ("k", k), ("v", v), ("o", o)):
        setattr(a, n, prnn.prnn_seq_t(t.data_ptr(), D, D, D))
    need = prnn.prnn_linear_attention_workspace(bytes(a), False)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), need
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    prnn.prnn_linear_attention_forward(bytes(a))
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end) / 1e3:.2f} s")
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK
    last = T - WARM - CHECKED
    at = torch.tensor([0] + [last * i // 63 for i in range(1, 64)], device="cuda")
    rows = at[None, :] + torch.arange(WARM + CHECKED, device="cuda")[:, None]
    kw, vw, ow = (x.view(T, D)[rows].double() for x in (k, v, o))
    want, S = windows(torch, kw, vw)
    M, MS = windows(torch, kw.abs(), vw.abs())
    fp32 = (D + WARM + CHECKED + 64) * U
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -15 + 2.0 ** -20 + fp32) * M
    assert bool(((ow[WARM:] - want).abs() <= bound).all())
    assert bool(((state[0, 0].double() - S[-1]).abs() <= fp32 * MS[-1]).all())
