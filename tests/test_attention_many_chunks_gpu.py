"""Linear attention whose blocks walk many chunks of tokens, against 64 bits: whole sequences of enough heads that time
is not cut (9 to 23 chunks a block), and cut ones whose runs are several chunks long, ragged, so that sequences
end in the middle of a run and, in reverse, begin with a partial chunk.

The tokens' magnitudes change by up to 2^10 from one 64-token block to the next: a tile, scale or state of another
chunk would show.  Bounds as for every call (tests/test_sequence_ops_gpu.py)."""
import pytest

from tests.attention_exact import exact
from tests.test_sequence_ops_gpu import (U, absolute, attention_tolerance, env, make, normal, rounding,  # noqa: F401
                                         types, within)

pytestmark = pytest.mark.gpu

CASES = [dict(T=1100, B=8, H=16, Hq=16, d=64, lens=None), dict(T=1100, B=8, H=16, Hq=4, d=128, lens=None),
         dict(T=1100, B=8, H=16, Hq=16, d=128, lens=[1100, 1, 0, 1099, 673, 672, 112, 897]),
         dict(T=2500, B=3, H=8, Hq=8, d=64, lens=[2500, 1777, 901]),
         dict(T=2500, B=3, H=8, Hq=2, d=128, lens=[2500, 1345, 2369]),
         dict(T=4000, B=3, H=4, Hq=4, d=128, lens=[3333, 4000, 130])]


def inputs(torch, T, B, H, Hq, d, lens, dt, seed):
    x = make(torch, T, B, H, Hq, d, d, dt, seed, state=True, lens=lens, decay=[-0.001, -0.01, -0.1, -1.5])
    gen = torch.Generator().manual_seed(seed)

    def vary(t, span):
        e = torch.randint(-span, span + 1, ((T + 63) // 64, B, t.shape[2]), generator=gen).cuda()
        return (t.float() * torch.exp2(e.float()).repeat_interleave(64, 0)[:T, :, :, None]).to(dt)
    for n, span in (("q", 1), ("k", 3), ("v", 2)):
        x[n] = vary(x[n], span)
    x["grad"] = vary(normal(torch, x["v"].shape, dt, seed + 5, 0.25), 5)
    return x


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_many_chunks(env, i, dtype):  # noqa: F811
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x = inputs(torch, **CASES[i], dt=dt, seed=3000 + 10 * i)
    grad = x.pop("grad")
    tol, tol32 = attention_tolerance(dtype, CASES[i]["T"], CASES[i]["d"])
    o, end = prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"], x["lens"])
    want, wend = exact(torch, **x)
    M, Mend = exact(torch, **absolute(x))
    assert float(want.abs().max()) < 3e4             # within fp16
    within(o, want, rounding(want, u) + tol * M + 1e-38, "o")
    within(end, wend, tol32 * Mend, "state")
    del want, M
    ds = normal(torch, x["state"].shape, torch.float32, 7)
    g = prnn.linear_attention_backward(grad, x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"], x["lens"], ds)
    want, M = exact(torch, **x, grad=grad, dstate=ds), exact(torch, **absolute(x, grad=grad, dstate=ds))
    for n in ("dq", "dk", "dv"):
        assert float(want[n].abs().max()) < 3e4
        within(g[n], want[n], rounding(want[n], u) + tol * M[n] + 1e-38, n)
    within(g["dstate"], want["dstate"], tol32 * M["dstate"], "dstate")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("i", [0, 3, 4])
def test_without_the_end_state(env, i, dtype):  # noqa: F811
    """state_out NULL (no entry for it in the tensor wrappers): the outputs alone, whole and cut, from zeros."""
    torch, prnn = env
    dt, u = types(torch)[dtype]
    c = CASES[i]
    x = inputs(torch, **c, dt=dt, seed=3200 + 10 * i)
    x.pop("grad")
    x["state"] = None
    o = torch.full_like(x["v"], 9.0)
    a = prnn.prnn_linear_attention_t(dtype={"f32": 0, "f16": 1, "bf16": 2}[dtype], T=c["T"], B=c["B"], heads=c["H"],
                                     qk_heads=c["Hq"], dk=c["d"], dv=c["d"], scale=x["scale"],
                                     log_decay=x["ld"].data_ptr(),
                                     lens=None if x["lens"] is None else x["lens"].data_ptr())
    for n, t in (("q", x["q"]), ("k", x["k"]), ("v", x["v"]), ("o", o)):
        setattr(a, n, prnn.prnn_seq_t(t.data_ptr(), *t.stride()[:3]))
    ws = torch.empty(prnn.prnn_linear_attention_workspace(bytes(a), False) + 16, dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    prnn.prnn_linear_attention_forward(bytes(a))
    want, M = exact(torch, **x)[0], exact(torch, **absolute(x))[0]
    tol, _ = attention_tolerance(dtype, c["T"], c["d"])
    within(o, want, rounding(want, u) + tol * M + 1e-38, "o")


STEPS = [(40, 16, 8, 128, 128), (20, 8, 4, 100, 100), (39, 4, 2, 256, 200), (160, 1, 1, 130, 36), (64, 4, 4, 96, 77),
         (152, 1, 1, 65, 68), (19, 8, 8, 255, 256), (96, 16, 8, 128, 128)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", STEPS, ids=str)
def test_step_of_a_serving_batch(env, sizes, dtype):  # noqa: F811
    """One token for enough sequences and heads that a block takes whole rows of a state, and for states with more
    rows than its threads hold at once; through a pool with padding rows, and with state b for sequence b."""
    torch, prnn = env
    dt, u = types(torch)[dtype]
    B, H, Hq, dk, dv = sizes
    x = make(torch, 1, B, H, Hq, dk, dv, dt, 3300, state=True)
    want, wend = exact(torch, **x)
    M, Mend = exact(torch, **absolute(x))
    args = (x["q"][0], x["k"][0], x["v"][0], x["ld"])
    state = x["state"].clone()
    o = prnn.linear_attention_step(*args, state, x["scale"])
    within(o, want[0], rounding(want[0], u) + (dk + 64) * U * M[0] + 1e-38, "o")
    within(state, wend, 8 * U * Mend, "state")
    n = B + B // 4 + 1
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(5))[:B].to(torch.int32).cuda()
    pool = torch.full((n, H, dk, dv), 9.0, device="cuda")
    pool[slots.long()] = x["state"]
    live = torch.ones(B, dtype=torch.bool, device="cuda")
    for row, slot in ((1, -1), (B // 2, n), (B - 1, -2 ** 31)):
        pool[slots[row].long()] = 9.0
        slots[row], live[row] = slot, False
    o2 = prnn.linear_attention_step(*args, pool, x["scale"], slots)
    assert torch.equal(o2[live], o[live]) and bool((o2[~live] == 0).all())
    assert torch.equal(pool[slots[live].long()], state[live])
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[slots[live].long()] = False
    assert bool((pool[rest] == 9).all())




def test_no_wait_has_run_out(env):  # noqa: F811
    torch, prnn = env
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK
