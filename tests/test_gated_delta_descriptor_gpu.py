"""The gated delta rule's C calls with one descriptor for both passes, as a C program keeps it: the forward call's outputs
are still named in it when the backward call runs, and the state is updated in place.  Sizes that go token by token
and in chunks.  Compared bit for bit with calls that name nothing besides."""
import pytest

pytestmark = pytest.mark.gpu
B, H, HQ = 3, 4, 2
CASES = [(20, 64, 64), (20, 40, 33), (200, 64, 64), (300, 128, 100), (40, 200, 136)]   # tokens, dk, dv


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    return torch, prnn


def inputs(torch, case, dtype):
    T, dk, dv = case
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(case))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    q, k = (torch.nn.functional.normalize(normal(T, B, HQ, dk), dim=-1).to(dtype) for _ in range(2))
    return {"q": q, "k": k, "v": normal(T, B, H, dv).to(dtype), "log_decay": -0.1 * normal(T, B, H).abs(),
            "beta": torch.sigmoid(normal(T, B, H)), "state": 0.3 * normal(B, H, dk, dv),
            "lens": torch.tensor([T, 0, T - 7], dtype=torch.int32, device="cuda"),
            "d_o": normal(T, B, H, dv).to(dtype), "d_state_out": 0.3 * normal(B, H, dk, dv)}


def descriptor(torch, prnn, case, dtype, tensors):
    """prnn_gated_delta_t of these tensors."""
    T, dk, dv = case
    code = {torch.float32: prnn.PRNN_F32, torch.float16: prnn.PRNN_F16, torch.bfloat16: prnn.PRNN_BF16}[dtype]
    a = prnn.prnn_gated_delta_t(dtype=code, T=T, B=B, heads=H, qk_heads=HQ, dk=dk, dv=dv, scale=0.2)
    for n, x in tensors.items():
        if n in ("lens", "state", "state_out", "d_state_out", "d_state"):
            setattr(a, n, x.data_ptr())
        else:
            setattr(a, n, prnn.prnn_seq_t(x.data_ptr(), *x.stride()[:3]))
    return a


def call(torch, prnn, a, backward):
    n = prnn.prnn_gated_delta_workspace(bytes(a), backward)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    (prnn.prnn_gated_delta_backward if backward else prnn.prnn_gated_delta_forward)(
        bytes(a), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_state_in_place(env, case, dtype):
    """state_out == state; a sequence of no tokens keeps its state's bits."""
    torch, prnn = env
    dt = getattr(torch, dtype)
    p = inputs(torch, case, dt)
    want, end = prnn.gated_delta_rule(p["q"], p["k"], p["v"], p["log_decay"], p["beta"], 0.2, p["state"], p["lens"])
    state, o = p["state"].clone(), torch.full_like(p["v"], 7.0)
    ins = {n: p[n] for n in ("q", "k", "v", "log_decay", "beta", "lens")}
    call(torch, prnn, descriptor(torch, prnn, case, dt, {**ins, "state": state, "state_out": state, "o": o}), 0)
    assert torch.equal(o, want) and torch.equal(state, end) and torch.equal(state[1], p["state"][1])


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward_leaves_the_forward_outputs(env, case, dtype):
    """o and state_out of the forward call keep what they hold by then, whatever that is: other values, the
    gradient of o, the state itself."""
    torch, prnn = env
    dt = getattr(torch, dtype)
    p = inputs(torch, case, dt)
    want = prnn.gated_delta_rule_backward(p["d_o"], p["q"], p["k"], p["v"], p["log_decay"], p["beta"], 0.2, p["state"],
                                          p["lens"], p["d_state_out"])
    names = {"d_q": "dq", "d_k": "dk", "d_v": "dv", "d_log_decay": "dlog_decay", "d_beta": "dbeta",
             "d_state": "dstate"}
    for o, state_out in ((torch.full_like(p["v"], 7.0), torch.full_like(p["state"], 7.0)),
                         (p["d_o"].clone(), p["state"].clone())):
        before = o.clone(), state_out.clone()
        same = bool(torch.equal(state_out, p["state"]))          # the second: d_o lies in o, state_out == state
        outs = {n: torch.full_like(want[m], 3.0) for n, m in names.items()}
        a = descriptor(torch, prnn, case, dt, {**p, **outs, "o": o, "state_out": state_out,
                                               **({"d_o": o, "state": state_out} if same else {})})
        call(torch, prnn, a, 1)
        for n, m in names.items():
            assert torch.equal(outs[n], want[m]), (n, same)
        assert torch.equal(o, before[0]) and torch.equal(state_out, before[1]), same


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_each_gradient_alone(env, case, dtype):
    """Gradients whose data is NULL are not computed; the others do not need them."""
    torch, prnn = env
    dt = getattr(torch, dtype)
    p = inputs(torch, case, dt)
    want = prnn.gated_delta_rule_backward(p["d_o"], p["q"], p["k"], p["v"], p["log_decay"], p["beta"], 0.2, p["state"],
                                          p["lens"], p["d_state_out"])
    for n, m in {"d_q": "dq", "d_k": "dk", "d_v": "dv", "d_log_decay": "dlog_decay", "d_beta": "dbeta",
                 "d_state": "dstate"}.items():
        out = torch.full_like(want[m], 3.0)
        call(torch, prnn, descriptor(torch, prnn, case, dt, {**p, n: out}), 1)
        assert torch.equal(out, want[m]), n
