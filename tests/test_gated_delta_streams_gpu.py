"""Calls of the sequence operators that run at once: blocks of several kernels share SMs, their shared memory and
their tensor memory.  Every result equals the same call's by itself, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    return torch, prnn


def make(torch, T, B, H, d, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    q, k = (normal(T, B, H, d) * d ** -0.5 for _ in range(2))
    return q, k, normal(T, B, H, d), -0.1 * torch.rand(T, B, H, generator=g, device="cuda"), \
        torch.rand(T, B, H, generator=g, device="cuda")


def test_calls_at_once(env):
    torch, prnn = env
    bf16, f32 = torch.bfloat16, torch.float32
    a, b, c = make(torch, 700, 3, 8, 128, bf16, 1), make(torch, 400, 2, 8, 64, f32, 2), make(torch, 60, 2, 4, 64, bf16, 3)
    decay = torch.full((8,), -0.01, device="cuda")
    x = torch.randn(5000, 1152, device="cuda", dtype=bf16)
    calls = [lambda: prnn.gated_delta_rule(*a, 0.1),
             lambda: tuple(prnn.gated_delta_rule_backward(a[2], *a, 0.1).values()),
             lambda: tuple(prnn.gated_delta_rule_backward(b[2], *b, 0.1).values()),
             lambda: prnn.gated_delta_rule(*c, 0.1),
             lambda: prnn.linear_attention(*a[:3], decay, 0.1),
             lambda: prnn.rms_norm_e4m3(x, residual=x)[:2]]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for turn in range(4):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for i in range(len(calls)):
            j = (i + turn) % len(calls)
            with torch.cuda.stream(streams[j]):
                got.append((j, calls[j]()))
        torch.cuda.synchronize()
        for j, outs in got:
            for u, v in zip(outs, want[j]):
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), (turn, j)
        del got
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK


def test_graphs_at_once(env):
    """Two captured graphs replayed on two streams: each has scratch of its own."""
    torch, prnn = env
    sets = [make(torch, 500, 2, 8, 128, torch.bfloat16, 10 + i) for i in range(2)]

    def both(p):
        o, end = prnn.gated_delta_rule(*p, 0.1)
        return (o, end, *prnn.gated_delta_rule_backward(o, *p, 0.1).values())
    want = [both(p) for p in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(both(p))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, expected in zip(outs, want):
        for u, v in zip(got, expected):
            assert torch.equal(u, v)
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK
