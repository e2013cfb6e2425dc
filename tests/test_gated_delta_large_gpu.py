"""The gated delta rule where sizes are large: scratch of more than one group of heads, offsets past 32 bits, and the
block that walks the most tokens.  Compared with the same call on a part of the batch, which the other tests hold against
64 bits: heads are independent of one another, so the results are equal bit for bit where the plan is the same."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 100e9:
        pytest.skip("100 GB of device memory are needed")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    yield torch, prnn
    torch.cuda.empty_cache()


def make(torch, T, B, H, d, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)
    q, k = (normal(T, B, H, d) * d ** -0.5 for _ in range(2))
    v = normal(T, B, H, d)
    gate = -torch.rand(T, B, H, generator=g, device="cuda") * 0.1
    beta = torch.rand(T, B, H, generator=g, device="cuda")
    return q, k, v, gate, beta


def test_more_heads_than_one_group_of_scratch(env):
    """T = 4096, 1088 heads of 32 x 32: the gradients' scratch of all heads would pass 8 GB."""
    torch, prnn = env
    T, B, H, d = 4096, 68, 16, 32
    ins = make(torch, T, B, H, d, torch.bfloat16, 1)
    do = torch.randn(T, B, H, d, device="cuda", dtype=torch.bfloat16)
    o, end = prnn.gated_delta_rule(*ins, 0.2)
    g = prnn.gated_delta_rule_backward(do, *ins, 0.2)
    for b in (slice(0, 12), slice(56, 68)):      # 192 heads: narrow and wide slices of columns are the same sums
        part = [x[:, b] for x in ins]
        o2, end2 = prnn.gated_delta_rule(*part, 0.2)
        assert torch.equal(o[:, b], o2) and torch.equal(end[b], end2)
        g2 = prnn.gated_delta_rule_backward(do[:, b], *part, 0.2)
        for n in g2:
            assert torch.equal(g[n][:, b], g2[n]), n
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK


def test_offsets_past_32_bits(env):
    """A sequence's tokens 2^33 bytes apart from its first: slices of a wide joint projection, batch-major."""
    torch, prnn = env
    T, H, d = 300, 2, 64
    wide = 3 * H * d + 7_200_000                   # elements of a row: 300 rows are 2.2e9 elements, 4.3 GB
    joint = torch.zeros(T, 1, wide, device="cuda", dtype=torch.bfloat16)
    ins = make(torch, T, 1, H, d, torch.bfloat16, 2)
    at = [joint[..., wide - (i + 1) * H * d:wide - i * H * d].view(T, 1, H, d) for i in range(3)]
    for x, y in zip(at, ins):
        x.copy_(y)
    o, end = prnn.gated_delta_rule(*at, *ins[3:], 0.2)
    want, wend = prnn.gated_delta_rule(*ins, 0.2)
    assert torch.equal(o, want) and torch.equal(end, wend)
    g = prnn.gated_delta_rule_backward(want, *at, *ins[3:], 0.2)
    for n, x in prnn.gated_delta_rule_backward(want, *ins, 0.2).items():
        assert torch.equal(g[n], x), n
    first, mid = prnn.gated_delta_rule(*(x[:20] for x in at), *(x[:20] for x in ins[3:]), 0.2)   # token by token
    wfirst, wmid = prnn.gated_delta_rule(*(x[:20] for x in ins), 0.2)
    assert torch.equal(first, wfirst) and torch.equal(mid, wmid)


def test_long_sequence_against_its_halves(env):
    """One sequence of 2^19 tokens and its two halves, cut at a chunk's end: the same chunks, the same bits."""
    torch, prnn = env
    T = 1 << 19
    ins = make(torch, T, 1, 1, 64, torch.float16, 3)
    o, end = prnn.gated_delta_rule(*ins, 0.2)
    first, mid = prnn.gated_delta_rule(*(x[:T // 2] for x in ins), 0.2)
    second, end2 = prnn.gated_delta_rule(*(x[T // 2:] for x in ins), 0.2, mid)
    assert torch.equal(o, torch.cat([first, second])) and torch.equal(end, end2)
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK


def test_norm_offsets_past_32_bits(env):
    """Root-mean-square norm of more than 2^32 values: the last rows as by themselves."""
    torch, prnn = env
    rows, cols = 1_100_000, 4096
    x = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    x[:1000].normal_()
    x[-1000:].normal_()
    x[1000:-1000] = 1.0
    y, _, rstd = prnn.rms_norm(x)
    want, _, wrstd = prnn.rms_norm(x[-1000:].clone())
    assert torch.equal(y[-1000:], want) and torch.equal(rstd[-1000:], wrstd)
    q, scale, _, _ = prnn.rms_norm_e4m3(x, residual=x, h=y)
    wq, wscale, _, _ = prnn.rms_norm_e4m3(x[-1000:].clone(), residual=x[-1000:].clone())
    assert torch.equal(q[-1000:].view(torch.uint8), wq.view(torch.uint8)) and torch.equal(scale[-1000:], wscale)
    dx, _ = prnn.rms_norm_backward(x, x, None, rstd, dx=y)
    wdx, _ = prnn.rms_norm_backward(x[-1000:].clone(), x[-1000:].clone(), None, wrstd)
    assert torch.equal(dx[-1000:], wdx)
