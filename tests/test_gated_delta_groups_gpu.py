"""The gated delta rule with more heads than one group of scratch holds, where the walk over states takes slices of 64
columns: two tiles of columns, ragged lengths, given states, and shared heads whose gradients are joined from fp32
parts.  Heads are independent of one another, so a part of the batch by itself gives the same bits where its plan is
the same; such parts the other tests hold against 64 bits."""
import pytest

pytestmark = pytest.mark.gpu


def test_groups_of_wide_slices(env):
    """T = 4096, 1056 heads of 128 x 128: scratch is 8.5 MB a head forward and 16.9 MB for the gradients, so 8 GB hold
    1004 and 507 of them, and the last batches are in a second and a third group of 52 and 42 heads.  More
    than 38 heads are more than 152 slices of 32 columns, so walks go by 64 in every group and every part."""
    torch, prnn = env
    T, B, H, Hq, d = 4096, 132, 8, 4, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)
    q, k = (normal(T, B, Hq, d) * d ** -0.5 for _ in range(2))
    v, do = normal(T, B, H, d), normal(T, B, H, d)
    gate = -0.1 * torch.rand(T, B, H, generator=g, device="cuda")
    beta = torch.rand(T, B, H, generator=g, device="cuda")
    state, dstate = (normal(B, H, d, d, dtype=torch.float32) * 0.1 for _ in range(2))
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    for b, n in ((0, 0), (1, 1), (5, 2049), (9, 4095), (60, 64), (64, 3000), (65, 129), (125, 0), (127, 4000), (131, 129)):
        lens[b] = n

    def call(b):
        x = [t[:, b] for t in (q, k, v, gate, beta)]
        o, end = prnn.gated_delta_rule(*x, 0.1, state[b], lens[b])
        return {"o": o, "end": end, **prnn.gated_delta_rule_backward(do[:, b], *x, 0.1, state[b], lens[b], dstate[b])}
    whole = call(slice(0, B))
    assert all(bool(x.isfinite().all()) for x in whole.values())
    # 80 to 96 heads, one group: in the first, across the gradients' first border (batch 63), in the last (from 125 and 126)
    for b in (slice(0, 10), slice(57, 68), slice(120, 132)):
        part = call(b)
        for n, x in part.items():
            assert torch.equal(whole[n][b] if n in ("end", "dstate") else whole[n][:, b], x), (n, b)
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK


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
