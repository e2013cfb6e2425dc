"""Offsets past 32 bits: the sequence operators on tensors and strides whose element offsets do not
fit 32-bit integers, against the same calls on packed copies (equal kernels give equal bits) or
against the generator's definition."""
import pytest

from tests.test_sequence_ops_gpu import normal, philox_words  # noqa: F401

pytestmark = pytest.mark.gpu
GIB = 1 << 30


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 64 * GIB:
        pytest.skip("needs 64 GiB of free device memory")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    yield torch, prnn
    torch.cuda.empty_cache()


def words_at(index, seed, offset):
    """The generator's word for one value, in Python integers."""
    m = 2 ** 32 - 1
    i = index // 4
    c, k = [i & m, i >> 32, offset & m, offset >> 32], [seed & m, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c[index % 4]


def test_dropout_past_the_block_counter(env):
    """2^34 + 9 values in place: the counter's high word becomes 1 at value 2^34."""
    torch, prnn = env
    n, seed, offset, p = 2 ** 34 + 9, 2 ** 40 + 17, 2 ** 33 + 5, 0.25
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    prnn.dropout(x, p, seed, offset, y=x)
    for at in (0, 5, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 3, 2 ** 34 - 1, 2 ** 34, 2 ** 34 + 4, n - 1):
        kept = words_at(at, seed, offset) >= round(p * 2 ** 32)
        assert (float(x[at]) != 0) == kept, at
    del x
    assert words_at(6, seed, offset) == philox_words(8, seed, offset)[6]


def test_layer_norm_far_rows(env):
    torch, prnn = env
    stride, cols = 2 ** 31 + 24, 1000
    base = torch.empty(2 * stride + cols, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((3, cols), (stride, 1))
    x.copy_(normal(torch, (3, cols), torch.bfloat16, 1))
    y, mean, rstd = prnn.layer_norm(x)
    want = prnn.layer_norm(x.contiguous())
    assert torch.equal(y, want[0]) and torch.equal(mean, want[1])
    dy = normal(torch, (3, cols), torch.bfloat16, 2)
    got = prnn.layer_norm_backward(dy, x, None, mean, rstd)
    ref = prnn.layer_norm_backward(dy, x.contiguous(), None, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_linear_attention_far_tokens(env, dtype):
    torch, prnn = env
    dt = getattr(torch, dtype)
    T, B, H, D, step = 130, 1, 2, 64, 2 ** 24 + 64
    base = torch.empty((T - 1) * step + H * D, dtype=dt, device="cuda")
    far = base.as_strided((T, B, H, D), (step, H * D, D, 1))
    q, k, v = (normal(torch, (T, B, H, D), dt, s, 0.3) for s in (3, 4, 5))
    ld = torch.tensor([-0.01, -0.2], device="cuda")
    want, end = prnn.linear_attention(q, k, v, ld)
    far.copy_(k)
    got = prnn.linear_attention(q, far, v, ld)
    assert torch.equal(got[0], want) and torch.equal(got[1], end)
    prnn.linear_attention(q, k, v, ld, o=far)
    assert torch.equal(far, want)


def test_linear_attention_step_far_slot(env):
    torch, prnn = env
    n, dk, dv = 2 ** 15 + 100, 256, 256
    pool = torch.empty(n, 1, dk, dv, device="cuda")
    slots = torch.tensor([n - 1, 2 ** 15 - 1], dtype=torch.int32, device="cuda")
    state = normal(torch, (2, 1, dk, dv), torch.float32, 6)
    pool[slots.long()] = state
    q, k, v = (normal(torch, (2, 1, dk), torch.float32, s) for s in (7, 8, 9))
    ld = torch.tensor([-0.1], device="cuda")
    got = prnn.linear_attention_step(q, k, v, ld, pool, 1.0, slots)
    want = prnn.linear_attention_step(q, k, v, ld, state, 1.0)
    assert torch.equal(got, want) and torch.equal(pool[slots.long()], state)
