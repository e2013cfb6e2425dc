"""Layer norm of one row of 2^31 - 1 columns, the most that its interface takes: column counters that step past
the last column leave 32 bits.

The row alternates between 1 and -1, so the sums over 2^21 values a thread are whole numbers and exact: the
mean is 2^-31 and the variance 1 within 2^-23, whatever the order.  With eps = 1e-5 the outputs are
+-(1 - 5e-6), which is +-1 in bf16 (spacing 2^-8 below 1); dx is what the projection leaves of dy = x,
rstd * 1e-5 at most with an error of a few 2^-22 in the two means; dgamma is 1 - 5e-6 and dbeta is dy."""
import pytest

pytestmark = pytest.mark.gpu
COLS = 2 ** 31 - 1


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


def test_one_row_of_all_columns(env):
    torch, prnn = env
    x = torch.ones(1, COLS, dtype=torch.bfloat16, device="cuda")
    x[:, 1::2] = -1
    y = torch.full_like(x, 7.0)
    y, mean, rstd = prnn.layer_norm(x, y=y)
    assert torch.equal(y, x)
    assert abs(float(mean)) <= 2.0 ** -20 and abs(float(rstd) - 1) <= 1e-5
    del y
    dx, dgamma, dbeta = prnn.layer_norm_backward(x, x, None, mean, rstd)
    assert float(dx.abs().max()) <= 2e-5
    del dx
    part = 1 << 28
    for lo in range(0, COLS, part):
        assert torch.equal(dbeta[lo:lo + part], x[0, lo:lo + part].float()), lo
        assert float((dgamma[lo:lo + part] - 1).abs().max()) <= 1e-5, lo
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK
