"""Layer norm and its gradient with more rows than the blocks take at once, against 64 bits: the plans of large
calls, every group of threads visiting enough rows to go round its ring of rows in shared memory more than once,
with last turns that are not full.

Bounds: those of tests/test_sequence_ops_gpu.py for the rows (no sum has more than 64 additions in a row: at
most 20 a thread, 5 in a warp, 32 over warps).  dgamma and dbeta are added row by row in a group, of which
there is at least one an SM of 132 or more, then over at most 16 groups and 160 blocks in 8 shares:
rows / 132 + 64 additions in a row."""
import pytest

from tests.test_sequence_ops_gpu import U, env, norm_reference, normal, rounding, types, within  # noqa: F401

pytestmark = pytest.mark.gpu

# rows enough for eight visits or more of every group (with 152 SMs), and not a multiple of the groups
SHAPES = [(31007, 31), (25013, 301), (8009, 700), (6007, 1152), (5003, 2001), (3001, 2501), (3001, 4096), (2003, 5760),
          (1501, 7001), (1213, 8192), (601, 12280), (607, 12287)]
# the register plans of the forward pass that these leave out
FORWARD = [(977, n) for n in (128, 256, 512, 768, 1024, 1280, 2048, 16384)] + [(305, 20000), (305, 32768), (311, 20001)]
# few rows, where a row is spread over many threads
FEW = [(3, 5761), (2, 8191), (5, 4097), (303, 1500)]


def laid(torch, shape, dtype, seed, layout, fill=None):
    """A tensor of `shape`: packed, or columns 1 .. of a wider one (rows at every alignment)."""
    rows, cols = shape
    x = normal(torch, shape, dtype, seed) + 0.5 if fill is None else torch.full(shape, fill, dtype=dtype, device="cuda")
    if layout == "packed":
        return x, None
    wide = torch.full((rows, cols + 3), 7.0, dtype=dtype, device="cuda")
    wide[:, 1:1 + cols] = x
    return wide[:, 1:1 + cols], wide


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("shape", SHAPES + FORWARD + FEW, ids=str)
def test_forward(env, shape, layout, dtype):  # noqa: F811
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x, _ = laid(torch, shape, dt, 1, layout)
    out, wide = laid(torch, shape, dt, 0, layout, fill=9.0)
    gamma, beta = normal(torch, shape[1:], torch.float32, 2), normal(torch, shape[1:], torch.float32, 3)
    y, mean, rstd = prnn.layer_norm(x, gamma, beta, 1e-5, y=out)
    want, wm, wr, M = norm_reference(torch, x, gamma, beta, 1e-5)
    within(y, want, rounding(want, u) + 128 * U * M, "y")
    within(mean, wm, 128 * U * x.double().abs().mean(-1), "mean")
    within(rstd, wr, wr * 128 * U * (1 + (wm * wr).abs()), "rstd")
    if wide is not None:
        assert bool((wide[:, 0] == 7).all()) and bool((wide[:, 1 + shape[1]:] == 7).all())
    assert torch.equal(prnn.layer_norm(x, gamma, beta, 1e-5, y=x)[0], y)      # in place
    ones, zeros = torch.ones_like(gamma), torch.zeros_like(beta)
    assert torch.equal(prnn.layer_norm(out)[0], prnn.layer_norm(out, ones, zeros)[0])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("shape", SHAPES + [(305, 20001)] + FEW, ids=str)
def test_backward(env, shape, layout, dtype):  # noqa: F811
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x, _ = laid(torch, shape, dt, 4, layout)
    dy = normal(torch, shape, dt, 5)
    if layout == "odd":                 # another phase than x's
        wide = torch.zeros(shape[0], shape[1] + 6, dtype=dt, device="cuda")
        wide[:, 3:3 + shape[1]] = dy
        dy = wide[:, 3:3 + shape[1]]
    gamma = normal(torch, shape[1:], torch.float32, 6)
    _, mean, rstd = prnn.layer_norm(x, gamma, None)
    for g in (gamma, None):
        dx, dg, db = prnn.layer_norm_backward(dy, x, g, mean, rstd)
        xd, dyd, r = x.double(), dy.double(), rstd.double()[:, None]
        xhat = (xd - mean.double()[:, None]) * r
        gd = dyd if g is None else dyd * g.double()
        want = r * (gd - gd.mean(-1, keepdim=True) - xhat * (gd * xhat).mean(-1, keepdim=True))
        wide_ = xhat.abs() + (xd.abs() + mean.double().abs()[:, None]) * r
        M = r * (gd.abs() + gd.abs().mean(-1, keepdim=True) + 2 * wide_ * (gd.abs() * wide_).mean(-1, keepdim=True))
        within(dx, want, rounding(want, u) + 128 * U * M, "dx")
        n = 64 + shape[0] / 132
        within(dg, (dyd * xhat).sum(0), n * U * (dyd.abs() * wide_).sum(0), "dgamma")
        within(db, dyd.sum(0), n * U * dyd.abs().sum(0), "dbeta")
        again = prnn.layer_norm_backward(dy, x, g, mean, rstd)
        assert all(torch.equal(a, b) for a, b in zip(again, (dx, dg, db)))


def test_no_wait_has_run_out(env):  # noqa: F811
    torch, prnn = env
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK
