"""Root-mean-square norm written in place where rows are too long for registers: the kernels of such rows read them
from memory more than once, so what is written over must not be needed again.  Widths on both sides of the plans'
borders, on and off 16-byte accesses, with more rows than the longest grid has blocks.  Every result equals the same call's
with tensors of its own, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu
# 4 blocks of the long rows' kernels an SM stay and go on to a row a grid away: 700 rows are more than 4 x 152
SHAPES = [(5, 8192), (700, 8193), (700, 8200), (3, 16384), (640, 16392), (2, 40001)]


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    return torch, prnn


def normal(torch, shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(env, shape, dtype):
    """dx over dy, over dh, and over both where they are one tensor."""
    torch, prnn = env
    dt = getattr(torch, dtype)
    h, dy, dh = (normal(torch, shape, dt, 1 + i) for i in range(3))
    w = normal(torch, shape[1:], torch.float32, 4)
    _, _, rstd = prnn.rms_norm(h, w)
    for other in (None, dh):
        dx, dw = prnn.rms_norm_backward(dy, h, w, rstd, other)
        place = dy.clone()
        got, dw2 = prnn.rms_norm_backward(place, h, w, rstd, other, dx=place)
        assert got is place and torch.equal(got, dx) and torch.equal(dw2, dw), "dx over dy"
    place = dh.clone()
    got, dw2 = prnn.rms_norm_backward(dy, h, w, rstd, place, dx=place)
    assert torch.equal(got, dx) and torch.equal(dw2, dw), "dx over dh"
    dx, dw = prnn.rms_norm_backward(dy, h, w, rstd, dy)
    place = dy.clone()
    got, dw2 = prnn.rms_norm_backward(place, h, w, rstd, place, dx=place)
    assert torch.equal(got, dx) and torch.equal(dw2, dw), "dx over dy and dh in one"


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(env, shape, dtype):
    """y over x and over the residual, h over x and over the residual, in both outputs' types."""
    torch, prnn = env
    dt = getattr(torch, dtype)
    x, r = (normal(torch, shape, dt, 5 + i) for i in range(2))
    w = normal(torch, shape[1:], torch.float32, 7)
    y, _, rstd = prnn.rms_norm(x, w)
    place = x.clone()
    got, _, rstd2 = prnn.rms_norm(place, w, y=place)
    assert torch.equal(got, y) and torch.equal(rstd2, rstd), "y over x"
    y, h, rstd = prnn.rms_norm(x, w, residual=r)
    for y_over_x in (False, True):
        a, b = x.clone(), r.clone()
        got, stream, rstd2 = prnn.rms_norm(a, w, residual=b, y=a if y_over_x else b, h=b if y_over_x else a)
        assert torch.equal(got, y) and torch.equal(stream, h) and torch.equal(rstd2, rstd), y_over_x
    for group in (0, 128):
        q, scale, h8, _ = prnn.rms_norm_e4m3(x, w, residual=r, group=group)
        assert torch.equal(h8, h)
        for over_x in (False, True):
            a, b = x.clone(), r.clone()
            q2, scale2, stream, rstd2 = prnn.rms_norm_e4m3(a, w, residual=b, group=group, h=a if over_x else b)
            assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scale2, scale)
            assert torch.equal(stream, h) and torch.equal(rstd2, rstd), (group, over_x)


def test_backward_in_a_joint_tensor(env):
    """dx over dy as a slice of wider rows, which no 16-byte access fits."""
    torch, prnn = env
    wide = normal(torch, (9, 9001), torch.bfloat16, 8)
    h, w = normal(torch, (9, 8500), torch.bfloat16, 9), normal(torch, (8500,), torch.float32, 10)
    _, _, rstd = prnn.rms_norm(h, w)
    place = wide.clone()
    dx, dw = prnn.rms_norm_backward(wide[:, 3:8503], h, w, rstd)
    got, dw2 = prnn.rms_norm_backward(place[:, 3:8503], h, w, rstd, dx=place[:, 3:8503])
    assert torch.equal(got, dx) and torch.equal(dw2, dw)
    assert torch.equal(place[:, :3], wide[:, :3]) and torch.equal(place[:, 8503:], wide[:, 8503:])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", [(700, 40), (33, 301), (700, 2304), *SHAPES], ids=str)
def test_one_gradient_alone(env, shape, dtype):
    """dx with dweight NULL and no workspace, over dy; dweight with dx NULL."""
    torch, prnn = env
    dt = getattr(torch, dtype)
    code = {torch.float32: prnn.PRNN_F32, torch.bfloat16: prnn.PRNN_BF16}[dt]
    (rows, cols), st = shape, torch.cuda.current_stream().cuda_stream
    h, dy, dh = (normal(torch, shape, dt, 11 + i) for i in range(3))
    w = normal(torch, (cols,), torch.float32, 14)
    _, _, rstd = prnn.rms_norm(h, w)
    dx, dw = prnn.rms_norm_backward(dy, h, w, rstd, dh)
    place = dy.clone()
    prnn.prnn_rms_norm_backward(code, rows, cols, place, cols, h, cols, w, rstd, dh, cols, place, cols, None, None, 0, st)
    assert torch.equal(place, dx)
    n = prnn.prnn_rms_norm_workspace(rows, cols)
    out, ws = torch.full_like(dw, 7.0), torch.empty(n, dtype=torch.uint8, device="cuda")
    prnn.prnn_rms_norm_backward(code, rows, cols, dy, cols, h, cols, w, rstd, dh, cols, None, 0, out, ws, n, st)
    assert torch.equal(out, dw)
