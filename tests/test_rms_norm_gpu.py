"""GPU tests of root-mean-square norm (with the residual's addition, in the data's type and in 8 bits, and its
gradient) against its definition in 64 bits.

Tolerances.  U = 2^-24 is the rounding of one fp32 operation, u (2^-24, 2^-11, 2^-8) that of an output.  The sum of
squares has terms of one sign and at most 64 additions in a row, the root and the products add a few: rstd and
y carry at most 72 U of themselves before y's one rounding.  The stream is a sum of two values of its type,
rounded once: it is compared bit for bit with the same sum in 64 bits.  A value in 8 bits is off by
half a step, 2^-4 of itself, or 2^-10 of the scale for subnormal ones.  A column's sum adds at most 256 + rows / 32
terms in a row in any order used here.
"""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
# every plan: rows in 8, 16 and 32 lanes, in a block with 1, 2, 4 and 8 packs a thread, and longer ones
SHAPES = [(1, 1), (3, 2), (5, 31), (7, 40), (300, 64), (33, 100), (2, 127), (9, 128), (1000, 129), (70, 256),
          (4, 301), (130, 1152), (4, 1792), (700, 1001), (650, 2304), (3, 2305), (1300, 4096), (2, 5760), (640, 5763),
          (1, 8192), (620, 8200), (2, 8193), (2, 16392), (2, 40001), (611, 33000)]


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    return torch, prnn


def typed(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def normal(torch, shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def within(got, want, bound, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - want).abs().max()))


def rounding(want, dtype):
    return (HALF[dtype] * want.abs()).clamp(min=LEAST[dtype])


def reference(torch, x, w, eps, res):
    h = x if res is None else (x.double() + res.double()).to(x.dtype)
    hd = h.double()
    rstd = (hd.pow(2).mean(-1) + eps).rsqrt()
    return hd * rstd[..., None] * (1.0 if w is None else w.double()), h, rstd


def check_e4m3(torch, q, scale, y, group, what):
    cols = y.shape[-1]
    width = group or cols
    tops = torch.stack([p.abs().amax(-1) for p in y.split(width, -1)], -1)
    want = torch.where(tops > 0, tops / 448, torch.ones_like(tops))
    within(scale, want, 80 * U * want, what + ": scale")
    wide = scale.double().repeat_interleave(width, -1)[..., :cols]
    within(q.double() * wide, y, 2.0 ** -4 * y.abs() + 2.0 ** -10 * wide + 80 * U * y.abs(), what + ": q")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(env, shape, dtype):
    torch, prnn = env
    dt = typed(torch, dtype)
    x, r = normal(torch, shape, dt, 1), normal(torch, shape, dt, 2, 2.0)
    w = normal(torch, shape[1:], torch.float32, 3)
    for weight, res in ((w, r), (None, None), (w, None), (None, r)):
        want, hw, rw = reference(torch, x, weight, 1e-6, res)
        y, h, rstd = prnn.rms_norm(x, weight, 1e-6, res)
        assert torch.equal(h, hw) and (res is not None or h is x)
        within(rstd, rw, 72 * U * rw, "rstd")
        within(y, want, rounding(want, dtype) + 72 * U * want.abs(), "y")
        for group in (0, 128):
            q, scale, h, r8 = prnn.rms_norm_e4m3(x, weight, 1e-6, res, group)
            assert torch.equal(h, hw) and torch.equal(r8, rstd) and q.dtype is torch.float8_e4m3fn
            check_e4m3(torch, q, scale, want, group, f"group {group}")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(env, shape, dtype):
    torch, prnn = env
    dt = typed(torch, dtype)
    h, dy, dh = (normal(torch, shape, dt, 4 + i) for i in range(3))
    w = normal(torch, shape[1:], torch.float32, 7)
    for weight, other in ((w, dh), (None, None), (w, None)):
        _, _, rstd = prnn.rms_norm(h, weight)
        dx, dw = prnn.rms_norm_backward(dy, h, weight, rstd, other)
        r = rstd.double()[:, None]
        xhat, dyd = h.double() * r, dy.double()
        g = dyd if weight is None else dyd * weight.double()
        want = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        M = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
        if other is not None:
            want, M = want + other.double(), M + other.double().abs()
        within(dx, want, rounding(want, dtype) + 80 * U * M, "dx")
        within(dw, (dyd * xhat).sum(0), (256 + shape[0] / 32) * U * (dyd * xhat).abs().sum(0), "dweight")


@pytest.mark.parametrize("residual", [False, True])
def test_gradient_against_differences(env, residual):
    """Central differences of the fp32 forward pass along random directions, h = 2^-7: the cubic term is about h^2 of
    the slope and rounding 2^-24 |L| / h, both below 1e-3 of the slope's scale."""
    torch, prnn = env
    shape = (6, 200)
    x, res, dy, dh = (normal(torch, shape, torch.float32, 10 + i) for i in range(4))
    w = normal(torch, shape[1:], torch.float32, 15)
    res = res if residual else None

    def loss(x, w):
        y, h, _ = prnn.rms_norm(x, w, 1e-6, res)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())
    _, h, rstd = prnn.rms_norm(x, w, 1e-6, res)
    dx, dw = prnn.rms_norm_backward(dy, h, w, rstd, dh)
    step = 2.0 ** -7
    for seed in range(3):
        d, e = normal(torch, shape, torch.float32, 20 + seed), normal(torch, shape[1:], torch.float32, 30 + seed)
        for got, grad, v in (((loss(x + step * d, w) - loss(x - step * d, w)) / (2 * step), dx, d),
                             ((loss(x, w + step * e) - loss(x, w - step * e)) / (2 * step), dw, e)):
            scale = float(grad.double().norm() * v.double().norm()) / v.numel() ** 0.5
            assert abs(got - float((grad.double() * v.double()).sum())) <= 2e-3 * scale + 1e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_places(env, dtype):
    """Rows of wider tensors at every alignment, outputs in place, and heads of a joint projection."""
    torch, prnn = env
    dt = typed(torch, dtype)
    wide, other = normal(torch, (9, 1000), dt, 40), normal(torch, (9, 1100), dt, 41)
    w = normal(torch, (1000,), torch.float32, 42)
    for lo, cols in ((0, 512), (8, 512), (1, 512), (3, 997), (2, 64), (16, 120)):
        x, r = wide[:, lo:lo + cols], other[:, lo:lo + cols]
        want, hw, _ = reference(torch, x, w[lo:lo + cols], 1e-6, r)
        y, h, rstd = prnn.rms_norm(x, w[lo:lo + cols], 1e-6, r)
        within(y, want, rounding(want, dtype) + 72 * U * want.abs(), (lo, cols))
        assert torch.equal(h, hw)
        out, stream = torch.full_like(other, 7.0), other.clone()
        prnn.rms_norm(x, w[lo:lo + cols], 1e-6, stream[:, lo:lo + cols], y=out[:, lo:lo + cols],
                      h=stream[:, lo:lo + cols])
        assert torch.equal(out[:, lo:lo + cols], y) and torch.equal(stream[:, lo:lo + cols], h)
        for t, before in ((out, torch.full_like(other, 7.0)), (stream, other)):
            assert torch.equal(t[:, :lo], before[:, :lo]) and torch.equal(t[:, lo + cols:], before[:, lo + cols:])
        q, scale, h8, _ = prnn.rms_norm_e4m3(x, w[lo:lo + cols], 1e-6, r, 128)
        assert torch.equal(h8, hw)
        check_e4m3(torch, q, scale, want, 128, "strided")
        both = x.clone(), r.clone()
        prnn.rms_norm(both[0], w[lo:lo + cols], 1e-6, both[1], y=both[1], h=both[0])
        assert torch.equal(both[1], y) and torch.equal(both[0], h)
        dy, dh = both[0].clone(), both[1].clone()
        dx, dw = prnn.rms_norm_backward(dy, x, w[lo:lo + cols], rstd, dh)
        for place in (dy.clone(), dh.clone()):
            a, b = (place, dh) if torch.equal(place, dy) else (dy, place)
            got, dw2 = prnn.rms_norm_backward(a, x, w[lo:lo + cols], rstd, b, dx=place)
            assert got is place and torch.equal(got, dx) and torch.equal(dw2, dw)
    qkv = normal(torch, (5, 3, 4, 96), dt, 43)
    q = qkv[..., 32:64]                       # [T, B, heads, 32] of a joint projection
    want, _, _ = reference(torch, q, None, 0.0, None)
    y, _, rstd = prnn.rms_norm(q, None, 0.0)
    assert rstd.shape == (5, 3, 4)
    within(y, want, rounding(want, dtype) + 72 * U * want.abs(), "heads")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [100, 128, 131, 2048, 2049, 40000])
def test_rows_of_zeros_infinities_and_nan(env, dtype, cols):
    """A row of zeros is 0 with scales 1; an infinity or NaN stays in its own row."""
    torch, prnn = env
    dt = typed(torch, dtype)
    x = normal(torch, (6, cols), dt, 50)
    clean, _, _ = prnn.rms_norm(x, None)
    x[1] = 0
    x[3, cols // 2] = float("inf")
    x[4, cols - 1] = float("nan")
    y, _, rstd = prnn.rms_norm(x, None)
    assert bool((y[1] == 0).all()) and torch.equal(y[[0, 2, 5]], clean[[0, 2, 5]])
    assert float(rstd[3]) == 0 and bool(y[3, cols // 2].isnan()) and bool(y[4].isnan().all())
    for group in (0, 128):
        q, scale, _, _ = prnn.rms_norm_e4m3(x, None, group=group)
        assert bool((q[1].float() == 0).all()) and bool((scale[1] == 1).all())
        assert bool(q[3, cols // 2].float().isnan()) and bool(q[4].float().isnan().all())
        assert bool(q[[0, 2, 5]].float().isfinite().all())


@pytest.mark.parametrize("cols", [100, 256, 301, 40000])
def test_values_too_small_for_a_scale(env, cols):
    """Outputs whose largest is 2^-100 and below become zeros with the scale 1, not infinities or NaN; just above that they
    keep their bits."""
    torch, prnn = env
    x = normal(torch, (3, cols), torch.float32, 80)
    x[:, ::7] = 0
    for power, zero in ((-140, True), (-125, True), (-110, True), (-97, False), (120, False)):
        w = torch.full((cols,), 2.0 ** power, device="cuda")
        want, _, _ = reference(torch, x, w, 1e-6, None)
        for group in (0, 128):
            q, scale, _, _ = prnn.rms_norm_e4m3(x, w, 1e-6, group=group)
            assert bool(q.float().isfinite().all())
            if zero:
                assert bool((q.float() == 0).all()) and bool((scale == 1).all())
            else:
                check_e4m3(torch, q, scale, want, group, f"2^{power}")


def test_empty_and_single(env):
    torch, prnn = env
    x = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16)
    y, h, rstd = prnn.rms_norm(x, None)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    q, scale, _, _ = prnn.rms_norm_e4m3(x)
    assert q.shape == (0, 64) and scale.shape == (0, 1)
    dx, dw = prnn.rms_norm_backward(x, x, None, rstd)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_refusals(env):
    torch, prnn = env
    x = normal(torch, (4, 64), torch.bfloat16, 60)
    w = torch.ones(64, device="cuda")
    for call in (lambda: prnn.rms_norm(x, w[:32]), lambda: prnn.rms_norm(x, w.half()),
                 lambda: prnn.rms_norm(x, w, 1e-6, x[:2]), lambda: prnn.rms_norm(x, w, 1e-6, x.float()),
                 lambda: prnn.rms_norm(x, w, h=x), lambda: prnn.rms_norm(x, w, y=x.float()),
                 lambda: prnn.rms_norm_e4m3(x, w, group=64), lambda: prnn.rms_norm(x.t(), w[:4]),
                 lambda: prnn.rms_norm(x.double()), lambda: prnn.rms_norm_backward(x, x, w, w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(Exception):
        prnn.rms_norm(x, w, -1.0)


def test_graph_and_streams(env):
    """Captured and replayed on new values; and on another stream with inputs dropped at once."""
    torch, prnn = env
    x, res = normal(torch, (300, 1152), torch.bfloat16, 70), normal(torch, (300, 1152), torch.bfloat16, 71)
    w = normal(torch, (1152,), torch.float32, 72)

    def all_of(x, res):
        y, h, rstd = prnn.rms_norm(x, w, 1e-6, res)
        return (y, h, rstd, *prnn.rms_norm_e4m3(x, w, 1e-6, res)[:2], *prnn.rms_norm_backward(y, h, w, rstd, x))
    all_of(x, res)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = all_of(x, res)
    x.copy_(normal(torch, x.shape, x.dtype, 73))
    want = all_of(x, res)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, rstd = prnn.rms_norm(x.clone(), w, 1e-6, res.clone(), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(h, want[1]) and torch.equal(rstd, want[2])
