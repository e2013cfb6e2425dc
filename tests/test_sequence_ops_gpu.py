"""GPU tests of the sequence operators (layer norm, dropout, linear attention with a decay per
head) against their definitions in 64 bits.

Tolerances, derived from the arithmetic.  u = 2^-24 for fp32, 2^-11 for fp16, 2^-8 for bf16 is the
rounding of an output (never less than half the spacing of the type's subnormal numbers, 2^-25 for
fp16), U = 2^-24 that of one fp32 operation.
  * layer norm: each value comes from sums of at most 8192 terms, taken as <= 64 additions in a
    row in any order used here, and a few products: u |y| + 128 U (|xhat gamma| + |beta| +
    |mean| rstd |gamma|), the last term for the cancellation in x - mean.
  * linear attention: u |out| + E M, with M the same sum over absolute values (no cancellation)
    and E = 2^-15 + 2^-13 (T / 128 + 1) 2^-10 for 16-bit data (products of factors held in two 16-bit
    parts, 2^-16 each, and fp32 sums) and n U, n = d + T + 64 additions, for fp32 data.  States are
    fp32 sums of exact products times a decay: n U M for either.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    return torch, prnn


def types(torch):
    return {"f32": (torch.float32, 2.0 ** -24), "f16": (torch.float16, 2.0 ** -11),
            "bf16": (torch.bfloat16, 2.0 ** -8)}


def normal(torch, shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def rounding(want, u):
    """Bound of one rounding to the type whose relative rounding is u."""
    return (u * want.abs()).clamp(min={2.0 ** -24: 2.0 ** -150, 2.0 ** -11: 2.0 ** -25, 2.0 ** -8: 2.0 ** -134}[u])


def within(got, want, bound, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - want).abs().max()))


# ---- layer norm -------------------------------------------------------------------
def norm_reference(torch, x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean) ** 2).mean(-1, keepdim=True).add(eps).rsqrt()
    g = 1.0 if gamma is None else gamma.double()
    b = torch.zeros_like(x[0]) if beta is None else beta.double()
    y = (x - mean) * rstd * g + b
    M = ((x - mean) * rstd * g).abs() + b.abs() + (mean.abs() * rstd) * (g if gamma is None else g.abs())
    return y, mean[..., 0], rstd[..., 0], M


NORM_SHAPES = [(1, 1), (3, 2), (5, 31), (4, 64), (7, 100), (2, 255), (33, 256), (9, 301), (4, 1792),
               (130, 1152), (3, 2305), (2, 4096), (300, 40), (2, 5760), (1, 8192), (2, 20001)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_layer_norm(env, shape, dtype):
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x = normal(torch, shape, dt, 1) + 0.5
    gamma, beta = normal(torch, shape[1:], torch.float32, 2), normal(torch, shape[1:], torch.float32, 3)
    for g, b in ((gamma, beta), (None, None), (gamma, None), (None, beta)):
        y, mean, rstd = prnn.layer_norm(x, g, b, 1e-5)
        want, wm, wr, M = norm_reference(torch, x, g, b, 1e-5)
        within(y, want, rounding(want, u) + 128 * U * M, (shape, dtype))
        within(mean, wm, 128 * U * x.double().abs().mean(-1), "mean")
        # rstd's relative error is half that of a sum of squares of differences
        within(rstd, wr, wr * 128 * U * (1 + (wm * wr).abs()), "rstd")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_layer_norm_backward(env, shape, dtype):
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x, dy = normal(torch, shape, dt, 4) + 0.25, normal(torch, shape, dt, 5)
    gamma = normal(torch, shape[1:], torch.float32, 6)
    for g in (gamma, None):
        _, mean, rstd = prnn.layer_norm(x, g, None)
        dx, dg, db = prnn.layer_norm_backward(dy, x, g, mean, rstd)
        xd, dyd, r = x.double(), dy.double(), rstd.double()[:, None]
        xhat = (xd - mean.double()[:, None]) * r
        gd = dyd if g is None else dyd * g.double()
        want = r * (gd - gd.mean(-1, keepdim=True) - xhat * (gd * xhat).mean(-1, keepdim=True))
        # xhat itself carries U (|x| + |mean|) rstd
        wide = xhat.abs() + (xd.abs() + mean.double().abs()[:, None]) * r
        M = r * (gd.abs() + gd.abs().mean(-1, keepdim=True) + 2 * wide * (gd.abs() * wide).mean(-1, keepdim=True))
        within(dx, want, rounding(want, u) + 128 * U * M, "dx")
        n = 64 + shape[0] / 32
        within(dg, (dyd * xhat).sum(0), n * U * (dyd.abs() * wide).sum(0), "dgamma")
        within(db, dyd.sum(0), n * U * dyd.abs().sum(0), "dbeta")


def test_layer_norm_gradient_against_differences(env):
    """Central differences of the fp32 kernel's own forward along random directions.
    Step h = 2^-7: the cubic term is about h^2 of the slope and rounding about 2^-24 |L| / h, both
    below 1e-3 of the slope's scale here."""
    torch, prnn = env
    x, dy = normal(torch, (6, 200), torch.float32, 7), normal(torch, (6, 200), torch.float32, 8)
    gamma, beta = normal(torch, (200,), torch.float32, 9), normal(torch, (200,), torch.float32, 10)
    _, mean, rstd = prnn.layer_norm(x, gamma, beta)
    dx, dg, db = prnn.layer_norm_backward(dy, x, gamma, mean, rstd)

    def loss(x, g, b):
        return float((prnn.layer_norm(x, g, b)[0].double() * dy.double()).sum())
    h = 2.0 ** -7
    for seed in range(3):
        d = normal(torch, x.shape, torch.float32, 20 + seed)
        e = normal(torch, gamma.shape, torch.float32, 30 + seed)
        for got, grad, v in (((loss(x + h * d, gamma, beta) - loss(x - h * d, gamma, beta)) / (2 * h), dx, d),
                             ((loss(x, gamma + h * e, beta) - loss(x, gamma - h * e, beta)) / (2 * h), dg, e),
                             ((loss(x, gamma, beta + h * e) - loss(x, gamma, beta - h * e)) / (2 * h), db, e)):
            scale = float(grad.double().norm() * v.double().norm()) / math.sqrt(v.numel())
            assert abs(got - float((grad.double() * v.double()).sum())) <= 2e-3 * scale + 1e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_strides_and_places(env, dtype):
    """Rows of a wider tensor, at every alignment; in place; a large common offset; equal rows."""
    torch, prnn = env
    dt, u = types(torch)[dtype]
    wide = normal(torch, (9, 1000), dt, 11)
    gamma = normal(torch, (997,), torch.float32, 12)
    for lo, cols in ((0, 512), (8, 512), (1, 512), (3, 997), (2, 64)):
        x = wide[:, lo:lo + cols]
        y, mean, rstd = prnn.layer_norm(x, gamma[:cols], None)
        want, _, _, M = norm_reference(torch, x, gamma[:cols], None, 1e-5)
        within(y, want, rounding(want, u) + 128 * U * M, (lo, cols))
        out = torch.full_like(wide, 7.0)
        prnn.layer_norm(x, gamma[:cols], None, y=out[:, lo:lo + cols])
        assert torch.equal(out[:, lo:lo + cols], y)
        assert bool((out[:, :lo] == 7).all()) and bool((out[:, lo + cols:] == 7).all())
        dx = prnn.layer_norm_backward(wide[:, lo:lo + cols], x, gamma[:cols], mean, rstd)
        ref = prnn.layer_norm_backward(x.contiguous(), x.contiguous(), gamma[:cols], mean, rstd)
        # another access width may add in another order
        within(dx[0], ref[0], 2 * u * ref[0].double().abs() + 256 * U * (1 + ref[0].double().abs().max()), lo)
    x = wide.clone()
    y = prnn.layer_norm(wide)[0]
    assert torch.equal(prnn.layer_norm(x, y=x)[0], y)
    big = (wide.float() + 1000.0).to(torch.float32)
    y, _, _ = prnn.layer_norm(big)
    want, _, _, M = norm_reference(torch, big, None, None, 1e-5)
    within(y, want, rounding(want, U) + 128 * U * M, "offset")
    flat = torch.full((3, 100), 2.0, dtype=dt, device="cuda")
    assert bool((prnn.layer_norm(flat)[0] == 0).all())


def test_layer_norm_rows_do_not_meet(env):
    """A row of infinities and NaN leaves the others' results as they are."""
    torch, prnn = env
    x = normal(torch, (8, 300), torch.float32, 13)
    y = prnn.layer_norm(x)[0]
    bad = x.clone()
    bad[3] = float("nan")
    bad[5, 7] = float("inf")
    got = prnn.layer_norm(bad)[0]
    keep = [0, 1, 2, 4, 6, 7]
    assert torch.equal(got[keep], y[keep])
    assert bool(got[3].isnan().all()) and bool(got[5].isnan().all())


# ---- dropout ----------------------------------------------------------------------
def philox_words(n, seed, offset):
    """Philox4x32-10 in Python integers."""
    m = 2 ** 32 - 1
    out = []
    for i in range((n + 3) // 4):
        c = [i & m, i >> 32, offset & m, offset >> 32]
        k = [seed & m, seed >> 32]
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
            k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
        out += c
    return out[:n]


def test_philox_against_published_vectors():
    """The known answers that accompany the generator's publication (all zeros, all ones)."""
    def block(c, k):
        m = 2 ** 32 - 1
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
            k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
        return c
    assert block([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert block([2 ** 32 - 1] * 4, [2 ** 32 - 1] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert philox_words(4, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 31, 1000, 4099])
def test_dropout(env, n, dtype):
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x, res = normal(torch, (n,), dt, n), normal(torch, (n,), dt, n + 1)
    for p, seed, offset in ((0.0, 5, 0), (0.1, 2 ** 63 + 12345, 2 ** 64 - 2), (0.5, 0, 2 ** 33 + 1)):
        words = torch.tensor(philox_words(n, seed, offset), dtype=torch.int64, device="cuda")
        kept = words >= round(p * 2 ** 32)
        want = torch.where(kept, x.double() / (1 - p), torch.zeros((), device="cuda", dtype=torch.float64))
        got = prnn.dropout(x, p, seed, offset)
        assert torch.equal(got != 0, kept & (x != 0))
        within(got, want, rounding(want, u) + 4 * U * want.abs(), (n, p))
        assert torch.equal(prnn.dropout_backward(x, p, seed, offset), got)
        both = prnn.dropout(x, p, seed, offset, res)
        sum_ = want + res.double()
        within(both, sum_, rounding(sum_, u) + 4 * U * (want.abs() + res.double().abs()), (n, p))
        for place in (x.clone(), res.clone()):
            a, r = (place, res) if torch.equal(place, x) else (x, place)
            assert torch.equal(prnn.dropout(a, p, seed, offset, r, y=place), both)


def test_dropout_alignment_and_counts(env):
    """Views at every alignment draw the mask of their own first value; the share dropped is p
    within five standard deviations; another offset is another mask."""
    torch, prnn = env
    base = torch.ones(100_003, dtype=torch.float16, device="cuda")
    whole = prnn.dropout(base.clone(), 0.3, 7, 1)
    for lo in (1, 2, 3, 4, 8):
        assert torch.equal(prnn.dropout(base[lo:], 0.3, 7, 1), whole[:base.numel() - lo])
    n = base.numel()
    dropped = int((whole == 0).sum())
    assert abs(dropped - 0.3 * n) <= 5 * math.sqrt(0.21 * n)
    other = prnn.dropout(base.clone(), 0.3, 7, 2)
    both = int(((whole == 0) & (other == 0)).sum())
    assert abs(both - 0.09 * n) <= 5 * math.sqrt(0.09 * 0.91 * n)


def test_dropout_drops_what_is_not_finite(env):
    torch, prnn = env
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::2] = float("inf")
    y = prnn.dropout(x, 0.5, 3, 4, torch.ones_like(x))
    kept = torch.tensor(philox_words(4096, 3, 4), device="cuda") >= 2 ** 31
    assert bool((y[~kept] == 1).all()) and not bool(torch.isfinite(y[kept]).any())


# ---- linear attention ---------------------------------------------------------------
def attention_reference(torch, q, k, v, ld, scale, state, lens, grad=None, dstate=None):
    """Token by token in 64 bits; with grad (d_o) the gradients instead."""
    f = torch.float64
    T, B, H, dv = v.shape
    g = H // q.shape[2]
    q, k, v = (x.to(f) for x in (q, k, v))
    q, k = q.repeat_interleave(g, 2), k.repeat_interleave(g, 2)
    dk = q.shape[3]
    l = ld.to(f).exp()
    lens = [T] * B if lens is None else [max(0, min(T, int(n))) for n in lens.tolist()]
    S = torch.zeros(B, H, dk, dv, dtype=f, device=v.device) if state is None else state.to(f).clone()
    o = torch.zeros(T, B, H, dv, dtype=f, device=v.device)
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    R = torch.zeros_like(S) if dstate is None else dstate.to(f).clone()
    for b in range(B):
        for t in range(lens[b]):
            S[b] = l[:, None, None] * S[b] + k[t, b][:, :, None] * v[t, b][:, None, :]
            o[t, b] = scale * torch.einsum("hd,hde->he", q[t, b], S[b])
            if grad is not None:
                dq[t, b] = scale * torch.einsum("hde,he->hd", S[b], grad[t, b].to(f))
        if grad is None:
            continue
        for t in reversed(range(lens[b])):
            R[b] += scale * q[t, b][:, :, None] * grad[t, b].to(f)[:, None, :]
            dkk[t, b] = torch.einsum("hde,he->hd", R[b], v[t, b])
            dvv[t, b] = torch.einsum("hde,hd->he", R[b], k[t, b])
            R[b] *= l[:, None, None]
    if grad is None:
        return o, S
    return {"dq": dq.reshape(T, B, H // g, g, dk).sum(3), "dk": dkk.reshape(T, B, H // g, g, dk).sum(3),
            "dv": dvv, "dstate": R}


def attention_tolerance(dtype, T, d):
    fp32 = (d + T + 64) * U
    return fp32 if dtype == "f32" else 2.0 ** -15 + 2.0 ** -23 * (T / 128 + 1) + fp32, fp32


def make(torch, T, B, H, Hq, dk, dv, dt, seed, state=False, lens=None, decay=None):
    x = dict(q=normal(torch, (T, B, Hq, dk), dt, seed), k=normal(torch, (T, B, Hq, dk), dt, seed + 1, dk ** -0.5),
             v=normal(torch, (T, B, H, dv), dt, seed + 2),
             ld=torch.tensor([(decay or [-0.002, -0.05, -0.7, -4.0])[h % len(decay or range(4))]
                              for h in range(H)], device="cuda"),
             scale=dk ** -0.5, state=normal(torch, (B, H, dk, dv), torch.float32, seed + 3) if state else None,
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return x


def absolute(x, **more):
    out = {n: v.abs() if n in ("q", "k", "v", "state", "grad", "dstate") and v is not None else v
           for n, v in {**x, **more}.items()}
    return out


def check_forward(env, x, dtype, what):
    torch, prnn = env
    u = types(torch)[dtype][1]
    o, end = prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"], x["lens"])
    want, wend = attention_reference(torch, **x)
    M, Mend = attention_reference(torch, **absolute(x))
    tol, tol32 = attention_tolerance(dtype, x["q"].shape[0], x["q"].shape[3])
    within(o, want, rounding(want, u) + tol * M + 1e-38, (what, "o"))
    within(end, wend, tol32 * Mend, (what, "state"))
    return o, end


def check_backward(env, x, dtype, what, seed, dstate=False):
    torch, prnn = env
    dt, u = types(torch)[dtype]
    do = normal(torch, x["v"].shape, dt, seed)
    ds = normal(torch, (x["v"].shape[1], x["v"].shape[2], x["q"].shape[3], x["v"].shape[3]), torch.float32,
                seed + 1) if dstate else None
    g = prnn.linear_attention_backward(do, x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"],
                                       x["lens"], ds)
    assert ("dstate" in g) == (x["state"] is not None)
    want = attention_reference(torch, **x, grad=do, dstate=ds)
    M = attention_reference(torch, **absolute(x, grad=do, dstate=ds))
    tol, tol32 = attention_tolerance(dtype, x["q"].shape[0], max(x["q"].shape[3], x["v"].shape[3]))
    for n in g:
        if n == "dstate":
            within(g[n], want[n], tol32 * M[n], (what, n))
        else:
            within(g[n], want[n], rounding(want[n], u) + tol * M[n] + 1e-38, (what, n))


SIZES = [dict(T=1, B=1, H=1, Hq=1, dk=1, dv=1), dict(T=1, B=3, H=2, Hq=2, dk=16, dv=16),
         dict(T=5, B=2, H=2, Hq=1, dk=7, dv=33), dict(T=31, B=1, H=4, Hq=4, dk=64, dv=64),
         dict(T=33, B=2, H=3, Hq=3, dk=64, dv=32), dict(T=64, B=2, H=2, Hq=2, dk=128, dv=128),
         dict(T=127, B=1, H=4, Hq=2, dk=128, dv=64), dict(T=128, B=1, H=2, Hq=2, dk=64, dv=128),
         dict(T=129, B=2, H=2, Hq=2, dk=64, dv=64), dict(T=300, B=2, H=4, Hq=4, dk=32, dv=96),
         dict(T=257, B=1, H=6, Hq=2, dk=72, dv=100), dict(T=140, B=1, H=2, Hq=2, dk=40, dv=136),
         dict(T=70, B=1, H=1, Hq=1, dk=256, dv=256), dict(T=600, B=1, H=4, Hq=1, dk=128, dv=128)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_linear_attention(env, i, dtype):
    torch, _ = env
    dt = types(torch)[dtype][0]
    check_forward(env, make(torch, **SIZES[i], dt=dt, seed=100 + 10 * i, state=i % 2 == 1), dtype, SIZES[i])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_linear_attention_backward(env, i, dtype):
    torch, _ = env
    dt = types(torch)[dtype][0]
    check_backward(env, make(torch, **SIZES[i], dt=dt, seed=300 + 10 * i, state=i % 2 == 1), dtype, SIZES[i],
                   500 + 10 * i, dstate=i % 4 == 1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_linear_attention_ragged_and_garbage_past_the_length(env, dtype):
    """Lengths of 0, 1, a chunk's edge and beyond T; NaN and infinities past them reach nothing."""
    torch, prnn = env
    dt = types(torch)[dtype][0]
    lens = [0, 1, 64, 128, 129, 150, 999, -5]
    x = make(torch, 150, 8, 2, 2, 64, 64, dt, 700, state=True, lens=lens)
    o, end = check_forward(env, x, dtype, "ragged")
    check_backward(env, x, dtype, "ragged", 710, dstate=True)
    y = dict(x)
    do = normal(torch, x["v"].shape, dt, 720)
    g = prnn.linear_attention_backward(do, x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"], x["lens"])
    for n, junk in (("q", float("nan")), ("k", float("inf")), ("v", float("nan"))):
        z = x[n].clone()
        for b, m in enumerate(lens):
            z[max(0, min(150, m)):, b] = junk
        y[n] = z
    for b, m in enumerate(lens):
        do[max(0, min(150, m)):, b] = float("nan")
    o2, end2 = prnn.linear_attention(y["q"], y["k"], y["v"], y["ld"], y["scale"], y["state"], y["lens"])
    assert torch.equal(o2, o) and torch.equal(end2, end)
    for b, m in enumerate(lens):
        assert bool((o2[max(0, min(150, m)):, b] == 0).all())
    assert torch.equal(end2[0], x["state"][0]) and torch.equal(end2[7], x["state"][7])
    g2 = prnn.linear_attention_backward(do, y["q"], y["k"], y["v"], y["ld"], y["scale"], y["state"], y["lens"])
    for n in g:
        assert torch.equal(g2[n], g[n]), n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_linear_attention_extreme_decays(env, dtype):
    """No forgetting, a half-life under a token, a decay that underflows within a chunk, and 0."""
    torch, _ = env
    dt = types(torch)[dtype][0]
    x = make(torch, 260, 1, 4, 4, 64, 64, dt, 800, state=True, decay=[0.0, -0.9, -60.0, float("-inf")])
    check_forward(env, x, dtype, "decays")
    check_backward(env, x, dtype, "decays", 810, dstate=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linear_attention_ranges(env, dtype):
    """Products and states far outside fp16's range, and gradients near its smallest normals, keep
    their accuracy: what is held between the products must not be the data's own type unscaled."""
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x = make(torch, 200, 1, 2, 2, 64, 64, dt, 900, state=True, decay=[-0.001, -0.1])
    x["q"], x["k"] = x["q"] * 100, x["k"] * 800
    x["state"] = x["state"] * 1e6
    x["scale"] = 1e-5
    check_forward(env, x, dtype, "large")
    x = make(torch, 200, 1, 2, 2, 64, 64, dt, 910, decay=[-0.001, -0.1])
    x["v"] = x["v"] * 2.0 ** -12
    x["k"] = x["k"] * 2.0 ** -6
    x["scale"] = 2.0 ** 14
    check_forward(env, x, dtype, "small")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_attention_strides(env, dtype):
    """Slices of a joint projection, batch-major and head-major layouts give the packed result, and
    write no element that is not theirs."""
    torch, prnn = env
    dt = types(torch)[dtype][0]
    T, B, H, D = 135, 2, 2, 64
    x = make(torch, T, B, H, H, D, D, dt, 1000)
    call = lambda q, k, v, **kw: prnn.linear_attention(q, k, v, x["ld"], x["scale"], **kw)
    o, end = call(x["q"], x["k"], x["v"])
    joint = torch.full((T, B, 4, H, D), 3.0, dtype=dt, device="cuda")
    joint[:, :, 0], joint[:, :, 1], joint[:, :, 2] = x["q"], x["k"], x["v"]
    o2, end2 = call(joint[:, :, 0], joint[:, :, 1], joint[:, :, 2], o=joint[:, :, 3])
    assert torch.equal(o2, o) and torch.equal(end2, end) and torch.equal(joint[:, :, 0], x["q"])
    major = {n: x[n].permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3) for n in ("q", "k", "v")}
    o3, _ = call(**major, o=torch.empty(B, T, H, D, dtype=dt, device="cuda").transpose(0, 1))
    assert torch.equal(o3, o)
    odd = torch.full((T, B, H, D + 1), 3.0, dtype=dt, device="cuda")
    odd[..., 1:] = x["q"]
    out = torch.full((T, B, H, D + 3), 5.0, dtype=dt, device="cuda")
    o4, end4 = call(odd[..., 1:], x["k"], x["v"], o=out[..., 1:D + 1])
    # another access width may run another kernel: the two differ by rounding at most
    within(o4, o.double(), 4 * types(torch)[dtype][1] * o.double().abs() + 1e-3 * float(o.abs().max()), "odd")
    assert bool((out[..., 0] == 5).all()) and bool((out[..., D + 1:] == 5).all())
    shared = x["q"][:1].expand(T, B, H, D)                       # stride 0 over time
    o5, _ = call(shared, x["k"], x["v"])
    assert torch.equal(o5, call(shared.contiguous(), x["k"], x["v"])[0])
    with pytest.raises(prnn.PrnnError):
        call(x["q"], x["k"], x["v"], o=x["v"])
    with pytest.raises(ValueError):
        call(x["q"].transpose(2, 3), x["k"], x["v"])
    with pytest.raises(ValueError):
        call(x["q"], x["k"].double(), x["v"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_attention_continues_and_repeats(env, dtype):
    """Equal calls give equal bits; a sequence cut in two, the state carried, agrees with the
    whole; few sequences (time split over blocks) agree with many."""
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x = make(torch, 1000, 2, 2, 2, 64, 64, dt, 1100, state=True)
    args = (x["ld"], x["scale"])
    o, end = prnn.linear_attention(x["q"], x["k"], x["v"], *args, x["state"])
    again = prnn.linear_attention(x["q"], x["k"], x["v"], *args, x["state"])
    assert torch.equal(o, again[0]) and torch.equal(end, again[1])
    cut = 333
    o1, s1 = prnn.linear_attention(x["q"][:cut], x["k"][:cut], x["v"][:cut], *args, x["state"])
    o2, s2 = prnn.linear_attention(x["q"][cut:], x["k"][cut:], x["v"][cut:], *args, s1)
    M, Mend = attention_reference(torch, **absolute(x))
    tol, tol32 = attention_tolerance(dtype, 1000, 64)
    within(torch.cat([o1, o2]), o.double(), 2 * u * o.double().abs() + 2 * tol * M, "cut")
    within(s2, end.double(), 2 * tol32 * Mend, "cut state")
    do = normal(torch, x["v"].shape, dt, 1110)
    a = prnn.linear_attention_backward(do, x["q"], x["k"], x["v"], *args, x["state"])
    b = prnn.linear_attention_backward(do, x["q"], x["k"], x["v"], *args, x["state"])
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_linear_attention_gradient_against_differences(env):
    """The output is linear in each of q, k, v and the state, so central differences of the fp32
    kernel's forward are exact but for rounding: 2^-24 n of the sum over absolute values."""
    torch, prnn = env
    x = make(torch, 70, 2, 4, 2, 24, 40, torch.float32, 1200, state=True, lens=[70, 37])
    do = normal(torch, x["v"].shape, torch.float32, 1210)
    ds = normal(torch, x["state"].shape, torch.float32, 1211)
    g = prnn.linear_attention_backward(do, x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"], x["lens"], ds)

    def loss(y):
        o, end = prnn.linear_attention(y["q"], y["k"], y["v"], y["ld"], y["scale"], y["state"], y["lens"])
        return float((o.double() * do.double()).sum() + (end.double() * ds.double()).sum())
    for n, grad in (("q", g["dq"]), ("k", g["dk"]), ("v", g["dv"]), ("state", g["dstate"])):
        d = normal(torch, x[n].shape, torch.float32, 1220)
        hi, lo = dict(x), dict(x)
        hi[n], lo[n] = x[n] + 0.5 * d, x[n] - 0.5 * d
        slope = loss(hi) - loss(lo)
        want = float((grad.double() * d.double()).sum())
        scale = float((grad.double() * d.double()).abs().sum())
        assert abs(slope - want) <= 1e-4 * scale, (n, slope, want, scale)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", [(1, 1, 1, 1, 1), (1, 8, 8, 64, 64), (3, 4, 2, 72, 100), (2, 3, 1, 33, 7),
                                   (5, 2, 2, 128, 128), (2, 1, 1, 256, 256), (40, 16, 8, 128, 64)], ids=str)
def test_linear_attention_step(env, sizes, dtype):
    torch, prnn = env
    dt, u = types(torch)[dtype]
    B, H, Hq, dk, dv = sizes
    x = make(torch, 1, B, H, Hq, dk, dv, dt, 1300, state=True)
    want, wend = attention_reference(torch, **x)
    M, Mend = attention_reference(torch, **absolute(x))
    state = x["state"].clone()
    o = prnn.linear_attention_step(x["q"][0], x["k"][0], x["v"][0], x["ld"], state, x["scale"])
    within(o, want[0], rounding(want[0], u) + (dk + 64) * U * M[0] + 1e-38, "o")
    within(state, wend, 8 * U * Mend, "state")
    # the same through a pool, with padding rows
    n = 2 * B + 1
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(5))[:B].to(torch.int32).cuda()
    pool = torch.full((n, H, dk, dv), 9.0, device="cuda")
    pool[slots.long()] = x["state"]
    live = torch.ones(B, dtype=torch.bool, device="cuda")
    if B > 2:
        pool[slots[1].long()], pool[slots[2].long()] = 9.0, 9.0
        slots[1], slots[2] = -1, n
        live[1:3] = False
    o2 = prnn.linear_attention_step(x["q"][0], x["k"][0], x["v"][0], x["ld"], pool, x["scale"], slots)
    assert torch.equal(o2[live], o[live]) and bool((o2[~live] == 0).all())
    assert torch.equal(pool[slots[live].long()], state[live])
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[slots[live].long()] = False
    assert bool((pool[rest] == 9).all())


def test_linear_attention_steps_follow_the_sequence(env):
    """Decoding token by token from a prompt's state gives the whole sequence's outputs."""
    torch, prnn = env
    x = make(torch, 40, 2, 2, 2, 64, 64, torch.float32, 1400)
    o, end = prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"])
    M, Mend = attention_reference(torch, **absolute(x))
    _, state = prnn.linear_attention(x["q"][:20], x["k"][:20], x["v"][:20], x["ld"], x["scale"])
    for t in range(20, 40):
        y = prnn.linear_attention_step(x["q"][t], x["k"][t], x["v"][t], x["ld"], state, x["scale"])
        within(y, o[t].double(), 2 * (64 + 40 + 64) * U * M[t], t)
    within(state, end.double(), 2 * (64 + 40 + 64) * U * Mend, "state")


# ---- all --------------------------------------------------------------------------
def test_empty_calls(env):
    torch, prnn = env
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = prnn.layer_norm(x)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dg, db = prnn.layer_norm_backward(x, x, None, mean, rstd)
    assert dx.shape == (0, 64) and bool((dg == 0).all()) and bool((db == 0).all())
    assert prnn.dropout(x, 0.5, 1).shape == (0, 64)
    ld = torch.zeros(2, device="cuda")
    s = normal(torch, (3, 2, 8, 8), torch.float32, 1)
    e = torch.empty(0, 3, 2, 8, device="cuda")
    o, end = prnn.linear_attention(e, e, e, ld, 1.0, s)
    assert o.shape == e.shape and torch.equal(end, s)
    assert bool((prnn.linear_attention(e, e, e, ld)[1] == 0).all())
    g = prnn.linear_attention_backward(e, e, e, e, ld, 1.0, s, None, s)
    assert torch.equal(g["dstate"], s)
    z = torch.empty(5, 0, 2, 8, device="cuda")
    assert prnn.linear_attention(z, z, z, ld)[0].shape == z.shape
    assert prnn.linear_attention_step(z[0], z[0], z[0], ld, torch.empty(0, 2, 8, 8, device="cuda")).shape == (0, 2, 8)


def test_another_stream(env):
    """Calls on a stream of their own, ordered by events, with memory reused meanwhile."""
    torch, prnn = env
    side = torch.cuda.Stream()
    x = make(torch, 500, 2, 4, 2, 64, 64, torch.bfloat16, 1500)
    do = normal(torch, x["v"].shape, torch.bfloat16, 1510)
    flat = x["v"].reshape(1000, 256)
    want = (prnn.linear_attention_backward(do, x["q"], x["k"], x["v"], x["ld"], x["scale"]),
            prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"]), prnn.layer_norm(flat),
            prnn.dropout(flat, 0.2, 3, 4))
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        got = (prnn.linear_attention_backward(do, x["q"], x["k"], x["v"], x["ld"], x["scale"], stream=side),
               prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"], stream=side),
               prnn.layer_norm(flat, stream=side), prnn.dropout(flat, 0.2, 3, 4, stream=side))
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]   # on the main stream
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(got[0][n], want[0][n]) for n in want[0])
        assert all(torch.equal(a, b) for a, b in zip(got[1] + got[2], want[1] + want[2]))
        assert torch.equal(got[3], want[3])
        del junk


def test_captured_in_a_graph(env):
    """Every call can be captured: no allocation of its own, no synchronisation."""
    torch, prnn = env
    x = make(torch, 300, 2, 2, 2, 64, 64, torch.bfloat16, 1600)
    flat = x["v"].reshape(600, 128)
    state = torch.zeros(2, 2, 64, 64, device="cuda")

    def run():
        y, m, r = prnn.layer_norm(flat)
        o, end = prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"])
        g = prnn.linear_attention_backward(o, x["q"], x["k"], x["v"], x["ld"], x["scale"])
        s = prnn.linear_attention_step(x["q"][0], x["k"][0], x["v"][0], x["ld"], state, x["scale"])
        return [y, *prnn.layer_norm_backward(flat, flat, None, m, r), prnn.dropout(flat, 0.1, 1, 2), o, end,
                g["dq"], g["dk"], g["dv"], s]
    want = run()
    state.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    state.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_attention_state_in_place(env, dtype):
    """state_out may be `state` itself: with few sequences and a long prompt, where time would
    otherwise be cut over blocks, the result is that of separate arrays."""
    torch, prnn = env
    dt = types(torch)[dtype][0]
    x = make(torch, 2000, 1, 2, 2, 64, 64, dt, 1700, state=True)
    o, end = prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"])
    place, o2 = x["state"].clone(), torch.empty_like(o)
    a = prnn.prnn_linear_attention_t(dtype={"f32": 0, "bf16": 2}[dtype], T=2000, B=1, heads=2, qk_heads=2,
                                     dk=64, dv=64, scale=x["scale"], log_decay=x["ld"].data_ptr(),
                                     state=place.data_ptr(), state_out=place.data_ptr())
    for n, t in (("q", x["q"]), ("k", x["k"]), ("v", x["v"]), ("o", o2)):
        setattr(a, n, prnn.prnn_seq_t(t.data_ptr(), *t.stride()[:3]))
    ws = torch.empty(prnn.prnn_linear_attention_workspace(bytes(a), False), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    prnn.prnn_linear_attention_forward(bytes(a))
    M, Mend = attention_reference(torch, **absolute(x))
    tol, tol32 = attention_tolerance(dtype, 2000, 64)
    u = types(torch)[dtype][1]
    within(o2, o.double(), 2 * u * o.double().abs() + 2 * tol * M, "o")
    within(place, end.double(), 2 * tol32 * Mend, "state")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_linear_attention_all_sequences_empty(env, dtype):
    torch, prnn = env
    dt = types(torch)[dtype][0]
    x = make(torch, 300, 3, 2, 1, 64, 40, dt, 1800, state=True, lens=[0, 0, -3])
    for n in ("q", "k", "v"):
        x[n].fill_(float("nan"))
    o, end = prnn.linear_attention(x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"], x["lens"])
    assert bool((o == 0).all()) and torch.equal(end, x["state"])
    g = prnn.linear_attention_backward(x["v"], x["q"], x["k"], x["v"], x["ld"], x["scale"], x["state"],
                                       x["lens"], x["state"])
    assert all(bool((g[n] == 0).all()) for n in ("dq", "dk", "dv")) and torch.equal(g["dstate"], x["state"])


def test_no_wait_has_run_out(env):
    """Every call of this file is behind it: none of the kernels' bounded waits gave up."""
    torch, prnn = env
    assert prnn.prnn_sequence_status() == prnn.PRNN_OK
