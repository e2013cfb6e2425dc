"""GPU tests of the gated delta rule (whole sequences, gradients, single tokens) against its definition in 64 bits.

Tolerances.  With keys of length one and beta in 0 .. 2 a step shrinks whatever error the state brings along, so
after T tokens it holds T independent roundings of sums of about dk terms: a standard deviation of at most 8 U
sqrt(T + 16) of the column's largest norm, U = 2^-24; E takes eight of them.  On 16-bit data, values computed in
between may enter products as sums of two or three 16-bit parts, 2^-16 each: E adds 2^-14.  A value is then
off by E times the norms of what it is a product of: an output by E scale |q| S, S the column's largest norm; a
gradient of a value by E |k| R; those that sum over columns by E times the sum of S |do| or of 5 S R;
dlog_decay adds the parts of up to 128 tokens, 16 times that in the mean.  Each output's own rounding u
comes on top.  Over a whole tensor the errors average out: relative to its 2-norm at most u / sqrt(3) times 1.25 and
64 U (fp32) or 2^-15 (16-bit data).
"""
import math

import pytest

from tests.delta_exact import exact

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    from persistent_rnn_recurrence_gb300 import prnn
    return torch, prnn


@pytest.fixture(autouse=True)
def no_wait_ran_out(env):
    yield
    assert env[1].prnn_sequence_status() == env[1].PRNN_OK


def typed(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def normal(torch, shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def problem(torch, dtype, T, B, H, Hq, dk, dv, lens=None, state=False, seed=0, rate=0.05):
    dt, f32 = typed(torch, dtype), torch.float32
    p = {"scale": dk ** -0.5}
    for i, n in enumerate(("q", "k")):
        x = normal(torch, (T, B, Hq, dk), f32, 100 * seed + i)
        p[n] = (x / x.norm(dim=-1, keepdim=True)).to(dt)
    p["v"] = normal(torch, (T, B, H, dv), dt, 100 * seed + 2)
    p["g"] = -rate * torch.nn.functional.softplus(normal(torch, (T, B, H), f32, 100 * seed + 3, 2.0))
    p["beta"] = torch.sigmoid(normal(torch, (T, B, H), f32, 100 * seed + 4, 2.0))
    p["do"] = normal(torch, (T, B, H, dv), dt, 100 * seed + 5)
    p["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    p["state"] = normal(torch, (B, H, dk, dv), f32, 100 * seed + 6, 0.3) if state else None
    p["dstate"] = normal(torch, (B, H, dk, dv), f32, 100 * seed + 7, 0.3) if state else None
    return p


def within(got, want, bound, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(off.max()), float((off / bound.clamp(min=1e-300)).max()))


def close(got, want, dtype, out_type, what, terms=None):
    """The whole tensor, relative to its 2-norm, and to that of the terms it is a sum of where those are given."""
    n = float(want.double().norm()) + (0.0 if terms is None else float(terms.norm()))
    off = float((got.double() - want.double()).norm())
    assert off <= n * (1.25 * HALF[out_type] / math.sqrt(3) + (64 * U if dtype == "f32" else 2.0 ** -15)) + 1e-30, \
        (what, off / max(n, 1e-300))


def error(T, dtype):
    return 64 * math.sqrt(T + 16) * U + (0.0 if dtype == "f32" else 2.0 ** -14)


def rounding(want, dtype):
    return (HALF[dtype] * want.abs()).clamp(min=LEAST[dtype])


def check_forward(torch, prnn, dtype, p, x=None):
    T, share = p["v"].shape[0], p["v"].shape[2] // p["q"].shape[2]
    x = x or exact(torch, p["q"], p["k"], p["v"], p["g"], p["beta"], p["scale"], p["state"], p["lens"])
    o, end = prnn.gated_delta_rule(p["q"], p["k"], p["v"], p["g"], p["beta"], p["scale"], p["state"], p["lens"])
    E = error(T, dtype)
    within(o, x["o"], rounding(x["o"], dtype) + E * p["scale"] * x["q"].norm(dim=-1, keepdim=True) * x["S"], "o")
    within(end, x["state"], E * x["S"][:, :, None, :].expand(x["state"].shape), "state")
    if T:
        assert bool((o[~x["live"].expand(o.shape)] == 0).all())
        close(o, x["o"], dtype, dtype, "o")
    close(end, x["state"], "f32", "f32", "state")
    return o, end


def check_backward(torch, prnn, dtype, p):
    T, B, H, dv = p["v"].shape
    Hq = p["q"].shape[2]
    x = exact(torch, p["q"], p["k"], p["v"], p["g"], p["beta"], p["scale"], p["state"], p["lens"], p["do"], p["dstate"])
    r = prnn.gated_delta_rule_backward(p["do"], p["q"], p["k"], p["v"], p["g"], p["beta"], p["scale"], p["state"],
                                       p["lens"], p["dstate"])
    assert ("dstate" in r) == (p["state"] is not None)
    E, S, R = error(T, dtype), x["S"], x["R"] + (x["do"].abs().amax(0) if T else 0)
    both = (S * R).sum(-1)                                              # [B, H]

    def shared(z):
        return z.reshape(T, B, Hq, H // Hq).sum(3)[..., None]
    kn = x["k"].norm(dim=-1, keepdim=True)
    within(r["dv"], x["dv"], rounding(x["dv"], dtype) + E * x["beta"][..., None] * kn * R, "dv")
    within(r["dq"], x["dq"], rounding(x["dq"], dtype) + E * shared((S * x["do"].abs()).sum(-1)), "dq")
    within(r["dk"], x["dk"], rounding(x["dk"], dtype) + E * shared(5 * both.expand(T, B, H)), "dk")
    within(r["dbeta"], x["dbeta"], 2 * E * both.expand(T, B, H) + 1e-37, "dbeta")
    within(r["dlog_decay"], x["dlog_decay"], 16 * 2 * E * both.expand(T, B, H) + 1e-37, "dlog_decay")
    if p["state"] is not None:
        within(r["dstate"], x["dstate"], E * R[:, :, None, :].expand(x["dstate"].shape), "dstate")
        close(r["dstate"], x["dstate"], "f32", "f32", "dstate")
    for n, t in (("dq", dtype), ("dk", dtype), ("dv", dtype), ("dlog_decay", "f32"), ("dbeta", "f32")):
        # dlog_decay is a sum over later tokens of o . do - v . dv, each rounded relative to itself: where they cancel
        # (to 0 at the first token of zeros as a state) the result's own norm says nothing of their roundings
        terms = (x["o"] * p["do"].double()).sum(-1).abs() + (p["v"].double() * x["dv"]).sum(-1).abs()
        close(r[n], x[n], dtype, t, n, torch.where(x["live"][..., 0], terms, 0.0) if n == "dlog_decay" else None)
        dead = ~(x["live"] if r[n].ndim == 4 else x["live"][..., 0]).expand(r[n].shape)
        assert bool((r[n][dead] == 0).all()), n
    return r


# (T, B, heads, qk_heads, dk, dv, lens, state)
CASES = [(1, 1, 1, 1, 1, 1, None, False), (3, 2, 2, 1, 5, 7, None, True), (16, 1, 3, 3, 16, 24, None, False),
         (17, 2, 2, 2, 64, 64, None, True), (64, 1, 4, 4, 64, 64, None, False), (100, 3, 4, 2, 48, 80, [100, 0, 1], True),
         (127, 1, 2, 2, 128, 128, None, False), (128, 2, 2, 1, 128, 128, None, True),
         (129, 2, 2, 2, 128, 128, [129, 128], True), (255, 2, 3, 1, 72, 100, [7, 255], True),
         (256, 1, 2, 2, 65, 33, None, False), (300, 3, 2, 2, 96, 128, [300, 127, 257], False),
         (513, 1, 2, 1, 128, 64, None, True), (700, 2, 2, 2, 37, 128, [700, 513], True),
         (40, 2, 2, 1, 200, 256, [40, 33], True), (150, 1, 2, 2, 256, 130, None, True), (1000, 1, 1, 1, 128, 128, None, True)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(env, case, dtype):
    torch, prnn = env
    check_forward(torch, prnn, dtype, problem(torch, dtype, *case))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(env, case, dtype):
    torch, prnn = env
    check_backward(torch, prnn, dtype, problem(torch, dtype, *case))


# more heads than fit the SMs in narrow slices, in every type; ragged, and with heads that share
MANY = [(200, 10, 16, 16, 64, 64, None, True), (130, 20, 16, 8, 128, 100, [130] * 10 + [0, 1, 127, 128, 129] * 2, False),
        (32, 3, 64, 64, 40, 33, None, True)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: str(c[:6]))
def test_many_heads(env, case, dtype):
    torch, prnn = env
    p = problem(torch, dtype, *case, seed=2)
    check_forward(torch, prnn, dtype, p)
    check_backward(torch, prnn, dtype, p)


def gates(torch, p, kind):
    """Gates and keys where the recurrence can go wrong."""
    if kind == "no decay":
        p["g"].zero_()
    elif kind == "forgets all":
        p["g"][::7] = -float("inf")
    elif kind == "strong":
        p["g"].mul_(100)
    elif kind == "writes nothing":
        p["beta"].zero_()
    elif kind == "one key":                    # every token overwrites the one before
        p["k"][:] = p["k"][:1]
        p["beta"].fill_(1.0)
        p["g"].zero_()
    elif kind == "two keys in turn":
        p["k"][0::2], p["k"][1::2] = p["k"][:1], p["k"][1:2]
        p["beta"].fill_(0.9)
    elif kind == "reflects":                   # beta = 2: what is held for a key changes sign
        p["beta"].fill_(2.0)
        p["g"].zero_()
    return p


KINDS = ["no decay", "forgets all", "strong", "writes nothing", "one key", "two keys in turn", "reflects"]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_gates(env, kind, dtype):
    torch, prnn = env
    p = gates(torch, problem(torch, dtype, 290, 2, 2, 1, 64, 64, [290, 150], True, seed=3), kind)
    if kind in ("one key", "two keys in turn", "reflects"):
        # lengths of one in the data's type, within its rounding: (1 + u)^2 a token would pass the bound over 290
        p["k"] = (p["k"].float() * (1 - 2.0 ** -7)).to(p["k"].dtype)
    check_forward(torch, prnn, dtype, p)
    check_backward(torch, prnn, dtype, p)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_against_differences(env, dtype):
    """Central differences of the forward pass of fp32 data along random directions, for every input: the cubic term
    is about h^2 = 2^-14 of the slope and rounding 2^-24 |L| / h, both below 2e-3 of the slope's scale."""
    torch, prnn = env
    p = problem(torch, "f32", 150, 2, 4, 2, 40, 48, [150, 70], True, seed=5, rate=0.2)
    weight = p["dstate"]

    def loss(**kw):
        x = {**p, **kw}
        o, end = prnn.gated_delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["scale"], x["state"], x["lens"])
        return float((o.double() * p["do"].double()).sum() + (end.double() * weight.double()).sum())
    r = prnn.gated_delta_rule_backward(p["do"], p["q"], p["k"], p["v"], p["g"], p["beta"], p["scale"], p["state"],
                                       p["lens"], weight)
    h = 2.0 ** -7
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("beta", "dbeta"), ("state", "dstate")):
        way = normal(torch, p[n].shape, torch.float32, 77)
        way = way / way.abs().max()
        got = (loss(**{n: p[n] + h * way}) - loss(**{n: p[n] - h * way})) / (2 * h)
        want = float((r[d].double() * way.double()).sum())
        scale = float(r[d].double().norm() * way.double().norm()) / math.sqrt(way.numel())
        assert abs(got - want) <= 4e-3 * scale + 2e-2, (n, got, want, scale)


def joint(torch, p):
    """q, k, v as slices of one projection, gates as slices of another, at offsets that no vector width fits."""
    T, B, H, dv = p["v"].shape
    Hq, dk = p["q"].shape[2:]
    wide = torch.full((T, B, Hq * 2 * dk + H * dv + 3), float("nan"), dtype=p["v"].dtype, device="cuda")
    parts, at = {}, 1
    for n, heads, d in (("q", Hq, dk), ("k", Hq, dk), ("v", H, dv)):
        x = wide[..., at:at + heads * d].view(T, B, heads, d)
        x.copy_(p[n])
        parts[n] = x
        at += heads * d
    two = torch.full((T, B, 2 * H + 1), float("nan"), device="cuda")
    two[..., :H], two[..., H + 1:] = p["g"], p["beta"]
    return {**p, **parts, "g": two[..., :H], "beta": two[..., H + 1:]}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strides(env, dtype):
    """Slices of joint projections, batch-major tensors, gates shared by stride 0: the same values as packed."""
    torch, prnn = env
    p = problem(torch, dtype, 140, 2, 4, 2, 64, 72, [140, 139], True, seed=7)
    args = ("q", "k", "v", "g", "beta", "scale", "state", "lens")
    want = prnn.gated_delta_rule(*(p[n] for n in args))
    grads = prnn.gated_delta_rule_backward(p["do"], *(p[n] for n in args), p["dstate"])
    major = {**p, **{n: p[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v", "g", "beta", "do")}}
    for x in (joint(torch, p), major):
        o, end = prnn.gated_delta_rule(*(x[n] for n in args))
        assert torch.equal(o, want[0]) and torch.equal(end, want[1])
        got = prnn.gated_delta_rule_backward(x["do"], *(x[n] for n in args), x["dstate"])
        for n in grads:
            assert torch.equal(got[n], grads[n]), n
    out = torch.full((140, 2, 4, 80), 7.0, dtype=p["v"].dtype, device="cuda")
    o, _ = prnn.gated_delta_rule(*(p[n] for n in args), o=out[..., 3:75])
    assert torch.equal(out[..., 3:75], want[0]) and bool((out[..., :3] == 7).all()) and bool((out[..., 75:] == 7).all())
    same = {**p, "beta": p["beta"][:1, :1].expand(140, 2, 4), "g": p["g"][:1].expand(140, 2, 4)}
    check_forward(torch, prnn, dtype, same)
    check_backward(torch, prnn, dtype, same)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_what_lies_past_the_length(env, dtype):
    """NaN behind each length, in every input, changes nothing; and outputs there are zeros."""
    torch, prnn = env
    p = problem(torch, dtype, 200, 3, 2, 2, 64, 64, [200, 130, 0], True, seed=8)
    args = ("q", "k", "v", "g", "beta", "scale", "state", "lens")
    want, grads = prnn.gated_delta_rule(*(p[n] for n in args)), \
        prnn.gated_delta_rule_backward(p["do"], *(p[n] for n in args), p["dstate"])
    for n in ("q", "k", "v", "g", "beta", "do"):
        p[n][130:, 1] = float("nan")
        p[n][:, 2] = float("nan")
    o, end = prnn.gated_delta_rule(*(p[n] for n in args))
    assert torch.equal(o, want[0]) and torch.equal(end, want[1]) and torch.equal(end[2], p["state"][2])
    got = prnn.gated_delta_rule_backward(p["do"], *(p[n] for n in args), p["dstate"])
    for n in grads:
        assert torch.equal(got[n], grads[n]), n
    assert torch.equal(got["dstate"][2], p["dstate"][2])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_an_infinity_or_nan_stays_in_its_sequence_and_head(env, dtype):
    torch, prnn = env
    for n in ("q", "k", "v", "g", "beta", "do"):
        p = problem(torch, dtype, 200, 2, 2, 2, 64, 64, None, True, seed=9)
        args = ("q", "k", "v", "g", "beta", "scale", "state", "lens")
        want, grads = prnn.gated_delta_rule(*(p[m] for m in args)), \
            prnn.gated_delta_rule_backward(p["do"], *(p[m] for m in args), p["dstate"])
        for bad in (float("nan"), float("inf")):
            x = {**p, n: p[n].clone()}
            x[n][150, 1, 1] = bad
            o, end = prnn.gated_delta_rule(*(x[m] for m in args))
            for a, b in ((o, want[0]), (end[None], want[1][None])):
                assert torch.equal(a[:, 0], b[:, 0]) and torch.equal(a[:, 1, 0], b[:, 1, 0]), n
            if n in ("k", "v", "g", "beta"):
                assert not bool(end[1, 1].isfinite().all()) and not bool(o[150:, 1, 1].isfinite().all()), n
                assert torch.equal(o[:150 - 127, 1, 1], want[0][:150 - 127, 1, 1]), n
            got = prnn.gated_delta_rule_backward(x["do"], *(x[m] for m in args), x["dstate"])
            for m in grads:
                a, b = (got[m][None], grads[m][None]) if m == "dstate" else (got[m], grads[m])
                assert torch.equal(a[:, 0], b[:, 0]) and torch.equal(a[:, 1, 0], b[:, 1, 0]), (n, m)


def test_states_pass_on(env):
    """A sequence in two calls, the state in place; and no tokens at all."""
    torch, prnn = env
    for dtype in ("f32", "bf16"):
        p = problem(torch, dtype, 256, 2, 2, 1, 64, 64, None, True, seed=10)
        args = ("q", "k", "v", "g", "beta")
        whole = prnn.gated_delta_rule(*(p[n] for n in args), p["scale"], p["state"])
        first, mid = prnn.gated_delta_rule(*(p[n][:128] for n in args), p["scale"], p["state"])
        second, end = prnn.gated_delta_rule(*(p[n][128:] for n in args), p["scale"], mid)
        assert torch.equal(torch.cat([first, second]), whole[0]) and torch.equal(end, whole[1])
        o, end = prnn.gated_delta_rule(*(p[n][:0] for n in args), p["scale"], p["state"])
        assert o.shape[0] == 0 and torch.equal(end, p["state"])
        g = prnn.gated_delta_rule_backward(p["do"][:0], *(p[n][:0] for n in args), p["scale"], p["state"], None,
                                           p["dstate"])
        assert torch.equal(g["dstate"], p["dstate"])
        o, end = prnn.gated_delta_rule(*(p[n][:, :0] for n in args), p["scale"])
        assert o.shape == (256, 0, 2, 64) and end.shape == (0, 2, 64, 64)


STEPS = [(1, 1, 1, 1, 1), (3, 2, 1, 5, 7), (2, 8, 8, 64, 64), (5, 4, 2, 72, 100), (96, 16, 8, 128, 128),
         (4, 3, 3, 128, 33), (2, 2, 1, 200, 256), (7, 2, 2, 256, 130), (40, 4, 4, 65, 64)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", STEPS, ids=str)
def test_step(env, case, dtype):
    """Three tokens one by one through a pool of slots with a padding row; what is not named keeps its bits."""
    torch, prnn = env
    B, H, Hq, dk, dv = case
    p = problem(torch, dtype, 3, B, H, Hq, dk, dv, None, True, seed=11)
    pool = normal(torch, (B + 3, H, dk, dv), torch.float32, 12, 0.3)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32).cuda()
    dead = B // 2 if B > 1 else -1
    pool[slots.long()] = p["state"]
    before = pool.clone()
    if dead >= 0:
        slots[dead] = -1 if B % 2 else B + 3
    x = exact(torch, p["q"], p["k"], p["v"], p["g"], p["beta"], p["scale"], p["state"])
    E = error(3, "f32")
    for t in range(3):
        o = prnn.gated_delta_rule_step(p["q"][t], p["k"][t], p["v"][t], p["g"][t], p["beta"][t], pool, p["scale"], slots)
        for b in range(B):
            if b == dead:
                assert bool((o[b] == 0).all())
                continue
            want = x["o"][t, b]
            within(o[b], want, rounding(want, dtype) + E * p["scale"] * x["q"][t, b].norm(dim=-1, keepdim=True)
                   * (2 * x["S"][b]), "o")
    named = [int(s) for s in slots if 0 <= int(s) < B + 3]
    for b, s in enumerate(slots.tolist()):
        if 0 <= s < B + 3:
            within(pool[s], x["state"][b], E * x["S"][b][:, None, :].expand(H, dk, dv), "state")
    for s in range(B + 3):
        if s not in named:
            assert torch.equal(pool[s], before[s])
    if B <= 7:
        plain = p["state"].clone()
        o = prnn.gated_delta_rule_step(p["q"][0], p["k"][0], p["v"][0], p["g"][0], p["beta"][0], plain, p["scale"])
        within(o, x["o"][0], rounding(x["o"][0], dtype) + 2 * E * p["scale"] * x["S"], "o without slots")


def test_prompt_then_tokens(env):
    """As it is served: heads normalised, a prompt as a sequence, then token by token from its state; against the
    whole sequence at once."""
    torch, prnn = env
    for dtype in ("f32", "bf16"):
        p = problem(torch, dtype, 160, 2, 4, 2, 64, 64, None, False, seed=13)
        unit = torch.full((64,), 64 ** -0.5, device="cuda")
        for n in ("q", "k"):
            p[n] = prnn.rms_norm(normal(torch, p[n].shape, p[n].dtype, 14), unit)[0]
        x = exact(torch, p["q"], p["k"], p["v"], p["g"], p["beta"], p["scale"])
        args = ("q", "k", "v", "g", "beta")
        whole, _ = prnn.gated_delta_rule(*(p[n] for n in args), p["scale"])
        first, state = prnn.gated_delta_rule(*(p[n][:150] for n in args), p["scale"])
        rest = [prnn.gated_delta_rule_step(*(p[n][t] for n in args), state, p["scale"]) for t in range(150, 160)]
        E = error(160, dtype)
        bound = rounding(x["o"], dtype) + E * p["scale"] * x["q"].norm(dim=-1, keepdim=True) * x["S"]
        within(torch.cat([first, torch.stack(rest)]), x["o"], bound, "prompt and tokens")
        within(whole, x["o"], bound, "whole")
        within(state, x["state"], E * x["S"][:, :, None, :].expand(x["state"].shape), "state")


def test_equal_calls_and_graphs(env):
    """Equal calls give equal bits; captured calls replayed on new values, two graphs that share nothing."""
    torch, prnn = env
    for dtype in ("f32", "bf16"):
        p = problem(torch, dtype, 270, 2, 4, 2, 64, 64, None, True, seed=15)
        args = ("q", "k", "v", "g", "beta", "scale", "state")
        pool = p["state"].clone()

        def every():
            o, end = prnn.gated_delta_rule(*(p[n] for n in args))
            g = prnn.gated_delta_rule_backward(p["do"], *(p[n] for n in args), None, p["dstate"])
            s = prnn.gated_delta_rule_step(*(p[n][0] for n in args[:5]), pool, p["scale"])
            return o, end, s, *g.values()
        first = every()
        pool.copy_(p["state"])
        for a, b in zip(first, every()):
            assert torch.equal(a, b)
        graphs, outs = [], []
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append(every())
        p["v"].copy_(normal(torch, p["v"].shape, p["v"].dtype, 16))
        pool.copy_(p["state"])
        want = every()
        for g, out in zip(graphs, outs):
            pool.copy_(p["state"])
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_streams(env):
    """On a stream of their own, inputs dropped while the call waits."""
    torch, prnn = env
    p = problem(torch, "bf16", 270, 2, 4, 2, 64, 64, None, True, seed=17)
    args = ("q", "k", "v", "g", "beta", "scale", "state")
    want = prnn.gated_delta_rule(*(p[n] for n in args))
    grads = prnn.gated_delta_rule_backward(p["do"], *(p[n] for n in args), None, p["dstate"])
    side = torch.cuda.Stream()
    copies = {n: x.clone() if hasattr(x, "clone") else x for n, x in p.items()}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = prnn.gated_delta_rule(*(copies[n] for n in args), stream=side)
    back = prnn.gated_delta_rule_backward(copies["do"], *(copies[n] for n in args), None, copies["dstate"], stream=side)
    copies.clear()
    junk = [torch.full((270, 2, 4, 64), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(8)]
    torch.cuda.synchronize()
    del junk
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n in grads:
        assert torch.equal(back[n], grads[n]), n


def test_refusals(env):
    torch, prnn = env
    p = problem(torch, "bf16", 8, 2, 4, 2, 16, 16, None, True)
    args = ("q", "k", "v", "g", "beta", "scale", "state")

    def call(**kw):
        x = {**p, **kw}
        return prnn.gated_delta_rule(*(x[n] for n in args), x["lens"])
    for kw in (dict(k=p["k"][:4]), dict(k=p["k"].float()), dict(v=p["v"][0]), dict(g=p["g"][..., :2]),
               dict(beta=p["beta"].bfloat16()), dict(beta=p["beta"].cpu()), dict(state=p["state"][:1]),
               dict(state=p["state"].half()), dict(lens=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(lens=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(q=p["q"].transpose(2, 3))):
        with pytest.raises(ValueError):
            call(**kw)
    wide = torch.zeros(4, 1, 1, 257, device="cuda")
    gate = torch.zeros(4, 1, 1, device="cuda")
    with pytest.raises(Exception):
        prnn.gated_delta_rule(wide, wide, wide, gate, gate)
    with pytest.raises(Exception):            # three value heads, two query heads
        prnn.gated_delta_rule(p["q"], p["k"], p["v"][:, :, :3], p["g"][..., :3], p["beta"][..., :3])
    with pytest.raises(Exception):            # the output lies upon an input
        prnn.gated_delta_rule(p["v"][:, :, :2], p["k"], p["v"], p["g"], p["beta"], o=p["v"])
