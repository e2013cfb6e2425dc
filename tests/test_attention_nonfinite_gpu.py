"""Linear attention with an infinity or NaN in one value within the length.

Where the 64-bit reference of such a call is finite, the value cannot depend on the bad one: the result is that
of the call without it, within the bounds of every call, or, up to 127 tokens away in the same sequence, NaN.
Where the reference is not finite, neither is the result: no infinity turns into a number."""
import pytest

from tests.attention_exact import exact
from tests.test_sequence_ops_gpu import (absolute, attention_tolerance, env,  # noqa: F401
                                         make, normal, rounding, types, within)

pytestmark = pytest.mark.gpu


def compare(torch, got, clean, dirty, bound, near, what):
    """near: where a NaN may stand for a finite value (None: nowhere)."""
    finite = torch.isfinite(dirty)
    g = got.double()
    assert not bool(torch.isfinite(g[~finite]).any()), (what, "an infinity became a number",
                                                        int(torch.isfinite(g[~finite]).sum()), int((~finite).sum()))
    fine = (g - clean).abs() <= bound
    if near is not None:
        fine |= g.isnan() & near
    bad = finite & ~fine
    assert not bool(bad.any()), (what, int(bad.sum()), int(finite.sum()))


def reach(torch, shape, b, j):
    """Tokens of sequence b up to 127 from token j."""
    near = torch.zeros(shape, dtype=torch.bool, device="cuda")
    near[max(0, j - 127):j + 128, b] = True
    return near


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 1)])
@pytest.mark.parametrize("j", [20, 130])
@pytest.mark.parametrize("name", ["q", "k", "v", "state"])
def test_forward(env, name, j, d, Hq, dtype):  # noqa: F811
    torch, prnn = env
    dt, u = types(torch)[dtype]
    T, B, H = 300, 2, 2
    x = make(torch, T, B, H, Hq, d, d, dt, 2100, state=True)
    clean, cend = exact(torch, **x)
    M, Mend = exact(torch, **absolute(x))
    tol, tol32 = attention_tolerance(dtype, T, d)
    for bad in (float("inf"), float("-inf"), float("nan")):
        y = dict(x)
        y[name] = x[name].clone()
        if name == "state":
            y[name][1, 0, 5, 17] = bad
        else:
            y[name][j, 1, 0, 7] = bad
        dirty, dend = exact(torch, **y)
        o, end = prnn.linear_attention(y["q"], y["k"], y["v"], y["ld"], y["scale"], y["state"])
        near = None if name == "state" else reach(torch, o.shape, 1, j)
        compare(torch, o, clean, dirty, rounding(clean, u) + tol * M + 1e-38, near, (name, bad, "o"))
        compare(torch, end, cend, dend, tol32 * Mend, None, (name, bad, "state"))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 1)])
@pytest.mark.parametrize("j", [20, 130])
@pytest.mark.parametrize("name", ["q", "k", "v", "grad", "state", "dstate"])
def test_backward(env, name, j, d, Hq, dtype):  # noqa: F811
    torch, prnn = env
    dt, u = types(torch)[dtype]
    T, B, H = 300, 2, 2
    x = make(torch, T, B, H, Hq, d, d, dt, 2200, state=True)
    x["grad"] = normal(torch, x["v"].shape, dt, 2210)
    x["dstate"] = normal(torch, x["state"].shape, torch.float32, 2211)
    clean, M = exact(torch, **x), exact(torch, **absolute(x))
    tol, tol32 = attention_tolerance(dtype, T, d)
    for bad in (float("inf"), float("nan")):
        y = dict(x)
        y[name] = x[name].clone()
        if name in ("state", "dstate"):
            y[name][1, 0, 5, 17] = bad
        else:
            y[name][j, 1, 0, 7] = bad
        dirty = exact(torch, **y)
        g = prnn.linear_attention_backward(y["grad"], y["q"], y["k"], y["v"], y["ld"], y["scale"], y["state"], None,
                                           y["dstate"])
        for n in g:
            bound = tol32 * M[n] if n == "dstate" else rounding(clean[n], u) + tol * M[n] + 1e-38
            near = None if n == "dstate" or name in ("state", "dstate") else reach(torch, g[n].shape, 1, j)
            compare(torch, g[n], clean[n], dirty[n], bound, near, (name, bad, n))
