"""Linear attention where one token's scores are 2^30 times the others': tokens that the mask keeps from seeing it, and
tokens that its decay has long made it nothing to, keep the accuracy that their own scores allow.

The bounds are those of every call (tests/test_sequence_ops_gpu.py): one rounding of the output and 2^-15 of the
sum over absolute values of what the token does see.  The 64-bit reference and that sum leave the large token out
of a token's result by causality, or weigh it with its decay (e^-4 a token: e^-48 of 2^30 after twelve)."""
import pytest

from tests.attention_exact import exact
from tests.test_sequence_ops_gpu import (absolute, attention_tolerance, env,  # noqa: F401
                                         make, normal, rounding, types, within)

pytestmark = pytest.mark.gpu
# the tensor with the large token, the result that must not feel it, whether time runs backwards in its sum
ROLES = [("k", "o", False), ("v", "dq", False), ("grad", "dk", True), ("q", "dv", True)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,d", [(40, 64), (150, 128)])
@pytest.mark.parametrize("large,result,back", ROLES)
@pytest.mark.parametrize("how", ["masked", "decayed"])
def test_one_large_token(env, how, large, result, back, T, d, dtype):  # noqa: F811
    torch, prnn = env
    dt, u = types(torch)[dtype]
    x = make(torch, T, 1, 2, 2, d, d, dt, 2000, decay=[-0.01, -0.03] if how == "masked" else [-4.0, -4.5])
    grad = normal(torch, x["v"].shape, dt, 2010)
    y = {**x, "grad": grad, "k": normal(torch, x["k"].shape, dt, 2011), "scale": 2.0 ** 10}
    at = {("masked", False): 25, ("masked", True): T - 26, ("decayed", False): 0, ("decayed", True): T - 1}[how, back]
    y[large] = (y[large].float() * 2.0 ** -17).to(dt)
    y[large][at] = normal(torch, y[large].shape[1:], dt, 2012, 2.0 ** 13)
    t = torch.arange(T, device="cuda")
    far = (at - t if back else t - at)              # > 0: this token sees the large one
    keep = far < 0 if how == "masked" else far >= 12
    grad = y.pop("grad")
    if result == "o":
        got = prnn.linear_attention(y["q"], y["k"], y["v"], y["ld"], y["scale"])[0]
        want, M = exact(torch, **y)[0], exact(torch, **absolute(y))[0]
    else:
        got = prnn.linear_attention_backward(grad, y["q"], y["k"], y["v"], y["ld"], y["scale"])[result]
        want = exact(torch, **y, grad=grad)[result]
        M = exact(torch, **absolute(y, grad=grad))[result]
    tol, _ = attention_tolerance(dtype, T, d)
    within(got[keep], want[keep], rounding(want[keep], u) + tol * M[keep] + 1e-38, (how, result))
