"""The example block around the gated delta rule: its operators and a recurrent layer run, differentiated and decoded
together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_rnn_recurrence_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("delta_block", os.path.join(ROOT, "examples", "delta_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return torch, mod


def test_block_trains(example):
    """Steps run and every number stays finite."""
    torch, mod = example
    block, losses = mod.train(steps=4)
    assert len(losses) == 4 and all(x == x and x < 1e3 for x in losses)
    assert all(bool(t.isfinite().all()) for t in block.p.values())


def test_block_gradient_against_differences(example):
    """Directional derivatives of the whole block: central differences with step 2^-9; kinks of the ReLU and rounding
    leave about 1 %."""
    torch, mod = example

    def normal(shape, seed):
        return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    block = mod.Block(mod.parameters(3))
    x, dy = normal((mod.T, mod.B, mod.W), 4), normal((mod.T, mod.B, mod.W), 5)
    block.forward(x)
    g, dx = block.backward(dy)

    def loss(x=x):
        return float((block.forward(x)[0].double() * dy.double()).sum())
    h = 2.0 ** -9
    for n in ("Wq", "Wk", "Wv", "Wa", "Wb", "a0", "Wo", "g1", "g2", "Wh", "Wy"):
        d = normal(block.p[n].shape, 6)
        d = d / d.norm()
        block.p[n] += h * d
        up = loss()
        block.p[n] -= 2 * h * d
        down = loss()
        block.p[n] += h * d
        want = float((g[n].double() * d.double()).sum())
        assert abs((up - down) / (2 * h) - want) <= 0.03 * float(g[n].norm()), n
    d = normal(x.shape, 7)
    d = d / d.norm()
    got = (loss(x + h * d) - loss(x - h * d)) / (2 * h)
    assert abs(got - float((dx.double() * d.double()).sum())) <= 0.03 * float(dx.norm())


def test_block_decodes(example):
    """Token by token from a prompt's state equals the whole sequence: both are within 2e-6 of the largest entry of the
    definition (64 roundings of 2^-24 at most, see the operator's own tests), so within 1e-5 of each other."""
    torch, mod = example
    block = mod.Block(mod.parameters(7))
    x = torch.randn(mod.T, mod.B, mod.W, device="cuda")
    _, whole, state = block.forward(x)
    for prompt in (1, 17, mod.T - 1):
        steps, end = mod.decode(block, x, prompt)
        assert float((steps - whole).abs().max()) <= 1e-5 * float(whole.abs().max())
        assert float((end - state).abs().max()) <= 1e-5 * float(state.abs().max())
