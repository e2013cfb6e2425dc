"""The example block: the sequence operators and a recurrent layer trained and decoded together."""
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
    spec = importlib.util.spec_from_file_location(
        "recurrent_block", os.path.join(ROOT, "examples", "recurrent_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return torch, mod


def test_block_learns(example):
    """Answering with the input of three steps ago: the loss starts near the target's variance (1) and
    falls by a third at least."""
    _, mod = example
    _, losses = mod.train(steps=40)
    assert losses[-1] < 0.67 * losses[0], losses


def test_block_gradient_against_differences(example):
    """Directional derivatives of the whole block without dropout's randomness (same seed): central
    differences with step 2^-9; kinks of the ReLU and rounding leave about 1 %."""
    torch, mod = example
    block = mod.Block(mod.parameters(3))
    x = torch.randn(mod.T, mod.B, mod.W, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    dy = torch.randn(mod.T, mod.B, mod.W, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    block.forward(x, seed=9)
    g, _ = block.backward(dy)

    def loss():
        return float((block.forward(x, seed=9)[0].double() * dy.double()).sum())
    h = 2.0 ** -9
    for n in ("Wq", "Wv", "Wo", "g1", "b2", "Wh", "Wy"):
        d = torch.randn(block.p[n].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
        d = d / d.norm()
        block.p[n] += h * d
        up = loss()
        block.p[n] -= 2 * h * d
        down = loss()
        block.p[n] += h * d
        want = float((g[n].double() * d.double()).sum())
        assert abs((up - down) / (2 * h) - want) <= 0.03 * float(g[n].norm()), n


def test_block_decodes(example):
    """Token by token from a prompt's state equals the whole sequence within fp32 rounding."""
    torch, mod = example
    block = mod.Block(mod.parameters(7))
    x = torch.randn(mod.T, mod.B, mod.W, device="cuda")
    _, whole, state = block.forward(x, seed=0)
    for prompt in (1, 17, mod.T - 1):
        steps, end = mod.decode(block, x, prompt)
        scale = float(whole.abs().max())
        assert float((steps - whole).abs().max()) <= 1e-5 * scale
        assert float((end - state).abs().max()) <= 1e-5 * float(state.abs().max())
