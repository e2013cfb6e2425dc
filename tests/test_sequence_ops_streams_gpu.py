"""Calls on a stream of their own whose inputs are let go at once: their memory must not be given to
the next allocation of the inputs' stream before the call has read it.

The side stream is held back by a wait of its own while the inputs are dropped and allocations of the same sizes
are made and overwritten on the main stream."""
import pytest

from tests.test_sequence_ops_gpu import env, make, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def held_back(torch, call, inputs):
    """call(stream, *clones of inputs), dropped and overwritten while the stream waits; its result.  Called twice:
    the first time loads kernels, which waits for the device."""
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()                         # nothing but the copies' memory is free to be given out
    copies = [None if t is None else t.clone() for t in inputs]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)               # about 0.1 s of clock ticks
    got = call(side, *copies)
    sizes = [t.untyped_storage().nbytes() for t in copies if t is not None]
    del copies
    junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    del junk
    return got


def flat(x):
    return [x[n] for n in sorted(x)] if isinstance(x, dict) else list(x) if isinstance(x, (list, tuple)) else [x]


CALLS = ["layer_norm", "layer_norm_backward", "dropout", "dropout_backward", "linear_attention",
         "linear_attention_backward", "linear_attention_step"]


@pytest.mark.parametrize("name", CALLS)
def test_inputs_let_go(env, name):  # noqa: F811
    torch, prnn = env
    x = normal(torch, (3000, 1024), torch.float32, 1)
    gamma, beta = normal(torch, (1024,), torch.float32, 2), normal(torch, (1024,), torch.float32, 3)
    _, mean, rstd = prnn.layer_norm(x, gamma, beta)
    a = make(torch, 300, 2, 2, 2, 64, 64, torch.bfloat16, 10, state=True, lens=[300, 211])
    do, ds = normal(torch, a["v"].shape, torch.bfloat16, 20), normal(torch, a["state"].shape, torch.float32, 21)
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    call, inputs = {
        "layer_norm": (lambda x, g, b, **s: prnn.layer_norm(x, g, b, **s), (x, gamma, beta)),
        "layer_norm_backward": (lambda d, x, g, m, r, **s: prnn.layer_norm_backward(d, x, g, m, r, **s),
                                (x * 0.5, x, gamma, mean, rstd)),
        "dropout": (lambda x, r, **s: prnn.dropout(x, 0.3, 5, 6, r, **s), (x, x * 2)),
        "dropout_backward": (lambda d, **s: prnn.dropout_backward(d, 0.3, 5, 6, **s), (x,)),
        "linear_attention": (lambda q, k, v, l, s0, n, **s: prnn.linear_attention(q, k, v, l, 0.5, s0, n, **s),
                             (a["q"], a["k"], a["v"], a["ld"], a["state"], a["lens"])),
        "linear_attention_backward": (
            lambda d, q, k, v, l, s0, n, e, **s: prnn.linear_attention_backward(d, q, k, v, l, 0.5, s0, n, e, **s),
            (do, a["q"], a["k"], a["v"], a["ld"], a["state"], a["lens"], ds)),
        "linear_attention_step": (lambda q, k, v, l, s0, sl, **s: prnn.linear_attention_step(q, k, v, l, s0, 0.5, sl, **s),
                                  (a["q"][0], a["k"][0], a["v"][0], a["ld"], a["state"], slots)),
    }[name]
    want = flat(call(*[t.clone() for t in inputs]))
    for _ in range(2):
        got = flat(held_back(torch, lambda side, *t: call(*t, stream=side), inputs))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_output_let_go(env):  # noqa: F811
    """An output given by the caller and dropped: what is allocated next on its stream is not written over."""
    torch, prnn = env
    x = normal(torch, (3000, 1024), torch.float32, 1)
    for _ in range(2):      # the first time loads kernels, which waits for the device
        side = torch.cuda.Stream()
        torch.cuda.empty_cache()
        y = torch.empty_like(x)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        prnn.dropout(x, 0.5, 1, 2, y=y, stream=side)
        del y
        others = [torch.full_like(x, 3.0) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((other == 3.0).all()) for other in others)
