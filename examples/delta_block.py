"""A residual block around the gated delta rule, trained and then decoded token by token.

    python examples/delta_block.py [--steps 60]

The block reads a sequence x [T, B, W]:

    n = rms_norm(x);  q, k, v = n Wq, n Wk, n Wv, the heads of q and k of length one (rms_norm once more)
    log_decay = -softplus(n Wa),  beta = sigmoid(n Wb)           (a value per token and head)
    a = gated_delta_rule(q, k, v, log_decay, beta) Wo
    z, u = rms_norm(a, residual=x)                               (u = x + a, the stream)
    y = ReLU RNN layer(z) Wy

Its gradient is written out from the library's backward calls; torch supplies the plain matrix products and
the memory.  The task: answer, at every step, with the input of `LAG` steps ago.  After training the delta
rule is decoded one token at a time from a prompt's state and compared with the whole sequence's result.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from persistent_rnn_recurrence_gb300 import prnn  # noqa: E402

T, B, W, HEADS, DIM, HIDDEN, LAG = 96, 8, 64, 4, 32, 128, 3


def parameters(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, std):
        return torch.randn(*shape, generator=g, device="cuda") * std
    p = {n: rand(W, HEADS * DIM, std=W ** -0.5) for n in ("Wq", "Wk", "Wv")}
    p.update({n: rand(W, HEADS, std=W ** -0.5) for n in ("Wa", "Wb")})
    p["Wo"] = rand(HEADS * DIM, W, std=(HEADS * DIM) ** -0.5)
    p["Wx"], p["Wh"] = rand(HIDDEN, W, std=W ** -0.5), rand(HIDDEN, HIDDEN, std=0.5 * HIDDEN ** -0.5)
    p["b"], p["Wy"] = torch.zeros(HIDDEN, device="cuda"), rand(HIDDEN, W, std=HIDDEN ** -0.5)
    p["a0"] = torch.linspace(-4.0, -1.0, HEADS, device="cuda")      # heads that forget at different rates
    for n in ("g1", "g2"):
        p[n] = torch.ones(W, device="cuda")
    return p


class Block:
    def __init__(self, p):
        self.p = p
        self.unit = torch.full((DIM,), DIM ** -0.5, device="cuda")
        self.rnn = prnn.Layer(HIDDEN, W, B, "f32")

    def inputs(self, x):
        """What the delta rule reads, and what its gradient needs besides."""
        p = self.p
        n, _, r1 = prnn.rms_norm(x, p["g1"])
        raw = [(n @ p[w]).view(*x.shape[:2], HEADS, DIM) for w in ("Wq", "Wk")]
        q, k = (prnn.rms_norm(z, self.unit) for z in raw)
        v = (n @ p["Wv"]).view(*x.shape[:2], HEADS, DIM)
        s = n @ p["Wa"] + p["a0"]
        return (q[0], k[0], v, -torch.nn.functional.softplus(s), torch.sigmoid(n @ p["Wb"])), \
            (n, r1, raw, (q[2], k[2]), s)

    def forward(self, x):
        p = self.p
        prnn.prnn_set_weights_dense(self.rnn.h, p["Wx"], p["Wh"], p["b"])
        ins, more = self.inputs(x)
        o, state = prnn.gated_delta_rule(*ins, DIM ** -0.5)
        flat = o.reshape(*x.shape[:2], -1)
        z, u, r2 = prnn.rms_norm((flat @ p["Wo"]), p["g2"], residual=x)
        h = self.rnn.forward(z)
        self.saved = (x, ins, more, flat, z, u, r2, h)
        return h @ p["Wy"], o, state

    def backward(self, dy):
        p = self.p
        x, ins, (n, r1, raw, norms, s), flat, z, u, r2, h = self.saved
        rows = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        g = {"Wy": rows(h).t() @ rows(dy)}
        r = self.rnn.backward(z, h, (dy @ p["Wy"].t()).contiguous())
        g["Wx"], g["Wh"], g["b"] = r["dWx"], r["dWh"], r["db"]
        du, g["g2"] = prnn.rms_norm_backward(r["dx"], u, p["g2"], r2)
        g["Wo"] = rows(flat).t() @ rows(du)
        d = prnn.gated_delta_rule_backward((du @ p["Wo"].t()).view_as(ins[2]), *ins, DIM ** -0.5)
        parts = {"Wv": d["dv"]}
        for w, z_, rstd, dz in zip(("Wq", "Wk"), raw, norms, (d["dq"], d["dk"])):
            parts[w] = prnn.rms_norm_backward(dz, z_, self.unit, rstd)[0]
        parts["Wa"] = -torch.sigmoid(s) * d["dlog_decay"]
        parts["Wb"] = ins[4] * (1 - ins[4]) * d["dbeta"]
        g["a0"] = rows(parts["Wa"]).sum(0)
        dn = 0
        for w, part in parts.items():
            part = rows(part.reshape(*x.shape[:2], -1))
            g[w] = rows(n).t() @ part
            dn = dn + part @ p[w].t()
        # the stream's gradient passes the block beside what comes through it
        dx, g["g1"] = prnn.rms_norm_backward(dn.view_as(x), x, p["g1"], r1, dh=du)
        return g, dx


def train(steps=60, lr=3e-3, seed=1):
    """Returns the block and the loss of every step (Adam)."""
    p = parameters()
    block = Block(p)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    m = {n: torch.zeros_like(t) for n, t in p.items()}
    s = {n: torch.zeros_like(t) for n, t in p.items()}
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(T, B, W, generator=gen, device="cuda")
        want = torch.zeros_like(x)
        want[LAG:] = x[:-LAG]
        y, _, _ = block.forward(x)
        diff = y - want
        losses.append(float((diff * diff).mean()))
        g, _ = block.backward(2.0 / diff.numel() * diff)
        for n in p:
            m[n].mul_(0.9).add_(g[n], alpha=0.1)
            s[n].mul_(0.99).addcmul_(g[n], g[n], value=0.01)
            p[n].sub_(lr * (m[n] / (1 - 0.9 ** step)) / ((s[n] / (1 - 0.99 ** step)).sqrt() + 1e-8))
    return block, losses


def decode(block, x, prompt):
    """The delta rule's outputs for x [T, B, W]: the prompt as a sequence, then token by token from its state."""
    ins, _ = block.inputs(x)
    first, state = prnn.gated_delta_rule(*(z[:prompt] for z in ins), DIM ** -0.5)
    rest = [prnn.gated_delta_rule_step(*(z[t] for z in ins), state, DIM ** -0.5) for t in range(prompt, x.shape[0])]
    return torch.cat([first, torch.stack(rest)]), state


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    block, losses = train(ap.parse_args().steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    x = torch.randn(T, B, W, device="cuda")
    _, whole, state = block.forward(x)
    steps, end = decode(block, x, T // 2)
    print(f"token by token against the whole sequence: outputs {float((steps - whole).abs().max()):.2e}, "
          f"state {float((end - state).abs().max()):.2e}")


if __name__ == "__main__":
    main()
