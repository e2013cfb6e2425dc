"""A residual recurrent block trained and then decoded token by token.

    python examples/recurrent_block.py [--steps 60]

The block reads a sequence x [T, B, W]:

    n = layer_norm(x);  q, k, v = n Wq, n Wk, n Wv            (heads of linear attention)
    a = linear_attention(q, k, v);  u = x + dropout(a Wo)
    h = ReLU RNN layer(layer_norm(u));  y = h Wy

Its gradient is written out from the library's backward calls; torch supplies the plain matrix
products and the memory.  The task: answer, at every step, with the input of `LAG` steps ago, which
needs a memory that spans the lag.  After training the attention half is decoded one token at a
time from a prompt's state and compared with the whole sequence's result.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from persistent_rnn_recurrence_gb300 import prnn  # noqa: E402

T, B, W, HEADS, DIM, HIDDEN, LAG = 64, 8, 64, 4, 32, 128, 3


def parameters(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, std):
        return torch.randn(*shape, generator=g, device="cuda") * std
    p = {n: rand(W, HEADS * DIM, std=W ** -0.5) for n in ("Wq", "Wk", "Wv")}
    p["Wo"] = rand(HEADS * DIM, W, std=(HEADS * DIM) ** -0.5)
    p["Wx"], p["Wh"] = rand(HIDDEN, W, std=W ** -0.5), rand(HIDDEN, HIDDEN, std=0.5 * HIDDEN ** -0.5)
    p["b"], p["Wy"] = torch.zeros(HIDDEN, device="cuda"), rand(HIDDEN, W, std=HIDDEN ** -0.5)
    for n in ("g1", "g2"):
        p[n] = torch.ones(W, device="cuda")
    for n in ("b1", "b2"):
        p[n] = torch.zeros(W, device="cuda")
    return p


# half-lives of 0.7 to 22 tokens: the heads look back over different spans
LOG_DECAY = torch.tensor([-1.0, -0.3, -0.1, -0.03])


class Block:
    def __init__(self, p, drop=0.1):
        self.p, self.drop = p, drop
        self.ld = LOG_DECAY.cuda()
        self.rnn = prnn.Layer(HIDDEN, W, B, "f32")

    def attend(self, x):
        p = self.p
        n, mean, rstd = prnn.layer_norm(x, p["g1"], p["b1"])
        q, k, v = ((n @ p[w]).view(*x.shape[:2], HEADS, DIM) for w in ("Wq", "Wk", "Wv"))
        return n, mean, rstd, q, k, v

    def forward(self, x, seed):
        p = self.p
        prnn.prnn_set_weights_dense(self.rnn.h, p["Wx"], p["Wh"], p["b"])
        n, m1, r1, q, k, v = self.attend(x)
        a, state = prnn.linear_attention(q, k, v, self.ld, DIM ** -0.5)
        flat = a.reshape(*x.shape[:2], -1)
        u = prnn.dropout(flat @ p["Wo"], self.drop, seed, 0, residual=x)
        z, m2, r2 = prnn.layer_norm(u, p["g2"], p["b2"])
        h = self.rnn.forward(z)
        self.saved = (x, seed, n, m1, r1, q, k, v, flat, u, z, m2, r2, h)
        return h @ p["Wy"], a, state

    def backward(self, dy):
        p = self.p
        x, seed, n, m1, r1, q, k, v, flat, u, z, m2, r2, h = self.saved
        rows = lambda t: t.reshape(-1, t.shape[-1])
        g = {"Wy": rows(h).t() @ rows(dy)}
        r = self.rnn.backward(z, h, (dy @ p["Wy"].t()).contiguous())
        g["Wx"], g["Wh"], g["b"] = r["dWx"], r["dWh"], r["db"]
        du, g["g2"], g["b2"] = prnn.layer_norm_backward(r["dx"], u, p["g2"], m2, r2)
        dproj = prnn.dropout_backward(du, self.drop, seed, 0)
        g["Wo"] = rows(flat).t() @ rows(dproj)
        da = (dproj @ p["Wo"].t()).view_as(v)
        d = prnn.linear_attention_backward(da, q, k, v, self.ld, DIM ** -0.5)
        dn = 0
        for name, w in (("dq", "Wq"), ("dk", "Wk"), ("dv", "Wv")):
            part = rows(d[name].reshape(*x.shape[:2], -1))
            g[w] = rows(n).t() @ part
            dn = dn + part @ p[w].t()
        dx, g["g1"], g["b1"] = prnn.layer_norm_backward(dn.view_as(x), x, p["g1"], m1, r1)
        return g, dx + du


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
        y, _, _ = block.forward(x, seed=step)
        diff = y - want
        losses.append(float((diff * diff).mean()))
        g, _ = block.backward(2.0 / diff.numel() * diff)
        for n in p:
            m[n].mul_(0.9).add_(g[n], alpha=0.1)
            s[n].mul_(0.99).addcmul_(g[n], g[n], value=0.01)
            p[n].sub_(lr * (m[n] / (1 - 0.9 ** step)) / ((s[n] / (1 - 0.99 ** step)).sqrt() + 1e-8))
    return block, losses


def decode(block, x, prompt):
    """Attention outputs of x [T, B, W]: the prompt as a sequence, then token by token from its state."""
    _, _, _, q, k, v = block.attend(x)
    first, state = prnn.linear_attention(q[:prompt], k[:prompt], v[:prompt], block.ld, DIM ** -0.5)
    rest = [prnn.linear_attention_step(q[t], k[t], v[t], block.ld, state, DIM ** -0.5)
            for t in range(prompt, x.shape[0])]
    return torch.cat([first, torch.stack(rest)]), state


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    block, losses = train(ap.parse_args().steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    x = torch.randn(T, B, W, device="cuda")
    _, whole, state = block.forward(x, seed=0)
    steps, end = decode(block, x, T // 2)
    print(f"token by token against the whole sequence: outputs {float((steps - whole).abs().max()):.2e}, "
          f"state {float((end - state).abs().max()):.2e}")


if __name__ == "__main__":
    main()
