"""Linear attention and its gradients in 64 bits, token by token, all sequences and heads at once: the same
definition as the reference in test_sequence_ops_gpu.py, fast enough for thousands of tokens."""


def exact(torch, q, k, v, ld, scale, state=None, lens=None, grad=None, dstate=None):
    """(o, end), or with grad (d_o) a dict of dq, dk, dv, dstate."""
    f = torch.float64
    T, B, H, dv = v.shape
    dk, g = q.shape[3], H // q.shape[2]
    q, k, v = q.to(f).repeat_interleave(g, 2), k.to(f).repeat_interleave(g, 2), v.to(f)
    decay = ld.to(f).exp()[None, :, None, None]
    lens = torch.full((B,), T, device=v.device) if lens is None else lens.long().clamp(0, T)
    whole = bool((lens == T).all())

    def live(t, new, old):
        return new if whole else torch.where((lens > t)[:, None, None, None], new, old)
    zero = torch.zeros((), dtype=f, device=v.device)
    S = torch.zeros(B, H, dk, dv, dtype=f, device=v.device) if state is None else state.to(f).clone()
    first = torch.zeros(T, B, H, dv if grad is None else dk, dtype=f, device=v.device)
    if grad is not None:
        grad = grad.to(f)
    for t in range(T):
        S = live(t, decay * S + k[t][..., :, None] * v[t][..., None, :], S)
        out = torch.matmul(q[t][..., None, :], S)[..., 0, :] if grad is None else \
            torch.matmul(S, grad[t][..., :, None])[..., 0]
        first[t] = scale * (out if whole else torch.where((lens > t)[:, None, None], out, zero))
    if grad is None:
        return first, S
    R = torch.zeros_like(S) if dstate is None else dstate.to(f).clone()
    dkk, dvv = torch.zeros_like(first), torch.zeros_like(v)
    for t in reversed(range(T)):
        full = R + scale * q[t][..., :, None] * grad[t][..., None, :]
        a, b = torch.matmul(full, v[t][..., :, None])[..., 0], torch.matmul(k[t][..., None, :], full)[..., 0, :]
        if not whole:
            on = (lens > t)[:, None, None]
            a, b = torch.where(on, a, zero), torch.where(on, b, zero)
        dkk[t], dvv[t] = a, b
        R = live(t, decay * full, R)
    shared = lambda z: z.reshape(T, B, H // g, g, dk).sum(3)  # noqa: E731
    return {"dq": shared(first), "dk": shared(dkk), "dv": dvv, "dstate": R}
