"""The gated delta rule and its gradients in 64 bits, token by token, with the largest norms that the states and
their gradients reach on the way: the tests' tolerances are relative to those."""


def exact(torch, q, k, v, g, beta, scale, state=None, lens=None, do=None, dstate=None):
    """dict of o, state, and with do the gradients; norms S [B,H,dv] and R [B,H,dv]: the largest 2-norm of a column
    of S_t (or value) and of R_t (or weighted d_o)."""
    f = torch.float64
    T, B, H, dv = v.shape
    dk, share = q.shape[3], H // q.shape[2]
    dev = v.device
    lens = torch.full((B,), T, device=dev) if lens is None else lens.long().clamp(0, T)
    live = torch.arange(T, device=dev)[:, None] < lens
    on = live[:, :, None, None]
    zero = torch.zeros((), dtype=f, device=dev)
    q, k, v = (torch.where(on, x.to(f), zero) for x in (q, k, v))
    q, k = q.repeat_interleave(share, 2), k.repeat_interleave(share, 2)
    a = torch.where(on[..., 0], g.to(f).exp(), torch.ones((), dtype=f, device=dev))
    beta = torch.where(on[..., 0], beta.to(f), zero)
    S = torch.zeros(B, H, dk, dv, dtype=f, device=dev) if state is None else state.to(f)
    o, kept = torch.zeros(T, B, H, dv, dtype=f, device=dev), []
    most = torch.maximum(S.norm(dim=2), v.abs().amax(0) if T else zero)
    for t in range(T):
        d = S * a[t][..., None, None]
        e = v[t] - torch.einsum("bhk,bhkv->bhv", k[t], d)
        u = beta[t][..., None] * e
        S = d + k[t][..., :, None] * u[..., None, :]
        o[t] = scale * torch.einsum("bhk,bhkv->bhv", q[t], S)
        most = torch.maximum(most, S.norm(dim=2))
        if do is not None:
            kept.append((d, e, u, S))
    out = {"o": torch.where(on, o, zero), "state": S, "S": most, "live": on, "q": q, "k": k, "beta": beta}
    if do is None:
        return out
    do = torch.where(on, do.to(f), zero) * scale
    R = torch.zeros_like(S) if dstate is None else dstate.to(f)
    rmost = R.norm(dim=2)
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a), torch.zeros_like(a)
    for t in reversed(range(T)):
        d, e, u, S = kept[t]
        dq[t] = torch.einsum("bhkv,bhv->bhk", S, do[t])
        R = R + q[t][..., :, None] * do[t][..., None, :]
        rmost = torch.maximum(rmost, R.norm(dim=2))
        du = torch.einsum("bhk,bhkv->bhv", k[t], R)
        dvv[t] = beta[t][..., None] * du
        db[t] = (e * du).sum(-1)
        dkk[t] = torch.einsum("bhkv,bhv->bhk", R, u) - torch.einsum("bhkv,bhv->bhk", d, dvv[t])
        R = R - k[t][..., :, None] * dvv[t][..., None, :]
        dg[t] = (d * R).sum((-1, -2))
        R = R * a[t][..., None, None]

    def shared(z):
        return torch.where(on, z, zero).reshape(T, B, H // share, share, dk).sum(3)
    out.update(dq=shared(dq), dk=shared(dkk), dv=torch.where(on, dvv, zero),
               dlog_decay=torch.where(on[..., 0], dg, zero), dbeta=torch.where(on[..., 0], db, zero), dstate=R, R=rmost,
               do=do)
    return out
