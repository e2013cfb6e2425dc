"""Measured cases of the gated delta rule (whole sequences, their gradients and
single tokens) and of the root-mean-square norm that feeds it (with the residual's
addition, in the data's type or in 8 bits with scales, and its gradient).

Each operator is written twice: the library's call (``own``) and its plain form in
elementary fp32 tensor operations.  ``exact`` is the definition in 64 bits, token by
token over time where the plain form works in chunks.  Sequences are time-major,
[T][B][...], as everywhere in this library.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PLAIN_CHUNK = 64
EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    return [
        # one token of 4 sequences through the norm of an H = 1792 layer (decoding: latency)
        {"name": "rms_step_bf16", "op": "rms", "dtype": "bf16", "rows": 4, "cols": 1792, "residual": True},
        # the residual stream of 256 steps of 32 sequences, in mixed precision
        {"name": "rms_seq_bf16", "op": "rms", "dtype": "bf16", "rows": 8192, "cols": 4096, "residual": True},
        # the widest layer's input for a product in 8 bits, a scale for every 128 columns
        {"name": "rms_e4m3_bf16", "op": "rms_e4m3", "dtype": "bf16", "rows": 8192, "cols": 5760,
         "residual": True, "group": 128},
        # a ragged batch of a layer whose size no vector width divides, a scale for each row
        {"name": "rms_e4m3_odd_f16", "op": "rms_e4m3", "dtype": "f16", "rows": 1285, "cols": 1001,
         "residual": False, "group": 0},
        # training a layer of H = 2304 in its own fp32, the residual's gradient added
        {"name": "rms_grad_f32", "op": "rms_grad", "dtype": "f32", "rows": 8192, "cols": 2304, "residual": True},
        # a short prompt of one user: few heads, one tile of time (latency)
        {"name": "delta_prompt_short_bf16", "op": "delta", "dtype": "bf16", "T": 64, "B": 1,
         "heads": 8, "qk_heads": 8, "dk": 64, "dv": 64, "ragged": False, "state": False},
        # long prompts of two users
        {"name": "delta_prompt_long_bf16", "op": "delta", "dtype": "bf16", "T": 8192, "B": 2,
         "heads": 16, "qk_heads": 16, "dk": 128, "dv": 128, "ragged": False, "state": False},
        # a ragged batch continuing from cached states in fp32: odd sizes, queries and keys shared by
        # three value heads, one sequence empty and one of a single token
        {"name": "delta_ragged_f32", "op": "delta", "dtype": "f32", "T": 700, "B": 5, "heads": 6,
         "qk_heads": 2, "dk": 72, "dv": 100, "ragged": True, "state": True},
        # a training step's gradients at ordinary length
        {"name": "delta_grad_bf16", "op": "delta_grad", "dtype": "bf16", "T": 2048, "B": 4,
         "heads": 16, "qk_heads": 16, "dk": 128, "dv": 128, "ragged": False, "state": False},
        # the gradients of a ragged batch with states, odd sizes and shared queries and keys
        {"name": "delta_grad_ragged_f16", "op": "delta_grad", "dtype": "f16", "T": 300, "B": 3,
         "heads": 4, "qk_heads": 2, "dk": 48, "dv": 80, "ragged": True, "state": True},
        # one token for one user (latency)
        {"name": "delta_token_one_f16", "op": "delta_token", "dtype": "f16", "B": 1, "heads": 8,
         "qk_heads": 8, "dk": 64, "dv": 64, "slots": False},
        # one token for each of a full serving batch whose states lie in a larger pool
        {"name": "delta_token_batch_bf16", "op": "delta_token", "dtype": "bf16", "B": 96, "heads": 16,
         "qk_heads": 8, "dk": 128, "dv": 128, "slots": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms", "rms_e4m3", "rms_grad", "delta", "delta", "delta_grad", "delta_grad", "delta_token"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op.startswith("rms"):
        # from the heads of a query to the widest layers
        cols = _log_uniform(rng, 48, 8192)
        if rng.random() < 0.6:
            cols = (cols + 7) // 8 * 8
        rows = _log_uniform(rng, 1, max(2, min(100_000, 18_000_000 // cols)))
        case = {"op": op, "dtype": dtype, "rows": rows, "cols": cols, "residual": rng.random() < 0.6}
        if op == "rms_e4m3":
            case["group"] = rng.choice([0, 128])
        return case
    qk_heads = rng.choice([1, 2, 3, 4, 8, 16])
    heads = qk_heads * rng.choice([1, 1, 1, 2, 4])
    dk = rng.choice([32, 64, 64, 96, 128, 128, rng.randint(16, 128)])
    dv = dk if rng.random() < 0.6 else rng.choice([64, 128, rng.randint(16, 128)])
    if op == "delta_token":
        most = max(2, 96 * 16 * 128 * 128 // (heads * dk * dv))
        return {"op": op, "dtype": dtype, "B": _log_uniform(rng, 1, min(128, most)),
                "heads": heads, "qk_heads": qk_heads, "dk": dk, "dv": dv, "slots": rng.random() < 0.5}
    B = _log_uniform(rng, 1, 16)
    most = (8_000_000 if op == "delta" else 4_000_000) * 4 // (B * heads * (dk + dv))
    T = _log_uniform(rng, 1, max(2, min(8192, most)))
    return {"op": op, "dtype": dtype, "T": T, "B": B, "heads": heads, "qk_heads": qk_heads,
            "dk": dk, "dv": dv, "ragged": rng.random() < 0.4, "state": rng.random() < 0.4}


# ---- inputs -------------------------------------------------------------------
def _log_decay(shape, gen, device):
    """Per token and head, minus a head's rate times softplus of a normal value: half-lives from about
    10 to 1400 tokens."""
    heads = shape[-1]
    h = torch.arange(heads, device=device, dtype=torch.float64)
    rate = torch.exp2(-4.0 - 7.0 * h / max(1, heads - 1)).to(torch.float32)
    return -rate * torch.nn.functional.softplus(torch.randn(shape, generator=gen, device=device))


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def unit(*shape):
        x = torch.randn(*shape, generator=gen, device=dev)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    op = case["op"]
    s = {"op": op}
    if op.startswith("rms"):
        rows, cols = case["rows"], case["cols"]
        s["weight"] = 1.0 + normal(cols, std=0.1, dtype=torch.float32)
        if op == "rms_grad":
            # the stream as the forward pass left it, the norm's gradient, and that of the stream itself
            s["h"], s["dy"] = normal(rows, cols), normal(rows, cols, std=0.02)
            s["dh"] = normal(rows, cols, std=0.02) if case["residual"] else None
            hf = s["h"].float()
            s["rstd"] = torch.rsqrt((hf * hf).mean(-1) + EPS)
        else:
            s["x"] = normal(rows, cols)
            s["residual"] = normal(rows, cols, std=2.0) if case["residual"] else None
            s["group"] = case.get("group")
        return s
    B, H, Hq, dk, dv = (case[n] for n in ("B", "heads", "qk_heads", "dk", "dv"))
    s["scale"] = dk ** -0.5
    # queries and keys come normalised to length one
    if op == "delta_token":
        s["q"], s["k"], s["v"] = unit(B, Hq, dk), unit(B, Hq, dk), normal(B, H, dv)
        s["log_decay"] = _log_decay((B, H), gen, dev)
        s["beta"] = torch.sigmoid(normal(B, H, dtype=torch.float32))
        if case["slots"]:
            n = B + B // 4 + 1
            slots = torch.randperm(n, generator=gen, device=dev)[:B].to(torch.int32)
            slots[B // 2] = -1          # a padding row of the batch
            s["slots"] = slots
        else:
            n, s["slots"] = B, None
        s["state"] = normal(n, H, dk, dv, std=0.3, dtype=torch.float32)
        return s
    T = case["T"]
    s["q"], s["k"], s["v"] = unit(T, B, Hq, dk), unit(T, B, Hq, dk), normal(T, B, H, dv)
    s["log_decay"] = _log_decay((T, B, H), gen, dev)
    s["beta"] = torch.sigmoid(normal(T, B, H, dtype=torch.float32))
    s["state"] = normal(B, H, dk, dv, std=0.3, dtype=torch.float32) if case["state"] else None
    s["lens"] = None
    if case["ragged"]:
        lens = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        lens[0] = T
        if B > 2:
            lens[1], lens[2] = 0, 1
        s["lens"] = lens
    if op == "delta_grad":
        s["do"] = normal(T, B, H, dv, std=0.02)
        s["dstate"] = normal(B, H, dk, dv, std=0.02, dtype=torch.float32) if case["state"] else None
    return s


# ---- plain forms --------------------------------------------------------------
def _rms(s):
    """(y in fp32, the stream, rstd): the stream x + residual is rounded to its type and normalised as stored."""
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    hf = h.float()
    rstd = 1.0 / torch.sqrt((hf * hf).sum(1) / hf.shape[1] + EPS)
    return hf * rstd[:, None] * s["weight"], h, rstd


def _rms_plain(s):
    y, h, rstd = _rms(s)
    return (y.to(h.dtype), rstd) if s["residual"] is None else (y.to(h.dtype), h, rstd)


def _rms_e4m3(s):
    y, h, rstd = _rms(s)
    rows, cols = y.shape
    width = s["group"] or cols
    n = -(-cols // width)
    padded = torch.zeros(rows, n * width, device=y.device)
    padded[:, :cols] = y
    groups = padded.reshape(rows, n, width)
    top = groups.abs().amax(2)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = (groups / scale[..., None]).reshape(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return (q, scale, rstd) if s["residual"] is None else (q, scale, h, rstd)


def _rms_grad(s):
    h, dy, r = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = h * r
    g = dy * s["weight"]
    dx = r * (g - xhat * ((g * xhat).sum(1) / h.shape[1])[:, None])
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["h"].dtype), (dy * xhat).sum(0)


def _unit_lower_inverse(a):
    """(I + a)^-1 for strictly lower triangular a [..., n, n], n a power of two: diagonal blocks of 1, 2,
    4, ... rows are inverted in turn, [[A, 0], [C, D]]^-1 = [[A^-1, 0], [-D^-1 C A^-1, D^-1]]."""
    n = a.shape[-1]
    out = torch.eye(n, device=a.device).expand(a.shape).contiguous()
    size = 1
    while size < n:
        blocks = n // (2 * size)
        view = out.reshape(-1, blocks, 2 * size, blocks, 2 * size).diagonal(dim1=1, dim2=3)      # [.., 2s, 2s, blocks]
        low = a.reshape(-1, blocks, 2 * size, blocks, 2 * size).diagonal(dim1=1, dim2=3).permute(0, 3, 1, 2)
        inv = view.permute(0, 3, 1, 2)
        first, second = inv[..., :size, :size], inv[..., size:, size:]
        view[:, size:, :size] = -torch.matmul(torch.matmul(second, low[..., size:, :size]), first).permute(0, 2, 3, 1)
        size *= 2
    return out


def _chunked(z, n, C):
    T = z.shape[0]
    z = torch.cat([z, z.new_zeros((n * C - T,) + z.shape[1:])]) if n * C > T else z
    z = z.reshape((n, C) + z.shape[1:])
    return z.permute(0, 2, 3, 1, 4) if z.dim() == 5 else z.permute(0, 2, 3, 1)


def _joined(z, T):
    """[n,B,H,C,...] back to [T,B,H,...]."""
    z = z.permute(0, 3, 1, 2, 4) if z.dim() == 5 else z.permute(0, 3, 1, 2)
    return z.reshape((-1,) + z.shape[2:])[:T]


def _delta_parts(s):
    """What the forward pass and its gradient share, per chunk [n,B,H,C,...] in fp32, zeros past each length."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    T, B, H = v.shape[:3]
    group = H // q.shape[2]
    if group > 1:
        q, k = q.repeat_interleave(group, 2), k.repeat_interleave(group, 2)
    g, beta = s["log_decay"], s["beta"]
    live = None
    if s["lens"] is not None:
        live = (torch.arange(T, device=v.device)[:, None] < s["lens"])[:, :, None]
        zero = torch.zeros((), device=v.device)
        q, k, v = (torch.where(live[..., None], z, zero) for z in (q, k, v))
        g, beta = torch.where(live, g, zero), torch.where(live, beta, zero)
    C = PLAIN_CHUNK
    n = -(-T // C)
    q, k, v, g, beta = (_chunked(z, n, C) for z in (q, k, v, g, beta))
    G = g.cumsum(-1)
    i = torch.arange(C, device=v.device)
    gap = G[..., :, None] - G[..., None, :]
    below = i[:, None] >= i[None, :]
    D = torch.where(below, torch.exp(torch.where(below, gap, torch.zeros((), device=v.device))),
                    torch.zeros((), device=v.device))
    M = torch.matmul(k, k.transpose(-1, -2)) * D * (i[:, None] > i[None, :])
    inv = _unit_lower_inverse(M * beta[..., None, :])
    up, last = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None]
    whole = torch.exp(G[..., -1])[..., None, None]
    p = {"q": q, "k": k, "v": v, "beta": beta[..., None], "D": D, "M": M, "inv": inv, "up": up, "down": last,
         "whole": whole, "W": torch.matmul(inv, k * up), "live": live, "T": T, "n": n}
    Ebar, ktail = torch.matmul(inv, v), (k * last * p["beta"]).transpose(-1, -2)
    S = s["state"] if s["state"] is not None else torch.zeros(B, H, k.shape[-1], v.shape[-1], device=v.device)
    before, E = [], []
    for m in range(n):
        before.append(S)
        E.append(Ebar[m] - torch.matmul(p["W"][m], S))
        S = S * whole[m] + torch.matmul(ktail[m], E[m])
    p["S"], p["E"], p["end"] = torch.stack(before), torch.stack(E), S
    p["U"] = p["E"] * p["beta"]
    return p


def _delta(s):
    p = _delta_parts(s)
    o = p["up"] * torch.matmul(p["q"], p["S"])
    o = o + torch.matmul(torch.matmul(p["q"], p["k"].transpose(-1, -2)) * p["D"], p["U"])
    return _joined(o * s["scale"], p["T"]).to(s["v"].dtype), p["end"]


def _delta_grad(s):
    p = _delta_parts(s)
    q, k, v, beta, D, U, T, n = (p[x] for x in ("q", "k", "v", "beta", "D", "U", "T", "n"))
    do = s["do"].float()
    if p["live"] is not None:
        do = torch.where(p["live"][..., None], do, torch.zeros((), device=do.device))
    do = _chunked(do, n, PLAIN_CHUNK) * s["scale"]
    X0 = torch.matmul((torch.matmul(q, k.transpose(-1, -2)) * D).transpose(-1, -2), do)
    add = torch.matmul((q * p["up"]).transpose(-1, -2), do)
    kdown, Wt = k * p["down"], p["W"].transpose(-1, -2)
    R = s["dstate"] if s["dstate"] is not None else torch.zeros_like(p["end"])
    after, X = [], []
    for m in reversed(range(n)):
        after.append(R)
        X.append(X0[m] + torch.matmul(kdown[m], R))
        R = R * p["whole"][m] + add[m] - torch.matmul(Wt[m], beta[m] * X[-1])
    R_end, X = torch.stack(after[::-1]), torch.stack(X[::-1])
    dv = torch.matmul(p["inv"].transpose(-1, -2), beta * X)
    du = X - torch.matmul(p["M"].transpose(-1, -2), dv)
    dbeta = (p["E"] * du).sum(-1)
    i = torch.arange(PLAIN_CHUNK, device=v.device)
    Z1 = torch.matmul(do, U.transpose(-1, -2)) * D
    Z2 = torch.matmul(dv, U.transpose(-1, -2)) * D * (i[:, None] > i[None, :])
    S0t = p["S"].transpose(-1, -2)
    dq = p["up"] * torch.matmul(do, S0t) + torch.matmul(Z1, k)
    dk = p["down"] * torch.matmul(U, R_end.transpose(-1, -2)) + torch.matmul(Z1.transpose(-1, -2), q) \
        - torch.matmul(Z2.transpose(-1, -2) + Z2, k) - p["up"] * torch.matmul(dv, S0t)
    # the log-decays' gradient: what later tokens of the chunk do with the state, and the state that leaves it
    after_S = torch.cat([p["S"][1:], p["end"][None]])
    leaves = (after_S.double() * R_end.double()).sum((-1, -2))[..., None]
    own_part = (q.double() * dq.double()).sum(-1) - (v.double() * dv.double()).sum(-1)
    dg = (own_part.flip(-1).cumsum(-1).flip(-1) + leaves).float()
    dq, dk, dv, dbeta, dg = (_joined(z, T) for z in (dq, dk, dv, dbeta, dg))
    if p["live"] is not None:
        zero = torch.zeros((), device=v.device)
        dq, dk, dv = (torch.where(p["live"][..., None], z, zero) for z in (dq, dk, dv))
        dbeta, dg = torch.where(p["live"], dbeta, zero), torch.where(p["live"], dg, zero)
    shared = s["q"].shape[2]
    if shared < v.shape[2]:
        dq, dk = (z.reshape(T, z.shape[1], shared, -1, z.shape[-1]).sum(3) for z in (dq, dk))
    dt = s["v"].dtype
    out = {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dlog_decay": dg, "dbeta": dbeta}
    if s["state"] is not None:
        out["dstate"] = R
    return out


def _delta_token(s):
    q, k, v, state = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    group = v.shape[1] // q.shape[1]
    if group > 1:
        q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    rows = torch.arange(v.shape[0], device=v.device)
    at = rows
    if s["slots"] is not None:
        live = s["slots"] >= 0
        rows, at = rows[live], s["slots"][live].long()
    S = state[at] * torch.exp(s["log_decay"][rows])[..., None, None]
    e = v[rows] - (S * k[rows][..., None]).sum(2)
    S = S + k[rows][..., None] * (s["beta"][rows][..., None] * e)[..., None, :]
    state[at] = S
    o = torch.zeros_like(v)
    o[rows] = (S * q[rows][..., None]).sum(2) * s["scale"]
    return o.to(s["v"].dtype), state


def run(s):
    if own:
        return _run_own(s)
    return {"rms": _rms_plain, "rms_e4m3": _rms_e4m3, "rms_grad": _rms_grad, "delta": _delta,
            "delta_grad": _delta_grad, "delta_token": _delta_token}[s["op"]](s)


def _run_own(s):
    from persistent_rnn_recurrence_gb300 import prnn
    op = s["op"]
    if op == "rms":
        y, h, rstd = prnn.rms_norm(s["x"], s["weight"], EPS, s["residual"])
        return (y, rstd) if s["residual"] is None else (y, h, rstd)
    if op == "rms_e4m3":
        q, scale, h, rstd = prnn.rms_norm_e4m3(s["x"], s["weight"], EPS, s["residual"], group=s["group"])
        return (q, scale, rstd) if s["residual"] is None else (q, scale, h, rstd)
    if op == "rms_grad":
        return prnn.rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dh"])
    if op == "delta":
        return prnn.gated_delta_rule(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["scale"],
                                     s["state"], s["lens"])
    if op == "delta_grad":
        return prnn.gated_delta_rule_backward(s["do"], s["q"], s["k"], s["v"], s["log_decay"], s["beta"],
                                              s["scale"], s["state"], s["lens"], s["dstate"])
    o = prnn.gated_delta_rule_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"],
                                   s["scale"], s["slots"])
    return o, s["state"]


# ---- what a pass cannot do without -------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op.startswith("rms"):
        rows, cols = case["rows"], case["cols"]
        n = rows * cols
        if op == "rms_grad":
            return {"bytes": (4 if case["residual"] else 3) * n * e + 8 * cols + 4 * rows, "flops": 9 * n}
        # the stream is written where something is added to it
        stream = (3 if case["residual"] else 1) * n * e
        if op == "rms":
            return {"bytes": stream + n * e + 4 * cols + 4 * rows, "flops": 5 * n}
        groups = -(-cols // case["group"]) if case["group"] else 1
        return {"bytes": stream + n + 4 * rows * groups + 4 * cols + 4 * rows, "flops": 8 * n}
    B, H, Hq, dk, dv = (case[n] for n in ("B", "heads", "qk_heads", "dk", "dv"))
    if op == "delta_token":
        live = B - 1 if case["slots"] else B
        return {"bytes": live * (8 * H * dk * dv + e * (2 * Hq * dk + H * dv) + 8 * H) + e * B * H * dv,
                "flops": 7 * live * H * dk * dv}
    T = case["T"]
    qk, vo, st, gates = T * B * Hq * dk * e, T * B * H * dv * e, 4 * B * H * dk * dv, 8 * T * B * H
    # one step: the decay of the state, its products with k and q, and a rank-one update, 7 dk dv
    if op == "delta":
        return {"bytes": 2 * qk + 2 * vo + gates + st * (2 if case["state"] else 1),
                "flops": 7 * T * B * H * dk * dv}
    # the states once more, and for the gradients 6 products with a state or its gradient, two rank-one
    # updates, a decay and an inner product of the two
    return {"bytes": 4 * qk + 3 * vo + 2 * gates + st * (3 if case["state"] else 0),
            "flops": 24 * T * B * H * dk * dv}


# ---- the definitions in 64 bits ----------------------------------------------------
def _exact_delta(s, grad):
    """Token by token.  Forward, with a = exp(log_decay): S' = a S_{t-1}, e_t = v_t - S'^T k_t,
    u_t = beta_t e_t, S_t = S' + k_t u_t^T, o_t = scale S_t^T q_t.  Gradients, with R the loss's by S_t:
    R += scale q_t do_t^T; du = R^T k_t; dv_t = beta_t du; dbeta_t = e_t . du;
    dS' = R - k_t dv_t^T; dk_t = R u_t - S' dv_t; dlog_decay_t = <S', dS'>; R for the token before = a dS'."""
    f = torch.float64
    q, k, v = s["q"].to(f), s["k"].to(f), s["v"].to(f)
    T, B, H, dv = v.shape
    dk, g = q.shape[3], H // q.shape[2]
    q, k = q.repeat_interleave(g, 2), k.repeat_interleave(g, 2)
    a, beta = torch.exp(s["log_decay"].to(f)), s["beta"].to(f)
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device=v.device)
    live = (torch.arange(T, device=v.device)[:, None] < lens)[:, :, None]
    # tokens past a length change nothing
    a, beta = torch.where(live, a, 1.0), torch.where(live, beta, 0.0)
    S = s["state"].to(f) if s["state"] is not None else torch.zeros(B, H, dk, dv, dtype=f, device=v.device)

    def step(S, t):
        d = S * a[t][..., None, None]
        e = v[t] - torch.matmul(k[t][..., None, :], d)[..., 0, :]
        u = beta[t][..., None] * e
        return d, e, u, d + k[t][..., :, None] * u[..., None, :]

    if not grad:
        o = torch.zeros_like(v)
        for t in range(T):
            S = step(S, t)[3]
            o[t] = s["scale"] * torch.matmul(q[t][..., None, :], S)[..., 0, :]
        return torch.where(live[..., None], o, 0.0), S
    every, kept = 64, []
    for t in range(T):
        if t % every == 0:
            kept.append(S)
        S = step(S, t)[3]
    do = torch.where(live[..., None], s["do"].to(f), 0.0) * s["scale"]
    R = s["dstate"].to(f) if s["dstate"] is not None else torch.zeros_like(S)
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a), torch.zeros_like(a)
    for m in reversed(range(len(kept))):
        S, run_ = kept[m], []
        for t in range(m * every, min(T, (m + 1) * every)):
            d, e, u, S = step(S, t)
            run_.append((t, d, e, u, S))
        for t, d, e, u, S in reversed(run_):
            dq[t] = torch.matmul(S, do[t][..., :, None])[..., 0]
            R = R + q[t][..., :, None] * do[t][..., None, :]
            du = torch.matmul(k[t][..., None, :], R)[..., 0, :]
            dvv[t] = beta[t][..., None] * du
            db[t] = (e * du).sum(-1)
            dkk[t] = torch.matmul(R, u[..., :, None])[..., 0] - torch.matmul(d, dvv[t][..., :, None])[..., 0]
            R = R - k[t][..., :, None] * dvv[t][..., None, :]
            dg[t] = (d * R).sum((-1, -2))
            R = R * a[t][..., None, None]
    z = torch.zeros((), dtype=f, device=v.device)
    dq, dkk, dvv = (torch.where(live[..., None], x, z) for x in (dq, dkk, dvv))
    out = {"dq": dq.reshape(T, B, H // g, g, dk).sum(3), "dk": dkk.reshape(T, B, H // g, g, dk).sum(3), "dv": dvv,
           "dlog_decay": torch.where(live, dg, z), "dbeta": torch.where(live, db, z)}
    if s["state"] is not None:
        out["dstate"] = R
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if op == "rms_grad":
        h, dy, r = s["h"].to(f), s["dy"].to(f), s["rstd"].to(f)[:, None]
        gx = dy * s["weight"].to(f)
        dot = torch.einsum("rc,rc->r", gx, h)[:, None] / h.shape[1]
        dx = r * gx - h * dot * r ** 3
        return dx if s["dh"] is None else dx + s["dh"].to(f), torch.einsum("rc,rc,r->c", dy, h, r[:, 0])
    if op.startswith("rms"):
        h = s["x"].to(f)
        if s["residual"] is not None:
            h = (h + s["residual"].to(f)).to(s["x"].dtype).to(f)
        rstd = (h.pow(2).mean(1) + EPS).rsqrt()
        y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].to(f))
        if op == "rms":
            return (y, rstd) if s["residual"] is None else (y, h, rstd)
        scales = torch.stack([part.abs().amax(1) for part in y.split(s["group"] or y.shape[1], 1)], 1) / 448.0
        # the values in 8 bits have no such value: one of two neighbours is theirs
        return (None, scales, rstd) if s["residual"] is None else (None, scales, h, rstd)
    if op in ("delta", "delta_grad"):
        if case["T"] > 16384:
            return None
        return _exact_delta(s, op == "delta_grad")
    state = s["state"].to(f)
    g = s["v"].shape[1] // s["q"].shape[1]
    o = torch.zeros(s["v"].shape, dtype=f, device=s["v"].device)
    for b in range(s["v"].shape[0]):
        at = b if s["slots"] is None else int(s["slots"][b])
        if at < 0:
            continue
        k, q = (s[n][b].to(f).repeat_interleave(g, 0) for n in ("k", "q"))
        S = torch.exp(s["log_decay"][b].to(f))[:, None, None] * state[at]
        e = s["v"][b].to(f) - torch.einsum("hd,hde->he", k, S)
        state[at] = S + torch.einsum("hd,he,h->hde", k, e, s["beta"][b].to(f))
        o[b] = s["scale"] * torch.einsum("hd,hde->he", q, state[at])
    return o, state
