"""Measured cases of the sequence operators around the recurrent layers: layer
normalisation, dropout with a residual, and linear attention with a decay per
head (whole sequences and single tokens).

Each operator is written twice: the library's call (``own``) and its plain form
in elementary fp32 tensor operations.  ``exact`` is the definition in 64 bits,
step by step over time where the plain form works in chunks.  Sequences are
time-major, [T][B][...], as everywhere in this library.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PLAIN_CHUNK = 64
EPS = 1e-5


def listed():
    return [
        # one time step of B = 4 sequences through the norm of an H = 1792 layer (decoding: latency)
        {"name": "norm_step_f32", "op": "norm", "dtype": "f32", "rows": 4, "cols": 1792},
        # the outputs of 256 steps of 32 sequences, normalised in mixed precision
        {"name": "norm_seq_bf16", "op": "norm", "dtype": "bf16", "rows": 8192, "cols": 4096},
        # training on a ragged batch of a layer whose size no vector width divides
        {"name": "norm_grad_odd_f16", "op": "norm_grad", "dtype": "f16", "rows": 1285, "cols": 301},
        # training the widest layer at full batch, in the layer's own fp32
        {"name": "norm_grad_f32", "op": "norm_grad", "dtype": "f32", "rows": 8192, "cols": 5760},
        # the gradient of dropout between two layers, 256 steps of 4 sequences
        {"name": "dropout_grad_f32", "op": "dropout_grad", "dtype": "f32", "rows": 1024,
         "cols": 1152, "p": 0.1, "residual": False},
        # dropout and residual over whole sequences at full batch, in mixed precision
        {"name": "dropout_seq_bf16", "op": "dropout", "dtype": "bf16", "rows": 8192, "cols": 5760,
         "p": 0.2, "residual": True},
        # a short prompt of one user: few heads, one tile of time (latency)
        {"name": "attn_prompt_short_bf16", "op": "attn", "dtype": "bf16", "T": 64, "B": 1,
         "heads": 8, "qk_heads": 8, "dk": 64, "dv": 64, "ragged": False, "state": False},
        # long prompts of two users
        {"name": "attn_prompt_long_bf16", "op": "attn", "dtype": "bf16", "T": 8192, "B": 2,
         "heads": 16, "qk_heads": 16, "dk": 128, "dv": 128, "ragged": False, "state": False},
        # a ragged batch continuing from cached states in fp32: odd sizes, queries and keys
        # shared by three value heads, one sequence empty and one of a single token
        {"name": "attn_ragged_f32", "op": "attn", "dtype": "f32", "T": 700, "B": 5, "heads": 6,
         "qk_heads": 2, "dk": 72, "dv": 100, "ragged": True, "state": True},
        # a training step's gradients at ordinary length
        {"name": "attn_grad_bf16", "op": "attn_grad", "dtype": "bf16", "T": 2048, "B": 4,
         "heads": 16, "qk_heads": 16, "dk": 128, "dv": 128, "ragged": False, "state": False},
        # one token for one user (latency)
        {"name": "token_one_f16", "op": "token", "dtype": "f16", "B": 1, "heads": 8, "qk_heads": 8,
         "dk": 64, "dv": 64, "slots": False},
        # one token for each of a full serving batch whose states lie in a larger pool
        {"name": "token_batch_bf16", "op": "token", "dtype": "bf16", "B": 96, "heads": 16,
         "qk_heads": 8, "dk": 128, "dv": 128, "slots": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dropout", "dropout_grad", "attn", "attn_grad", "token"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("norm", "norm_grad", "dropout", "dropout_grad"):
        cols = _log_uniform(rng, 64, 8192)
        if rng.random() < 0.5:
            cols = (cols + 7) // 8 * 8
        rows = _log_uniform(rng, 1, max(2, min(65536, 40_000_000 // cols)))
        case = {"op": op, "dtype": dtype, "rows": rows, "cols": cols}
        if op in ("dropout", "dropout_grad"):
            case["p"] = rng.choice([0.0, 0.1, 0.25, 0.5])
            case["residual"] = op == "dropout" and rng.random() < 0.5
        return case
    qk_heads = rng.choice([1, 2, 3, 4, 8, 16])
    heads = qk_heads * rng.choice([1, 1, 1, 2, 4])
    dk = rng.choice([32, 64, 64, 96, 128, 128, rng.randint(16, 128)])
    dv = dk if rng.random() < 0.6 else rng.choice([64, 128, rng.randint(16, 128)])
    if op == "token":
        most = max(2, 96 * 16 * 128 * 128 // (heads * dk * dv))
        return {"op": op, "dtype": dtype, "B": _log_uniform(rng, 1, min(128, most)),
                "heads": heads, "qk_heads": qk_heads, "dk": dk, "dv": dv,
                "slots": rng.random() < 0.5}
    B = _log_uniform(rng, 1, 32)
    most = (4_000_000 if op == "attn" else 2_000_000) * 4 // (B * heads * (dk + dv))
    T = _log_uniform(rng, 1, max(2, min(16384, most)))
    return {"op": op, "dtype": dtype, "T": T, "B": B, "heads": heads, "qk_heads": qk_heads,
            "dk": dk, "dv": dv, "ragged": rng.random() < 0.4, "state": rng.random() < 0.4}


# ---- inputs -------------------------------------------------------------------
def _log_decay(heads, device):
    """Each head forgets at its own rate: half-lives from about 20 to 2800 tokens."""
    h = torch.arange(heads, device=device, dtype=torch.float64)
    return torch.log1p(-torch.exp2(-5.0 - 7.0 * h / max(1, heads - 1))).to(torch.float32)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    s = {"op": case["op"], "seed": int(seed)}
    if case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        # a residual stream: an offset common to the row beside the varying part
        x = torch.randn(rows, cols, generator=gen, device=dev)
        s["x"] = (x + 0.5 * torch.randn(rows, 1, generator=gen, device=dev)).to(dt)
        s["gamma"] = 1.0 + normal(cols, std=0.1, dtype=torch.float32)
        s["beta"] = normal(cols, std=0.1, dtype=torch.float32)
        if case["op"] == "norm_grad":
            s["dy"] = normal(rows, cols, std=0.02)
            xf = s["x"].float()
            s["mean"] = xf.mean(-1)
            s["rstd"] = torch.rsqrt(xf.var(-1, unbiased=False) + EPS)
    elif case["op"] in ("dropout", "dropout_grad"):
        # the gradient's mask is the forward pass's, so x stands for dy there
        s["x"] = normal(case["rows"], case["cols"])
        s["residual"] = normal(case["rows"], case["cols"]) if case["residual"] else None
        s["p"] = case["p"]
        s["offset"] = 1 + (int(seed) % 1000)
    else:
        B, H, Hq, dk, dv = (case[n] for n in ("B", "heads", "qk_heads", "dk", "dv"))
        s["scale"] = dk ** -0.5
        s["log_decay"] = _log_decay(H, dev)
        if case["op"] == "token":
            s["q"], s["k"] = normal(B, Hq, dk), normal(B, Hq, dk, std=dk ** -0.5)
            s["v"] = normal(B, H, dv)
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
        s["q"], s["k"] = normal(T, B, Hq, dk), normal(T, B, Hq, dk, std=dk ** -0.5)
        s["v"] = normal(T, B, H, dv)
        s["state"] = normal(B, H, dk, dv, std=0.3, dtype=torch.float32) if case["state"] else None
        s["lens"] = None
        if case["ragged"]:
            lens = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            lens[0] = T
            if B > 2:
                lens[1], lens[2] = 0, 1
            s["lens"] = lens
        if case["op"] == "attn_grad":
            s["do"] = normal(T, B, H, dv, std=0.02)
            s["dstate"] = normal(B, H, dk, dv, std=0.02, dtype=torch.float32) \
                if case["state"] else None
    return s


# ---- plain forms --------------------------------------------------------------
def _norm(s):
    x = s["x"].float()
    n = x.shape[1]
    mean = x.sum(1) / n
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).sum(1) / n + EPS)
    return (c * rstd[:, None] * s["gamma"] + s["beta"]).to(s["x"].dtype), mean, rstd


def _norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    n = x.shape[1]
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"]
    dx = s["rstd"][:, None] * (g - (g.sum(1) / n)[:, None] - xhat * ((g * xhat).sum(1) / n)[:, None])
    return dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)


def _random_words(n, seed, offset, device):
    """The first n 32-bit words of Philox4x32-10 (Salmon et al., 2011) under the
    key `seed`: block i has the counter (i, offset), each 64 bits wide."""
    m32 = 0xFFFFFFFF
    i = torch.arange((n + 3) // 4, device=device, dtype=torch.int64)
    c0, c1 = i & m32, i >> 32
    c2, c3 = torch.full_like(i, offset & m32), torch.full_like(i, (offset >> 32) & m32)
    k0, k1 = seed & m32, (seed >> 32) & m32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m32) ^ c1 ^ k0, p1 & m32, ((p0 >> 32) & m32) ^ c3 ^ k1, p0 & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _dropout(s):
    x = s["x"].float()
    words = _random_words(x.numel(), s["seed"], s["offset"], x.device).reshape(x.shape)
    kept = words >= round(s["p"] * 2 ** 32)
    y = torch.where(kept, x * (1.0 / (1.0 - s["p"])), torch.zeros_like(x))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _powers(ld, e):
    """decay^e for log-decays [H] and exponents e [...]: [H, ...]."""
    return torch.exp(ld.reshape((-1,) + (1,) * e.dim()) * e)


def _mix(a, b, c, ld, x0=None):
    """out_t = sum_{s <= t} decay^(t-s) (a_t . b_s) c_s + decay^(t+1) a_t X0, in chunks:
    a, b [T,B,H,d], c [T,B,H,e], x0 [B,H,d,e]; fp32."""
    T, B, H, d = a.shape
    C = min(PLAIN_CHUNK, T)
    n = -(-T // C)

    def chunks(z):
        z = torch.cat([z, z.new_zeros((n * C - T,) + z.shape[1:])]) if n * C > T else z
        return z.reshape(n, C, B, H, z.shape[3]).permute(0, 2, 3, 1, 4)      # [n,B,H,C,d]

    a, b, c = chunks(a), chunks(b), chunks(c)
    i = torch.arange(C, device=a.device, dtype=torch.float32)
    gap = i[:, None] - i[None, :]
    mask = torch.where(gap >= 0, _powers(ld, gap.clamp(min=0)), torch.zeros((), device=a.device))
    out = torch.matmul(torch.matmul(a, b.transpose(-1, -2)) * mask, c)
    add = torch.matmul((b * _powers(ld, C - 1 - i)[..., None]).transpose(-1, -2), c)
    whole = _powers(ld, torch.full((1, 1), float(C), device=a.device))
    x, before = x0, []
    for m in range(n):
        before.append(x if x is not None else torch.zeros_like(add[0]))
        x = add[m] if x is None else x * whole + add[m]
    out = out + torch.matmul(a, torch.stack(before)) * _powers(ld, i + 1)[..., None]
    return out.permute(0, 3, 1, 2, 4).reshape(n * C, B, H, c.shape[-1])[:T]


def _attn_inputs(s):
    """fp32 copies with one query and key head per value head, zeros past each length;
    lengths [B]; 1 where a token counts [T,B,1,1]."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    T, B, H = v.shape[:3]
    g = H // q.shape[2]
    if g > 1:
        q, k = q.repeat_interleave(g, 2), k.repeat_interleave(g, 2)
    lens = s["lens"].float() if s["lens"] is not None else torch.full((B,), float(T), device=v.device)
    t = torch.arange(T, device=v.device, dtype=torch.float32)
    live = (t[:, None] < lens)[:, :, None, None]
    if s["lens"] is not None:
        zero = torch.zeros((), device=v.device)
        q, k, v = (torch.where(live, z, zero) for z in (q, k, v))
    return q, k, v, lens, live


def _attn(s):
    q, k, v, lens, live = _attn_inputs(s)
    T, ld = v.shape[0], s["log_decay"]
    o = _mix(q, k, v, ld, s["state"]) * s["scale"]
    t = torch.arange(T, device=v.device, dtype=torch.float32)
    w = _powers(ld, (lens - 1 - t[:, None]).clamp(min=0)).permute(1, 2, 0)[..., None]   # [T,B,H,1]
    end = torch.matmul((k * w).permute(1, 2, 3, 0), v.permute(1, 2, 0, 3))
    if s["state"] is not None:
        end = end + s["state"] * _powers(ld, lens).t()[..., None, None]
    if s["lens"] is not None:
        o = torch.where(live, o, torch.zeros((), device=o.device))
    return o.to(s["v"].dtype), end


def _attn_grad(s):
    q, k, v, lens, live = _attn_inputs(s)
    T, B, H = v.shape[:3]
    ld, scale = s["log_decay"], s["scale"]
    do = torch.where(live, s["do"].float(), torch.zeros((), device=v.device)) * scale
    t = torch.arange(T, device=v.device, dtype=torch.float32)
    x0 = s["state"].transpose(-1, -2) if s["state"] is not None else None
    dq = _mix(do, v, k, ld, x0)
    dk = _mix(v.flip(0), do.flip(0), q.flip(0), ld).flip(0)
    dv = _mix(k.flip(0), q.flip(0), do.flip(0), ld).flip(0)
    out = {}
    if s["state"] is not None:
        w = _powers(ld, (lens - 1 - t[:, None]).clamp(min=0)).permute(1, 2, 0)[..., None]
        end = s["dstate"]
        dk = dk + torch.matmul(v.permute(1, 2, 0, 3), end.transpose(-1, -2)).permute(2, 0, 1, 3) * w
        dv = dv + torch.matmul(k.permute(1, 2, 0, 3), end).permute(2, 0, 1, 3) * w
        u = _powers(ld, t + 1).t()[:, None, :, None]                                      # [T,1,H,1]
        out["dstate"] = torch.matmul((q * u).permute(1, 2, 3, 0), do.permute(1, 2, 0, 3)) \
            + end * _powers(ld, lens).t()[..., None, None]
    zero = torch.zeros((), device=v.device)
    dq, dk, dv = (torch.where(live, z, zero) for z in (dq, dk, dv))
    shared = s["q"].shape[2]
    if shared < H:
        dq, dk = (z.reshape(T, B, shared, H // shared, -1).sum(3) for z in (dq, dk))
    dt = s["v"].dtype
    out.update(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt))
    return out


def _token(s):
    q, k, v, state = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    g = v.shape[1] // q.shape[1]
    if g > 1:
        q, k = q.repeat_interleave(g, 1), k.repeat_interleave(g, 1)
    decay = torch.exp(s["log_decay"])[:, None, None]
    rows = torch.arange(v.shape[0], device=v.device)
    at = rows
    if s["slots"] is not None:
        live = s["slots"] >= 0
        rows, at = rows[live], s["slots"][live].long()
    new = state[at] * decay + k[rows][..., None] * v[rows][..., None, :]
    state[at] = new
    o = torch.zeros_like(v)
    o[rows] = (new * q[rows][..., None]).sum(2) * s["scale"]
    return o.to(s["v"].dtype), state


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm, "norm_grad": _norm_grad, "dropout": _dropout,
            "dropout_grad": _dropout, "attn": _attn, "attn_grad": _attn_grad, "token": _token}[s["op"]](s)


def _run_own(s):
    from persistent_rnn_recurrence_gb300 import prnn
    op = s["op"]
    if op == "norm":
        return prnn.layer_norm(s["x"], s["gamma"], s["beta"], EPS)
    if op == "norm_grad":
        return prnn.layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])
    if op == "dropout":
        return prnn.dropout(s["x"], s["p"], s["seed"], s["offset"], s["residual"])
    if op == "dropout_grad":
        return prnn.dropout_backward(s["x"], s["p"], s["seed"], s["offset"])
    if op == "attn":
        return prnn.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["scale"],
                                     s["state"], s["lens"])
    if op == "attn_grad":
        g = prnn.linear_attention_backward(s["do"], s["q"], s["k"], s["v"], s["log_decay"],
                                           s["scale"], s["state"], s["lens"], s["dstate"])
        if s["state"] is None:
            g.pop("dstate", None)
        return g
    o = prnn.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"],
                                   s["scale"], s["slots"])
    return o, s["state"]


# ---- what a pass cannot do without -------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op in ("norm", "norm_grad", "dropout", "dropout_grad"):
        n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
        if op == "norm":
            return {"bytes": 2 * n * e + 8 * cols + 8 * rows, "flops": 8 * n}
        if op == "norm_grad":
            return {"bytes": 3 * n * e + 12 * cols + 8 * rows, "flops": 14 * n}
        return {"bytes": (3 if case["residual"] else 2) * n * e, "flops": 3 * n}
    B, H, Hq, dk, dv = (case[n] for n in ("B", "heads", "qk_heads", "dk", "dv"))
    if op == "token":
        live = B - 1 if case["slots"] else B
        return {"bytes": live * (8 * H * dk * dv + e * (2 * Hq * dk + H * dv)) + e * B * H * dv,
                "flops": 5 * live * H * dk * dv}
    T = case["T"]
    qk, vo, st = T * B * Hq * dk * e, T * B * H * dv * e, 4 * B * H * dk * dv
    # one step costs a decayed rank-one update and a product with the state: 5 dk dv
    if op == "attn":
        return {"bytes": 2 * qk + 2 * vo + st * (2 if case["state"] else 1),
                "flops": 5 * T * B * H * dk * dv}
    return {"bytes": 4 * qk + 3 * vo + st * (3 if case["state"] else 0),
            "flops": 13 * T * B * H * dk * dv}


# ---- the definitions in 64 bits ----------------------------------------------------
def _exact_attn(s, grad):
    """Token by token.  Forward: S_t = decay S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.
    Gradients: dq_t = scale S_t do_t; with R_t = decay R_{t+1} + scale q_t do_t^T and
    R past the end = the gradient of the final state / decay: dk_t = R_t v_t,
    dv_t = R_t^T k_t, and the initial state's gradient is decay R_0."""
    f = torch.float64
    q, k, v = s["q"].to(f), s["k"].to(f), s["v"].to(f)
    T, B, H, dv = v.shape
    dk, g = q.shape[3], H // q.shape[2]
    head = torch.arange(H, device=v.device) // g
    decay = torch.exp(s["log_decay"].to(f))[None, :, None, None]
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device=v.device)
    S = s["state"].to(f).clone() if s["state"] is not None else torch.zeros(B, H, dk, dv, dtype=f,
                                                                         device=v.device)
    o = torch.zeros(T, B, H, dk if grad else dv, dtype=f, device=v.device)
    whole = s["lens"] is None
    for t in range(T):
        r = slice(None) if whole else (lens > t).nonzero()[:, 0]
        kt, vt = k[t][r][:, head], v[t][r]
        S[r] = S[r] * decay + kt[..., None] * vt[..., None, :]
        if grad:
            o[t, r] = s["scale"] * torch.matmul(S[r], s["do"][t][r].to(f)[..., None])[..., 0]
        else:
            o[t, r] = s["scale"] * torch.matmul(q[t][r][:, head][..., None, :], S[r])[..., 0, :]
    if not grad:
        return o, S
    dq, dkk, dvv = o, torch.zeros_like(o), torch.zeros(T, B, H, dv, dtype=f, device=v.device)
    # R is carried with the next decay already applied: R_t = carried + scale q_t do_t^T
    R = s["dstate"].to(f).clone() if s["dstate"] is not None else torch.zeros_like(S)
    for t in reversed(range(T)):
        r = slice(None) if whole else (lens > t).nonzero()[:, 0]
        full = R[r] + s["scale"] * q[t][r][:, head][..., None] * s["do"][t][r].to(f)[..., None, :]
        dkk[t, r] = torch.matmul(full, v[t][r][..., None])[..., 0]
        dvv[t, r] = torch.matmul(k[t][r][:, head][..., None, :], full)[..., 0, :]
        R[r] = full * decay
    out = {"dq": dq.reshape(T, B, H // g, g, dk).sum(3), "dk": dkk.reshape(T, B, H // g, g, dk).sum(3),
           "dv": dvv}
    if s["state"] is not None:
        out["dstate"] = R
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if op == "norm":
        x = s["x"].to(f)
        mean, var = x.mean(1), x.var(1, unbiased=False)
        rstd = (var + EPS).rsqrt()
        y = (x - mean[:, None]).mul_(rstd[:, None]).mul_(s["gamma"].to(f)).add_(s["beta"].to(f))
        return y, mean, rstd
    if op == "norm_grad":
        dy, gamma = s["dy"].to(f), s["gamma"].to(f)
        mean, rstd = s["mean"].to(f)[:, None], s["rstd"].to(f)[:, None]
        xhat = (s["x"].to(f) - mean) * rstd
        dgamma, dbeta = torch.einsum("rc,rc->c", dy, xhat), dy.sum(0)
        g = dy * gamma
        dot = torch.einsum("rc,rc->r", g, xhat) / g.shape[1]
        return (g - g.mean(1, keepdim=True) - xhat * dot[:, None]) * rstd, dgamma, dbeta
    if op in ("dropout", "dropout_grad"):
        # Philox4x32-10 once more, on unsigned 64-bit host integers
        import numpy as np
        n = s["x"].numel()
        if n > 100_000_000:
            return None
        u = np.uint64
        m32, sh = u(0xFFFFFFFF), u(32)
        kept = np.empty((n + 3) // 4 * 4, dtype=bool)
        limit = u(round(s["p"] * 2 ** 32))
        for lo in range(0, (n + 3) // 4, 1 << 20):
            c = np.zeros((4, min(1 << 20, (n + 3) // 4 - lo)), dtype=u)
            i = np.arange(lo, lo + c.shape[1], dtype=u)
            c[0], c[1], c[2], c[3] = i & m32, i >> sh, s["offset"] & 0xFFFFFFFF, s["offset"] >> 32
            key = [s["seed"] & 0xFFFFFFFF, (s["seed"] >> 32) & 0xFFFFFFFF]
            for _ in range(10):
                a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
                c = np.stack([(b >> sh) ^ c[1] ^ u(key[0]), b & m32, (a >> sh) ^ c[3] ^ u(key[1]), a & m32])
                key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
            kept[4 * lo:4 * (lo + c.shape[1])] = (c.T >= limit).reshape(-1)
        keep = torch.from_numpy(kept[:n]).to(s["x"].device).reshape(s["x"].shape)
        y = s["x"].to(f) / (1.0 - s["p"]) * keep
        return y if s["residual"] is None else y + s["residual"].to(f)
    if op in ("attn", "attn_grad"):
        return _exact_attn(s, op == "attn_grad")
    state = s["state"].to(f)
    g = s["v"].shape[1] // s["q"].shape[1]
    o = torch.zeros(s["v"].shape, dtype=f, device=s["v"].device)
    decay = torch.exp(s["log_decay"].to(f))
    for b in range(s["v"].shape[0]):
        at = b if s["slots"] is None else int(s["slots"][b])
        if at < 0:
            continue
        k, q = (s[n][b].to(f).repeat_interleave(g, 0) for n in ("k", "q"))
        state[at] = decay[:, None, None] * state[at] + torch.einsum("hd,he->hde", k, s["v"][b].to(f))
        o[b] = s["scale"] * torch.einsum("hd,hde->he", q, state[at])
    return o, state
