"""What the gated delta rule and the layer norm of this library are measured on.

The gated delta rule keeps one headdim x dstate fp32 state S per sequence and head:

    S' = exp(a_t) S,   e_t = v_t - S' k_t,   S = S' + beta_t e_t k_t^T,   y_t = scale S q_t

(the state-space dual with the delta correction: what S already answers for the key is
taken off the value before it is written).  The layer norm is the norm in front of such a
mixer (rows of the model's width) and behind it (one row per token and head):

    y = (x - mean) rstd weight + bias,   rstd = 1 / sqrt(var + eps)

``run`` computes them from elementary torch operations in 32 bits (``own`` false) or
calls the library (``own`` true).  The plain delta rule is the chunked form: everything
inside chunks of 64 tokens is a batched product, and only the state goes from chunk to
chunk in a loop, which the recurrence cannot do without.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64
EPS = 1e-5


def listed():
    return [
        # one layer of a 130m-sized model over its training batch (24 heads of 64, state 128)
        {"name": "fwd_block", "op": "delta_fwd", "batch": 8, "L": 2048, "heads": 24, "qk_heads": 24, "P": 64, "N": 128,
         "dtype": "bf16", "carried": False},
        # the prefill of one long prompt, continued from a carried state, key heads shared by two
        {"name": "fwd_long", "op": "delta_fwd", "batch": 1, "L": 32749, "heads": 16, "qk_heads": 8, "P": 128, "N": 128,
         "dtype": "bf16", "carried": True},
        # a short fp32 prompt: latency
        {"name": "fwd_short", "op": "delta_fwd", "batch": 2, "L": 37, "heads": 8, "qk_heads": 2, "P": 64, "N": 64,
         "dtype": "fp32", "carried": True},
        # the training step's backward of fwd_block
        {"name": "bwd_block", "op": "delta_bwd", "batch": 8, "L": 2048, "heads": 24, "qk_heads": 24, "P": 64, "N": 128,
         "dtype": "bf16", "carried": False},
        # fp32 gradients through a carried state, ragged length, shared key heads
        {"name": "bwd_ragged", "op": "delta_bwd", "batch": 3, "L": 1021, "heads": 8, "qk_heads": 4, "P": 128, "N": 64,
         "dtype": "fp32", "carried": True},
        # one decode token of a serving batch
        {"name": "step_batch", "op": "delta_step", "batch": 256, "ntok": 1, "heads": 24, "qk_heads": 24, "P": 64,
         "N": 128, "dtype": "bf16"},
        # a few drafted tokens of one sequence: latency
        {"name": "step_one", "op": "delta_step", "batch": 1, "ntok": 4, "heads": 16, "qk_heads": 8, "P": 128, "N": 128,
         "dtype": "bf16"},
        # the norm in front of the mixer, 16384 tokens of width 768
        {"name": "ln_fwd_block", "op": "ln_fwd", "rows": 16384, "dim": 768, "dtype": "bf16"},
        # the norm of the mixer's output, one row per token and head
        {"name": "ln_fwd_heads", "op": "ln_fwd", "rows": 393216, "dim": 64, "dtype": "bf16"},
        # one decode step's rows: latency
        {"name": "ln_fwd_few", "op": "ln_fwd", "rows": 8, "dim": 2560, "dtype": "fp32"},
        # the training step's norm gradient at width 2560
        {"name": "ln_bwd_wide", "op": "ln_bwd", "rows": 16384, "dim": 2560, "dtype": "bf16"},
        # fp32 gradients, an odd number of rows
        {"name": "ln_bwd_ragged", "op": "ln_bwd", "rows": 997, "dim": 5120, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_bwd", "delta_step", "ln_fwd", "ln_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("ln"):
        dim = _log_int(rng, 32, 8192)
        dim = dim if rng.random() < 0.3 else -(-dim // 64) * 64
        return {"op": op, "rows": _log_int(rng, 1, 24_000_000 // dim), "dim": dim, "dtype": dtype}
    qk = _log_int(rng, 1, 16)
    c = {"op": op, "heads": qk * rng.choice([1, 1, 2, 4]), "qk_heads": qk, "P": rng.choice([32, 64, 64, 96, 128, 128]),
         "N": rng.choice([32, 64, 64, 96, 128, 128]), "dtype": dtype}
    size = c["heads"] * c["P"] * c["N"]
    if op == "delta_step":
        c["batch"], c["ntok"] = _log_int(rng, 1, max(1, 50_000_000 // size)), rng.choice([1, 1, 1, 2, 4, 7])
        return c
    c["batch"], c["carried"] = rng.choice([1, 1, 2, 3, 8]), rng.random() < 0.5
    most = 3_000_000_000 if op == "delta_fwd" else 1_500_000_000     # token x state elements
    c["L"] = _log_int(rng, 1, max(1, min(32768 if op == "delta_fwd" else 8192, most // (size * c["batch"]))))
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    if case["op"].startswith("ln"):
        rows, dim = case["rows"], case["dim"]
        x = torch.randn((rows, dim), device="cuda", generator=g) * 1.5
        x += 0.5 * torch.randn(dim, device="cuda", generator=g)
        s = {"case": case, "x": x.to(dt), "weight": 1 + 0.2 * torch.randn(dim, device="cuda", generator=g),
             "bias": 0.2 * torch.randn(dim, device="cuda", generator=g)}
        if case["op"] == "ln_bwd":       # a training step holds the forward's statistics
            xd = s["x"].double()
            mean = xd.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (xd.sub_(mean[:, None]).square_().mean(1) + EPS).rsqrt().float()
            s["dy"] = torch.randn((rows, dim), device="cuda", generator=g).to(dt)
        return s
    H, K, P, N = case["heads"], case["qk_heads"], case["P"], case["N"]
    lead = (case["ntok"], case["batch"]) if case["op"] == "delta_step" else (case["batch"], case["L"])

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    # queries and keys of unit length, as such a mixer normalises them; heads that forget
    # within a few tokens beside heads that keep for a thousand
    s = {"case": case, "scale": N ** -0.5}
    for n in ("q", "k"):
        t = normal(*lead, K, N)
        s[n] = (t / t.norm(dim=-1, keepdim=True)).to(dt)
    s["v"] = normal(*lead, H, P).to(dt)
    rate = torch.exp(torch.empty(H, device="cuda").uniform_(math.log(1e-3), 0.0, generator=g))
    s["a"] = -torch.nn.functional.softplus(normal(*lead, H)) * rate
    s["beta"] = torch.sigmoid(normal(*lead, H))
    if case["op"] == "delta_step":
        s["state"] = 0.3 * normal(case["batch"], H, P, N)
        return s
    s["initial_state"] = 0.3 * normal(case["batch"], H, P, N) if case["carried"] else None
    if case["op"] == "delta_bwd":
        s["dy"] = normal(*lead, H, P).to(dt)
        s["dfinal_state"] = 0.3 * normal(case["batch"], H, P, N) if case["carried"] else None
    return s


# ---- plain forms ----------------------------------------------------------------------


def _per_head(t, heads):
    """[..., qk_heads, N] -> [..., heads, N]: head h reads key head h // (heads // qk_heads)."""
    return t.repeat_interleave(heads // t.shape[-2], dim=-2)


def _cut(t, C):
    """[batch, L, heads, ...] -> [batch, heads, chunks, C, ...] fp32, the tail zero."""
    t = t.float().transpose(1, 2)
    pad = -t.shape[2] % C
    if pad:
        t = torch.cat([t, t.new_zeros((*t.shape[:2], pad, *t.shape[3:]))], 2)
    return t.reshape(*t.shape[:2], t.shape[2] // C, C, *t.shape[3:])


def _join(t, L, dtype):
    """[batch, heads, chunks, C, ...] -> [batch, L, heads, ...]."""
    t = t.reshape(*t.shape[:2], t.shape[2] * t.shape[3], *t.shape[4:])[:, :, :L]
    return t.transpose(1, 2).contiguous().to(dtype)


def _chunk_parts(s):
    """The products inside the chunks: q, k, v, beta cut; the decays to, from and inside a
    chunk; the masked key and query products; and T, the inverse that solves for e."""
    H = s["v"].shape[2]
    C = CHUNK
    q, k = _cut(_per_head(s["q"], H), C) * s["scale"], _cut(_per_head(s["k"], H), C)
    v, beta = _cut(s["v"], C), _cut(s["beta"], C)
    G = _cut(s["a"], C).double().cumsum(-1)                  # differences of long sums: 64 bits
    lower = torch.ones(C, C, device=v.device).tril()
    ratio = torch.exp((G[..., :, None] - G[..., None, :]) * lower).float() * lower
    gam, end = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float()
    KK = (k @ k.transpose(-1, -2)) * ratio * lower.tril(-1)
    QK = (q @ k.transpose(-1, -2)) * ratio
    power = KK * beta[..., None, :]
    T = torch.eye(C, device=v.device) - power
    for _ in range(int(math.log2(C)) - 1):                   # (I + n)^-1 = (I - n)(I + n^2)(I + n^4) ...
        power = power @ power
        T = T + T @ power
    return q, k, v, beta, gam, end, KK, QK, T


def _forward(s, parts):
    """e of every token, the state before every chunk, and the last one."""
    q, k, v, beta, gam, end, KK, QK, T = parts
    W, V = T @ (k * gam[..., None]), T @ v
    write = (k * (beta * end)[..., None]).transpose(-1, -2)
    b, H, n = v.shape[:3]
    S = v.new_zeros((b, H, k.shape[-1], v.shape[-1]))        # [N, P]
    if s["initial_state"] is not None:
        S = s["initial_state"].transpose(-1, -2).contiguous()
    states, e = [], []
    for c in range(n):
        states.append(S)
        e.append(V[:, :, c] - W[:, :, c] @ S)
        S = gam[:, :, c, -1, None, None] * S + write[:, :, c] @ e[-1]
    return torch.stack(e, 2), torch.stack(states, 2), S


def _plain_fwd(s):
    q, k, v, beta, gam, end, KK, QK, T = parts = _chunk_parts(s)
    e, S0, S = _forward(s, parts)
    y = (q * gam[..., None]) @ S0 + QK @ (e * beta[..., None])
    return {"y": _join(y, s["v"].shape[1], s["v"].dtype), "final_state": S.transpose(-1, -2).contiguous()}


def _plain_bwd(s):
    q, k, v, beta, gam, end, KK, QK, T = parts = _chunk_parts(s)
    e, S0, S = _forward(s, parts)
    L, dt = s["v"].shape[1], s["v"].dtype
    do = _cut(s["dy"], CHUNK)
    b, H, n = v.shape[:3]
    # the adjoint of the state behind every chunk, and w = beta x (the adjoint of beta e)
    local = QK.transpose(-1, -2) @ do
    Tt = T.transpose(-1, -2)
    kend = k * end[..., None]
    read, wrote = (q * gam[..., None]).transpose(-1, -2), (k * gam[..., None]).transpose(-1, -2)
    dS = torch.zeros_like(S) if s["dfinal_state"] is None else s["dfinal_state"].transpose(-1, -2).contiguous()
    dends, ws = [None] * n, [None] * n
    for c in reversed(range(n)):
        dends[c] = dS
        ws[c] = Tt[:, :, c] @ (beta[:, :, c, :, None] * (kend[:, :, c] @ dS + local[:, :, c]))
        dS = gam[:, :, c, -1, None, None] * dS + read[:, :, c] @ do[:, :, c] - wrote[:, :, c] @ ws[c]
    dE, w = torch.stack(dends, 2), torch.stack(ws, 2)
    u = e * beta[..., None]
    lower = torch.ones(CHUNK, CHUNK, device=v.device).tril()
    G = _cut(s["a"], CHUNK).double().cumsum(-1)
    ratio = torch.exp((G[..., :, None] - G[..., None, :]) * lower).float() * lower
    M1 = (do @ u.transpose(-1, -2)) * ratio
    M2 = (w @ u.transpose(-1, -2)) * ratio * lower.tril(-1)
    from_start = gam[..., None] * (do @ S0.transpose(-1, -2))
    out_start = gam[..., None] * (w @ S0.transpose(-1, -2))
    to_end = end[..., None] * (e @ dE.transpose(-1, -2))
    dq = s["scale"] * (from_start + M1 @ k)
    dk = to_end * beta[..., None] + M1.transpose(-1, -2) @ q - out_start - M2.transpose(-1, -2) @ k - M2 @ k
    Xe = (do @ e.transpose(-1, -2)) * QK - (w @ e.transpose(-1, -2)) * KK
    Fe = (to_end * k).sum(-1)
    dbeta = Fe + Xe.sum(-2)
    # da_t is <adjoint, state> of the decayed state: what starts before t (a pair's source,
    # or the chunk's start) and ends at t or later (a pair's sink, or the chunk's end)
    X = Xe * beta[..., None, :]
    later = X.flip(-2).cumsum(-2).flip(-2)                   # sinks t' >= t of source s
    pairs = (later * lower.tril(-1)).sum(-1)
    starts = ((from_start * q).sum(-1) - (out_start * k).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    F = Fe * beta
    da = pairs + starts + (F.cumsum(-1) - F) + gam[..., -1:] * (dE * S0).sum((-1, -2))[..., None]
    K = s["k"].shape[2]

    def grouped(t):                                          # shared key heads: sum over their heads
        return _join(t.reshape(b, K, H // K, *t.shape[2:]).sum(2), L, dt)

    d = {"dq": grouped(dq), "dk": grouped(dk), "dv": _join(w, L, dt), "da": _join(da, L, torch.float32),
         "dbeta": _join(dbeta, L, torch.float32)}
    if s["initial_state"] is not None:
        d["dinitial_state"] = dS.transpose(-1, -2).contiguous()
    return d


def _plain_step(s):
    H, S, y = s["v"].shape[2], s["state"], torch.empty_like(s["v"])
    q, k, v = _per_head(s["q"], H).float(), _per_head(s["k"], H).float(), s["v"].float()
    alpha, beta = torch.exp(s["a"]), s["beta"]
    for t in range(v.shape[0]):
        S = S * alpha[t, :, :, None, None]
        e = v[t] - (S @ k[t, :, :, :, None])[..., 0]
        S = S + (beta[t, :, :, None] * e)[..., None] * k[t, :, :, None, :]
        y[t] = (s["scale"] * (S @ q[t, :, :, :, None])[..., 0]).to(y.dtype)
    s["state"].copy_(S)
    return {"y": y, "state": s["state"]}


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    return {"y": (c * rstd[:, None] * s["weight"] + s["bias"]).to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


_PLAIN = {"delta_fwd": _plain_fwd, "delta_bwd": _plain_bwd, "delta_step": _plain_step, "ln_fwd": _plain_ln_fwd,
          "ln_bwd": _plain_ln_bwd}


# ---- the library's calls --------------------------------------------------------------


def _own(s):
    import selective_state_space_45_b200 as ssm

    op = s["case"]["op"]
    if op == "delta_fwd":
        y, fs = ssm.delta_rule(s["q"], s["k"], s["v"], s["a"], s["beta"], initial_state=s["initial_state"],
                               scale=s["scale"], out_dtype=s["v"].dtype)
        return {"y": y, "final_state": fs}
    if op == "delta_bwd":
        d = ssm.delta_rule_bwd(s["dy"], s["q"], s["k"], s["v"], s["a"], s["beta"], initial_state=s["initial_state"],
                               dfinal_state=s["dfinal_state"], scale=s["scale"])
        return {n: t for n, t in d.items() if t is not None}
    if op == "delta_step":
        y = ssm.delta_rule_step(s["state"], s["q"], s["k"], s["v"], s["a"], s["beta"], scale=s["scale"],
                                out_dtype=s["v"].dtype)
        return {"y": y, "state": s["state"]}
    if op == "ln_fwd":
        y, mean, rstd = ssm.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, return_stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    return ssm.layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    size = {"bf16": 2, "fp32": 4}[case["dtype"]]
    if case["op"].startswith("ln"):
        rows, dim = case["rows"], case["dim"]
        if case["op"] == "ln_fwd":
            return {"bytes": 2 * rows * dim * size + 8 * dim + 8 * rows, "flops": 8 * rows * dim}
        return {"bytes": 3 * rows * dim * size + 12 * dim + 8 * rows, "flops": 14 * rows * dim}
    H, K, P, N = case["heads"], case["qk_heads"], case["P"], case["N"]
    if case["op"] == "delta_step":
        tok = case["ntok"] * case["batch"]
        # the state once in and out; per token two reads of the state and a rank-1 update
        return {"bytes": 8 * case["batch"] * H * P * N + tok * (2 * size * (K * N + H * P) + 8 * H),
                "flops": 7 * tok * H * P * N}
    tok = case["batch"] * case["L"]
    states = case["batch"] * H * P * N * 4
    if case["op"] == "delta_fwd":
        return {"bytes": tok * (2 * size * (K * N + H * P) + 8 * H) + states * (2 if case["carried"] else 1),
                "flops": 7 * tok * H * P * N}
    # q, k, v, dy, a, beta in; dq, dk, dv, da, dbeta out; the states are recomputed (one read
    # and one update), the adjoint is read twice and updated twice, the state read twice
    return {"bytes": tok * (size * (4 * K * N + 3 * H * P) + 16 * H) + states * (3 if case["carried"] else 0),
            "flops": 17 * tok * H * P * N}


# ---- the definition in 64 bits --------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(s)
    H = s["v"].shape[2]
    group = torch.arange(H, device="cuda") // (H // s["k"].shape[2])
    q, k, v = s["q"].double()[:, :, group], s["k"].double()[:, :, group], s["v"].double()
    alpha, beta, scale = s["a"].double().exp(), s["beta"].double(), s["scale"]

    def token(S, t, axis):
        """S before the token -> S after it, and e."""
        at = (lambda x: x[t]) if axis == 0 else (lambda x: x[:, t])
        S = S * at(alpha)[..., None, None]
        e = at(v) - torch.einsum("bhpn,bhn->bhp", S, at(k))
        return S + (at(beta)[..., None] * e)[..., None] * at(k)[..., None, :], e

    if case["op"] == "delta_step":
        S, y = s["state"].double(), torch.empty_like(v)
        for t in range(v.shape[0]):
            S, _ = token(S, t, 0)
            y[t] = scale * torch.einsum("bhpn,bhn->bhp", S, q[t])
        return {"y": y, "state": S}
    b, L, _, P = v.shape
    N = k.shape[-1]
    start = torch.zeros(b, H, P, N, device="cuda", dtype=torch.float64)
    if s["initial_state"] is not None:
        start = s["initial_state"].double()
    if case["op"] == "delta_fwd":
        S, y = start, torch.empty_like(v)
        for t in range(L):
            S, _ = token(S, t, 1)
            y[:, t] = scale * torch.einsum("bhpn,bhn->bhp", S, q[:, t])
        return {"y": y, "final_state": S}
    if b * L * H * P * N > 4e9:
        return None
    every, S, saved = 64, start, []
    for t in range(L):
        if t % every == 0:
            saved.append(S)
        S, _ = token(S, t, 1)
    dy = s["dy"].double()
    mu = torch.zeros_like(start) if s["dfinal_state"] is None else s["dfinal_state"].double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    da, dbeta = torch.empty_like(alpha), torch.empty_like(beta)
    for c in reversed(range(len(saved))):
        states, es = [saved[c]], []
        for t in range(c * every, min(L, (c + 1) * every)):
            S, e = token(states[-1], t, 1)
            states.append(S)
            es.append(e)
        for t in reversed(range(c * every, min(L, (c + 1) * every))):
            i = t - c * every
            before = states[i] * alpha[:, t, :, None, None]
            dq[:, t] = scale * torch.einsum("bhpn,bhp->bhn", states[i + 1], dy[:, t])
            lam = mu + scale * dy[:, t][..., None] * q[:, t][..., None, :]           # adjoint of S_t
            lk = torch.einsum("bhpn,bhn->bhp", lam, k[:, t])
            de = beta[:, t][..., None] * lk
            dbeta[:, t] = (lk * es[i]).sum(-1)
            dv[:, t] = de
            dk[:, t] = torch.einsum("bhpn,bhp->bhn", lam, beta[:, t][..., None] * es[i]) - torch.einsum(
                "bhpn,bhp->bhn", before, de)
            lam = lam - de[..., None] * k[:, t][..., None, :]                        # adjoint of S'
            da[:, t] = (lam * before).sum((-1, -2))
            mu = alpha[:, t, :, None, None] * lam
    Kh = s["k"].shape[2]
    d = {"dq": dq.reshape(b, L, Kh, H // Kh, N).sum(3), "dk": dk.reshape(b, L, Kh, H // Kh, N).sum(3), "dv": dv,
         "da": da, "dbeta": dbeta}
    if s["initial_state"] is not None:
        d["dinitial_state"] = mu
    return d


def _exact_ln(s):
    x, w = s["x"].double(), s["weight"].double()
    if s["case"]["op"] == "ln_fwd":
        mean = x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)
        return {"y": (x - mean) * rstd * w + s["bias"].double(), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    # with respect to x through the given statistics' definitions
    dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    h = (x - mean) * rstd
    gw = dy * w
    n = x.shape[1]
    dx = (gw - gw.sum(1, keepdim=True) / n - h * (gw * h).sum(1, keepdim=True) / n) * rstd
    return {"dx": dx, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}
