"""The gated delta rule and what prepares its queries and keys, as cases to be timed and compared.

Each case is one call of one operator:
  delta            S_t = e^g_t S_{t-1} + beta_t (v_t - e^g_t S_{t-1} k_t) k_t^T, o_t = scale S_t q_t over [B, H, T, d],
                   or over sequences packed along T
  delta_backward   its gradient (dq, dk, dv, dg, dbeta, dS0)
  delta_step       one token of it on a cache of states
  rotary           RMS norm of each head of queries and keys, and the rotation by position, token rows to head rows
  rotary_backward  its gradient (dq, dk, and those of the two weights)

`own` chooses between the plain form (elementary torch operations in 32 bits, the angles in 64) and the framework's
calls.  H heads of values share Hk heads of queries and keys.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
CHUNK = 64  # tokens that the plain form takes at once


def listed():
    return [
        # a short prompt in 32 bits, with the state of what came before it
        {"name": "delta_short", "op": "delta", "B": 1, "H": 4, "Hk": 4, "T": 150, "dk": 64, "dv": 64, "dtype": "f32", "gate": "f32"},
        # prefill: 8 prompts of 4096 tokens
        {"name": "delta_prompt", "op": "delta", "B": 8, "H": 16, "Hk": 16, "T": 4096, "dk": 128, "dv": 128, "dtype": "bf16", "gate": "f32"},
        # a long single sequence
        {"name": "delta_long", "op": "delta", "B": 1, "H": 16, "Hk": 16, "T": 65536, "dk": 128, "dv": 128, "dtype": "bf16", "gate": "f32"},
        # serving: 37 prompts of mixed lengths in one call, four heads of values to each head of keys
        {"name": "delta_packed", "op": "delta", "B": 37, "H": 16, "Hk": 4, "T": 9001, "dk": 128, "dv": 128, "dtype": "bf16", "gate": "bf16", "packed": True},
        # training: 8 sequences of 4096 tokens
        {"name": "delta_backward", "op": "delta_backward", "B": 8, "H": 16, "Hk": 16, "T": 4096, "dk": 128, "dv": 128, "dtype": "bf16", "gate": "f32"},
        # training in 32 bits, ragged, shared heads of keys, values wider than keys
        {"name": "delta_backward_ragged", "op": "delta_backward", "B": 2, "H": 6, "Hk": 3, "T": 777, "dk": 64, "dv": 128, "dtype": "f32", "gate": "f32"},
        # decoding: 256 sequences of 16 heads, one token each
        {"name": "delta_step", "op": "delta_step", "B": 256, "H": 16, "Hk": 16, "dk": 128, "dv": 128, "dtype": "bf16", "gate": "f32"},
        # decoding one sequence
        {"name": "delta_step_one", "op": "delta_step", "B": 1, "H": 16, "Hk": 8, "dk": 128, "dv": 128, "dtype": "bf16", "gate": "bf16"},
        # prefill: 8 prompts of 4096 tokens, heads between the gates' and values' columns of one projection
        {"name": "rotary_prompt", "op": "rotary", "B": 8, "T": 4096, "H": 16, "Hk": 16, "d": 128, "rot": 128, "pairs": "halves", "dtype": "bf16"},
        # decoding: 256 sequences far into their contexts, one token each
        {"name": "rotary_step", "op": "rotary", "B": 256, "T": 1, "H": 16, "Hk": 4, "d": 128, "rot": 64, "pairs": "halves", "dtype": "bf16"},
        # training: 8 sequences of 4096 tokens
        {"name": "rotary_backward", "op": "rotary_backward", "B": 8, "T": 4096, "H": 16, "Hk": 16, "d": 128, "rot": 128, "pairs": "halves", "dtype": "bf16"},
        # training in 32 bits, a head width that is no power of two, a part of it rotated in neighbouring pairs
        {"name": "rotary_backward_ragged", "op": "rotary_backward", "B": 3, "T": 517, "H": 6, "Hk": 2, "d": 80, "rot": 32, "pairs": "neighbours", "dtype": "f32"},
    ]


def _log(rng, low, high):
    return max(1, int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high)))))))


def draw(rng):
    op = rng.choice(("delta", "delta", "delta", "delta_backward", "delta_backward", "delta_step", "rotary", "rotary_backward"))
    c = {"op": op, "dtype": rng.choice(("f32", "bf16", "bf16"))}
    c["Hk"] = rng.choice((1, 2, 3, 4, 8, 16))
    c["H"] = c["Hk"] * rng.choice((1, 1, 2, 3)) if c["Hk"] <= 8 else c["Hk"]
    if op.startswith("rotary"):
        c["d"], c["pairs"] = rng.choice((32, 64, 80, 128, 128, 256)), rng.choice(("halves", "neighbours"))
        c["rot"] = rng.choice((c["d"], c["d"] // 2 // 16 * 16))
        c["B"] = _log(rng, 1, 64)
        c["T"] = _log(rng, 1, min(8192, 2 ** 26 // ((c["H"] + c["Hk"]) * c["d"] * c["B"])))
        return c
    c["gate"], c["dk"], c["dv"] = rng.choice(("f32", "bf16")), rng.choice((32, 64, 128, 128)), rng.choice((32, 64, 128, 128))
    if op == "delta_step":
        c["B"] = _log(rng, 1, 256)
        return c
    c["B"] = _log(rng, 1, 64)
    c["T"] = _log(rng, 1, min(16384, 2 ** 25 // (c["B"] * c["H"] * c["dv"])))
    if op == "delta" and rng.random() < 0.3:
        c["packed"], c["T"] = True, c["T"] * c["B"]
    return c


# ---------------------------------------------------------------- inputs

def _lengths(n, total, g):
    """n lengths of very different sizes with that sum"""
    w = torch.rand(n, generator=g, device="cuda").double().mul(-3).exp().cumsum(0)
    ends = (w / w[-1] * total).round().int()
    ends[-1] = total
    return torch.cat((ends.new_zeros(1), ends))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    op, t, B, H, Hk = case["op"], TYPES[case["dtype"]], case["B"], case["H"], case["Hk"]
    st = {"case": case}
    if op.startswith("rotary"):
        T, d, rot = case["T"], case["d"], case["rot"]
        z = normal(B, T, 8 + (H + Hk) * d + 64).to(t)  # token rows of a projection: gates, q, k, values
        st["q"] = z[..., 8:8 + H * d].unflatten(-1, (H, d))
        st["k"] = z[..., 8 + H * d:8 + (H + Hk) * d].unflatten(-1, (Hk, d))
        st["q_weight"], st["k_weight"] = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d)
        first = torch.randint(0, 100000, (B, 1), generator=g, device="cuda", dtype=torch.int32)
        st["position"] = first + torch.arange(T, device="cuda", dtype=torch.int32)
        st["inv_freq"] = 10000.0 ** (-2 * torch.arange(rot // 2, device="cuda") / max(rot, 1))
        if op == "rotary_backward":
            st["dq"], st["dk"] = normal(B, H, T, d).to(t), normal(B, Hk, T, d).to(t)
            for n in "qk":
                st[n + "_rstd"] = (st[n].float().square().mean(-1) + EPS).rsqrt().transpose(1, 2).contiguous()
        return st
    dk, dv, tg = case["dk"], case["dv"], TYPES[case["gate"]]
    if op == "delta_step":
        lead, S_lead = ((B, Hk), (B, H)), B
    elif case.get("packed"):
        st["cu_seqlens"] = _lengths(B, case["T"], g)
        st["lengths"] = st["cu_seqlens"].diff().tolist()
        lead, S_lead = ((Hk, case["T"]), (H, case["T"])), B
    else:
        lead, S_lead = ((B, Hk, case["T"]), (B, H, case["T"])), B
    st["q"] = torch.nn.functional.normalize(normal(*lead[0], dk), dim=-1).to(t)
    st["k"] = torch.nn.functional.normalize(normal(*lead[0], dk), dim=-1).to(t)
    st["v"] = normal(*lead[1], dv).to(t)
    rate = 0.02 if case.get("T", 1) > 8192 else 0.1
    st["g"] = (-rate * torch.nn.functional.softplus(normal(*lead[1]))).to(tg)
    st["beta"] = torch.sigmoid(normal(*lead[1])).to(tg)
    st["S0"] = 0.3 * normal(S_lead, H, dv, dk)
    if op == "delta_backward":
        st["do"], st["dS_T"] = normal(*lead[1], dv).to(t), 0.3 * normal(B, H, dv, dk)
    return st


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    import kalman_filter_memory_amd as kdn

    op = st["case"]["op"]
    if op == "delta":
        if "cu_seqlens" in st:
            return kdn.gated_delta_varlen(st["q"], st["k"], st["v"], st["g"], st["beta"], st["cu_seqlens"], st["S0"])
        return kdn.gated_delta(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"])
    if op == "delta_backward":
        return kdn.gated_delta_backward(st["q"], st["k"], st["v"], st["g"], st["beta"], st["do"], st["S0"], st["dS_T"])
    if op == "delta_step":
        return kdn.gated_delta_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"]), st["S0"]
    a = (st["q"], st["k"], st["q_weight"], st["k_weight"])
    how = {"eps": EPS, "interleaved": st["case"]["pairs"] == "neighbours"}
    if op == "rotary":
        return kdn.qk_norm_rotary(*a, st["position"], st["inv_freq"], **how)
    del how["eps"]
    return kdn.qk_norm_rotary_backward(st["dq"], st["dk"], *a, st["position"], st["inv_freq"], st["q_rstd"], st["k_rstd"], **how)


# ---------------------------------------------------------------- the plain form

def _to_chunks(x, T):
    """[B, H, T, ...] -> [B, H, chunks, CHUNK, ...] in 32 bits, zeros behind the last token: they leave a state as it is."""
    n = -(-T // CHUNK)
    x = torch.cat((x.float(), x.new_zeros(*x.shape[:2], n * CHUNK - T, *x.shape[3:], dtype=torch.float32)), 2)
    return x.unflatten(2, (n, CHUNK))


def _inverse(A):
    """(1 + A)^-1 of strictly lower triangular matrices: pairs of inverted diagonal blocks are joined, 1, 2, 4 .. rows at a time."""
    n = A.shape[-1]
    X = torch.eye(n, device=A.device).expand(A.shape).clone()
    s = 1
    while s < n:
        i = torch.arange(n, device=A.device)
        low = ((i[:, None] // s == i[None] // s + 1) & (i[:, None] // (2 * s) == i[None] // (2 * s))).float()
        X = X - X @ (A * low) @ X
        s *= 2
    return X


class _Plain:
    """What every chunk needs apart from the state, for all chunks at once."""

    def __init__(self, q, k, v, g, beta, T):
        r = v.shape[1] // k.shape[1]
        self.q, self.k = (_to_chunks(x.repeat_interleave(r, 1), T) for x in (q, k))
        self.v, self.g, self.beta = (_to_chunks(x, T) for x in (v, g, beta))
        self.scale = q.shape[-1] ** -0.5
        G = self.g.cumsum(-1)
        i = torch.arange(CHUNK, device=q.device)
        self.keep, self.before = i[:, None] >= i[None], i[:, None] > i[None]
        self.ratio = torch.where(self.keep, G[..., :, None] - G[..., None, :], 0).exp() * self.keep
        self.gamma, self.rest, self.last = G.exp(), (G[..., -1:] - G).exp(), G[..., -1].exp()
        self.L = (self.k @ self.k.transpose(-1, -2).contiguous()) * self.ratio * self.before
        self.X = _inverse(self.beta[..., None] * self.L)
        self.P = self.scale * (self.q @ self.k.transpose(-1, -2).contiguous()) * self.ratio

    def states(self, S):
        """U of every chunk, the states before them and the last one (S here [dk, dv])"""
        V = self.X @ (self.beta[..., None] * self.v)
        W = self.X @ ((self.beta * self.gamma)[..., None] * self.k)
        K = (self.rest[..., None] * self.k).transpose(-1, -2).contiguous()
        U, before = torch.empty_like(V), S.new_empty(*S.shape[:2], V.shape[2], *S.shape[2:])
        for c in range(V.shape[2]):
            before[:, :, c] = S
            U[:, :, c] = V[:, :, c] - W[:, :, c] @ S
            S = self.last[:, :, c, None, None] * S + K[:, :, c] @ U[:, :, c]
        return U, before, S


def _plain_delta(q, k, v, g, beta, S0):
    T = q.shape[2]
    p = _Plain(q, k, v, g, beta, T)
    U, S, last = p.states(S0.transpose(-1, -2).contiguous())
    o = p.scale * p.gamma[..., None] * (p.q @ S) + p.P @ U
    return o.flatten(2, 3)[:, :, :T].to(v.dtype), last.transpose(-1, -2).contiguous()


def _plain_delta_backward(q, k, v, g, beta, do, S0, dS_T):
    T, r = q.shape[2], v.shape[1] // q.shape[1]
    p = _Plain(q, k, v, g, beta, T)
    U, S, last = p.states(S0.transpose(-1, -2).contiguous())
    do = _to_chunks(do, T)
    Kt, Xt = (x.transpose(-1, -2).contiguous() for x in (p.k, p.X))
    from_o = p.P.transpose(-1, -2).contiguous() @ do
    into_S = (p.scale * p.gamma[..., None] * p.q).transpose(-1, -2).contiguous() @ do
    bg, K = (p.beta * p.gamma)[..., None], p.rest[..., None] * p.k
    X, after = torch.empty_like(p.v), torch.empty_like(S)  # gradients of beta (v - ..) and of the state behind each chunk
    D = dS_T.transpose(-1, -2).contiguous()
    for c in reversed(range(X.shape[2])):
        after[:, :, c] = D
        X[:, :, c] = Xt[:, :, c] @ (from_o[:, :, c] + K[:, :, c] @ D)
        D = p.last[:, :, c, None, None] * D + into_S[:, :, c] - Kt[:, :, c] @ (bg[:, :, c] * X[:, :, c])
    St, Dt, Ut = (x.transpose(-1, -2).contiguous() for x in (S, after, U))
    dv = p.beta[..., None] * X
    dP = (p.scale * (do @ Ut)) * p.ratio
    dL = -(dv @ Ut) * p.ratio * p.before
    from_S = p.scale * p.gamma[..., None] * (do @ St)
    dq = from_S + dP @ p.k
    to_S = p.rest[..., None] * (U @ Dt)
    error_S = p.gamma[..., None] * (p.k @ S)  # what the state says of v
    dk = dP.transpose(-1, -2).contiguous() @ p.q + to_S - p.gamma[..., None] * (dv @ St) + dL @ p.k + dL.transpose(-1, -2).contiguous() @ p.k
    dbeta = (X * (p.v - error_S - p.L @ U)).sum(-1)
    # log gamma_t: through o_t and the right side of row t, and as the divisor of u_t
    dlog = (dq * p.q).sum(-1) - (dv * p.v).sum(-1)
    end = torch.cat((S[:, :, 1:], last[:, :, None]), 2)
    dg = dlog.flip(-1).cumsum(-1).flip(-1) + (after * end).sum((-1, -2))[..., None]
    flat = lambda x, t: x.flatten(2, 3)[:, :, :T].to(t)  # noqa: E731
    shared = lambda x: x.unflatten(1, (-1, r)).sum(2)  # noqa: E731
    t = q.dtype
    return {"dq": flat(shared(dq), t), "dk": flat(shared(dk), t), "dv": flat(dv, t), "dg": flat(dg, t), "dbeta": flat(dbeta, t),
            "dS0": D.transpose(-1, -2).contiguous()}


def _padded(st):
    """Packed inputs as a batch: zeros behind each sequence, and where each row comes from."""
    longest = max(st["lengths"])
    at = st["cu_seqlens"][:-1, None] + torch.arange(longest, device="cuda")
    real = at < st["cu_seqlens"][1:, None]
    at = torch.where(real, at, 0).long()
    batch = lambda x: (x[:, at].transpose(0, 1) * real.view(real.shape[0], 1, longest, *[1] * (x.dim() - 2)))  # noqa: E731
    return at, real, [batch(st[n]) for n in ("q", "k", "v", "g", "beta")]


def _angles(st):
    a = st["position"].double()[..., None] * st["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, rot, pairs):
    """x [B, T, H, d], its first `rot` columns turned by the angles, cos and sin [B, T, rot / 2]"""
    cos, sin, head = cos[:, :, None], sin[:, :, None], x[..., :rot]
    if pairs == "halves":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., rot:]), -1)


def run(st):
    if own:
        return _own(st)
    c = st["case"]
    op = c["op"]
    if op == "delta":
        if "cu_seqlens" not in st:
            return _plain_delta(*(st[n] for n in ("q", "k", "v", "g", "beta", "S0")))
        at, real, x = _padded(st)
        o, S = _plain_delta(*x, st["S0"])
        out = torch.empty_like(st["v"])
        out[:, at[real]] = o.transpose(0, 1)[:, real]
        return out, S
    if op == "delta_backward":
        return _plain_delta_backward(*(st[n] for n in ("q", "k", "v", "g", "beta", "do", "S0", "dS_T")))
    if op == "delta_step":
        r = c["H"] // c["Hk"]
        q, k = (st[n].float().repeat_interleave(r, 1)[:, :, None] for n in "qk")
        S = st["S0"] * st["g"].float().exp()[..., None, None]
        u = st["beta"].float()[..., None] * (st["v"].float() - (S * k).sum(-1))
        st["S0"].copy_(S + u[..., None] * k)
        return (c["dk"] ** -0.5 * (st["S0"] * q).sum(-1)).to(st["v"].dtype), st["S0"]
    cos, sin = _angles(st)
    if op == "rotary":
        out, rstds = [], []
        for n in "qk":
            x = st[n].float()
            rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
            y = _rotate(x * rstd * st[n + "_weight"], cos, sin, c["rot"], c["pairs"])
            out.append(y.to(st[n].dtype).transpose(1, 2).contiguous())
            rstds.append(rstd[..., 0].transpose(1, 2).contiguous())
        return (*out, *rstds)
    dx, dw = [], []
    for n in "qk":
        xhat = st[n].float() * st[n + "_rstd"].transpose(1, 2)[..., None]
        dn = _rotate(st["d" + n].float().transpose(1, 2), cos, -sin, c["rot"], c["pairs"])
        dw.append((dn * xhat).sum((0, 1, 2)))
        dn = dn * st[n + "_weight"]
        d = st[n + "_rstd"].transpose(1, 2)[..., None] * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
        dx.append(d.to(st[n].dtype))
    return (*dx, *dw)


# ---------------------------------------------------------------- 64 bits

def _exact_tokens(q, k, v, a, beta, S, at, n):
    """The recurrence over tokens at .. at + n, from S: o, the states before each token and the last one."""
    o, kept = [], []
    for t in range(at, at + n):
        kept.append(S)
        kt = k[:, :, t, :, None]
        S = S * a[:, :, t, None, None]
        S = torch.baddbmm(S.flatten(0, 1), (beta[:, :, t, None, None] * (v[:, :, t, :, None] - S @ kt)).flatten(0, 1),
                          kt.flatten(0, 1).transpose(1, 2).contiguous()).view(S.shape)
        o.append((S @ q[:, :, t, :, None])[..., 0])
    return o, kept, S


def _exact_delta(q, k, v, g, beta, S):
    r, T = v.shape[1] // k.shape[1], v.shape[2]
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    a, o = g.exp(), torch.empty_like(v)
    for at in range(0, T, 64):
        n = min(64, T - at)
        part, _, S = _exact_tokens(q, k, v, a, beta, S, at, n)
        o[:, :, at:at + n] = torch.stack(part, 2) / math.sqrt(q.shape[-1])
    return o, S


def _exact_delta_backward(q, k, v, g, beta, do, S, dS):
    """Token by token from the last: the states between are computed again, 64 tokens at a time."""
    r, T = v.shape[1] // k.shape[1], v.shape[2]
    q, k, v, g, beta, do, S, D = (x.double() for x in (q, k, v, g, beta, do, S, dS))
    q, k, do = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1), do / math.sqrt(q.shape[-1])
    a, starts = g.exp(), []
    for at in range(0, T, 64):
        starts.append(S)
        S = _exact_tokens(q, k, v, a, beta, S, at, min(64, T - at))[2]
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, g, beta))
    for at in reversed(range(0, T, 64)):
        n = min(64, T - at)
        _, kept, S = _exact_tokens(q, k, v, a, beta, starts[at // 64], at, n)
        for t in reversed(range(at, at + n)):
            kt, qt, dot = k[:, :, t, :, None], q[:, :, t, :, None], do[:, :, t, :, None]
            dq[:, :, t] = (dot.transpose(2, 3).contiguous() @ S)[:, :, 0]
            D = D + dot * qt.transpose(2, 3)
            old = kept[t - at] * a[:, :, t, None, None]  # the state that token t corrects
            e = v[:, :, t, :, None] - old @ kt
            Dk, b = D @ kt, beta[:, :, t, None, None]
            db[:, :, t] = (Dk * e).sum((2, 3))
            dv[:, :, t] = (b * Dk)[..., 0]
            dk[:, :, t] = (b * ((e.transpose(2, 3).contiguous() @ D) - (Dk.transpose(2, 3).contiguous() @ old)))[:, :, 0]
            D = D - (b * Dk) * kt.transpose(2, 3)
            dg[:, :, t] = (D * old).sum((2, 3))
            D = D * a[:, :, t, None, None]
            S = kept[t - at]
    shared = lambda x: x.unflatten(1, (-1, r)).sum(2)  # noqa: E731
    return {"dq": shared(dq), "dk": shared(dk), "dv": dv, "dg": dg, "dbeta": db, "dS0": D}


def _exact_turn(st):
    """cos and sin as the complex numbers that a pair is multiplied by, [B, T, 1, rot / 2]"""
    a = st["position"].double()[..., None] * st["inv_freq"].double()
    return torch.polar(torch.ones_like(a), a)[:, :, None]


def _exact_pairs(x, c, turn):
    rot, y = c["rot"], x.clone()
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if c["pairs"] == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "delta":
        names = ("q", "k", "v", "g", "beta")
        if "cu_seqlens" not in st:
            return _exact_delta(*(st[n] for n in names), st["S0"])
        if case["T"] > 100000:
            return None
        o, S, at = torch.empty(st["v"].shape, dtype=torch.float64, device="cuda"), st["S0"].double(), 0
        for i, n in enumerate(st["lengths"]):
            part = _exact_delta(*(st[x][None, :, at:at + n] for x in names), st["S0"][i:i + 1])
            o[:, at:at + n], S[i], at = part[0][0], part[1][0], at + n
        return o, S
    if op == "delta_backward":
        return _exact_delta_backward(*(st[n] for n in ("q", "k", "v", "g", "beta", "do", "S0", "dS_T")))
    if op == "delta_step":
        names = ("q", "k", "v", "g", "beta")
        o, S = _exact_delta(*(st[n][:, :, None] for n in names), st["S0"])
        return o[:, :, 0], S
    turn = _exact_turn(st)
    if op == "rotary":
        out, rstds = [], []
        for n in "qk":
            x = st[n].double()
            rstd = 1 / torch.sqrt((x * x).sum(-1) / case["d"] + EPS)
            out.append(_exact_pairs(torch.einsum("bthd,bth,d->bthd", x, rstd, st[n + "_weight"].double()), case, turn).transpose(1, 2))
            rstds.append(rstd.transpose(1, 2))
        return (*out, *rstds)
    dx, dw = [], []
    for n in "qk":
        # y = turn(x r w) with r = (mean x^2 + eps)^(-1/2), dr/dx = -r^3 x / d, at the kept r
        x, r, w = st[n].double(), st[n + "_rstd"].double().transpose(1, 2)[..., None], st[n + "_weight"].double()
        back = _exact_pairs(st["d" + n].double().transpose(1, 2), case, turn.conj())
        dw.append((back * x * r).sum((0, 1, 2)))
        along = (back * w * x).sum(-1, keepdim=True)
        dx.append(back * w * r - x * (along * r ** 3 / case["d"]))
    return (*dx, *dw)


def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    e, B, H, Hk = size[case["dtype"]], case["B"], case["H"], case["Hk"]
    if op.startswith("rotary"):
        rows, d = B * case["T"] * (H + Hk), case["d"]
        side = 4 * B * case["T"] + 4 * rows + 8 * d + 2 * case["rot"]
        if op == "rotary":
            return {"bytes": 2 * rows * d * e + side, "flops": 8 * rows * d}
        return {"bytes": 3 * rows * d * e + side + 8 * d, "flops": 16 * rows * d}
    dk, dv, eg = case["dk"], case["dv"], size[case["gate"]]
    states = 4 * B * H * dk * dv
    tokens = B if op == "delta_step" else case["T"] if case.get("packed") else B * case["T"]
    rows = e * tokens * (2 * Hk * dk + 2 * H * dv) + 2 * eg * tokens * H
    if op != "delta_backward":
        # per token and head: the correction, the write and the read-out are dk dv products each
        return {"bytes": rows + 2 * states, "flops": 6 * tokens * H * dk * dv}
    # read q, k, v, do, the gates and two states; write dq, dk, dv, dg, dbeta and a state
    return {"bytes": rows + e * tokens * (2 * Hk * dk + H * dv) + 2 * e * tokens * H + 3 * states, "flops": 18 * tokens * H * dk * dv}
