"""The gated delta rule and its gradient in 64 bits, token by token, and bounds on the
float32 kernels' errors (used by the tests of gated_delta and its backward)."""
from __future__ import annotations

import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def shared(x, H):
    """heads of queries and keys, one for each head of values"""
    return x.repeat_interleave(H // x.shape[1], 1) if x.shape[1] else x.new_zeros(x.shape[0], H, *x.shape[2:])


def delta(q, k, v, g, beta, S0=None, scale=None):
    """(o, S_T, all states) in 64 bits; q, k [B,Hk,T,dk]"""
    H, T = v.shape[1], v.shape[2]
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    q, k, v, g, beta = (x.double() for x in (shared(q, H), shared(k, H), v, g, beta))
    S = v.new_zeros(*v.shape[:2], v.shape[-1], q.shape[-1]) if S0 is None else S0.double()
    o, kept = torch.empty_like(v), [S]
    for t in range(T):
        kt = k[:, :, t, None, :]
        S = S * g[:, :, t, None, None].exp()
        S = S + beta[:, :, t, None, None] * (v[:, :, t, :, None] - (S * kt).sum(-1, keepdim=True)) * kt
        o[:, :, t] = scale * (S * q[:, :, t, None, :]).sum(-1)
        kept.append(S)
    return o, S, kept


def delta_gradients(q, k, v, g, beta, do, S0=None, dS_T=None, scale=None):
    """Gradients of <do, o> + <dS_T, S_T> in 64 bits by the chain rule of one token"""
    H, T = v.shape[1], v.shape[2]
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    _, _, kept = delta(q, k, v, g, beta, S0, scale)
    Hk = q.shape[1]
    q, k, v, g, beta, do = (x.double() for x in (shared(q, H), shared(k, H), v, g, beta, do))
    D = torch.zeros_like(kept[0]) if dS_T is None else dS_T.double()
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    for t in reversed(range(T)):
        kt, qt, w = k[:, :, t, None, :], q[:, :, t, None, :], scale * do[:, :, t, :, None]
        dq[:, :, t] = (kept[t + 1] * w).sum(-2)
        D = D + w * qt
        old = kept[t] * g[:, :, t, None, None].exp()
        e = v[:, :, t, :, None] - (old * kt).sum(-1, keepdim=True)
        Dk, b = (D * kt).sum(-1, keepdim=True), beta[:, :, t, None, None]
        db[:, :, t] = (Dk * e).sum((2, 3))
        dv[:, :, t] = (b * Dk)[..., 0]
        dk[:, :, t] = (b * (e * D - Dk * old)).sum(-2)
        D = D - b * Dk * kt
        dg[:, :, t] = (D * old).sum((2, 3))
        D = D * g[:, :, t, None, None].exp()
    r = H // Hk
    return {"dq": dq.unflatten(1, (Hk, r)).sum(2), "dk": dk.unflatten(1, (Hk, r)).sum(2), "dv": dv, "dg": dg,
            "dbeta": db, "dS0": D}


def state_errors(q, k, v, g, beta, kept):
    """(D, s): per head, a bound on |error of S_t|_F for each t, and the largest |S_t|_F.

    For beta |k|^2 <= 2 a token's map S -> a S (I - beta k k^T) does not lengthen S, so
    errors add up: D_t = a_t D_{t-1} + new.  In a block of 32 tokens the kernels solve
    (I + L beta) E = V - gamma K S.  A dot product of up to 128 terms in planes costs at
    most 70 u of its |.||.| (4 x 6 accumulations of a 32-term sum, the dropped products
    below 2^-24, and the sum's own tree); decays from differences of sums of logarithms
    up to 32 |g| / ln 2 < 64 cost 64 u 2.  With |T| <= kappa (rows of |inverse|, below) the
    errors of e are within kappa 200 u (s + |v|) and enter S through beta |k| <= 2, with 70 u
    of the sums over the block: 600 u kappa (s + |v|) for each token covers both."""
    H = v.shape[1]
    q, k = shared(q, H).double(), shared(k, H).double()
    a, b = g.double().exp(), beta.double()
    s = torch.stack([S.flatten(2).norm(dim=-1) for S in kept]).amax(0)
    size = s + (v.double().norm(dim=-1).amax(-1) if v.shape[2] else 0)
    kappa = torch.ones_like(s)
    for at in range(0, v.shape[2], 32):
        kk, gg = k[:, :, at:at + 32], g[:, :, at:at + 32].double().clamp_min(-88.0).cumsum(-1)
        L = (kk @ kk.transpose(-1, -2).contiguous()) * (gg[..., :, None] - gg[..., None, :]).tril(-1).exp()
        L = L.tril(-1) * b[:, :, None, at:at + 32]
        inverse = torch.linalg.inv(torch.eye(L.shape[-1], dtype=L.dtype, device=L.device) + L)
        kappa = torch.maximum(kappa, inverse.abs().sum(-1).amax(-1))
    D, out = torch.zeros_like(s), []
    for t in range(v.shape[2]):
        D = a[:, :, t] * D + 600 * U * kappa * size
        out.append(D)
    return (torch.stack(out, 2) if out else s[..., None][..., :0]), s


def inputs(B, H, Hk, T, dk, dv, dtype, gate, seed, kind="decay", device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    t, tg = TYPES[dtype], TYPES[gate]
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    k = rand(B, Hk, T, dk)
    if kind == "alike":  # keys near one direction: a system far from the identity
        k = k + 3 * rand(B, Hk, 1, dk)
    q, k, v = unit(rand(B, Hk, T, dk)).to(t), (0.99 * unit(k)).to(t), rand(B, H, T, dv).to(t)
    gate_ = -0.2 * torch.nn.functional.softplus(rand(B, H, T))
    beta = torch.sigmoid(rand(B, H, T))
    if kind == "resets":  # g = -inf forgets, g = 0 keeps, beta = 0 writes nothing, beta = 1 everything
        r = rand(B, H, T)
        gate_ = torch.where(r > 1.5, -float("inf"), torch.where(r > 0, 0.0, gate_))
        beta = torch.where(rand(B, H, T) > 1, 0.0, torch.where(rand(B, H, T) > 1, 1.0, beta))
    return q, k, v, gate_.to(tg), beta.to(tg), rand(B, H, dv, dk)


def _blocks(T, n):
    return [(at, min(n, T - at)) for at in range(0, T, n)]


def rounding_bounds(q, k, v, g, beta, do, S0, dS_T, half, scale=None):
    """Bounds on what rounding the operands of the last products to a type with that half
    step costs each element of dq, dk, dg and dbeta (in groups of 64 tokens): every product's
    sum of absolute values, times the roundings on its way.  E, dV, S and D are rounded
    once, U = beta E once more, and the weights dP and M behind U (and dV):
      dO S: 1   dP K, dP Q: E, U, dP 3   M K: E, U, dV, M 4   U D: E, U, D 3   dV S: 2   X E: 1."""
    H, T = v.shape[1], v.shape[2]
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    grads = delta_gradients(q, k, v, g, beta, do, S0, dS_T, scale)
    _, _, kept = delta(q, k, v, g, beta, S0, scale)
    Hk, r = q.shape[1], H // q.shape[1]
    q, k, v, g, beta, do = (x.double() for x in (shared(q, H), shared(k, H), v, g, beta, do))
    # e_t from the states: S_t - a S_{t-1} = u_t k_t^T
    E, X = torch.zeros_like(v), torch.zeros_like(v)
    D = [None] * (T + 1)
    D[T] = torch.zeros_like(kept[0]) if dS_T is None else dS_T.double()
    for t in reversed(range(T)):
        old = kept[t] * g[:, :, t, None, None].exp()
        E[:, :, t] = v[:, :, t] - (old * k[:, :, t, None, :]).sum(-1)
        now = D[t + 1] + scale * do[:, :, t, :, None] * q[:, :, t, None, :]
        X[:, :, t] = (now * k[:, :, t, None, :]).sum(-1)
        D[t] = (now - (beta[:, :, t, None] * X[:, :, t])[..., None] * k[:, :, t, None, :]) * g[:, :, t, None, None].exp()
    U, dv = (beta[..., None] * E).abs(), grads["dv"].abs()
    out = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dg", g))}
    out["dbeta"] = (X.abs() * E.abs()).sum(-1)
    mm = lambda x, y: x @ y.contiguous()  # noqa: E731
    for at, n in _blocks(T, 64):
        sl = slice(at, at + n)
        G = g[:, :, sl].clamp_min(-700).cumsum(-1)
        gam, rest = G.exp()[..., None], (G[..., -1:] - G).exp()[..., None]
        ratio = (G[..., :, None] - G[..., None, :]).tril().exp().tril()
        Q, K, O, W, u = q[:, :, sl].abs(), k[:, :, sl].abs(), do[:, :, sl].abs(), dv[:, :, sl], U[:, :, sl]
        S, De = kept[at].abs(), D[at + n].abs()
        P, M = scale * mm(O, u.transpose(-1, -2)) * ratio, (mm(W, u.transpose(-1, -2)) * ratio).tril(-1)
        os, vs, ud = scale * gam * mm(O, S), gam * mm(W, S), rest * mm(u, De)
        out["dq"][:, :, sl] = os + 3 * mm(P, K)
        out["dk"][:, :, sl] = 3 * mm(P.transpose(-1, -2), Q) + 4 * (mm(M, K) + mm(M.transpose(-1, -2), K)) + 3 * ud + 2 * vs
        A, B = (Q * os).sum(-1) + 2 * (K * vs).sum(-1), 3 * (K * ud).sum(-1)
        w = 3 * P * (q[:, :, sl] @ k[:, :, sl].transpose(-1, -2).contiguous()).abs() \
            + 4 * M * (k[:, :, sl] @ k[:, :, sl].transpose(-1, -2).contiguous()).abs()
        for t in range(n):
            out["dg"][:, :, at + t] = (2 * (De * S).sum((-1, -2)) * gam[:, :, -1, 0] + A[:, :, t:].sum(-1) + B[:, :, :t].sum(-1)
                                       + w[:, :, t:, :t].sum((-1, -2)))
    out["dq"], out["dk"] = (out[n].unflatten(1, (Hk, r)).sum(2) for n in ("dq", "dk"))
    return grads, {n: half * out[n] for n in out}
