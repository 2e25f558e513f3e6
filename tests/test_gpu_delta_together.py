"""The gated delta rule as a model uses it: the projection's rows, head norms with rotation,
the recurrence; a prompt against its tokens one by one, and a training step against
differences."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from delta_reference import delta
from gpu_util import say

pytestmark = pytest.mark.gpu


def _setup(B, T, H, Hk, dk, dv, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    z = rand(B, T, 2 * Hk * dk + H * dv).to(dtype)
    position = torch.arange(T, device="cuda", dtype=torch.int32).expand(B, T).contiguous() + 1000
    inv_freq = 1e4 ** (-2 * torch.arange(dk // 2, device="cuda") / dk)
    weight = torch.full((dk,), dk ** -0.5, device="cuda") * (1 + 0.1 * rand(dk)).clamp(0.8, 1.0)
    gate, beta = -0.1 * torch.nn.functional.softplus(rand(B, H, T)), torch.sigmoid(rand(B, H, T))
    return rand, z, position, inv_freq, weight, gate, beta


def _heads(z, H, Hk, dk, dv):
    q, k, v = z.split((Hk * dk, Hk * dk, H * dv), -1)
    return q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (H, dv))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv", [(2, 50, 4, 2, 64, 128), (1, 100, 2, 2, 128, 64)])
def test_prompt_equals_its_tokens(B, T, H, Hk, dk, dv, dtype):
    """The step's kernels add in another order: float32 1e-5 of the largest (a few hundred
    roundings); bfloat16 outputs are roundings of values that near: one step, 2^-7."""
    rand, z, position, inv_freq, weight, gate, beta = _setup(B, T, H, Hk, dk, dv, dtype, T)
    q, k, v = _heads(z, H, Hk, dk, dv)
    say(f"[gpu] delta together {B, T, H, Hk, dk, dv, dtype}")
    qh, kh, _, _ = kdn.qk_norm_rotary(q, k, weight, weight, position, inv_freq)
    o, S_T = kdn.gated_delta(qh, kh, v.transpose(1, 2).contiguous(), gate, beta)
    S, got = torch.zeros(B, H, dv, dk, device="cuda"), []
    for t in range(T):
        qt, kt, vt = _heads(z[:, t:t + 1], H, Hk, dk, dv)
        qt, kt, _, _ = kdn.qk_norm_rotary(qt, kt, weight, weight, position[:, t:t + 1].contiguous(), inv_freq)
        got.append(kdn.gated_delta_step(qt[:, :, 0], kt[:, :, 0], vt[:, 0].contiguous(), gate[..., t].contiguous(),
                                        beta[..., t].contiguous(), S))
    got = torch.stack(got, 2).double()
    tol = 1e-5 * o.double().abs().max() + (2.0 ** -7 * o.double().abs() if dtype == torch.bfloat16 else 0)
    assert ((got - o.double()).abs() <= tol).all()
    assert (S - S_T).abs().max() <= 1e-5 * S_T.abs().max()


def test_training_step_against_differences():
    """loss = <c, o> + <d, S_T> of norm, rotation and recurrence: its gradient by the backward
    calls along random directions against central differences in 64 bits (h = 1e-5), 1e-4 of
    the sum of absolute values; q's and k's gradients go into the projection's rows."""
    B, T, H, Hk, dk, dv = 2, 40, 4, 2, 32, 64
    rand, z, position, inv_freq, weight, gate, beta = _setup(B, T, H, Hk, dk, dv, torch.float32, 3)
    weight_k = weight * 0.9
    S0, c, d = 0.3 * rand(B, H, dv, dk), rand(B, H, T, dv), 0.3 * rand(B, H, dv, dk)

    def turned(x, w):
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = n.chunk(2, -1)
        angle = (position.double()[..., None] * inv_freq.double())[:, :, None]
        return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1).transpose(1, 2)

    def loss(z, wq, wk, gate, beta, S0):
        q, k, v = _heads(z, H, Hk, dk, dv)
        o, S, _ = delta(turned(q, wq), turned(k, wk), v.transpose(1, 2), gate, beta, S0)
        return (o * c.double()).sum() + (S * d.double()).sum()

    q, k, v = _heads(z, H, Hk, dk, dv)
    vh = v.transpose(1, 2).contiguous()
    qh, kh, qr, kr = kdn.qk_norm_rotary(q, k, weight, weight_k, position, inv_freq)
    g = kdn.gated_delta_backward(qh, kh, vh, gate, beta, c, S0, d)
    dz = torch.empty_like(z)
    dq, dk_, dv_ = _heads(dz, H, Hk, dk, dv)
    _, _, dwq, dwk = kdn.qk_norm_rotary_backward(g["dq"], g["dk"], q, k, weight, weight_k, position, inv_freq, qr, kr,
                                                 out=(dq, dk_))
    dv_.copy_(g["dv"].transpose(1, 2))
    leaves = (z, weight, weight_k, gate, beta, S0)
    grads = (dz, dwq, dwk, g["dg"], g["dbeta"], g["dS0"])
    for _ in range(3):
        e = [rand(*t.shape).double() for t in leaves]
        plus, minus = (loss(*(t.double() + s * 1e-5 * v for t, v in zip(leaves, e))) for s in (1, -1))
        parts = [p.double() * v for p, v in zip(grads, e)]
        got, size = sum(p.sum() for p in parts), sum(p.abs().sum() for p in parts)
        assert abs(got - (plus - minus) / 2e-5) <= 1e-4 * size


def test_heads_feed_the_filter_too():
    """The same head rows are forward()'s q and k: with the weight d^(-1/2) the norm is the
    layer's, and a head's result does not depend on a rotation by position 0."""
    B, T, H, d = 1, 70, 2, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v = rand(B, T, H, d), rand(B, T, H, d), rand(B, H, T, d)
    w = torch.full((d,), d ** -0.5, device="cuda")
    a, nu, r = torch.sigmoid(2 + rand(B, H, T)), 0.05 * rand(B, H, T).abs(), 0.5 + rand(B, H, T).abs()
    here = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    inv_freq = 1e4 ** (-2 * torch.arange(d // 2, device="cuda") / d)
    plain = kdn.qk_norm_rotary(q, k, w, w, None, None, eps=0.0)
    turned = kdn.qk_norm_rotary(q, k, w, w, here, inv_freq, eps=0.0)
    assert torch.equal(plain[0], turned[0]) and torch.equal(plain[1], turned[1])
    unit = [torch.nn.functional.normalize(x.double(), dim=-1).float().transpose(1, 2).contiguous() for x in (q, k)]
    for x, y in zip(kdn.forward(*plain[:2], v, a, nu, r, chunk=32), kdn.forward(*unit, v, a, nu, r, chunk=32)):
        assert (x - y).abs().max() <= 1e-4 * y.abs().max()
