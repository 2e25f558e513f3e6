"""The operators as a model uses them: a pre-norm block of a gated recurrence with
8-bit projections, its prompt against its tokens one by one, and its training step
(in the input's type) against differences."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu


def _gates(z, H, d):
    """token rows [B,T,2 H d] -> x (1 - a) and a, [B,H,T,d]"""
    B, T, _ = z.shape
    x, g = z.view(B, T, 2, H, d).permute(2, 0, 3, 1, 4).float()
    a = torch.sigmoid(g + 2)
    return ((1 - a) * x).contiguous(), a.contiguous()


@pytest.mark.parametrize("B,T,H,d,D", [(2, 70, 4, 32, 256), (1, 300, 3, 64, 208), (3, 33, 2, 128, 1040)])
def test_prompt_equals_its_tokens(B, T, H, d, D):
    """Two blocks on a residual stream.  The kernels for one token add in another order
    than those for a prompt (about 1e-6 relative in float32), which the two roundings to
    8 bits on the way turn into whole steps of a few elements: a share of 2 e / 2^-4 of
    them moves by at most 2^-3, so with e = 1e-5 the 2-norm changes by 2.2e-3 per
    rounding, four in all: 1e-2."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    blocks = [(1 + 0.1 * rand(D), kdn.quantize(rand(2 * H * d, D) * D ** -0.5, 128),
               kdn.quantize(rand(D, H * d) * (H * d) ** -0.5, 128)) for _ in range(2)]
    x = rand(B, T, D)
    say(f"[gpu] two blocks {B, T, H, d, D}")

    def read_out(h, down):
        rows = h.transpose(1, 2).reshape(*h.shape[:1], h.shape[2], H * d).contiguous()
        return kdn.quant_matmul(*kdn.quantize(rows), *down, out_dtype=torch.float32)

    y, res = x, torch.zeros_like(x)
    for w, up, down in blocks:
        q, s, res = kdn.rms_norm_quant(y, w, res)
        u, a = _gates(kdn.quant_matmul(q, s, *up, out_dtype=torch.float32), H, d)
        h, _ = kdn.gated_scan(u, a)
        y = read_out(h, down)
    want = y + res

    states = [torch.zeros(B, H, d, device="cuda") for _ in blocks]
    got = []
    for t in range(T):
        y, res = x[:, t:t + 1].contiguous(), torch.zeros(B, 1, D, device="cuda")
        for (w, up, down), state in zip(blocks, states):
            q, s, res = kdn.rms_norm_quant(y, w, res, in_place=True)
            u, a = _gates(kdn.quant_matmul(q, s, *up, out_dtype=torch.float32), H, d)
            o = kdn.gated_scan_step(u[:, :, 0].contiguous(), a[:, :, 0].contiguous(), state)
            y = read_out(o[:, :, None], down)
        got.append(y + res)
    got = torch.cat(got, 1)
    assert (got - want).double().norm() <= 1e-2 * want.double().norm()


def test_training_step_against_differences():
    """loss = <c, y> + <k, s>, y the scan of the norm of s = x + r: its gradient by the
    backward calls along random directions, against central differences in 64 bits (h =
    1e-5, truncation below 1e-9; float32 sums over 2 x 40 x 64 elements: 1e-4 of the sum
    of absolute values)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    B, T, d = 2, 40, 64
    x, r, c, k = (rand(B, T, d) for _ in range(4))
    w, a = 1 + 0.1 * rand(d), torch.sigmoid(rand(B, T, d) + 2)

    def loss(x, r, w, a):
        s = x + r
        n = s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-6) * w
        h, out = torch.zeros(B, d, dtype=n.dtype, device="cuda"), 0.0
        for t in range(T):
            h = a[:, t] * h + n[:, t]
            out = out + (h * c[:, t].double()).sum()
        return out + (s * k.double()).sum()

    n, s, rstd = kdn.rms_norm(x, w, r)
    h, _ = kdn.gated_scan(n[:, None], a[:, None])
    gs = kdn.gated_scan_backward(a[:, None], h, c[:, None])
    dx, dw = kdn.rms_norm_backward(gs["dx"][:, 0], s, w, rstd, k)
    grads = (dx, dx, dw, gs["da"][:, 0])
    for _ in range(3):
        e = [torch.randn(t.shape, generator=g, device="cuda").double() for t in (x, r, w, a)]
        plus, minus = (loss(*(t.double() + z * 1e-5 * v for t, v in zip((x, r, w, a), e))) for z in (1, -1))
        parts = [(p.double() * v) for p, v in zip(grads, e)]
        got, size = sum(p.sum() for p in parts), sum(p.abs().sum() for p in parts)
        assert abs(got - (plus - minus) / 2e-5) <= 1e-4 * size
