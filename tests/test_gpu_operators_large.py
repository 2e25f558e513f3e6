"""The operators beyond 2^32 bytes and elements, and over very long sequences: what
lies at the far end equals the same rows computed on their own (the same kernel on the
same rows: bit for bit), or a result that is exact."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_norm_and_quantiser_beyond_32_bit_offsets():
    rows, d = (1 << 20) + 3, 4104  # 4.3e9 elements
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn(d, device="cuda")
    say(f"[gpu] norm of {rows} x {d}")
    q, scale, s = kdn.rms_norm_quant(x, w, x)
    tail = x[-7:].clone()
    q2, scale2, s2 = kdn.rms_norm_quant(tail, w, tail)
    assert torch.equal(q[-7:].view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(scale[-7:], scale2) and torch.equal(s[-7:], s2)
    del q, scale, s
    for block_rows in (1, 128):
        n = 7 if block_rows == 1 else rows % 128
        q, scale = kdn.quantize(x, block_rows=block_rows)
        q2, scale2 = kdn.quantize(x[-n:].clone(), block_rows=block_rows)
        assert torch.equal(q[-n:].view(torch.uint8), q2.view(torch.uint8))
        assert torch.equal(scale[-scale2.shape[0]:], scale2)
        del q, scale


def test_norm_backward_beyond_32_bit_offsets():
    rows, d = (1 << 20) + 3, 4104
    s = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_()
    rstd = torch.ones(rows, device="cuda")
    w = torch.randn(d, device="cuda")
    say(f"[gpu] norm backward of {rows} x {d}")
    dx, dw = kdn.rms_norm_backward(s, s, w, rstd)
    dx2, _ = kdn.rms_norm_backward(s[-7:].clone(), s[-7:].clone(), w, rstd[-7:].clone())
    assert torch.equal(dx[-7:], dx2) and torch.isfinite(dw).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_product_beyond_32_bit_offsets(dtype):
    """A of 4.3e9 bytes, and C of 4.4e9 elements: small whole numbers and scales of one,
    so every sum is exact, whichever kernel computes it."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def whole(r, k):
        return torch.randint(-2, 3, (r, k), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16).to(torch.float8_e4m3fn)

    for M, N, K in (((1 << 20) + 5, 72, 4112), ((1 << 21) + 5, 2104, 48)):
        say(f"[gpu] product {M} x {N} x {K}")
        a, b = whole(M, K), whole(N, K)
        kb = -(-K // 128)
        c = kdn.quant_matmul(a, torch.ones(M, kb, device="cuda"), b, torch.ones(-(-N // 128), kb, device="cuda"),
                             out_dtype=dtype)
        for rows in (slice(0, 50), slice(M // 2, M // 2 + 50), slice(M - 50, M)):
            want = (a[rows].double() @ b.double().t().contiguous()).to(dtype)
            assert torch.equal(c[rows], want)
        del a, c


def test_scan_beyond_32_bit_offsets():
    """2.2e9 elements: a = 1 and a few tokens that are not zero, so the state is a
    whole number, exact in bfloat16."""
    T, d = 17_000_000, 128
    x = torch.zeros(1, 1, T, d, dtype=torch.bfloat16, device="cuda")
    a = torch.ones(1, 1, T, d, dtype=torch.bfloat16, device="cuda")
    at = [0, 255, 256, 2047, 2048, 16_777_215, 16_777_216, T - 1]
    for t in at:
        x[0, 0, t] = 1
    h0 = torch.arange(d, device="cuda", dtype=torch.float32).view(1, 1, d) % 8
    say(f"[gpu] scan of {T} tokens")
    h, h_T = kdn.gated_scan(x, a, h0)
    probe = sorted({0, 1, 254, 255, 256, 2046, 2047, 2048, 9_000_000, 16_777_214, 16_777_215, 16_777_216, T - 2, T - 1})
    for t in probe:
        want = h0[0, 0] + sum(u <= t for u in at)
        assert torch.equal(h[0, 0, t].float(), want), t
    assert torch.equal(h_T[0, 0], h0[0, 0] + len(at))
    g = kdn.gated_scan_backward(a, h, x, h0, h0)
    for t in probe:
        dx = h0[0, 0] + sum(u >= t for u in at)
        before = h[0, 0, t - 1].float() if t else h0[0, 0]
        assert torch.equal(g["dx"][0, 0, t], dx) and torch.equal(g["da"][0, 0, t], dx * before), t
    assert torch.equal(g["dh0"][0, 0], h0[0, 0] + len(at))


@pytest.mark.parametrize("T,d", [(1_000_003, 8), (300_001, 40), (65_536, 200)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_long_scans_are_exact_on_whole_numbers(T, d, dtype):
    """a = 1 but for a few zeros, x of whole numbers: running sums from the last zero,
    below 2^24, so float32's are exact (bfloat16's rounded once)."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randint(-3, 4, (1, 1, T, d), generator=g, device="cuda")
    a = (torch.rand(1, 1, T, d, generator=g, device="cuda") > 2e-5).long()
    total = x.cumsum(2)
    # the sum before the last zero of a, carried along
    idx = torch.where(a == 0, torch.arange(T, device="cuda").view(1, 1, T, 1), 0).cummax(2).values
    before = torch.cat((torch.zeros_like(total[:, :, :1]), total[:, :, :-1]), 2)
    want = total - torch.where((a == 0).cumsum(2) > 0, before.gather(2, idx), 0)
    h, h_T = kdn.gated_scan(x.to(dtype), a.to(dtype))
    assert torch.equal(h, want.float().to(dtype)) and torch.equal(h_T, want[:, :, -1].float())
    # backwards: the same sums from the other end, one token later
    flip = lambda v: v.flip(2).to(dtype)  # noqa: E731
    back = kdn.gated_scan_backward(flip(a), flip(torch.zeros_like(x)), flip(x))
    # m_t = a_t (dh_t + m_{t+1}); dx_t = dh_t + m_{t+1}: m and dx are zero where a is
    m = torch.cat((torch.zeros_like(want[:, :, :1]), _runs(a, x)[:, :, :-1]), 2)
    assert torch.equal(back["dx"], (x + m).flip(2).float()) and (back["da"] == 0).all()


def _runs(a, x):
    """m_t = a_t (x_t + m_{t-1}) in whole numbers: the sum since the last zero of a."""
    T = x.shape[2]
    total = x.cumsum(2)
    idx = torch.where(a == 0, torch.arange(T, device=x.device).view(1, 1, T, 1), 0).cummax(2).values
    seen = (a == 0).cumsum(2) > 0
    return torch.where(a == 0, 0, total - torch.where(seen, total.gather(2, idx), 0))
