"""The gated recurrence of one sequence, alone and inside a batch: the same bits, however
the batch is spread over the GPU (a workgroup per tile where there are few sequences, one
that walks along its sequence where there are many)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _chains(B, H, T, d, dtype, gate, backward):
    """Whether the call needs a workspace: only tiles that hand their state on do."""
    s = kdn.make_scan_desc(B, H, T, d, kdn._dtype_code(dtype), kdn._dtype_code(gate))
    lib = kdn.load_library()
    f = lib.kdn_gated_scan_backward_workspace_bytes if backward else lib.kdn_gated_scan_workspace_bytes
    return f(ctypes.byref(s)) > 16


# tiles of 64 to 1024 tokens: up to one group of 16 tiles, just beyond one, several groups
@pytest.mark.parametrize("dtype,gate", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,d", [(4096, 128), (4097, 128), (5300, 72), (1200, 200), (20000, 32)])
def test_a_sequence_gives_the_same_bits_alone_and_in_a_batch(T, d, dtype, gate):
    B = 128 if d > 128 else 256
    t, tg = TYPES[dtype], TYPES[gate]
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    say(f"[gpu] gated scan alone and in a batch {B, T, d, dtype, gate}")
    x, dh, a = rand(B, 1, T, d).to(t), rand(B, 1, T, d).to(t), torch.sigmoid(4 + rand(B, 1, T, d)).to(tg)
    h0, dh_T = rand(B, 1, d), rand(B, 1, d)
    for back in (False, True):
        assert _chains(1, 1, T, d, t, tg, back) and _chains(2, 1, T, d, t, tg, back)
        assert not _chains(B, 1, T, d, t, tg, back)
    h, h_T = kdn.gated_scan(x, a, h0)
    grads = kdn.gated_scan_backward(a, h, dh, h0, dh_T)
    for part in (slice(0, 1), slice(B - 2, B)):
        h1, h_T1 = kdn.gated_scan(x[part], a[part], h0[part])
        assert torch.equal(h1, h[part]) and torch.equal(h_T1, h_T[part])
        for n, v in kdn.gated_scan_backward(a[part], h[part], dh[part], h0[part], dh_T[part]).items():
            assert torch.equal(v, grads[n][part]), n
