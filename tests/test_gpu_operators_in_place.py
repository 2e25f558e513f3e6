"""The outputs that may be an input's own buffer, at every width and in every form of the
kernels: the same bits as into a buffer of their own."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

WIDTHS = [8, 512, 520, 1024, 1032, 2056, 4104, 8200, 16384]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)]
IDS = ["f32", "bf16", "bf16-f32"]


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("d", WIDTHS)
def test_the_residual_stream(d, types):
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(37, d, generator=g, device="cuda").to(types[0])
    r = torch.randn(37, d, generator=g, device="cuda").to(types[1])
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    say(f"[gpu] norm in place {d} {types}")
    for call in (kdn.rms_norm, kdn.rms_norm_quant):
        want = call(x, w, r)
        at = r.clone()
        got = call(x, w, at, in_place=True)
        s = 1 if call is kdn.rms_norm else 2
        assert got[s].data_ptr() == at.data_ptr()
        for p, q in zip(want, got):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
        if types[0] == types[1]:  # x is its own residual, written over
            want = call(x, w, x.clone())
            at = x.clone()
            got = call(at, w, at, in_place=True)
            for p, q in zip(want, got):
                assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("d", WIDTHS)
def test_the_norms_gradient_over_its_own_ds(d, types):
    g = torch.Generator(device="cuda").manual_seed(d)
    rows = 1500  # more than one row for a wave or a workgroup
    dy = torch.randn(rows, d, generator=g, device="cuda").to(types[0])
    s = torch.randn(rows, d, generator=g, device="cuda").to(types[1])
    w, ds = torch.randn(d, generator=g, device="cuda"), torch.randn(rows, d, generator=g, device="cuda")
    rstd = 1 + torch.rand(rows, generator=g, device="cuda")
    say(f"[gpu] norm backward in place {d} {types}")
    dx, dw = kdn.rms_norm_backward(dy, s, w, rstd, ds)
    n = kdn._norm_desc(dy, "dy", w, s.dtype, 0.0)
    lib = kdn.load_library()
    ws = torch.empty(lib.kdn_rms_norm_backward_workspace_bytes(ctypes.byref(n)), dtype=torch.uint8, device="cuda")
    dw2 = torch.empty_like(dw)
    assert lib.kdn_rms_norm_backward(ctypes.byref(n), dy.data_ptr(), s.data_ptr(), w.data_ptr(), rstd.data_ptr(),
                                     ds.data_ptr(), ds.data_ptr(), dw2.data_ptr(), ws.data_ptr(), ws.numel(), _stream()) == 0
    assert torch.equal(ds, dx) and torch.equal(dw2, dw)


# a walk of one tile and of several, a chain of several groups; one and two channel blocks
@pytest.mark.parametrize("B,T,d", [(3, 40, 72), (300, 1500, 72), (1024, 700, 32), (2, 9000, 128), (2, 5000, 200), (130, 2000, 200)])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_the_state_of_a_scan(B, T, d, types):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(B, 1, T, d, generator=g, device="cuda").to(types[0])
    a = torch.rand(B, 1, T, d, generator=g, device="cuda").to(types[1])
    h0 = torch.randn(B, 1, d, generator=g, device="cuda")
    say(f"[gpu] gated scan in place {B, T, d, types}")
    want, want_T = kdn.gated_scan(x, a, h0)
    lib = kdn.load_library()
    s = kdn.make_scan_desc(B, 1, T, d, kdn._dtype_code(x.dtype), kdn._dtype_code(a.dtype))
    need = lib.kdn_gated_scan_workspace_bytes(ctypes.byref(s))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    h = torch.empty_like(x)
    state = h0.clone()
    assert lib.kdn_gated_scan(ctypes.byref(s), x.data_ptr(), a.data_ptr(), state.data_ptr(), h.data_ptr(),
                              state.data_ptr(), ws.data_ptr(), need, _stream()) == 0
    assert torch.equal(h, want) and torch.equal(state, want_T)
