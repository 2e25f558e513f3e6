"""The layer in 8 bits at its empty sizes: without heads the residual stream is still
written and y is zero; an empty batch gives empty results."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1004)


def _args(**kw):
    a = dict(x=FAKE, residual=FAKE, rd=kdn.F32, nw=FAKE, eps=1e-6, wi=None, wis=None, bg=None, wo=None, wos=None,
             l0=None, s0=None, y=FAKE, s=FAKE, st=None, lt=None, ws=FAKE, n=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


def test_without_heads_the_stream_is_still_checked():
    d = ctypes.byref(kdn.make_layer_desc(2, 5, 0, 64, 32, 32, 16, "diagonal", kdn.F32))
    call = kdn.load_library().kdn_layer_quant_forward
    for n in ("x", "nw", "y", "s", "residual", "ws"):
        assert call(d, *_args(**{n: None})) == 1, n
    for n in ("x", "residual", "nw", "y", "s", "ws"):
        assert call(d, *_args(**{n: ODD})) == 5, n
    assert call(d, *_args(n=0)) == 4


def _weights(H, D):
    n_in = H * (2 * 32 + 32) + 3 * H
    return (*kdn.quantize(torch.randn(n_in, D).cuda(), 128), torch.zeros(3 * H).cuda(),
            *kdn.quantize(torch.randn(D, 32 * H).cuda(), 128))


@pytest.mark.gpu
@pytest.mark.parametrize("variant", ["diagonal", "isotropic"])
@pytest.mark.parametrize("dtype,res", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                       (torch.bfloat16, torch.bfloat16), (torch.float32, None)])
@pytest.mark.parametrize("B,T,D", [(2, 5, 64), (1, 1, 16), (1, 700, 2048)])
def test_without_heads(B, T, D, dtype, res, variant):
    g = torch.Generator().manual_seed(D)
    x = torch.randn(B, T, D, generator=g).to(dtype).cuda()
    r = None if res is None else torch.randn(B, T, D, generator=g).to(res).cuda()
    want = x if r is None else (x.float() + r.float()).to(res)
    args = (x, torch.ones(D).cuda(), *_weights(0, D), 0, 32, 32)
    for in_place in (False, True):
        torch.full((B, T, D), 7.0, device="cuda", dtype=dtype)  # (what a new tensor of y's size may find)
        y, s, S_T, lam = kdn.layer_quant_forward(*args, residual=r, variant=variant, chunk=16, in_place=in_place)
        assert y.dtype == dtype and int((y != 0).sum()) == 0 and not torch.isnan(y.float()).any()
        assert torch.equal(s, want)
        assert S_T.shape == (B, 0, 32, 32) and lam.numel() == 0


@pytest.mark.parametrize("B,T,H", [(0, 5, 2), (0, 0, 2), (2, 0, 0), (0, 0, 0)])
def test_empty_sizes_are_valid_descriptors(B, T, H):
    """0 bytes of workspace are the answer for an invalid descriptor alone."""
    d = kdn.make_layer_desc(B, T, H, 64, 32, 32, 16, "diagonal", kdn.F32)
    assert kdn.layer_quant_workspace_bytes(d) > 0
    args = _args(**{n: None for n in ("x", "residual", "nw", "y", "s", "ws")}, n=0)
    assert kdn.load_library().kdn_layer_quant_forward(ctypes.byref(d), *args) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H", [(0, 5, 2), (0, 0, 2), (2, 0, 0), (2, 0, 2), (0, 3, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_empty_batches(B, T, H, residual):
    D = 64
    x = torch.empty(B, T, D).cuda()
    S0 = torch.randn(B, H, 32, 32).cuda()
    y, s, S_T, lam = kdn.layer_quant_forward(x, torch.ones(D).cuda(), *_weights(H, D), H, 32, 32,
                                             residual=x.clone() if residual else None, S0=S0, chunk=16)
    assert y.shape == s.shape == x.shape and torch.equal(S_T, S0) and lam.shape == (B, H, 32)
