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
