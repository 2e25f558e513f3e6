"""The layer without heads: y is a product of depth 0, all zeros."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn

FAKE = ctypes.c_void_p(0x1000)


def test_without_heads_y_is_checked():
    d = ctypes.byref(kdn.make_layer_desc(2, 5, 0, 64, 32, 32, 16, "diagonal", kdn.F32))
    call = kdn.load_library().kdn_layer_forward
    for y, code in ((None, 1), (ctypes.c_void_p(0x1004), 5)):
        assert call(d, FAKE, FAKE, None, None, None, None, None, y, None, None, FAKE, 1 << 30, None) == code


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (2, 5, 72), (1, 9000, 2048)])
def test_without_heads(B, T, D, dtype):
    x = torch.randn(B, T, D, device="cuda").to(dtype)
    none = torch.empty(0, D, dtype=dtype, device="cuda"), torch.empty(D, 0, dtype=dtype, device="cuda")
    y0, _, _ = kdn.layer_forward(x, none[0], torch.empty(0).cuda(), none[1], 0, 32, 32, chunk=16)
    assert y0.shape == x.shape and int((y0 != 0).sum()) == 0 and not torch.isnan(y0.float()).any()
    d = kdn.make_layer_desc(B, T, 0, D, 32, 32, 16, "diagonal", kdn._dtype_code(dtype))
    y = torch.full((B * T + 1, D), 7.0, dtype=dtype, device="cuda")
    assert kdn.load_library().kdn_layer_forward(
        ctypes.byref(d), kdn.blas_handle(), x.data_ptr(), None, None, None, None, None, y.data_ptr(), None, None,
        None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert int((y[:-1] != 0).sum()) == 0 and int((y[-1] != 7).sum()) == 0
