"""Host-side checks of the gated delta rule: workspace queries and refusals, all before any
GPU work."""
import ctypes
import os

import pytest
import torch

import kalman_filter_memory_amd as kdn

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kdn.LIB_PATH):
        from kalman_filter_memory_amd import build
        build.build()
    return kdn.load_library()


def _desc(B=2, H=4, Hk=2, T=10, d_k=64, d_v=32, dtype=kdn.BF16, gate_dtype=kdn.F32, scale=0.125):
    return kdn.KdnDeltaDesc(B, H, Hk, T, d_k, d_v, dtype, gate_dtype, scale)


BAD = [
    (dict(B=-1), 2), (dict(H=-4), 2), (dict(Hk=-2), 2), (dict(T=-1), 2), (dict(Hk=3), 2), (dict(Hk=0), 2),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
    (dict(d_k=0), 3), (dict(d_k=48), 3), (dict(d_v=256), 3), (dict(dtype=2), 3), (dict(gate_dtype=-1), 3),
    (dict(B=1 << 20, H=1, Hk=1), 3),
]


@pytest.mark.parametrize("kw,code", BAD, ids=[str(k) for k, _ in BAD])
def test_refuses_descriptors(lib, kw, code):
    d = ctypes.byref(_desc(**kw))
    for packed in (0, 1):
        assert lib.kdn_gated_delta_workspace_bytes(d, packed) == 0
    assert lib.kdn_gated_delta(d, None, *([FAKE] * 9), 1 << 40, None) == code
    assert lib.kdn_gated_delta_step(d, *([FAKE] * 6), None, 0, FAKE, None) == code
    for packed in (0, 1):
        assert lib.kdn_gated_delta_backward_workspace_bytes(d, packed) == 0
    assert lib.kdn_gated_delta_backward(d, None, *([FAKE] * 15), 1 << 40, None) == code


def test_refuses_too_many_tokens(lib):
    d = ctypes.byref(_desc(T=(1 << 30) + 1))
    assert lib.kdn_gated_delta_workspace_bytes(d, 0) == 0
    assert lib.kdn_gated_delta(d, None, *([FAKE] * 9), 1 << 40, None) == 3


def test_refuses_arguments(lib):
    d = ctypes.byref(_desc())
    need = lib.kdn_gated_delta_workspace_bytes(d, 0)
    assert need == 16  # none
    assert lib.kdn_gated_delta(None, None, *([FAKE] * 9), need, None) == 1
    for i in (0, 1, 2, 3, 4, 6):  # q, k, v, g, beta, o
        args = [FAKE] * 9
        args[i] = None
        assert lib.kdn_gated_delta(d, None, *args, need, None) == 1
    for i in (0, 1, 2, 5, 6, 7, 8):  # q, k, v, S0, o, S_T, ws
        args = [FAKE] * 9
        args[i] = ODD
        assert lib.kdn_gated_delta(d, None, *args, need, None) == 5
    assert lib.kdn_gated_delta_step(None, *([FAKE] * 6), None, 0, FAKE, None) == 1
    assert lib.kdn_gated_delta_step(d, *([FAKE] * 6), FAKE, -1, FAKE, None) == 2
    for i in range(6):
        args = [FAKE] * 6
        args[i] = None
        assert lib.kdn_gated_delta_step(d, *args, None, 0, FAKE, None) == 1
    assert lib.kdn_gated_delta_step(d, *([FAKE] * 6), None, 0, None, None) == 1
    for i in (0, 1, 5):
        args = [FAKE] * 6
        args[i] = ODD
        assert lib.kdn_gated_delta_step(d, *args, None, 0, FAKE, None) == 5


def test_backward_refuses_arguments(lib):
    d = ctypes.byref(_desc())
    need = lib.kdn_gated_delta_backward_workspace_bytes(d, 0)
    # E, states before and gradients behind each 64 tokens, a row of dbeta for 16 columns
    assert need == 2 * 4 * 10 * 32 * 2 + 2 * (2 * 4 * 32 * 64 * 2) + 2 * 4 * 10 * 2 * 4 + 128 + 16
    assert lib.kdn_gated_delta_backward_workspace_bytes(d, 1) > 0
    assert lib.kdn_gated_delta_backward(d, None, *([FAKE] * 15), need - 1, None) == 4
    assert lib.kdn_gated_delta_backward(None, None, *([FAKE] * 15), need, None) == 1
    for i in (0, 1, 2, 3, 4, 6, 8, 9, 10, 11, 12, 14):  # not S0, dS_T, dS0
        args = [FAKE] * 15
        args[i] = None
        assert lib.kdn_gated_delta_backward(d, None, *args, need, None) == 1
    for i in (0, 1, 2, 5, 6, 7, 8, 9, 10, 13, 14):  # not g, beta, dg, dbeta
        args = [FAKE] * 15
        args[i] = ODD
        assert lib.kdn_gated_delta_backward(d, None, *args, need, None) == 5
    # more groups of tokens than a launch takes
    many = ctypes.byref(_desc(B=1, H=16, Hk=16, T=1 << 26))
    assert lib.kdn_gated_delta_backward_workspace_bytes(many, 0) == 0
    assert lib.kdn_gated_delta_backward(many, None, *([FAKE] * 15), 1 << 60, None) == 3
    assert lib.kdn_gated_delta_backward(ctypes.byref(_desc(B=0)), None, *([None] * 15), 0, None) == 0


def test_nothing_to_do(lib):
    for kw in (dict(B=0), dict(H=0), dict(H=0, Hk=0)):
        d = ctypes.byref(_desc(**kw))
        assert lib.kdn_gated_delta(d, None, *([None] * 9), 0, None) == 0
        assert lib.kdn_gated_delta_step(d, *([None] * 6), None, 0, None, None) == 0


def _cpu(T=4, H=4, Hk=2, dk=32, dv=64, B=2):
    return [torch.zeros(B, Hk, T, dk), torch.zeros(B, Hk, T, dk), torch.zeros(B, H, T, dv), torch.zeros(B, H, T),
            torch.zeros(B, H, T)]


def test_binding_refuses_cpu_tensors():
    x = _cpu()
    with pytest.raises(kdn.KdnError):
        kdn.gated_delta(*x)
    with pytest.raises(kdn.KdnError):
        kdn.gated_delta_step(*(t[:, :, 0].contiguous() for t in x), torch.zeros(2, 4, 64, 32))
    with pytest.raises(ValueError):
        kdn.gated_delta_varlen(*(t[0] for t in x), None)


@pytest.mark.parametrize("change", [
    lambda x: x.__setitem__(1, x[1][..., :16]), lambda x: x.__setitem__(2, x[2][:, :3]), lambda x: x.__setitem__(3, x[3][:, :, 1:]),
    lambda x: x.__setitem__(4, x[4].to(torch.bfloat16)), lambda x: x.__setitem__(2, x[2].to(torch.bfloat16)),
    lambda x: x.__setitem__(2, x[2][:1]), lambda x: x.__setitem__(0, x[0][0])])
def test_binding_refuses_shapes_and_types(change):
    """(the checks of shapes, which need no GPU)"""
    x = _cpu()
    change(x)
    with pytest.raises((ValueError, TypeError)):
        kdn._delta_desc(*x, None)
