"""Host-side checks of the head norm with rotation: workspace queries and refusals, all
before any GPU work."""
import ctypes
import os

import pytest

import kalman_filter_memory_amd as kdn

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kdn.LIB_PATH):
        from kalman_filter_memory_amd import build
        build.build()
    return kdn.load_library()


def _desc(B=2, T=10, H=4, Hk=2, d=64, rot=32, dtype=kdn.BF16, interleaved=0, eps=1e-6, strides=None):
    s = strides or (H * d * T, H * d, d)
    return kdn.KdnRotaryDesc(B, T, H, Hk, d, rot, dtype, interleaved, eps, *s, *s, *s, *s)


BAD = [
    (dict(B=-1), 2), (dict(T=-1), 2), (dict(H=-1), 2), (dict(Hk=-1), 2), (dict(d=-8), 2), (dict(rot=-16), 2), (dict(rot=80), 2),
    (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2),
    (dict(d=0, rot=0), 3), (dict(d=12, rot=0), 3), (dict(d=264), 3), (dict(rot=24), 3), (dict(dtype=2), 3), (dict(dtype=-1), 3),
    (dict(B=1 << 13, T=1 << 13), 3), (dict(H=(1 << 16) + 1), 3),
    (dict(strides=(2560, 256, 36)), 5), (dict(strides=(2560, 257, 64)), 5), (dict(strides=(2561, 256, 64)), 5),
]


@pytest.mark.parametrize("kw,code", BAD, ids=[str(k) for k, _ in BAD])
def test_refuses_descriptors(lib, kw, code):
    d = ctypes.byref(_desc(**kw))
    assert lib.kdn_qk_norm_rotary(d, *([FAKE] * 10), None) == code
    assert lib.kdn_qk_norm_rotary_backward_workspace_bytes(d) == 0
    assert lib.kdn_qk_norm_rotary_backward(d, *([FAKE] * 14), 1 << 40, None) == code


def test_refuses_arguments(lib):
    d = ctypes.byref(_desc())
    assert lib.kdn_qk_norm_rotary(None, *([FAKE] * 10), None) == 1
    for i in range(8):  # not the rstds
        args = [FAKE] * 10
        args[i] = None
        assert lib.kdn_qk_norm_rotary(d, *args, None) == 1
    for i in (0, 1, 2, 3, 6, 7):
        args = [FAKE] * 10
        args[i] = ODD
        assert lib.kdn_qk_norm_rotary(d, *args, None) == 5
    need = lib.kdn_qk_norm_rotary_backward_workspace_bytes(d)
    assert need == 20 * 2 * 64 * 4  # a workgroup per token, a row for each of the two weights
    assert lib.kdn_qk_norm_rotary_backward(None, *([FAKE] * 14), need, None) == 1
    assert lib.kdn_qk_norm_rotary_backward(d, *([FAKE] * 14), need - 1, None) == 4
    for i in range(14):
        args = [FAKE] * 14
        args[i] = None
        assert lib.kdn_qk_norm_rotary_backward(d, *args, need, None) == 1
    for i in (0, 1, 2, 3, 4, 5, 10, 11, 12, 13):
        args = [FAKE] * 14
        args[i] = ODD
        assert lib.kdn_qk_norm_rotary_backward(d, *args, need, None) == 5


def test_nothing_to_do(lib):
    for kw in (dict(B=0), dict(T=0), dict(H=0, Hk=0)):
        assert lib.kdn_qk_norm_rotary(ctypes.byref(_desc(**kw)), *([None] * 10), None) == 0
