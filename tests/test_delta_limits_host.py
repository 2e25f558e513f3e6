"""Host-side refusals of the gated delta rule at the edges of its ranges."""
import ctypes

import kalman_filter_memory_amd as kdn

FAKE = ctypes.c_void_p(0x1000)


def test_backward_refuses_heads_of_keys_without_values():
    """(dq and dk would stay unwritten)"""
    lib = kdn.load_library()
    d = ctypes.byref(kdn.KdnDeltaDesc(2, 0, 2, 10, 64, 32, kdn.BF16, kdn.F32, 0.125))
    assert lib.kdn_gated_delta_backward_workspace_bytes(d, 0) == 0
    assert lib.kdn_gated_delta_backward(d, None, *([FAKE] * 15), 1 << 40, None) == 2
    none = ctypes.byref(kdn.KdnDeltaDesc(2, 0, 0, 10, 64, 32, kdn.BF16, kdn.F32, 0.125))
    assert lib.kdn_gated_delta_backward(none, None, *([None] * 15), 0, None) == 0
