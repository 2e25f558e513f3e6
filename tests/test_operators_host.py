"""Host-side checks of the norm, the 8-bit operands and the gated recurrence:
workspace queries and refusals, all before any GPU work."""
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


def _norm(rows=10, d=64, dtype=kdn.BF16, residual_dtype=kdn.BF16, eps=1e-6):
    n = kdn.KdnNormDesc()
    n.rows, n.d, n.dtype, n.residual_dtype, n.eps = rows, d, dtype, residual_dtype, eps
    return n


def _quant(rows=10, d=64, block_rows=1, dtype=kdn.BF16):
    n = kdn.KdnQuantDesc()
    n.rows, n.d, n.block_rows, n.dtype = rows, d, block_rows, dtype
    return n


NORM_BAD = [
    (dict(rows=-1), 2), (dict(d=-8), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(d=0), 3), (dict(d=12), 3), (dict(d=16392), 3), (dict(rows=1 << 24), 3),
    (dict(dtype=7), 3), (dict(residual_dtype=-1), 3), (dict(dtype=kdn.F32), 3),
]


@pytest.mark.parametrize("kw,code", NORM_BAD, ids=[str(k) for k, _ in NORM_BAD])
def test_norm_refuses_descriptors(lib, kw, code):
    n = ctypes.byref(_norm(**kw))
    assert lib.kdn_rms_norm(n, *([FAKE] * 6), None) == code
    assert lib.kdn_rms_norm_quant(n, *([FAKE] * 7), None) == code
    assert lib.kdn_rms_norm_backward_workspace_bytes(n) == 0
    assert lib.kdn_rms_norm_backward(n, *([FAKE] * 8), 1 << 40, None) == code


def test_norm_refuses_arguments(lib):
    n = ctypes.byref(_norm())
    assert lib.kdn_rms_norm(None, *([FAKE] * 6), None) == 1
    for i in (0, 2, 3):  # x, weight, y
        args = [FAKE] * 6
        args[i] = None
        assert lib.kdn_rms_norm(n, *args, None) == 1
    # s exactly when there is a residual
    assert lib.kdn_rms_norm(n, FAKE, None, FAKE, FAKE, FAKE, None, None) == 1
    assert lib.kdn_rms_norm(n, FAKE, FAKE, FAKE, FAKE, None, None, None) == 1
    for i in (0, 1, 2, 3, 4):
        args = [FAKE] * 6
        args[i] = ODD
        assert lib.kdn_rms_norm(n, *args, None) == 5
    assert lib.kdn_rms_norm_quant(n, FAKE, None, FAKE, FAKE, None, None, None, None) == 1
    assert lib.kdn_rms_norm_quant(n, FAKE, None, FAKE, ODD, FAKE, None, None, None) == 5
    need = lib.kdn_rms_norm_backward_workspace_bytes(n)
    assert need == 3 * 64 * 4  # 10 rows, four to a workgroup, one row of dw each
    assert lib.kdn_rms_norm_backward(n, *([FAKE] * 8), need - 1, None) == 4
    for i in (0, 1, 2, 3, 5, 6, 7):
        args = [FAKE] * 8
        args[i] = None
        assert lib.kdn_rms_norm_backward(n, *args, need, None) == 1
    for i in (0, 1, 2, 4, 5, 7):
        args = [FAKE] * 8
        args[i] = ODD
        assert lib.kdn_rms_norm_backward(n, *args, need, None) == 5
    # no rows: nothing to do
    assert lib.kdn_rms_norm(ctypes.byref(_norm(rows=0)), *([None] * 6), None) == 0


QUANT_BAD = [
    (dict(rows=-1), 2), (dict(d=-8), 2), (dict(d=12), 3), (dict(block_rows=0), 3),
    (dict(block_rows=64), 3), (dict(dtype=9), 3), (dict(rows=1 << 33), 3),
    (dict(rows=(1 << 31) - 1, d=1024), 3),
    # the last multiple of 8 below 2^31: 2^24 blocks, counted without passing 32 bits
    (dict(rows=1, d=(1 << 31) - 8, block_rows=128), 3),
    (dict(rows=16, d=(1 << 31) - 8), 3),
]


@pytest.mark.parametrize("kw,code", QUANT_BAD, ids=[str(k) for k, _ in QUANT_BAD])
def test_quantize_refuses(lib, kw, code):
    assert lib.kdn_quantize(ctypes.byref(_quant(**kw)), FAKE, FAKE, FAKE, None) == code


def test_quantize_refuses_arguments(lib):
    n = ctypes.byref(_quant())
    assert lib.kdn_quantize(None, FAKE, FAKE, FAKE, None) == 1
    assert lib.kdn_quantize(n, None, FAKE, FAKE, None) == 1
    assert lib.kdn_quantize(n, FAKE, None, FAKE, None) == 1
    assert lib.kdn_quantize(n, FAKE, FAKE, None, None) == 1
    assert lib.kdn_quantize(n, ODD, FAKE, FAKE, None) == 5
    assert lib.kdn_quantize(n, FAKE, ODD, FAKE, None) == 5
    assert lib.kdn_quantize(ctypes.byref(_quant(rows=0)), None, None, None, None) == 0
    assert lib.kdn_quantize(ctypes.byref(_quant(d=0)), None, None, None, None) == 0


SCAN_BAD = [
    (dict(B=-1), 2), (dict(T=-1), 2), (dict(d=-8), 2), (dict(d=0), 3), (dict(d=12), 3),
    (dict(dtype=5), 3), (dict(gate_dtype=5), 3), (dict(B=1 << 12, H=1 << 12), 3),
    (dict(T=(1 << 30) + 1), 3), (dict(B=4096, H=1024, d=1024), 3), (dict(d=(1 << 20) + 8), 3),
]


def _scan(B=2, H=3, T=50, d=64, dtype=kdn.BF16, gate_dtype=kdn.F32):
    return kdn.make_scan_desc(B, H, T, d, dtype, gate_dtype)


@pytest.mark.parametrize("kw,code", SCAN_BAD, ids=[str(k) for k, _ in SCAN_BAD])
def test_scan_refuses_descriptors(lib, kw, code):
    s = ctypes.byref(_scan(**kw))
    assert lib.kdn_gated_scan_workspace_bytes(s) == 0
    assert lib.kdn_gated_scan_backward_workspace_bytes(s) == 0
    assert lib.kdn_gated_scan(s, *([FAKE] * 6), 1 << 40, None) == code
    assert lib.kdn_gated_scan_backward(s, *([FAKE] * 9), 1 << 40, None) == code


def test_scan_refuses_arguments(lib):
    s = ctypes.byref(_scan(T=5000))
    need = lib.kdn_gated_scan_workspace_bytes(s)
    back = lib.kdn_gated_scan_backward_workspace_bytes(s)
    assert need > 16 and back > 16  # few sequences, several tiles: the state travels through it
    assert lib.kdn_gated_scan_workspace_bytes(ctypes.byref(_scan())) == 16
    assert lib.kdn_gated_scan(None, *([FAKE] * 6), need, None) == 1
    for i in (0, 1, 3, 5):  # x, a, h, ws (h0 and h_T may be NULL)
        args = [FAKE] * 6
        args[i] = None
        assert lib.kdn_gated_scan(s, *args, need, None) == 1
    for i in range(6):
        args = [FAKE] * 6
        args[i] = ODD
        assert lib.kdn_gated_scan(s, *args, need, None) == 5
    assert lib.kdn_gated_scan(s, *([FAKE] * 6), need - 1, None) == 4
    for i in (0, 1, 3, 5, 6, 8):
        args = [FAKE] * 9
        args[i] = None
        assert lib.kdn_gated_scan_backward(s, *args, back, None) == 1
    for i in range(9):
        args = [FAKE] * 9
        args[i] = ODD
        assert lib.kdn_gated_scan_backward(s, *args, back, None) == 5
    assert lib.kdn_gated_scan_backward(s, *([FAKE] * 9), back - 1, None) == 4
    assert lib.kdn_gated_scan(ctypes.byref(_scan(B=0)), *([None] * 6), 0, None) == 0
    # one tile, or two: no workspace
    assert lib.kdn_gated_scan_backward_workspace_bytes(ctypes.byref(_scan())) == 16
    assert lib.kdn_gated_scan_workspace_bytes(ctypes.byref(_scan(T=2048))) > 16
    assert lib.kdn_gated_scan_workspace_bytes(ctypes.byref(_scan(T=512))) == 16
    step = lib.kdn_gated_scan_step
    for i in (0, 1, 2):
        args = [FAKE] * 4
        args[i] = None
        assert step(s, *args, 1, FAKE, None) == 1
        args[i] = ODD
        assert step(s, *args, 1, FAKE, None) == 5
    assert step(s, *([FAKE] * 4), 1, None, None) == 1
    assert step(s, *([FAKE] * 4), -1, FAKE, None) == 2
    assert step(ctypes.byref(_scan(d=4)), *([FAKE] * 4), 1, FAKE, None) == 3
    assert step(ctypes.byref(_scan(B=0)), *([None] * 4), 1, None, None) == 0


def test_binding_refuses_sizes_beyond_the_descriptors(lib):
    """Sizes that a 32-bit field would cut are refused, not cut (tensors without
    storage stand in for ones of that size)."""
    import torch
    big = (1 << 32) + 64
    with pytest.raises(ValueError):
        kdn._int32(big)
    with pytest.raises(ValueError):
        kdn.make_scan_desc(1, 1, big, 64, kdn.F32, kdn.F32)
    with pytest.raises(ValueError):
        kdn._norm_desc(torch.empty(1, big, device="meta"), "x", torch.empty(big, device="meta"),
                       torch.float32, 1e-6)
    assert kdn._int32(5, (1 << 31) - 1) == (5, (1 << 31) - 1)


def test_binding_refuses_cpu_tensors(lib):
    import torch
    x = torch.zeros(2, 64)
    w = torch.ones(64)
    y = torch.zeros(1, 1, 4, 64)
    for call in (lambda: kdn.rms_norm(x, w), lambda: kdn.rms_norm_quant(x, w),
                 lambda: kdn.rms_norm_backward(x, x, w, w), lambda: kdn.quantize(x),
                 lambda: kdn.gated_scan(y, y), lambda: kdn.gated_scan_backward(y, y, y),
                 lambda: kdn.gated_scan_step(y[0], y[0], y[0])):
        with pytest.raises(kdn.KdnError):
            call()


GEMM_BAD = [
    (dict(M=-1), 2), (dict(N=-1), 2), (dict(K=-16), 2), (dict(ldc=199), 2), (dict(K=24), 3),
    (dict(dtype=2), 3), (dict(K=(1 << 23) + 16), 3), (dict(M=(1 << 26) + 1), 3), (dict(N=(1 << 26) + 1, ldc=(1 << 26) + 1), 3), (dict(ldc=(1 << 26) + 1), 3),
    (dict(M=1 << 20, N=1 << 20, ldc=1 << 20), 3),
]


def _gemm(M=20, N=200, K=256, ldc=200, dtype=kdn.BF16):
    d = kdn.KdnGemmDesc()
    d.M, d.N, d.K, d.ldc, d.dtype = M, N, K, ldc, dtype
    return d


@pytest.mark.parametrize("kw,code", GEMM_BAD, ids=[str(k) for k, _ in GEMM_BAD])
def test_quant_gemm_refuses_descriptors(lib, kw, code):
    assert lib.kdn_quant_gemm(ctypes.byref(_gemm(**kw)), *([FAKE] * 5), None) == code


def test_quant_gemm_refuses_arguments(lib):
    d = ctypes.byref(_gemm())
    assert lib.kdn_quant_gemm(None, *([FAKE] * 5), None) == 1
    for i in range(5):
        args = [FAKE] * 5
        args[i] = None
        assert lib.kdn_quant_gemm(d, *args, None) == 1
    for i in (0, 2, 4):
        args = [FAKE] * 5
        args[i] = ODD
        assert lib.kdn_quant_gemm(d, *args, None) == 5
    assert lib.kdn_quant_gemm(ctypes.byref(_gemm(M=0)), *([None] * 5), None) == 0
    assert lib.kdn_quant_gemm(ctypes.byref(_gemm(N=0)), *([None] * 5), None) == 0


def test_layer_in_8_bits_host_side_checks(lib):
    def desc(B=1, T=16, H=2, D=64, dk=32, dv=32, chunk=16, dtype=kdn.F32):
        return kdn.make_layer_desc(B, T, H, D, dk, dv, chunk, "diagonal", dtype)

    d = desc()
    need = kdn.layer_quant_workspace_bytes(d)
    core = kdn.forward_workspace_bytes(kdn.make_desc(1, 2, 16, 32, 32, 16, "diagonal", kdn.F32, kdn.F32))
    # Z (198 columns in rows of 256), 8 bits and scales, q k v o, three gates
    expect = 16 * 256 * 4 + 16 * 64 + 16 * 4 + 4 * 2 * 16 * 32 * 4 + 3 * 2 * 16 * 4 + core
    assert expect <= need <= expect + 11 * 256
    for kw in (dict(D=40), dict(D=16400), dict(dk=48), dict(H=90), dict(dtype=7), dict(B=1 << 15, T=1 << 15)):
        assert kdn.layer_quant_workspace_bytes(desc(**kw)) == 0, kw
    call = lib.kdn_layer_quant_forward

    def args(**kw):
        a = dict(x=FAKE, residual=FAKE, rd=kdn.F32, nw=FAKE, eps=1e-6, wi=FAKE, wis=FAKE, bg=FAKE, wo=FAKE,
                 wos=FAKE, l0=None, s0=None, y=FAKE, s=FAKE, st=None, lt=None, ws=FAKE, n=need, stream=None)
        a.update(kw)
        return list(a.values())

    assert call(None, *args()) == 1
    for n in ("x", "nw", "wi", "wis", "bg", "wo", "wos", "y", "s", "residual", "ws"):
        assert call(ctypes.byref(d), *args(**{n: None})) == 1, n
    for n in ("x", "residual", "nw", "wi", "wo", "y", "s", "ws"):
        assert call(ctypes.byref(d), *args(**{n: ODD})) == 5, n
    assert call(ctypes.byref(d), *args(n=need - 1)) == 4
    assert call(ctypes.byref(d), *args(eps=-1.0)) == 2
    assert call(ctypes.byref(d), *args(rd=kdn.BF16)) == 3
    assert call(ctypes.byref(desc(D=40)), *args()) == 3
    assert call(ctypes.byref(desc(B=0)), *([None] * 2), kdn.F32, None, 1e-6, *([None] * 12), 0, None) == 0
