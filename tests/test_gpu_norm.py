"""RMS norm with the residual's addition (in the input's type and in 8 bits), its
backward and the quantiser, on the GPU against the formulas in 64 bits.

u = 2^-24 is float32's half step, relative.  A row's sum of squares passes at most
64 additions in a thread and 8 across threads, all of positive terms, and its
products round once each: 74 u; rstd takes half of that and 4 more roundings, y two
products: 48 u in all."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _inputs(rows, d, dtype, res, seed):
    g = _gen(seed)
    x = torch.randn(rows, d, generator=g).to(TYPES[dtype])
    r = None if res is None else (3 * torch.randn(rows, d, generator=g)).to(TYPES[res])
    w = 1 + 0.3 * torch.randn(d, generator=g)
    return x, r, w


def _plain(x, r, w):
    s = x if r is None else (x.float() + r.float()).to(r.dtype)
    f = s.double()
    rstd = 1 / torch.sqrt(f.square().mean(1) + EPS)
    return s, rstd, f * rstd[:, None] * w.double()


def _cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


# rows, d, dtype, residual's dtype: one row, one vector, ragged blocks, a wave per
# row up to 1024 columns and a workgroup per row beyond, the widest row
SHAPES = [
    (1, 8, "f32", None), (1, 8, "bf16", "bf16"), (3, 64, "bf16", "f32"), (5, 120, "bf16", "bf16"),
    (7, 136, "f32", "f32"), (130, 512, "bf16", None), (9, 520, "bf16", "f32"), (2, 1024, "f32", "f32"),
    (33, 1032, "bf16", "bf16"), (6, 2048, "bf16", "bf16"), (5, 2056, "f32", "f32"),
    (3, 4096, "bf16", "f32"), (4, 4104, "bf16", "bf16"), (2, 8192, "f32", None),
    (2, 8200, "bf16", "bf16"), (3, 16384, "f32", "f32"), (3, 16384, "bf16", "f32"),
]
IDS = ["-".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_norm_matches_the_formula(shape):
    rows, d, dtype, res = shape
    x, r, w = _inputs(rows, d, dtype, res, 11)
    s0, rstd0, y0 = _plain(x, r, w)
    say(f"[gpu] rms_norm {shape}")
    y, s, rstd = kdn.rms_norm(*_cuda(x, w), *_cuda(r), eps=EPS)
    assert y.dtype == x.dtype and torch.equal(s.cpu(), s0)
    assert ((rstd.cpu().double() - rstd0).abs() <= 42 * U * rstd0).all()
    tol = 48 * U + (HALF[y.dtype] if dtype == "bf16" else 0)
    assert ((y.cpu().double() - y0).abs() <= tol * y0.abs() + 1e-37).all()


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_norm_in_8_bits_matches_the_formula(shape):
    rows, d, dtype, res = shape
    x, r, w = _inputs(rows, d, dtype, res, 12)
    s0, _, y0 = _plain(x, r, w)
    say(f"[gpu] rms_norm_quant {shape}")
    q, scale, s = kdn.rms_norm_quant(*_cuda(x, w), *_cuda(r), eps=EPS)
    assert torch.equal(s.cpu(), s0)
    _check_quantized(q, scale, y0, 1, 48 * U)


def _check_quantized(q, scale, x, block_rows, rel):
    """x in 64 bits, `rel` how far the values that were rounded may be off it.  The
    scale is a maximum over 448: one more rounding.  An element is off by half a
    step (2^-4 relative, or half of the smallest step 2^-9 times the scale), on a
    value that is `rel` off and was multiplied by a reciprocal (3 u)."""
    rows, d = x.shape
    nr, nb = -(-rows // block_rows), -(-d // 128)
    pad = torch.zeros(nr * block_rows, nb * 128, dtype=torch.float64)
    pad[:rows, :d] = x
    amax = pad.view(nr, block_rows, nb, 128).abs().amax(dim=(1, 3))
    s0 = (amax / 448).clamp_min(2.0 ** -126)
    s = scale.cpu().double().view(nr, nb)
    assert ((s - s0).abs() <= (rel + 2 * U) * s0).all()
    wide = s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :d]
    got = q.cpu().view(rows, d).to(torch.float64) * wide
    assert torch.isfinite(got).all()
    off = (got - x).abs()
    assert (off <= (2.0 ** -4 + 2 * rel + 8 * U) * x.abs() + 2.0 ** -10 * (1 + 1e-5) * wide).all()


def test_norm_in_place_and_without_rstd():
    x, r, w = _inputs(19, 264, "bf16", "f32", 13)
    s0, _, _ = _plain(x, r, w)
    xd, rd, wd = _cuda(x, r, w)
    y, s, _ = kdn.rms_norm(xd, wd, rd.clone(), eps=EPS)
    at = rd.clone()
    y2, s2, _ = kdn.rms_norm(xd, wd, at, eps=EPS, in_place=True)
    assert s2.data_ptr() == at.data_ptr()
    assert torch.equal(y, y2) and torch.equal(s.cpu(), s0) and torch.equal(s2, s)
    n = kdn._norm_desc(xd, "x", wd, torch.float32, EPS)
    y3, s3 = torch.empty_like(y), torch.empty_like(s)
    assert kdn.load_library().kdn_rms_norm(ctypes.byref(n), xd.data_ptr(), rd.data_ptr(),
                                           wd.data_ptr(), y3.data_ptr(), s3.data_ptr(), None,
                                           torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y3, y) and torch.equal(s3, s)


def test_norm_of_zero_rows_and_zero_values():
    w = torch.ones(64).cuda()
    y, s, rstd = kdn.rms_norm(torch.empty(0, 64).cuda(), w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    q, scale, _ = kdn.rms_norm_quant(torch.zeros(3, 64).cuda(), w)
    assert (q.float() == 0).all() and (scale == 2.0 ** -126).all()
    dx, dw = kdn.rms_norm_backward(torch.empty(0, 64).cuda(), torch.empty(0, 64).cuda(), w,
                                   torch.empty(0).cuda())
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_quantize_keeps_nan_and_infinity():
    x = torch.randn(4, 256, generator=_gen(1))
    x[0, 3], x[1, 200], x[2, 5] = float("nan"), float("inf"), float("-inf")
    q, scale = (t.cpu() for t in kdn.quantize(x.cuda()))
    v = q.float() * scale.repeat_interleave(128, 1)
    assert torch.isnan(scale[0, 0]) and torch.isnan(v[0, :128]).all()
    assert torch.isinf(scale[1, 1]) and torch.isinf(scale[2, 0])
    assert torch.isnan(v[1, 200]) and torch.isnan(v[2, 5])
    assert torch.isfinite(v[0, 128:]).all() and torch.isfinite(v[3]).all()
    assert torch.isfinite(v[1, :128]).all() and torch.isfinite(v[2, 128:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 128), (129, 136), (127, 1000), (300, 2048)])
def test_quantize_matches_the_formula(rows, d, block_rows, dtype):
    x = torch.randn(rows, d, generator=_gen(rows + d))
    x *= 10.0 ** torch.linspace(-30, 30, rows)[:, None]  # blocks of every size
    x[:, ::7] = 0
    x = x.to(TYPES[dtype])
    say(f"[gpu] quantize {rows} {d} {block_rows} {dtype}")
    q, scale = kdn.quantize(x.cuda(), block_rows=block_rows)
    _check_quantized(q, scale, x.double(), block_rows, 0.0)


@pytest.mark.parametrize("shape", SHAPES + [(3000, 64, "bf16", "bf16"), (5000, 2056, "bf16", "f32")],
                         ids=IDS + ["3000-64", "5000-2056"])
@pytest.mark.parametrize("with_ds", [False, True])
def test_norm_backward_matches_the_formula(shape, with_ds):
    """dx: the mean over a row is off by at most 90 u of the mean of the absolute
    values (64 additions in a thread, 8 across, the products' own roundings), each
    of the other terms by at most 8 u.  dw: an element passes its wave's rows, 3
    additions across waves, ceil(groups / 128) + 7 across workgroups."""
    rows, d, dtype, res = shape
    g = _gen(21)
    s = torch.randn(rows, d, generator=g).to(TYPES[res or dtype])
    dy = torch.randn(rows, d, generator=g).to(TYPES[dtype])
    w = 1 + 0.3 * torch.randn(d, generator=g)
    ds = torch.randn(rows, d, generator=g) if with_ds else None
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + EPS)).float()
    say(f"[gpu] rms_norm_backward {shape} ds {with_ds}")
    args = _cuda(dy, s, w, rstd, ds)
    dx, dw = kdn.rms_norm_backward(*args)
    r = rstd.double()[:, None]
    xh, dn = s.double() * r, dy.double() * w.double()
    p = dn * xh
    dx0 = r * (dn - xh * p.mean(1, keepdim=True)) + (0 if ds is None else ds.double())
    tol = U * (8 * r * dn.abs() + 98 * r * xh.abs() * p.abs().mean(1, keepdim=True)
               + (0 if ds is None else 2 * ds.abs().double()))
    assert ((dx.cpu().double() - dx0).abs() <= tol).all()
    t = dy.double() * xh
    rpb = 4 if d <= 1024 else 1  # rows of a workgroup
    units = -(-rows // rpb)
    groups = min(units, 512 if units < 4096 else 1024)
    steps = -(-rows // (groups * rpb)) + 3 + -(-groups // 128) + 7 + 3
    assert ((dw.cpu().double() - t.sum(0)).abs() <= steps * U * t.abs().sum(0)).all()
    again = kdn.rms_norm_backward(*args)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_norm_backward_against_differences():
    """The gradient along random directions against central differences of the
    formula in 64 bits (h = 1e-5: truncation about h^2 = 1e-10, cancellation about
    1e-16 / h = 1e-11, both relative to a loss of order 10; the kernel's float32
    sums over 5 x 72 elements of order 1: 1e-4)."""
    g = _gen(5)
    s, w, c, cs = (torch.randn(5, 72, generator=g) for _ in range(4))
    w = w[0]

    def loss(s, w):
        return ((s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * w) * c.double()).sum() + (s * cs.double()).sum()

    sd, _, rstd = kdn.rms_norm(s.cuda(), w.cuda(), eps=EPS)
    dx, dw = kdn.rms_norm_backward(c.cuda(), s.cuda(), w.cuda(), rstd, cs.cuda())
    for k in range(4):
        es, ew = torch.randn(5, 72, generator=g).double(), torch.randn(72, generator=g).double()
        h = 1e-5
        diff = (loss(s.double() + h * es, w.double() + h * ew)
                - loss(s.double() - h * es, w.double() - h * ew)) / (2 * h)
        got = (dx.cpu().double() * es).sum() + (dw.cpu().double() * ew).sum()
        assert abs(got - diff) <= 1e-4 * max(1.0, abs(diff))


def test_norm_backward_over_its_own_ds():
    g = _gen(9)
    s, dy, ds = (torch.randn(40, 1032, generator=g).cuda() for _ in range(3))
    w = torch.ones(1032).cuda()
    _, _, rstd = kdn.rms_norm(s, w)
    dx, dw = kdn.rms_norm_backward(dy, s, w, rstd, ds)
    lib = kdn.load_library()
    n = kdn._norm_desc(dy, "dy", w, torch.float32, 0.0)
    ws = torch.empty(lib.kdn_rms_norm_backward_workspace_bytes(ctypes.byref(n)), dtype=torch.uint8, device="cuda")
    dw2 = torch.empty_like(dw)
    assert lib.kdn_rms_norm_backward(ctypes.byref(n), dy.data_ptr(), s.data_ptr(), w.data_ptr(),
                                     rstd.data_ptr(), ds.data_ptr(), ds.data_ptr(), dw2.data_ptr(),
                                     ws.data_ptr(), ws.numel(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(ds, dx) and torch.equal(dw, dw2)


def test_norm_refuses_mismatched_tensors():
    x, w = torch.zeros(4, 64).cuda(), torch.ones(64).cuda()
    for bad, err in (
            (lambda: kdn.rms_norm(x, w[:32]), ValueError),
            (lambda: kdn.rms_norm(x, w.bfloat16()), ValueError),
            (lambda: kdn.rms_norm(x, w, x[:2]), ValueError),
            (lambda: kdn.rms_norm(x, w, x.bfloat16()), ValueError),
            (lambda: kdn.rms_norm(x.t(), torch.ones(4).cuda()), ValueError),
            (lambda: kdn.rms_norm(x.half(), w), TypeError),
            (lambda: kdn.rms_norm(x, w.cpu()), kdn.KdnError),
            (lambda: kdn.rms_norm(x[:, :20].contiguous(), torch.ones(20).cuda()), kdn.KdnError),
            (lambda: kdn.quantize(x, block_rows=2), kdn.KdnError),
            (lambda: kdn.quantize(x[None], block_rows=128), ValueError),
            (lambda: kdn.rms_norm_backward(x, x[:2], w, torch.ones(4).cuda()), ValueError),
            (lambda: kdn.rms_norm_backward(x, x, w, torch.ones(3).cuda()), ValueError),
            (lambda: kdn.rms_norm_backward(x, x, w, torch.ones(4).cuda(), x.bfloat16()), ValueError)):
        with pytest.raises(err):
            bad()


def test_norm_in_a_captured_graph():
    """Forward and backward replayed on new inputs, with eager work between."""
    g = _gen(3)
    x, r = torch.randn(70, 520, generator=g).cuda().bfloat16(), torch.randn(70, 520, generator=g).cuda()
    w, dy = torch.randn(520, generator=g).cuda(), torch.randn(70, 520, generator=g).cuda().bfloat16()

    def step():
        y, s, rstd = kdn.rms_norm(x, w, r)
        q, scale, _ = kdn.rms_norm_quant(x, w, r)
        return (y, s, q.float(), scale, *kdn.rms_norm_backward(dy, s, w, rstd, r))

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(torch.randn(70, 520, generator=g).cuda())
        r.copy_(torch.randn(70, 520, generator=g).cuda())
        torch.cuda.synchronize()
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), k
