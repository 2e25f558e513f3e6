"""The matrix product of 8-bit operands on the GPU against the formula in 64 bits.

Tolerance: u = 2^-24.  A block's 128 products are exact in float32 and their sum
passes 128 additions, each off by at most a whole step (2 u) whichever way the matrix
unit rounds; scaling rounds twice, and a block's part passes at most ceil(K / 128) + 16
additions afterwards: u (258 + ceil(K / 128) + 16) of the sum of absolute values.

A result in bfloat16 is rounded once more (2^-8), and its products go through the 8-bit
matrix instruction, which adds 8 of them aligned to the largest and drops what lies
below 2^-14 of the largest's power of two: with |p| the largest product of a group, at
most 7 products lose less than 2^-14 |p| each, and |p| is at most the group's sum of
absolute values, so 7 2^-14 of the sum of absolute values in all.  Where the signs are
random the losses cancel, so the 2-norm of the error is held to the rounding's alone,
2^-8 (1 + 1/16) of the result's, where there are 4096 results and more."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _operands(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(M, K, generator=g, device="cuda")
    a *= 10.0 ** (torch.rand(M, 1, generator=g, device="cuda") * 4 - 2)  # rows of every size
    b = torch.randn(N, K, generator=g, device="cuda")
    return (*kdn.quantize(a), *kdn.quantize(b, block_rows=128))


def _wide(q, s, block_rows):
    r, k = q.shape
    return q.double() * s.double().repeat_interleave(block_rows, 0)[:r].repeat_interleave(128, 1)[:, :k]


def _check(c, a, sa, b, sb):
    K = a.shape[1]
    A, B = _wide(a, sa, 1), _wide(b, sb, 128)
    want, size = A @ B.t().contiguous(), A.abs() @ B.abs().t().contiguous()
    tol = U * (258 + -(-K // 128) + 16) * size
    if c.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs() + 7 * 2.0 ** -14 * size
    off = (c.double() - want).abs()
    assert (off <= tol).all(), float((off - tol).max())
    if c.numel() >= 4096:
        assert off.norm() <= 2.0 ** -8 * 17 / 16 * want.norm()


# one row to many; columns that are no multiple of anything; k below, at and just
# beyond whole blocks; few columns; sizes for each tile
SHAPES = [
    (1, 1, 16), (1, 16, 128), (1, 200, 2048), (3, 130, 144), (16, 128, 256), (17, 257, 1040),
    (32, 64, 112), (33, 100, 128), (64, 1000, 8192), (65, 65, 16), (65, 300, 272), (100, 129, 4112),
    (128, 128, 128), (129, 1, 384), (257, 513, 640), (509, 2048, 2064), (2000, 2100, 400),
    (40, 70, 1024), (200, 300, 1040), (300, 190, 1168), (64, 64, 3200), (448, 4000, 2048), (450, 4100, 1040),
    (2048, 2048, 2048), (4095, 4100, 1168), (4096, 4096, 256), (70, 6192, 2048), (5000, 24, 96),
    (4, 4500, 1040), (7, 4500, 1040), (8, 5000, 272), (20, 130, 1040), (40, 6001, 2064), (257, 2100, 4112),
    (4090, 4093, 144), (4096, 4095, 272),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_product_matches_the_formula(shape, dtype):
    ops = _operands(*shape, seed=41)
    say(f"[gpu] quant_matmul {shape} {dtype}")
    c = kdn.quant_matmul(*ops, out_dtype=dtype)
    assert c.shape == shape[:2] and c.dtype == dtype
    _check(c, *ops)
    assert torch.equal(c, kdn.quant_matmul(*ops, out_dtype=dtype))


def test_product_of_small_whole_numbers_is_exact():
    """Scales of one and whole numbers up to 8: every sum is a whole number below
    2^24, so the product has to be exact."""
    g = torch.Generator().manual_seed(2)
    for M, N, K in ((5, 40, 400), (300, 200, 1040), (4096, 4096, 272)):
        a = torch.randint(-8, 9, (M, K), generator=g).float().cuda()
        b = torch.randint(-8, 9, (N, K), generator=g).float().cuda()
        kb = -(-K // 128)
        c = kdn.quant_matmul(a.to(torch.float8_e4m3fn), torch.ones(M, kb).cuda(),
                             b.to(torch.float8_e4m3fn), torch.ones(-(-N // 128), kb).cuda(),
                             out_dtype=torch.float32)
        assert torch.equal(c.double(), a.double() @ b.double().t().contiguous())


def test_product_uses_each_scale_where_it_belongs():
    """Operands of ones: C[m][n] = sum over blocks of (width of the block) sA sB, with
    scales that are powers of two, so exactly."""
    M, N, K = 300, 400, 336
    kb, nb = 3, 4
    ones = lambda r: torch.ones(r, K).cuda().to(torch.float8_e4m3fn)  # noqa: E731
    sa = 2.0 ** torch.randint(-3, 4, (M, kb)).float().cuda()
    sb = 2.0 ** torch.randint(-3, 4, (nb, kb)).float().cuda()
    width = torch.tensor([128.0, 128.0, 80.0]).cuda()
    want = (sa * width) @ sb.t().repeat_interleave(128, 1)[:, :N]
    for m in (1, 20, 60, 300):
        c = kdn.quant_matmul(ones(m), sa[:m].contiguous(), ones(N), sb, out_dtype=torch.float32)
        assert torch.equal(c, want[:m])


@pytest.mark.parametrize("M", [3, 64, 200, 5000])
def test_product_into_wider_rows(M):
    """ldc > N: what lies behind the columns stays (aligned and odd rows)."""
    N, K = 1000, 272
    a, sa, b, sb = _operands(M, N, K, seed=43)
    lib = kdn.load_library()
    for ldc, td, code in ((1008, torch.bfloat16, kdn.BF16), (1003, torch.bfloat16, kdn.BF16), (1001, torch.float32, kdn.F32)):
        d = kdn.KdnGemmDesc()
        d.M, d.N, d.K, d.ldc, d.dtype = M, N, K, ldc, code
        c = torch.full((M + 1, ldc), 7.0, dtype=td, device="cuda")
        assert lib.kdn_quant_gemm(ctypes.byref(d), a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(),
                                  c.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(c[:M, :N], kdn.quant_matmul(a, sa, b, sb, out_dtype=td))
        assert (c[M] == 7).all() and (c[:M, N:] == 7).all()


def test_product_keeps_nan_to_its_row_and_column():
    for M in (10, 300):
        a, sa, b, sb = _operands(M, 200, 256, seed=44)
        clean = kdn.quant_matmul(a, sa, b, sb)
        sa[3, 1] = float("nan")
        bad = b.view(torch.uint8).clone()
        bad[150, 7] = 0x7F  # NaN
        c = kdn.quant_matmul(a, sa, bad.view(torch.float8_e4m3fn), sb)
        assert torch.isnan(c[3]).all() and torch.isnan(c[:, 150]).all()
        rows, cols = [i for i in range(M) if i != 3], [i for i in range(200) if i != 150]
        assert torch.equal(c[rows][:, cols], clean[rows][:, cols])


def test_product_with_an_infinite_scale():
    """A row whose scale is infinite is infinite (or NaN where its sum in that block is
    zero), in tiles as in the kernel for few rows, also where the blocks are shared out
    and one share has one less; the others stay."""
    for K in (1040, 1168, 1152, 272):
        a, sa, b, sb = _operands(100, 200, K, seed=47)
        a = torch.where(a.float() == 0, 1.0, a.float()).to(a.dtype)
        b = torch.where(b.float() == 0, 1.0, b.float()).to(b.dtype)
        clean = kdn.quant_matmul(a, sa, b, sb)
        sa[7, -1] = float("inf")
        c = kdn.quant_matmul(a, sa, b, sb)
        assert not torch.isfinite(c[7]).any()
        s = kdn.quant_matmul(a[7:8].contiguous(), sa[7:8].contiguous(), b, sb)
        assert torch.equal(torch.isnan(c[7]), torch.isnan(s[0]))
        assert torch.equal(c[7][~torch.isnan(c[7])], s[0][~torch.isnan(s[0])])
        keep = [i for i in range(100) if i != 7]
        assert torch.equal(c[keep], clean[keep])


def test_product_of_no_rows_columns_or_depth():
    e = lambda r, k: torch.empty(r, k, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    s = lambda r, k: torch.ones(r, k, device="cuda")  # noqa: E731
    assert kdn.quant_matmul(e(0, 64), s(0, 1), e(9, 64), s(1, 1)).shape == (0, 9)
    assert kdn.quant_matmul(e(9, 64), s(9, 1), e(0, 64), s(0, 1)).shape == (9, 0)
    for m in (9, 500):
        assert (kdn.quant_matmul(e(m, 0), s(m, 0), e(40, 0), s(1, 0)) == 0).all()
    ops = _operands(12, 40, 64, seed=45)
    c = kdn.quant_matmul(ops[0].view(3, 4, 64), ops[1].view(3, 4, 1), *ops[2:])
    assert torch.equal(c.view(12, 40), kdn.quant_matmul(*ops))


def test_product_refuses_mismatched_tensors():
    a, sa, b, sb = _operands(20, 200, 256, seed=46)
    for bad, err in (
            (lambda: kdn.quant_matmul(a.float(), sa, b, sb), TypeError),
            (lambda: kdn.quant_matmul(a, sa, b[:, :128].contiguous(), sb), ValueError),
            (lambda: kdn.quant_matmul(a, sa[:, :1].contiguous(), b, sb), ValueError),
            (lambda: kdn.quant_matmul(a, sa, b, sb[:1]), ValueError),
            (lambda: kdn.quant_matmul(a, sa.double(), b, sb), ValueError),
            (lambda: kdn.quant_matmul(a, sa, b, sb, out_dtype=torch.float16), TypeError),
            (lambda: kdn.quant_matmul(a, sa, b.cpu(), sb), kdn.KdnError),
            (lambda: kdn.quant_matmul(a.view(40, 128)[::2], sa, b, sb), ValueError),
            (lambda: kdn.quant_matmul(a.view(640, 8), torch.ones(640, 1).cuda(), b.view(6400, 8),
                                      torch.ones(50, 1).cuda()), kdn.KdnError)):
        with pytest.raises(err):
            bad()


def test_norm_quantised_into_products_in_a_captured_graph():
    """As in a model: norm with the residual, 8 bits, a projection and another one of
    its quantised result, replayed with eager work between."""
    g = torch.Generator(device="cuda").manual_seed(6)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r, w = rand(70, 512).bfloat16(), rand(70, 512), 1 + 0.1 * rand(512)
    up, down = kdn.quantize(rand(1040, 512), 128), kdn.quantize(rand(512, 1040), 128)

    def step():
        q, s, res = kdn.rms_norm_quant(x, w, r)
        h = kdn.quant_matmul(q, s, *up)
        return h, kdn.quant_matmul(*kdn.quantize(h), *down), res

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(rand(70, 512))
        torch.cuda.synchronize()
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q), k
