"""What the sums of the 8-bit product are, where they cancel: every eight neighbouring k
hold 448 448, -448 448 and a few small products, whose sum is what is left.

Small products are whole numbers and C's exact value is below 2^24, so float32 sums give
it exactly: a float32 C, and a bfloat16 C of few rows (rounded once).  A bfloat16 C of more
rows goes through the 8-bit matrix instruction, which drops of each of eight products what
lies below 2^-14 of the largest: at most 7 2^-14 of the sum of absolute values, beside C's
own rounding (2^-8)."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def _cancelling(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-3, 4, (M, K), generator=g).float()
    b = torch.randint(-3, 4, (N, K), generator=g).float()
    i, j = seed % 8, (seed + 3) % 8
    a[:, i::8], a[:, j::8] = 448.0, 448.0
    b[:, i::8], b[:, j::8] = 448.0, -448.0
    kb = -(-K // 128)
    ops = (a.to(FP8).cuda(), torch.ones(M, kb).cuda(), b.to(FP8).cuda(), torch.ones(-(-N // 128), kb).cuda())
    return ops, a.double() @ b.double().t(), a.double().abs() @ b.double().abs().t()


# few rows by each rule that takes them (up to 4; up to 16 with at most 4096 columns; up to
# 32 with a short K too), and tiles of every size
FEW = [(1, 40, 48), (1, 6192, 2048), (4, 5000, 272), (12, 300, 400), (16, 4096, 128), (20, 130, 1024), (32, 200, 512)]
TILES = [(33, 100, 128), (64, 200, 2048), (300, 500, 1040), (500, 1000, 4112), (2000, 2100, 400), (4096, 4096, 272)]


def _id(s):
    return "x".join(map(str, s))


@pytest.mark.parametrize("seed", [1, 6])
@pytest.mark.parametrize("shape", FEW + TILES, ids=_id)
def test_float32_results_cancel_exactly(shape, seed):
    ops, want, _ = _cancelling(*shape, seed)
    say(f"[gpu] cancelling product {shape} f32")
    c = kdn.quant_matmul(*ops, out_dtype=torch.float32).cpu()
    assert int((c.double() != want).sum()) == 0


@pytest.mark.parametrize("seed", [1, 6])
@pytest.mark.parametrize("shape", FEW, ids=_id)
def test_bfloat16_results_of_few_rows_cancel_exactly(shape, seed):
    ops, want, _ = _cancelling(*shape, seed)
    say(f"[gpu] cancelling product {shape} bf16")
    c = kdn.quant_matmul(*ops).cpu()
    assert int((c != want.float().bfloat16()).sum()) == 0


@pytest.mark.parametrize("seed", [1, 6])
@pytest.mark.parametrize("shape", TILES, ids=_id)
def test_bfloat16_results_stay_within_the_stated_bound(shape, seed):
    ops, want, size = _cancelling(*shape, seed)
    say(f"[gpu] cancelling product {shape} bf16")
    c = kdn.quant_matmul(*ops).cpu().double()
    off = (c - want).abs()
    say(f"[gpu] largest error {float((off / size).max()):.3g} of the sum of absolute values")
    assert int((off > 7 * 2.0 ** -14 * size + 2.0 ** -8 * want.abs()).sum()) == 0
