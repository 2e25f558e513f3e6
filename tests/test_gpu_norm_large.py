"""The norm's backward over many rows per workgroup: small whole numbers and rstd = 1, so
that dweight's sums stay below 2^24 and are exact in any order; a row that is dropped,
doubled or taken from elsewhere shows."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


# rows of a wave and of a workgroup, each width of a thread's columns; many rounds per
# workgroup with a last one that is not full; just above and below the rule for 1024
@pytest.mark.parametrize("rows,d", [(4_000_003, 72), (700_001, 1024), (1_500_001, 1032), (300_007, 4096),
                                    ((1 << 20) + 3, 4104), (70_001, 16384), (4095, 2048), (4097, 2048), (16_381, 512),
                                    (16_389, 512)])
@pytest.mark.parametrize("types", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)], ids=["bf16", "bf16-f32"])
def test_dweight_is_exact_on_whole_numbers(rows, d, types):
    t, ts = types
    g = torch.Generator(device="cuda").manual_seed(rows)
    whole = lambda td: torch.randint(-1, 3, (rows, d), generator=g, device="cuda", dtype=torch.int8).to(td)  # noqa: E731
    dy, s = whole(t), whole(ts)
    say(f"[gpu] norm backward of {rows} x {d} {types}")
    dx, dw = kdn.rms_norm_backward(dy, s, torch.ones(d, device="cuda"), torch.ones(rows, device="cuda"))
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, 1 << 16):
        want += (dy[lo:lo + (1 << 16)].double() * s[lo:lo + (1 << 16)].double()).sum(0)
    assert float(want.abs().max()) < 2 ** 24 and float(want.min()) > 0
    assert int((dw.double() != want).sum()) == 0
    # dx = dn - xhat mean(dn xhat): 90 u of the mean, and the last roundings, as in a single row
    for lo in (0, rows // 2, rows - 50):
        a, b = dy[lo:lo + 50].double(), s[lo:lo + 50].double()
        p = a * b
        want_dx = a - b * p.mean(1, keepdim=True)
        tol = 2.0 ** -24 * (8 * a.abs() + 98 * b.abs() * p.abs().mean(1, keepdim=True))
        assert ((dx[lo:lo + 50].double() - want_dx).abs() <= tol).all()
