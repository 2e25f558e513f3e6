"""8-bit operands bit for bit: the quantiser and the norm's 8-bit output against the
format's definition in elementary float32 operations,
    scale = max(max |x| * (1 / 448), 2^-126),   element = e4m3(x / scale),
each rounded once, to nearest even (on the CPU, whose products and quotients are
IEEE's).  No tolerance: equal bits."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def _blocks(x, block_rows):
    rows, d = x.shape
    nr, nb = -(-rows // block_rows), -(-d // 128)
    pad = torch.nn.functional.pad(x.float(), (0, nb * 128 - d, 0, nr * block_rows - rows))
    return pad.view(nr, block_rows, nb, 128)


def _expect(x, block_rows):
    """(elements as bytes [rows, d], scale [blocks of rows, blocks of columns])"""
    rows, d = x.shape
    g = _blocks(x, block_rows)
    scale = (g.abs().amax(dim=(1, 3)) * torch.tensor(1 / 448)).clamp_min(2.0 ** -126)
    q = (g / scale[:, None, :, None]).clamp(-448, 448)
    return q.reshape(g.shape[0] * block_rows, -1)[:rows, :d].to(FP8).view(torch.uint8), scale


def _same(got, want):
    q, scale = (t.cpu() for t in got)
    q0, scale0 = want
    assert torch.equal(scale.view(scale0.shape), scale0)
    share = (q.view(torch.uint8).view(q0.shape) != q0).float().mean().item()
    assert share == 0, share


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,d", [(1, 8), (129, 136), (700, 1000), (1100, 2056)])
def test_quantize_gives_the_definitions_bits(rows, d, block_rows, dtype):
    x = torch.randn(rows, d, generator=torch.Generator().manual_seed(rows)).to(dtype)
    say(f"[gpu] quantize {rows} {d} {block_rows} {dtype}")
    _same(kdn.quantize(x.cuda(), block_rows=block_rows), _expect(x, block_rows))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_gives_the_definitions_bits_in_every_binade(block_rows, dtype):
    """Blocks from the smallest numbers (scale 2^-126, and just above it) to the largest,
    with elements far below their block's largest, and zeros of both signs."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(128 * 64, 128, generator=g)
    x *= 2.0 ** (-20 * torch.rand(x.shape, generator=g))  # inside a block
    size = torch.linspace(-150, 124, 64).repeat_interleave(128)[:, None]
    x = (x * 2.0 ** (size / 2) * 2.0 ** (size / 2)).to(dtype)
    x[::3, ::5], x[1::3, ::5] = 0.0, -0.0
    assert torch.isfinite(x).all()
    _same(kdn.quantize(x.cuda(), block_rows=block_rows), _expect(x, block_rows))


def test_quantize_gives_the_definitions_bits_on_borders():
    """Quotients on and next to the borders between two elements: x = border * scale,
    rounded, and its float32 neighbours."""
    e = torch.arange(127, dtype=torch.uint8).view(FP8).float()  # all elements, ascending
    border = (e[1:] + e[:-1]) / 2
    rows = []
    g = torch.Generator().manual_seed(4)
    for top in (1 + torch.rand(40, generator=g)) * 2.0 ** torch.randint(-100, 100, (40,), generator=g):
        s = top * torch.tensor(1 / 448)
        at = border * s
        for v in (at, torch.nextafter(at, torch.tensor(0.0)), torch.nextafter(at, torch.tensor(3e38))):
            v = torch.where(v <= top, v, 0.0)
            rows.append(torch.cat((top[None], -v, torch.zeros(1))))
    x = torch.stack(rows)
    assert x.shape == (120, 128)
    _same(kdn.quantize(x.cuda()), _expect(x, 1))


def test_quantize_of_infinities_gives_the_definitions_bits():
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(5))
    x[0, 3], x[2, 140] = float("inf"), float("-inf")
    q, scale = (t.cpu() for t in kdn.quantize(x.cuda()))
    q0, scale0 = _expect(x, 1)
    assert torch.equal(scale, scale0)
    nan = torch.isnan(q.float())
    assert torch.equal(nan, torch.isnan(q0.view(FP8).float())) and nan.sum() == 2
    assert torch.equal(q.view(torch.uint8)[~nan], q0[~nan])


@pytest.mark.parametrize("rows,d", [(5, 8), (70, 520), (33, 1032), (9, 4104), (5, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_in_8_bits_is_the_norm_quantised(rows, d, residual):
    """In float32 the 8-bit output is the definition's, of the same y."""
    g = torch.Generator().manual_seed(d)
    x, w = torch.randn(rows, d, generator=g), 1 + 0.3 * torch.randn(d, generator=g)
    r = torch.randn(rows, d, generator=g).cuda() if residual else None
    say(f"[gpu] rms_norm_quant {rows} {d} {residual}")
    y, s, _ = kdn.rms_norm(x.cuda(), w.cuda(), r)
    q, scale, s2 = kdn.rms_norm_quant(x.cuda(), w.cuda(), r)
    assert torch.equal(s, s2)
    _same((q, scale), _expect(y.cpu(), 1))
