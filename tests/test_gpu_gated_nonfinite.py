"""Infinities and NaN in the gated recurrence: they stay in their channel, reach every
state behind their token (every gradient before it) and none before."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

BAD = {"inf": float("inf"), "-inf": float("-inf"), "nan": float("nan")}


def _inputs(B, T, d, seed, gates):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # "slow": products stay in range for a while; "fast": below float32's range within a tile
    a = torch.sigmoid((3 if gates == "slow" else -4) + rand(B, 1, T, d))
    return rand(B, 1, T, d), a, rand(B, 1, d)


# one tile; a chain of tiles; a walk of several tiles (one sequence in a batch)
@pytest.mark.parametrize("B,T,d", [(1, 50, 32), (1, 5000, 64), (256, 1500, 64)])
@pytest.mark.parametrize("gates", ["slow", "fast"])
@pytest.mark.parametrize("what", list(BAD))
def test_forward(B, T, d, gates, what):
    x, a, h0 = _inputs(B, T, d, 7, gates)
    say(f"[gpu] gated scan with {what} {B, T, d, gates}")
    clean, clean_T = kdn.gated_scan(x, a, h0)
    for at in (-1, 0, 13, T // 2, T - 1):  # -1: in the state that enters
        xb, hb = x.clone(), h0.clone()
        if at < 0:
            hb[B - 1, 0, 3] = BAD[what]
        else:
            xb[B - 1, 0, at, 3] = BAD[what]
        h, h_T = kdn.gated_scan(xb, a, hb)
        bad = torch.zeros_like(h, dtype=torch.bool)
        bad[B - 1, 0, max(at, 0):, 3] = True
        assert not torch.isfinite(h[bad]).any() and not torch.isfinite(h_T[B - 1, 0, 3])
        assert torch.equal(h[~bad], clean[~bad])
        keep = torch.ones_like(h_T, dtype=torch.bool)
        keep[B - 1, 0, 3] = False
        assert torch.equal(h_T[keep], clean_T[keep])


@pytest.mark.parametrize("B,T,d", [(1, 50, 32), (1, 5000, 64), (256, 1500, 64)])
@pytest.mark.parametrize("gates", ["slow", "fast"])
@pytest.mark.parametrize("what", list(BAD))
def test_backward(B, T, d, gates, what):
    x, a, h0 = _inputs(B, T, d, 8, gates)
    say(f"[gpu] gated scan backward with {what} {B, T, d, gates}")
    h, _ = kdn.gated_scan(x, a, h0)
    clean = kdn.gated_scan_backward(a, h, x, h0, h0)
    for at in (0, 13, T // 2, T - 1, T):  # T: in the gradient of the state that leaves
        dh, dh_T = x.clone(), h0.clone()
        if at == T:
            dh_T[B - 1, 0, 5] = BAD[what]
        else:
            dh[B - 1, 0, at, 5] = BAD[what]
        g = kdn.gated_scan_backward(a, h, dh, h0, dh_T)
        bad = torch.zeros_like(h, dtype=torch.bool)
        bad[B - 1, 0, :at + 1, 5] = True
        for n in ("dx", "da"):
            assert not torch.isfinite(g[n][bad]).any() and torch.equal(g[n][~bad], clean[n][~bad]), n
        keep = torch.ones_like(h0, dtype=torch.bool)
        keep[B - 1, 0, 5] = False
        assert not torch.isfinite(g["dh0"][B - 1, 0, 5]) and torch.equal(g["dh0"][keep], clean["dh0"][keep])
