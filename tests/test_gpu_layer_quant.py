"""The layer in 8 bits (kdn_layer_quant_forward) on the GPU.

Against the calls it is made of: the same kernels in the same order, so q, k, v and
the gates differ only by how they are rebuilt here (float32 arithmetic: 1e-6 relative,
or one rounding to bfloat16), and the read-out o by the recurrence's own bar.  An
element of o in 8 bits moves by a step (at most 2^-3 relative) where a difference of
e relative crosses a border, and borders lie 2^-4 relative apart or more, so a share
of at most 2 e / 2^-4 moves: with e = 1e-5 the 2-norm changes by 2^-3 sqrt(3.2e-4) =
2.2e-3, with e = 2e-2 by 2^-3 sqrt(0.64) = 0.1, beside the bar itself.

Against the oracle: the oracle takes the 8-bit operands as the values they stand for,
but not the rounding of o to 8 bits, which is off by 2^-4 |o| + 2^-10 scale per
element; with the recurrence's bar that bounds every element of y, and the 2-norm of
y's error is held to 2^-4 times 1.5 (o's own is below 2^-4, and a random W_out keeps
the ratio up to its sampling)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import TOL_BF16, TOL_F32, host, normwise, say
from kdn_inputs import layer_inputs
from oracle.layer import layer_forward as oracle_layer

pytestmark = pytest.mark.gpu

CASES = [
    # B, T, H, D, dk, dv, variant, dtype, chunk, residual's dtype
    (2, 100, 2, 64, 32, 32, "diagonal", "f32", 64, "f32"),
    (1, 130, 4, 144, 64, 32, "isotropic", "f32", 32, None),
    (2, 77, 3, 96, 32, 64, "diagonal", "bf16", 16, "f32"),
    (1, 64, 2, 256, 128, 128, "isotropic", "bf16", 64, "bf16"),
    (1, 1, 3, 32, 32, 32, "diagonal", "f32", 16, "f32"),
    (1, 300, 16, 2048, 128, 128, "diagonal", "bf16", 64, "bf16"),
]
IDS = [f"B{c[0]}T{c[1]}H{c[2]}D{c[3]}dk{c[4]}dv{c[5]}{c[6][:4]}{c[7]}res{c[9]}" for c in CASES]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _setup(case):
    B, T, H, D, dk, dv, variant, dtype, chunk, res = case
    p = layer_inputs(B, T, H, D, dk, dv, variant=variant, dtype=dtype, seed=37)
    t = {"x": torch.from_numpy(p["x"]).cuda().to(TYPES[dtype])}
    rng = np.random.default_rng(38)
    t["r"] = None if res is None else torch.from_numpy(rng.standard_normal((B, T, D), np.float32)).cuda().to(TYPES[res])
    t["w"] = torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).cuda()
    for n in ("W_in", "W_out"):
        t[n], t[n + "_scale"] = kdn.quantize(torch.from_numpy(np.ascontiguousarray(p[n].T)).cuda(), 128)
    t.update({n: torch.from_numpy(p[n]).cuda() for n in ("b_gate", "lambda0", "S0")})
    return p, t


def _run(case, t, **kw):
    _, _, H, _, dk, dv, variant, _, chunk, _ = case
    return kdn.layer_quant_forward(t["x"], t["w"], t["W_in"], t["W_in_scale"], t["b_gate"], t["W_out"],
                                   t["W_out_scale"], H, dk, dv, residual=t["r"], lambda0=t["lambda0"],
                                   S0=t["S0"], variant=variant, chunk=chunk, **kw)


def _wide(q, s):
    r, k = q.shape
    return q.double() * s.double().repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :k]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_in_8_bits_is_its_parts(case):
    B, T, H, D, dk, dv, variant, dtype, chunk, res = case
    say(f"[gpu] layer in 8 bits {case}")
    p, t = _setup(case)
    y, s, S_T, lam = _run(case, t)
    td = TYPES[dtype]
    q8, scale, s2 = kdn.rms_norm_quant(t["x"], t["w"], t["r"])
    assert torch.equal(s, s2)
    Z = kdn.quant_matmul(q8, scale, t["W_in"], t["W_in_scale"], out_dtype=td).float()

    def heads(lo, d):
        return Z[..., lo:lo + H * d].reshape(B, T, H, d).transpose(1, 2)

    q, k, v = heads(0, dk), heads(H * dk, dk), heads(2 * H * dk, dv)
    q, k = (x / x.square().sum(-1, keepdim=True).clamp_min(1e-12).sqrt() for x in (q, k))
    g = (Z[..., H * (2 * dk + dv):] + t["b_gate"]).reshape(B, T, 3, H).permute(2, 0, 3, 1)
    gates = [torch.sigmoid(g[0]), torch.nn.functional.softplus(g[1]), torch.nn.functional.softplus(g[2])]
    args = [x.to(td).contiguous() for x in (q, k, v, *gates)]
    o, S2, lam2 = kdn.forward(*args, t["lambda0"], t["S0"], variant=variant, chunk=chunk)
    rows = o.transpose(1, 2).reshape(B, T, H * dv).contiguous()
    y2 = kdn.quant_matmul(*kdn.quantize(rows), t["W_out"], t["W_out_scale"], out_dtype=td)
    bar = TOL_F32 if dtype == "f32" else TOL_BF16
    assert normwise(host(S_T), host(S2)) <= bar
    assert normwise(host(lam), host(lam2)) <= bar
    off, size = (y.double() - y2.double()).norm(), y2.double().norm()
    assert off <= (3e-3 if dtype == "f32" else 0.12) * size


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_in_8_bits_matches_the_oracle(case):
    B, T, H, D, dk, dv, variant, dtype, chunk, res = case
    p, t = _setup(case)
    y, s, S_T, lam = _run(case, t)
    q8, scale, _ = kdn.rms_norm_quant(t["x"], t["w"], t["r"])
    x = q8.double() * scale.double().repeat_interleave(128, -1)[..., :D]
    W_in, W_out = _wide(t["W_in"], t["W_in_scale"]), _wide(t["W_out"], t["W_out_scale"])
    ref = oracle_layer(x.cpu().numpy(), W_in.cpu().numpy().T, p["b_gate"], W_out.cpu().numpy().T, H, dk, dv,
                       p["lambda0"], p["S0"], variant, debug=True)
    bar = 1.5 * TOL_F32 if dtype == "f32" else 3e-2  # (3e-2: with Z rounded to bfloat16, as in the layer)
    assert normwise(host(S_T), ref["S_T"]) <= bar
    o = ref["o"].transpose(0, 2, 1, 3).reshape(B, T, H * dv)
    top = np.abs(ref["o"]).max(axis=(2, 3))  # [B, H]
    n = -(-H * dv // 128)
    pad = np.zeros((B, T, n * 128))
    pad[..., :H * dv] = np.abs(o)
    step = np.repeat(pad.reshape(B, T, n, 128).max(-1) / 448, 128, -1)[..., :H * dv]
    off_o = (2.0 ** -4 * np.abs(o) + 2.0 ** -10 * step
             + (1 + 2.0 ** -3) * bar * np.repeat(top[:, None, :], dv, -1))
    tol = off_o @ np.abs(W_out.cpu().numpy().T) + (2.0 ** -8 * np.abs(ref["y"]) if dtype == "bf16" else 0)
    off = np.abs(host(y) - ref["y"])
    say(f"[gpu] layer in 8 bits {case}: 2-norm {np.linalg.norm(off) / np.linalg.norm(ref['y']):.3g}")
    assert (off <= 1.01 * tol).all()
    if T > 1:
        assert np.linalg.norm(off) <= 1.5 * 2.0 ** -4 * np.linalg.norm(ref["y"])


def test_layer_in_8_bits_in_place_and_again():
    case = CASES[2]
    _, t = _setup(case)
    want = _run(case, t)
    again = _run(case, t)
    for a, b in zip(want, again):
        assert torch.equal(a, b)
    t["r"] = t["r"].clone()
    got = _run(case, t, in_place=True)
    assert got[1].data_ptr() == t["r"].data_ptr()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_layer_in_8_bits_token_by_token():
    """Prompt, then one token at a time from the kept state: the rows of a longer
    prompt, up to the 8-bit rounding's borders (float32: 2.2e-3 in the 2-norm, as
    above)."""
    case = (2, 40, 2, 64, 32, 32, "diagonal", "f32", 16, "f32")
    _, t = _setup(case)
    y, s, S_T, lam = _run(case, t)
    part = dict(t, x=t["x"][:, :32].contiguous(), r=t["r"][:, :32].contiguous())
    _, _, S, la = _run(case, part)
    rows = []
    for i in range(32, 40):
        one = dict(t, x=t["x"][:, i:i + 1].contiguous(), r=t["r"][:, i:i + 1].contiguous(), S0=S, lambda0=la)
        yi, _, S, la = _run(case, one)
        rows.append(yi)
    got = torch.cat(rows, 1).double()
    assert (got - y[:, 32:].double()).norm() <= 3e-3 * y[:, 32:].double().norm()
    assert normwise(host(S), host(S_T)) <= TOL_F32


def test_layer_in_8_bits_without_tokens():
    case = CASES[0]
    _, t = _setup(case)
    t["x"], t["r"] = t["x"][:, :0].contiguous(), t["r"][:, :0].contiguous()
    y, _, S_T, lam = _run(case, t)
    assert y.shape == (2, 0, 64) and torch.equal(S_T, t["S0"]) and torch.equal(lam, t["lambda0"])


def test_layer_in_8_bits_refuses():
    case = CASES[0]
    _, t = _setup(case)
    for k, v, err in (("w", t["w"][:32], ValueError), ("W_in", t["W_in"].float(), ValueError),
                      ("W_in_scale", t["W_in_scale"][:1], ValueError), ("r", t["r"][:1], ValueError),
                      ("r", t["r"].bfloat16(), ValueError), ("W_out", t["W_out"][:32], ValueError),
                      ("b_gate", t["b_gate"].double(), ValueError), ("x", t["x"][0], ValueError),
                      ("S0", t["S0"].cpu(), kdn.KdnError)):
        with pytest.raises(err):
            _run(case, dict(t, **{k: v}))
    with pytest.raises(kdn.KdnError):  # an odd width: d_model a multiple of 8 but not of 16
        kdn.layer_quant_forward(torch.zeros(1, 2, 40).cuda(), torch.ones(40).cuda(), *kdn.quantize(torch.zeros(99, 40).cuda(), 128),
                                torch.zeros(3).cuda(), *kdn.quantize(torch.zeros(40, 32).cuda(), 128), 1, 32, 32)


def test_layer_in_8_bits_in_a_captured_graph():
    case = CASES[3]
    _, t = _setup(case)
    ws = torch.empty(kdn.layer_quant_workspace_bytes(
        kdn.make_layer_desc(1, 64, 2, 256, 128, 128, 64, "isotropic", kdn.BF16)), dtype=torch.uint8, device="cuda")
    _run(case, t, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(case, t, workspace=ws)
    g = torch.Generator(device="cuda").manual_seed(3)
    for k in range(3):
        t["x"].copy_(torch.randn(t["x"].shape, generator=g, device="cuda"))
        want = [v.clone() for v in _run(case, t)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), k
