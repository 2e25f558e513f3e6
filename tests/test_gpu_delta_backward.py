"""Gradients of the gated delta rule on the GPU against the chain rule of one token in 64
bits, and against differences.  Tolerances: float32 1e-4 of the head's largest (the
library's acceptance for gradients); bfloat16 each element's delta_reference.rounding_bounds,
the result's own half step, and 1e-4 of the head's largest for the float32 part."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn
from delta_reference import HALF, delta, delta_gradients, inputs, rounding_bounds
from gpu_util import say

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")
SHAPES = [
    (1, 1, 1, 1, 32, 32, "f32", "f32"), (2, 3, 1, 5, 32, 64, "bf16", "bf16"), (1, 2, 2, 32, 64, 32, "bf16", "f32"),
    (1, 4, 2, 33, 128, 128, "f32", "bf16"), (3, 1, 1, 64, 128, 64, "bf16", "bf16"), (2, 6, 3, 101, 64, 128, "f32", "f32"),
    (1, 5, 5, 150, 128, 32, "bf16", "f32"), (1, 2, 1, 129, 32, 128, "f32", "f32"), (5, 3, 3, 31, 128, 128, "bf16", "bf16"),
    (1, 1, 1, 200, 128, 128, "bf16", "f32"), (2, 2, 1, 63, 64, 64, "f32", "bf16"), (1, 6, 2, 65, 64, 64, "bf16", "f32"),
    (1, 2, 2, 70, 32, 32, "f32", "f32"), (1, 2, 1, 96, 128, 64, "f32", "f32"), (1, 2, 2, 97, 32, 128, "bf16", "bf16"),
    (1, 1, 1, 40, 128, 32, "f32", "f32"), (1, 2, 2, 75, 64, 128, "bf16", "bf16"), (1, 1, 1, 66, 32, 32, "bf16", "f32"),
]
IDS = ["-".join(map(str, s)) for s in SHAPES]


def _all(shape, seed, kind="decay"):
    *x, S0 = inputs(*shape, seed=seed, kind=kind)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    do = torch.randn(x[2].shape, generator=g, device="cuda").to(x[2].dtype)
    return x, do, S0, torch.randn(S0.shape, generator=g, device="cuda")


def _check(got, want, bounds, dtype):
    for n in NAMES:
        x, y = got[n].double(), want[n]
        t = torch.float32 if n == "dS0" else dtype
        assert got[n].dtype == t and x.shape == y.shape, n
        top = y.abs().flatten(2).amax(-1) if y.numel() else y.new_zeros(y.shape[:2])
        tol = 1e-4 * top.view(*top.shape, *[1] * (y.dim() - 2)).expand(y.shape).clone()
        if t == torch.bfloat16:
            tol += HALF[t] * y.abs() + bounds.get(n, 0.0)
        wrong = int(((x - y).abs() > tol).sum())
        assert wrong == 0, (n, wrong)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("kind", ["decay", "resets", "alike"])
def test_matches_the_formula(shape, kind):
    x, do, S0, dS_T = _all(shape, 51, kind)
    say(f"[gpu] gated_delta_backward {shape} {kind}")
    got = kdn.gated_delta_backward(*x, do, S0, dS_T)
    _check(got, *rounding_bounds(*x, do, S0, dS_T, HALF[x[2].dtype]), x[2].dtype)
    again = kdn.gated_delta_backward(*x, do, S0, dS_T)
    for n in NAMES:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("shape", [
    (1, 1, 1, 1500, 64, 64, "f32", "f32"), (1, 2, 1, 1203, 128, 32, "bf16", "f32"), (1, 1, 1, 1100, 128, 128, "bf16", "bf16"),
    (1, 2, 2, 1300, 32, 64, "bf16", "f32"), (1, 1, 1, 1001, 128, 64, "f32", "f32")])
def test_few_heads_over_long_sequences(shape):
    """Both recurrences cut into segments, also with dS0 over dS_T's own buffer"""
    x, do, S0, dS_T = _all(shape, 52)
    B, H, Hk, T, dk, dv, dtype, gate = shape
    code = {"f32": kdn.F32, "bf16": kdn.BF16}
    few, many = (kdn.make_delta_desc(b, H, Hk, T, dk, dv, code[dtype], code[gate]) for b in (1, 512))
    need = [kdn.load_library().kdn_gated_delta_backward_workspace_bytes(ctypes.byref(d), 0) for d in (few, many)]
    assert need[0] > 1.02 * need[1] / 512  # (maps and states of segments)
    say(f"[gpu] gated_delta_backward in segments {shape}")
    got = kdn.gated_delta_backward(*x, do, S0, dS_T)
    _check(got, *rounding_bounds(*x, do, S0, dS_T, HALF[x[2].dtype]), x[2].dtype)
    out = {n: torch.empty_like(t) for n, t in got.items()}
    out["dS0"] = dS_T.clone()
    kdn.gated_delta_backward(*x, do, S0, out["dS0"], out=out)
    for n in NAMES:
        assert torch.equal(out[n], got[n]), n


def test_long_packed_sequences_of_few_heads():
    lengths = (700, 3, 0, 900, 33)
    x, do, _, _ = _all((1, 1, 1, sum(lengths), 64, 64, "f32", "f32"), 18)
    x, do = [t[0] for t in x], do[0]
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    S0, dS_T = torch.randn(2, len(lengths), 1, 64, 64, device="cuda")
    got = kdn.gated_delta_backward(*x, do, S0, dS_T, cu_seqlens=cu)
    at = 0
    for i, n in enumerate(lengths):
        part = [t[None, :, at:at + n].contiguous() for t in (*x, do)]
        one = {m: got[m][None, :, at:at + n] for m in NAMES[:5]} | {"dS0": got["dS0"][i:i + 1]}
        if n:
            _check(one, delta_gradients(*part, S0[i:i + 1], dS_T[i:i + 1]), {}, torch.float32)
        else:
            assert torch.equal(got["dS0"][i], dS_T[i])
        at += n


def test_without_states_and_with_another_scale():
    x, do, S0, _ = _all((2, 2, 1, 70, 64, 64, "f32", "f32"), 6)
    zero = torch.zeros_like(S0)
    p, q = kdn.gated_delta_backward(*x, do), kdn.gated_delta_backward(*x, do, zero, zero)
    for n in NAMES:
        assert torch.equal(p[n], q[n])
    got = kdn.gated_delta_backward(*x, do, S0, S0, scale=-1.5)
    _check(got, delta_gradients(*x, do, S0, S0, scale=-1.5), {}, torch.float32)


def test_against_differences():
    """Central differences of <do, o> + <dS_T, S_T> in 64 bits along random directions (h =
    1e-5: truncation below 1e-8); float32 gradients: 1e-4 of the sum of absolute values."""
    x, do, S0, dS_T = _all((1, 4, 2, 70, 32, 64, "f32", "f32"), 7)
    g = torch.Generator(device="cuda").manual_seed(3)
    got = kdn.gated_delta_backward(*x, do, S0, dS_T)

    def loss(*y):
        o, S, _ = delta(*y)
        return (o * do.double()).sum() + (S * dS_T.double()).sum()

    leaves = (*x, S0)
    for n, i in zip(NAMES, range(6)):
        e = torch.randn(leaves[i].shape, generator=g, device="cuda").double()
        sides = [loss(*(t.double() + (z * 1e-5 * e if j == i else 0) for j, t in enumerate(leaves))) for z in (1, -1)]
        parts = got[n].double() * e
        assert abs(parts.sum() - (sides[0] - sides[1]) / 2e-5) <= 1e-4 * parts.abs().sum(), n


@pytest.mark.parametrize("lengths,H,Hk,dk,dv,dtype", [
    ((1, 0, 31, 32, 33, 64, 2, 0, 65), 4, 2, 64, 64, "bf16"), ((100,), 3, 1, 128, 32, "f32"),
    ((0, 0), 2, 2, 32, 64, "f32"), ((5, 130, 7, 64, 64), 2, 1, 128, 128, "bf16"), ((63, 1, 64), 2, 2, 32, 32, "bf16")])
def test_packed_sequences_are_each_their_own(lengths, H, Hk, dk, dv, dtype):
    T = sum(lengths) + 3
    x, do, _, _ = _all((1, H, Hk, T, dk, dv, dtype, "f32"), 8)
    x, do = [t[0] for t in x], do[0]
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    S0, dS_T = torch.randn(2, len(lengths), H, dv, dk, device="cuda")
    say(f"[gpu] gated_delta_backward packed {lengths}")
    out = {n: torch.full_like(t, 7.0, dtype=do.dtype) for n, t in zip(NAMES, x)}
    out["dS0"] = torch.empty_like(S0)
    got = kdn.gated_delta_backward(*x, do, S0, dS_T, cu_seqlens=cu, out=out)
    at = 0
    for i, n in enumerate(lengths):
        part = [t[None, :, at:at + n].contiguous() for t in (*x, do)]
        one = kdn.gated_delta_backward(*part, S0[i:i + 1], dS_T[i:i + 1])
        for name in NAMES[:5]:
            assert torch.equal(got[name][:, at:at + n], one[name][0]), name
        assert torch.equal(got["dS0"][i], one["dS0"][0])
        at += n
    for name in NAMES[:5]:
        assert (out[name][:, at:] == 7.0).all()


def test_wrong_offsets_stay_inside():
    x, do, _, _ = _all((1, 2, 2, 90, 32, 32, "f32", "f32"), 8)
    S0 = torch.randn(2, 2, 32, 32, device="cuda")
    cu = torch.tensor([-5, 1000, 3], dtype=torch.int32, device="cuda")
    whole = kdn.gated_delta_backward(*x, do, S0[:1], S0[:1])
    got = kdn.gated_delta_backward(*(t[0] for t in x), do[0], S0, S0, cu_seqlens=cu)
    for n in NAMES[:5]:
        assert torch.equal(got[n], whole[n][0])
    assert torch.equal(got["dS0"][1], S0[1])


def test_no_tokens_and_in_place():
    x, do, S0, dS_T = _all((2, 2, 1, 0, 32, 64, "bf16", "f32"), 1)
    assert torch.equal(kdn.gated_delta_backward(*x, do, S0, dS_T)["dS0"], dS_T)
    x, do, S0, dS_T = _all((2, 2, 1, 50, 32, 64, "bf16", "f32"), 1)
    want = kdn.gated_delta_backward(*x, do, S0, dS_T)
    out = {n: torch.empty_like(t) for n, t in want.items()}
    out["dS0"] = dS_T.clone()
    kdn.gated_delta_backward(*x, do, S0, out["dS0"], out=out)
    for n in NAMES:
        assert torch.equal(out[n], want[n])


def test_training_step_in_a_graph_with_the_forward():
    x, do, S0, dS_T = _all((2, 4, 2, 100, 128, 128, "bf16", "f32"), 30)
    eager = (*kdn.gated_delta(*x, S0), *kdn.gated_delta_backward(*x, do, S0, dS_T).values())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = kdn.gated_delta_backward(*x, do, S0, dS_T)
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(other.values(), eager[2:]):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*kdn.gated_delta(*x, S0), *kdn.gated_delta_backward(*x, do, S0, dS_T).values())
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, eager):
            assert torch.equal(p, q)


def test_c_entry_without_the_state_gradient():
    x, do, S0, _ = _all((1, 2, 2, 40, 32, 32, "f32", "f32"), 2)
    want = kdn.gated_delta_backward(*x, do, S0)
    d = kdn.make_delta_desc(1, 2, 2, 40, 32, 32, kdn.F32, kdn.F32)
    lib = kdn.load_library()
    need = lib.kdn_gated_delta_backward_workspace_bytes(ctypes.byref(d), 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in x]
    code = lib.kdn_gated_delta_backward(ctypes.byref(d), None, *(t.data_ptr() for t in x), S0.data_ptr(), do.data_ptr(), None,
                                        *(t.data_ptr() for t in out), None, ws.data_ptr(), need,
                                        torch.cuda.current_stream().cuda_stream)
    assert code == 0
    for n, t in zip(NAMES, out):
        assert torch.equal(t, want[n])
