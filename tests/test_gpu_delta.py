"""The gated delta rule on the GPU (a batch, packed sequences, one token) against the
recurrence in 64 bits.  Tolerances: delta_reference.state_errors; o = scale S q adds 70
u of |q| s, and in bfloat16 the third planes left out of the read-out (at most 2^-14 of
|q| (s + the block's writes), which are within 2 s + |v|) and its half step."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn
from delta_reference import HALF, U, delta, inputs, shared, state_errors
from gpu_util import say

pytestmark = pytest.mark.gpu

# B, H, Hk, T, d_k, d_v, type, gates' type: one token, less than a block of 32, whole
# blocks, ragged ones, every width, shared heads, an odd number of workgroups
SHAPES = [
    (1, 1, 1, 1, 32, 32, "f32", "f32"), (2, 3, 1, 5, 32, 64, "bf16", "bf16"), (1, 2, 2, 32, 64, 32, "bf16", "f32"),
    (1, 4, 2, 33, 128, 128, "f32", "bf16"), (3, 1, 1, 64, 128, 64, "bf16", "bf16"), (2, 6, 3, 101, 64, 128, "f32", "f32"),
    (1, 5, 5, 150, 128, 32, "bf16", "f32"), (1, 2, 1, 257, 32, 128, "f32", "f32"), (5, 3, 3, 31, 128, 128, "bf16", "bf16"),
    (1, 1, 1, 700, 128, 128, "bf16", "f32"), (2, 2, 1, 63, 64, 64, "f32", "bf16"),
]
IDS = ["-".join(map(str, s)) for s in SHAPES]


def _compare(x, S0, o, S_T, scale=None, times=1):
    q, k, v, g, beta = x
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    want, last, kept = delta(q, k, v, g, beta, S0, scale)
    D, s = state_errors(q, k, v, g, beta, kept)
    D = times * D
    assert o.dtype == v.dtype and o.shape == v.shape and S_T.dtype == torch.float32
    size = s + (v.double().norm(dim=-1).amax(-1) if v.shape[2] else 0)
    tol = D + 70 * U * s[..., None] + (2.0 ** -14 * 2 * size[..., None] if v.dtype == torch.bfloat16 else 0)
    tol = (tol * abs(scale) * shared(q, v.shape[1]).double().norm(dim=-1))[..., None] + HALF[v.dtype] * want.abs()
    assert ((o.double() - want).abs() <= tol).all()
    end = D[..., -1] if v.shape[2] else torch.zeros_like(s)
    assert ((S_T.double() - last).flatten(2).norm(dim=-1) <= end + U * s).all()


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("kind", ["decay", "resets", "alike"])
def test_matches_the_recurrence(shape, kind):
    *x, S0 = inputs(*shape, seed=41, kind=kind)
    say(f"[gpu] gated_delta {shape} {kind}")
    o, S_T = kdn.gated_delta(*x, S0)
    _compare(x, S0, o, S_T)
    again = kdn.gated_delta(*x, S0)
    assert torch.equal(o, again[0]) and torch.equal(S_T, again[1])


def test_without_a_state_and_with_another_scale():
    *x, S0 = inputs(2, 2, 1, 70, 64, 64, "f32", "f32", seed=6)
    for p, q in zip(kdn.gated_delta(*x), kdn.gated_delta(*x, torch.zeros_like(S0))):
        assert torch.equal(p, q)
    _compare(x, S0, *kdn.gated_delta(*x, S0, scale=-1.5), scale=-1.5)


@pytest.mark.parametrize("dtype,top", [("f32", 2 ** 21), ("bf16", 64)])
@pytest.mark.parametrize("dk,dv", [(32, 128), (64, 32), (128, 64)])
def test_exact_on_whole_numbers(dtype, top, dk, dv):
    """Unit vectors as keys, beta 1 and no decay but a few -inf: every token overwrites one
    column of the state.  Corrections and their sums are whole numbers below 4 top + 1, the
    inverse holds 0 and +-1, so nothing is rounded - also where a float32 needs all three
    planes (2^23) - and what is forgotten is 0."""
    B, H, T = 2, 2, 130
    g = torch.Generator(device="cuda").manual_seed(dk)
    ints = lambda *s: torch.randint(-top, top + 1, s, generator=g, device="cuda").float()  # noqa: E731
    one = lambda: torch.nn.functional.one_hot(torch.randint(0, dk, (B, H, T), generator=g, device="cuda"), dk).to(t)  # noqa: E731
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    q, k, v, S0 = one(), one(), ints(B, H, T, dv).to(t), ints(B, H, dv, dk)
    gate = torch.zeros(B, H, T, device="cuda")
    gate[0, 0, 50] = gate[1, 1, 96] = -float("inf")
    say(f"[gpu] gated_delta whole numbers {dtype} {dk} {dv}")
    want, last, _ = delta(q, k, v, gate, torch.ones_like(gate), S0, 1.0)
    o, S_T = kdn.gated_delta(q, k, v, gate, torch.ones_like(gate), S0, scale=1.0)
    wrong = int((S_T.double() != last).sum()), int((o.double() != want).sum())
    assert wrong == (0, 0)


def _packed(lengths, H, Hk, dk, dv, dtype, gate, seed, gap=0):
    """Packed inputs, their offsets, and a state per sequence; `gap` rows in no sequence at the end"""
    T = sum(lengths) + gap
    *x, _ = inputs(1, H, Hk, T, dk, dv, dtype, gate, seed)
    x = [t[0] for t in x]
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    S0 = torch.randn(len(lengths), H, dv, dk, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    return x, cu, S0


@pytest.mark.parametrize("lengths,H,Hk,dk,dv,dtype", [
    ((1, 0, 31, 32, 33, 64, 2, 0), 4, 2, 64, 64, "bf16"), ((100,), 3, 1, 128, 32, "f32"), ((0, 0), 2, 2, 32, 64, "f32"),
    ((5, 200, 7, 65), 2, 1, 128, 128, "bf16")])
def test_packed_sequences_are_each_their_own(lengths, H, Hk, dk, dv, dtype):
    x, cu, S0 = _packed(lengths, H, Hk, dk, dv, dtype, "f32", 3, gap=3)
    say(f"[gpu] gated_delta_varlen {lengths}")
    o, S_T = torch.full_like(x[2], 7.0), torch.empty_like(S0)
    kdn.gated_delta_varlen(*x, cu, S0, out=(o, S_T))
    at = 0
    for i, n in enumerate(lengths):
        part = [t[None, :, at:at + n].contiguous() for t in x]
        one, last = kdn.gated_delta(*part, S0[i:i + 1])
        assert torch.equal(o[:, at:at + n], one[0]) and torch.equal(S_T[i], last[0])
        at += n
    assert (o[:, at:] == 7.0).all()


def test_wrong_offsets_stay_inside():
    x, _, S0 = _packed((40, 50), 2, 2, 32, 32, "f32", "f32", 8)
    o, S_T = torch.full_like(x[2], 7.0), torch.empty_like(S0)
    cu = torch.tensor([-5, 1000, 3], dtype=torch.int32, device="cuda")  # clamped to 0 .. 90, then empty
    kdn.gated_delta_varlen(*x, cu, S0, out=(o, S_T))
    whole = kdn.gated_delta(*(t[None] for t in x), S0[:1])
    assert torch.equal(o, whole[0][0]) and torch.equal(S_T[0], whole[1][0]) and torch.equal(S_T[1], S0[1])


@pytest.mark.parametrize("shape", [
    (1, 1, 1, 2100, 128, 128, "bf16", "f32"), (1, 2, 1, 1999, 64, 32, "bf16", "bf16"), (2, 1, 1, 1600, 32, 128, "f32", "f32"),
    (1, 1, 1, 1700, 128, 64, "f32", "bf16"), (1, 3, 3, 2900, 32, 64, "bf16", "f32"), (1, 1, 1, 1537, 64, 64, "f32", "f32")])
def test_few_heads_over_long_sequences(shape):
    """Cut into segments (a workspace is asked for), also over the first state's own buffer.
    The composition adds the maps' errors, which each are a state's: twice the bound."""
    *x, S0 = inputs(*shape, seed=44)
    B, H, Hk, T, dk, dv, dtype, gate = shape
    code = {"f32": kdn.F32, "bf16": kdn.BF16}
    d = kdn.make_delta_desc(B, H, Hk, T, dk, dv, code[dtype], code[gate])
    assert kdn.load_library().kdn_gated_delta_workspace_bytes(ctypes.byref(d), 0) > 16
    say(f"[gpu] gated_delta in segments {shape}")
    o, S_T = kdn.gated_delta(*x, S0)
    _compare(x, S0, o, S_T, times=2)
    S, again = S0.clone(), torch.empty_like(o)
    kdn.gated_delta(*x, S, out=(again, S))
    assert torch.equal(again, o) and torch.equal(S, S_T)


def test_long_packed_sequences_of_few_heads():
    lengths = (1500, 3, 0, 1100, 33)
    x, cu, S0 = _packed(lengths, 1, 1, 64, 64, "f32", "f32", 13)
    o, S_T = kdn.gated_delta_varlen(*x, cu, S0)
    at = 0
    for i, n in enumerate(lengths):
        part = [t[None, :, at:at + n].contiguous() for t in x]
        _compare(part, S0[i:i + 1], o[None, :, at:at + n], S_T[i:i + 1], times=2)
        at += n


def test_no_tokens():
    *x, S0 = inputs(2, 2, 1, 0, 32, 64, "bf16", "f32", seed=1)
    o, S_T = kdn.gated_delta(*x, S0)
    assert o.shape == (2, 2, 0, 64) and torch.equal(S_T, S0)
    assert (kdn.gated_delta(*x)[1] == 0).all()
    *x, S0 = inputs(0, 2, 1, 5, 32, 64, "bf16", "f32", seed=1)
    assert kdn.gated_delta(*x, S0)[0].numel() == 0


def test_state_in_place():
    *x, S0 = inputs(2, 4, 2, 90, 64, 128, "bf16", "f32", seed=9)
    o, S_T = kdn.gated_delta(*x, S0)
    S = S0.clone()
    o2 = torch.empty_like(o)
    kdn.gated_delta(*x, S, out=(o2, S))
    assert torch.equal(S, S_T) and torch.equal(o, o2)


def test_what_is_not_finite_stays_in_its_head():
    *x, S0 = inputs(2, 2, 2, 100, 64, 64, "f32", "f32", seed=12)
    o, S_T = kdn.gated_delta(*x, S0)
    for which, bad in ((2, float("nan")), (1, float("inf")), (0, float("nan")), (3, float("nan"))):
        y = [t.clone() for t in x]
        y[which][0, 1, 40] = bad
        p, S = kdn.gated_delta(*y, S0)
        assert torch.equal(p[0, 0], o[0, 0]) and torch.equal(p[1], o[1]) and torch.equal(S[1], S_T[1])
        assert torch.equal(p[0, 1, :32], o[0, 1, :32])  # the blocks before
        assert not torch.isfinite(p[0, 1, 40]).any()
        if which:
            assert not torch.isfinite(p[0, 1, 64:]).any() and not torch.isfinite(S[0, 1]).any()
    # a value's column alone, from its block on
    y = [t.clone() for t in x]
    y[2][0, 1, 40, 5] = float("nan")
    p, S = kdn.gated_delta(*y, S0)
    rest = [i for i in range(64) if i != 5]
    assert torch.equal(p[..., rest], o[..., rest]) and torch.equal(S[:, :, rest], S_T[:, :, rest])
    assert not torch.isfinite(p[0, 1, 40:, 5]).any() and torch.equal(p[0, 1, :32, 5], o[0, 1, :32, 5])


# ------------------------------------------------------------------------- one token

@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("dtype,gate", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_step_matches_the_recurrence(dk, dv, dtype, gate):
    """A dot product of d_k terms in float32 is within (d_k / 16 + 8) u of its |.||.| (four
    products a lane, five exchanges), well below the 70 u of state_errors."""
    *x, S0 = inputs(3, 4, 2, 1, dk, dv, dtype, gate, seed=21)
    S = S0.clone()
    o = kdn.gated_delta_step(*(t[:, :, 0].contiguous() for t in x), S)
    _compare(x, S0, o[:, :, None], S)


def test_steps_equal_the_sequence():
    B, H, T = 2, 4, 45
    *x, S0 = inputs(B, H, 2, T, 64, 128, "f32", "f32", seed=22)
    S, got = S0.clone(), []
    for t in range(T):
        got.append(kdn.gated_delta_step(*(y[:, :, t].contiguous() for y in x), S))
    _compare(x, S0, torch.stack(got, 2), S)


def test_step_on_a_cache_of_slots():
    *x, S0 = inputs(4, 2, 1, 1, 128, 64, "bf16", "f32", seed=23)
    x = [t[:, :, 0].contiguous() for t in x]
    cache = torch.randn(7, 2, 64, 128, device="cuda")
    before = cache.clone()
    slot = torch.tensor([5, -1, 0, 7], dtype=torch.int32, device="cuda")
    out = torch.full_like(x[2], 3.0)
    assert kdn.gated_delta_step(*x, cache, slot, out=out) is out
    S = before[[5, 5, 0, 0]].contiguous()
    o = kdn.gated_delta_step(*x, S)
    for n, s in ((0, 5), (2, 0)):
        assert torch.equal(out[n], o[n]) and torch.equal(cache[s], S[n])
    assert (out[1] == 3.0).all() and (out[3] == 3.0).all()
    for s in (1, 2, 3, 4, 6):
        assert torch.equal(cache[s], before[s])


# --------------------------------------------------------------- streams, graphs, C entry

def test_on_another_stream_and_in_a_graph():
    *x, S0 = inputs(2, 4, 2, 100, 128, 128, "bf16", "f32", seed=30)
    o, S_T = kdn.gated_delta(*x, S0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p, P_T = kdn.gated_delta(*x, S0)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, p) and torch.equal(S_T, P_T)
    one = [t[:, :, 0].contiguous() for t in x]
    S = S0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, P_T = kdn.gated_delta(*x, S0)
        r = kdn.gated_delta_step(*one, S)
    S.copy_(S0)
    eager = S0.clone()
    for _ in range(3):
        graph.replay()
        want = kdn.gated_delta_step(*one, eager)
        torch.cuda.synchronize()
        assert torch.equal(o, p) and torch.equal(S_T, P_T)
        assert torch.equal(r, want) and torch.equal(S, eager)


def test_c_entry_without_a_last_state():
    *x, S0 = inputs(1, 2, 2, 40, 32, 32, "f32", "f32", seed=2)
    want, _ = kdn.gated_delta(*x, S0)
    d = kdn.make_delta_desc(1, 2, 2, 40, 32, 32, kdn.F32, kdn.F32)
    o = torch.empty_like(x[2])
    code = kdn.load_library().kdn_gated_delta(ctypes.byref(d), None, *(t.data_ptr() for t in x), S0.data_ptr(), o.data_ptr(),
                                              None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert torch.equal(o, want)
