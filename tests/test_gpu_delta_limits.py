"""The gated delta rule and the head norms with rotation where offsets pass 32 bits (what lies
at the far end equals the same rows computed alone: the same kernel on the same rows, bit for
bit), two calls at once, and segments in a graph."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from delta_reference import inputs
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_no_tokens_for_many_states():
    """2^32 elements of states pass through"""
    B, H, d = 16389, 16, 128
    x = [torch.empty(B, H, 0, d, device="cuda") for _ in range(3)] + [torch.empty(B, H, 0, device="cuda") for _ in range(2)]
    S0 = torch.zeros(B, H, d, d, device="cuda")
    S0[-1] = 3.0
    S0[0, 0] = 2.0
    say(f"[gpu] {B} x {H} states without tokens")
    S_T = kdn.gated_delta(*x, S0)[1]
    assert torch.equal(S_T[-1], S0[-1]) and torch.equal(S_T[0], S0[0])


def _far(B, H, T, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=g)

    q, k = normal(B, H, T, d), normal(B, H, T, d).mul_(0.5 * d ** -0.5)
    gates = torch.empty(B, H, T, device="cuda").uniform_(-0.2, 0, generator=g)
    return q, k, normal(B, H, T, d), gates, torch.empty(B, H, T, device="cuda").uniform_(0, 1, generator=g)


@pytest.mark.parametrize("B,H,T,dtype", [(70, 1000, 480, torch.bfloat16), (35, 1000, 480, torch.float32)], ids=["bf16", "f32"])
def test_sequences_beyond_32_bit_offsets(B, H, T, dtype):
    """More than 2^32 elements in bfloat16, 2^31 in float32; T is short of what is cut into
    segments, so that the last head takes the same path alone."""
    x = _far(B, H, T, 128, dtype)
    alone = [t[-1:, -1:].clone() for t in x]
    say(f"[gpu] forward {B} x {H} x {T}")
    o, S_T = kdn.gated_delta(*x)
    p, P_T = kdn.gated_delta(*alone)
    assert torch.equal(o[-1:, -1:], p) and torch.equal(S_T[-1:, -1:], P_T)
    del o, S_T
    say("[gpu] packed")
    rows = [t.view(B, H * T, *t.shape[3:]) for t in x]  # B heads of H sequences
    cu = torch.arange(0, H * T + 1, T, dtype=torch.int32, device="cuda")
    o, S_T = kdn.gated_delta_varlen(*rows, cu)
    assert torch.equal(o[-1:, -T:], p[0]) and torch.equal(S_T[-1:, -1:], P_T)
    del o, S_T
    say("[gpu] backward")
    r = kdn.gated_delta_backward(*x, x[2])
    a = kdn.gated_delta_backward(*alone, alone[2])
    for n in a:
        assert torch.equal(r[n][-1:, -1:], a[n]), n


def test_step_on_a_cache_beyond_32_bit_offsets():
    n, H, d = 16389, 16, 128  # 4.3e9 elements
    S = torch.zeros(n, H, d, d, device="cuda")
    S[-1].normal_()
    q, k, v = (torch.randn(1, H, d, device="cuda", dtype=torch.bfloat16) * d ** -0.5 for _ in range(3))
    g, beta = -torch.rand(1, H, device="cuda"), torch.rand(1, H, device="cuda")
    alone = S[-1:].clone()
    say(f"[gpu] step on {n} x {H} states")
    slot = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    o = kdn.gated_delta_step(q, k, v, g, beta, S, slot)
    assert torch.equal(o, kdn.gated_delta_step(q, k, v, g, beta, alone)) and torch.equal(S[-1:], alone)
    assert not S[0].any() and not S[-2].any()


def test_rotary_beyond_32_bit_offsets():
    B, T, H, d = 1, (1 << 20) + 3, 32, 128  # 4.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.empty(B, T, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k = torch.empty(B, T, 1, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.randn(d, device="cuda", generator=g)
    position = torch.arange(T, dtype=torch.int32, device="cuda").view(1, T)
    inv = 1e4 ** (-torch.arange(0, d // 2, device="cuda") * 2.0 / d)
    say(f"[gpu] rotary {T} x {H}")
    n = 5
    last = (q[:, -n:].clone(), k[:, -n:].clone(), w, w, position[:, -n:].clone(), inv)
    full = kdn.qk_norm_rotary(q, k, w, w, position, inv)
    alone = kdn.qk_norm_rotary(*last)
    for x, y in zip(full, alone):
        assert torch.equal(x[:, :, -n:], y)
    say("[gpu] rotary backward")
    dq, dk, dw, _ = kdn.qk_norm_rotary_backward(full[0], full[1], q, k, w, w, position, inv, full[2], full[3])
    eq, ek, _, _ = kdn.qk_norm_rotary_backward(alone[0], alone[1], *last, alone[2], alone[3])
    assert torch.equal(dq[:, -n:], eq) and torch.equal(dk[:, -n:], ek) and torch.isfinite(dw).all()


def test_rotary_refuses_outputs_that_overlap():
    q, k = torch.randn(1, 4, 2, 32, device="cuda"), torch.randn(1, 4, 1, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    qo, ko, qr, kr = kdn.qk_norm_rotary(q, k, w, w, None, None)
    one = torch.empty(1, 4, 1, 32, device="cuda")
    with pytest.raises(ValueError):
        kdn.qk_norm_rotary_backward(qo, ko, q, k, w, w, None, None, qr, kr, out=(one.expand(1, 4, 2, 32), torch.empty_like(k)))
    # heads that share their rows are fine to read
    shared = one.normal_().expand(1, 4, 2, 32)
    a, b = kdn.qk_norm_rotary(shared, k, w, w, None, None), kdn.qk_norm_rotary(shared.contiguous(), k, w, w, None, None)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def _run(x, S0, dO):
    o, S_T = kdn.gated_delta(*x, S0)
    return [o, S_T, *kdn.gated_delta_backward(*x, dO, S0, S0).values()]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_two_calls_at_once(kind):
    """segments, each call with its own workspace"""
    work = []
    for seed in (1, 2):
        *x, S0 = inputs(1, 2, 1, 3000, 64, 64, kind, "f32", seed=seed)
        work.append((x, S0, torch.randn_like(x[2])))
    want = [_run(*w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_run(*work[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_segments_in_two_graphs(kind):
    *x, S0 = inputs(1, 2, 1, 3000, 64, 64, kind, "f32", seed=3)
    dO = torch.randn_like(x[2])
    _run(x, S0, dO)
    torch.cuda.synchronize()
    graphs = []
    pool = None
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = _run(x, S0, dO)
        pool = graph.pool()
        graphs.append((graph, out))
    for n in range(3):
        x[2].normal_()
        want = _run(x, S0, dO)
        for graph, out in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), n
