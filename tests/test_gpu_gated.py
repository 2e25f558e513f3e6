"""The gated linear recurrence on the GPU (forward, backward, one step) against the
recurrence in 64 bits.

Tolerance: a term a_t .. a_{s+1} x_s of h_t passes at most 2 (t - s) + 20 roundings of
half a step u = 2^-24 (t - s products, an addition for each token or fold it crosses,
and the last few folds), so |error of h_t| <= u N_t with H_t = |a_t| H_{t-1} + |x_t| and
N_t = |a_t| (N_{t-1} + 2 H_{t-1}) + 20 |x_t|, whatever the bracketing."""
from __future__ import annotations

import ctypes

import pytest
import torch

import kalman_filter_memory_amd as kdn
from gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _recurrence(a, x, h0):
    """(h, N) along dim 2, in 64 bits"""
    h, H, N = h0.clone(), h0.abs(), 20 * h0.abs()
    hs, Ns = torch.empty_like(x), torch.empty_like(x)
    for t in range(x.shape[2]):
        at, xt = a[:, :, t], x[:, :, t]
        h = at * h + xt
        N = at.abs() * (N + 2 * H) + 20 * xt.abs()
        H = at.abs() * H + xt.abs()
        hs[:, :, t], Ns[:, :, t] = h, N
    return hs, Ns, h, N


def _inputs(B, H, T, d, dtype, gate, seed, kind="decay"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    a = torch.sigmoid(3 + rand(B, H, T, d))
    if kind == "signs":
        a = a * torch.sign(rand(B, H, T, d))
    if kind == "resets":  # a = 0 starts anew, a = 1 keeps
        a = torch.where(rand(B, H, T, d) > 1.5, 0.0, torch.where(rand(B, H, T, d) > 0, 1.0, a))
    return rand(B, H, T, d).to(TYPES[dtype]), a.to(TYPES[gate]), rand(B, H, d)


# B, H, T, d, x's type, a's type.  Tiles are 64 to 1024 tokens: one token, less than
# a strip, one tile, a few tiles and several groups of tiles in a chain, two
# channel blocks, and as many sequences as CUs or more, so that a workgroup walks along
# its own.
SHAPES = [
    (1, 1, 1, 8, "f32", "f32"), (2, 3, 5, 32, "bf16", "bf16"), (1, 2, 257, 64, "bf16", "f32"),
    (1, 1, 4500, 128, "bf16", "bf16"), (2, 1, 2100, 200, "f32", "bf16"), (1, 1, 9000, 32, "bf16", "bf16"),
    (1, 1, 9000, 24, "f32", "f32"), (3, 1, 1024, 128, "bf16", "bf16"), (1, 2, 1025, 128, "f32", "f32"),
    (64, 16, 300, 128, "bf16", "bf16"), (512, 2, 530, 40, "bf16", "f32"), (1, 1, 700, 1000, "bf16", "bf16"),
    (250, 1, 700, 72, "bf16", "f32"), (3, 1, 400, 128, "f32", "f32"),
]
IDS = ["-".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("kind", ["decay", "signs", "resets"])
def test_scan_matches_the_recurrence(shape, kind):
    x, a, h0 = _inputs(*shape, seed=31, kind=kind)
    say(f"[gpu] gated_scan {shape} {kind}")
    h, h_T = kdn.gated_scan(x, a, h0)
    hs, Ns, hl, Nl = _recurrence(a.double(), x.double(), h0.double())
    assert h.dtype == x.dtype
    assert ((h.double() - hs).abs() <= U * Ns + HALF[h.dtype] * hs.abs()).all()
    assert ((h_T.double() - hl).abs() <= U * Nl).all()
    again = kdn.gated_scan(x, a, h0)
    assert torch.equal(h, again[0]) and torch.equal(h_T, again[1])


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("kind", ["decay", "resets"])
def test_scan_backward_matches_the_formula(shape, kind):
    x, a, h0 = _inputs(*shape, seed=32, kind=kind)
    dh, _, dh_T = _inputs(*shape, seed=33)
    h, _ = kdn.gated_scan(x, a, h0)
    say(f"[gpu] gated_scan_backward {shape} {kind}")
    g = kdn.gated_scan_backward(a, h, dh, h0, dh_T)
    # m_t = a_t m_{t+1} + a_t dh_t from the last token to the first
    ad, dd = a.double().flip(2), dh.double().flip(2)
    m, N, m1, N1 = _recurrence(ad, ad * dd, dh_T.double())
    m, N = m.flip(2), N.flip(2)
    after = torch.cat((m[:, :, 1:], dh_T.double()[:, :, None]), 2)
    slack = torch.cat((N[:, :, 1:], dh_T.double().abs()[:, :, None]), 2)
    before = torch.cat((h0.double()[:, :, None], h[:, :, :-1].double()), 2)
    dx = dh.double() + after
    tol = U * (2 * slack + 2 * dx.abs())  # (a_t (dh_t + m): one rounding more per token)
    assert ((g["dx"].double() - dx).abs() <= tol).all()
    assert ((g["da"].double() - dx * before).abs() <= tol * before.abs() + U * (dx * before).abs()).all()
    assert ((g["dh0"].double() - m1).abs() <= 2 * U * N1).all()
    again = kdn.gated_scan_backward(a, h, dh, h0, dh_T)
    for n in g:
        assert torch.equal(g[n], again[n])


def test_scan_without_states():
    x, a, h0 = _inputs(2, 2, 700, 64, "f32", "f32", seed=5)
    zero = torch.zeros_like(h0)
    for p, q in zip(kdn.gated_scan(x, a), kdn.gated_scan(x, a, zero)):
        assert torch.equal(p, q)
    h, _ = kdn.gated_scan(x, a)
    p, q = kdn.gated_scan_backward(a, h, x), kdn.gated_scan_backward(a, h, x, zero, zero)
    for n in p:
        assert torch.equal(p[n], q[n])


def test_scan_of_no_tokens_passes_the_state_on():
    x = torch.empty(2, 3, 0, 64).cuda()
    h0 = torch.randn(2, 3, 64).cuda()
    h, h_T = kdn.gated_scan(x, x, h0)
    assert h.shape == x.shape and torch.equal(h_T, h0)
    assert (kdn.gated_scan(x, x)[1] == 0).all()
    g = kdn.gated_scan_backward(x, h, x, h0, h0)
    assert g["dx"].shape == x.shape and torch.equal(g["dh0"], h0)
    e = torch.empty(0, 3, 5, 64).cuda()
    assert kdn.gated_scan(e, e)[0].shape == e.shape


@pytest.mark.parametrize("T", [40, 5000])
def test_scan_writes_the_last_state_over_the_first(T):
    """h_T in h0's buffer, h0 and h_T NULL: through the C ABI."""
    x, a, h0 = _inputs(1, 2, T, 128, "bf16", "f32", seed=7)
    want = kdn.gated_scan(x, a, h0)
    lib = kdn.load_library()
    s = kdn.make_scan_desc(1, 2, T, 128, kdn.BF16, kdn.F32)
    ws = torch.empty(lib.kdn_gated_scan_workspace_bytes(ctypes.byref(s)), dtype=torch.uint8, device="cuda")
    h = torch.empty_like(x)
    state = h0.clone()
    stream = torch.cuda.current_stream().cuda_stream
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731

    def call(first, last):
        assert lib.kdn_gated_scan(ctypes.byref(s), P(x), P(a), P(first), P(h), P(last), P(ws),
                                  ws.numel(), stream) == 0

    call(state, state)
    assert torch.equal(h, want[0]) and torch.equal(state, want[1])
    call(h0, None)
    assert torch.equal(h, want[0])


def test_scan_leaves_what_lies_behind_its_outputs():
    """The rows behind the last token and the channels of the next head."""
    x, a, _ = _inputs(1, 1, 300, 40, "bf16", "bf16", seed=8)
    big = torch.full((1, 1, 320, 40), 7.0, device="cuda", dtype=torch.bfloat16)
    lib = kdn.load_library()
    s = kdn.make_scan_desc(1, 1, 300, 40, kdn.BF16, kdn.BF16)
    ws = torch.empty(lib.kdn_gated_scan_workspace_bytes(ctypes.byref(s)), dtype=torch.uint8, device="cuda")
    assert lib.kdn_gated_scan(ctypes.byref(s), x.data_ptr(), a.data_ptr(), None, big.data_ptr(), None,
                              ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(big[:, :, :300], kdn.gated_scan(x, a)[0]) and (big[:, :, 300:] == 7).all()


def test_scan_keeps_nan_to_its_channel():
    x, a, h0 = _inputs(1, 1, 3000, 128, "f32", "f32", seed=9)
    clean, _ = kdn.gated_scan(x, a, h0)
    x[0, 0, 700, 5] = float("nan")
    x[0, 0, 900, 6] = torch.tensor(-1, dtype=torch.int32, device="cuda").view(torch.float32)  # a NaN of all ones
    h, h_T = kdn.gated_scan(x, a, h0)
    assert torch.isnan(h[0, 0, 700:, 5]).all() and torch.isnan(h[0, 0, 900:, 6]).all()
    assert torch.isnan(h_T[0, 0, 5:7]).all()
    keep = [i for i in range(128) if i not in (5, 6)]
    assert torch.equal(h[..., keep], clean[..., keep])


def test_scan_backward_against_differences():
    """Along random directions, against central differences of the recurrence in 64
    bits (h = 1e-5; the kernel's float32 sums over 2 x 150 x 16 elements of order 1
    to 10: 1e-4 of the sum of absolute values)."""
    B, H, T, d = 1, 2, 150, 16
    x, a, h0 = _inputs(B, H, T, d, "f32", "f32", seed=10)
    c, _, cT = _inputs(B, H, T, d, "f32", "f32", seed=11)

    def loss(x, a, h0):
        hs, _, hl, _ = _recurrence(a, x, h0)
        return (hs * c.double()).sum() + (hl * cT.double()).sum()

    h, _ = kdn.gated_scan(x, a, h0)
    g = kdn.gated_scan_backward(a, h, c, h0, cT)
    for k in range(3):
        e = [torch.randn(t.shape, device="cuda", dtype=torch.float64) for t in (x, a, h0)]
        s = 1e-5
        plus = loss(*(t.double() + s * v for t, v in zip((x, a, h0), e)))
        minus = loss(*(t.double() - s * v for t, v in zip((x, a, h0), e)))
        parts = [(g[n].double() * v) for n, v in zip(("dx", "da", "dh0"), e)]
        got = sum(p.sum() for p in parts)
        assert abs(got - (plus - minus) / (2 * s)) <= 1e-4 * sum(p.abs().sum() for p in parts)


@pytest.mark.parametrize("shape", [(1, 1, 8, "f32", "f32"), (5, 3, 40, "bf16", "f32"),
                                   (256, 16, 128, "bf16", "bf16"), (3, 2, 64, "f32", "bf16")])
def test_step_equals_one_token_of_the_scan(shape):
    B, H, d, dtype, gate = shape
    x, a, h0 = _inputs(B, H, 3, d, dtype, gate, seed=12)
    h, h_T = kdn.gated_scan(x, a, h0)
    state = h0.clone()
    for t in range(3):
        o = kdn.gated_scan_step(x[:, :, t].contiguous(), a[:, :, t].contiguous(), state)
        assert torch.equal(o, h[:, :, t])  # three tokens of one strip: the same operations
    assert torch.equal(state, h_T)


def test_step_over_cache_slots():
    B, H, d, n = 6, 2, 32, 9
    x, a, _ = _inputs(B, H, 1, d, "bf16", "f32", seed=13)
    x, a = x[:, :, 0].contiguous(), a[:, :, 0].contiguous()
    cache = torch.randn(n, H, d).cuda()
    slot = torch.tensor([3, -1, 0, 8, 9, 5], dtype=torch.int32).cuda()
    out = torch.full((B, H, d), 7.0, device="cuda", dtype=torch.bfloat16)
    before = cache.clone()
    kdn.gated_scan_step(x, a, cache, slot=slot, out=out)
    for b, s in enumerate(slot.tolist()):
        if 0 <= s < n:
            want = torch.addcmul(x[b].double(), a[b].double(), before[s].double())
            assert ((cache[s].double() - want).abs() <= U * want.abs()).all()  # one fma
            assert torch.equal(out[b], cache[s].bfloat16())
        else:
            assert (out[b] == 7).all()
    idle = [i for i in range(n) if i not in slot.tolist()]
    assert torch.equal(cache[idle], before[idle])


def test_scan_refuses_mismatched_tensors():
    x, h0 = torch.zeros(2, 2, 10, 64).cuda(), torch.zeros(2, 2, 64).cuda()
    for bad, err in (
            (lambda: kdn.gated_scan(x, x[:, :, :5].contiguous()), ValueError),
            (lambda: kdn.gated_scan(x, x[..., 0].contiguous()), ValueError),
            (lambda: kdn.gated_scan(x[0], x[0]), ValueError),
            (lambda: kdn.gated_scan(x, x, h0.bfloat16()), ValueError),
            (lambda: kdn.gated_scan(x, x, h0[:1]), ValueError),
            (lambda: kdn.gated_scan(x.transpose(1, 2), x.transpose(1, 2)), ValueError),
            (lambda: kdn.gated_scan(x.half(), x), TypeError),
            (lambda: kdn.gated_scan(x, x.cpu()), kdn.KdnError),
            (lambda: kdn.gated_scan(x[..., :4].contiguous(), x[..., :4].contiguous()), kdn.KdnError),
            (lambda: kdn.gated_scan_backward(x, x, x.bfloat16()), ValueError),
            (lambda: kdn.gated_scan_backward(x, x, x, h0, h0.bfloat16()), ValueError),
            (lambda: kdn.gated_scan_step(h0, h0, h0.bfloat16()), ValueError),
            (lambda: kdn.gated_scan_step(h0, h0, h0[:1]), ValueError),
            (lambda: kdn.gated_scan_step(h0, h0, h0, slot=torch.zeros(2).cuda()), ValueError),
            (lambda: kdn.gated_scan_step(h0, h0, h0, out=h0.bfloat16()), ValueError)):
        with pytest.raises(err):
            bad()


def test_scan_in_captured_graphs():
    """Two graphs (a chain of tiles each, forward and backward) replayed in turn and
    against each other on two streams, with eager work between."""
    g = torch.Generator(device="cuda").manual_seed(4)
    sets = [_inputs(1, 2, 3000, 128, "bf16", "bf16", seed=s) for s in (14, 15)]

    def step(x, a, h0):
        h, h_T = kdn.gated_scan(x, a, h0)
        return (h, h_T, *kdn.gated_scan_backward(a, h, x, h0, h0).values())

    for s in sets:
        step(*s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(*s))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    for k in range(3):
        for x, a, h0 in sets:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        want = [[t.clone() for t in step(*s)] for s in sets]
        torch.cuda.synchronize()
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for p, q in zip(o, w):
                assert torch.equal(p, q), k


def test_scans_on_two_streams_at_once():
    sets = [_inputs(1, 4, 20000, 128, "bf16", "bf16", seed=s) for s in (16, 17)]
    want = [kdn.gated_scan(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for st, s in zip(streams, sets):
        with torch.cuda.stream(st):
            got.append([kdn.gated_scan(*s) for _ in range(4)])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])
