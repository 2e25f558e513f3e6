"""Head norm with rotation by position on the GPU (forward and backward) against the
formulas in 64 bits.

Tolerances in u = 2^-24: the mean square is a sum of up to eight products a lane and five
exchanges, its root and quotient round four times (17 u, half of it in the inverse root),
two products follow: 12 u of |x r w|.  Angles: 64-bit products reduced to a turn in float32,
2 pi 2^-25 = 4 u, and four ulps of sine and cosine, 8 u; two products and a sum, 3 u.  So
|error of y| <= 30 u (|a| + |b|) of the pair, and the result's half step."""
from __future__ import annotations

import pytest
import torch

import kalman_filter_memory_amd as kdn
from delta_reference import HALF, TYPES, U
from gpu_util import say

pytestmark = pytest.mark.gpu
EPS = 1e-6

# B, T, H, Hk, d, rot, type, interleaved: every width of a lane group, heads whose width is
# no power of two, partly turned and not turned, one token, a tile and a ragged one (8
# tokens from 4096 on)
SHAPES = [
    (1, 1, 1, 1, 8, 0, "f32", False), (2, 3, 3, 1, 16, 16, "bf16", True), (1, 5, 2, 2, 32, 32, "f32", False),
    (3, 7, 4, 2, 64, 32, "bf16", False), (1, 33, 5, 1, 80, 80, "f32", False), (2, 9, 1, 3, 80, 32, "f32", True),
    (2, 17, 16, 4, 128, 128, "bf16", False), (1, 6, 2, 1, 128, 64, "f32", True), (2, 4, 3, 2, 256, 256, "bf16", False),
    (1, 3, 2, 2, 200, 112, "f32", False), (1, 4101, 2, 1, 32, 32, "bf16", True), (3, 1500, 1, 2, 128, 96, "bf16", False),
    (1, 2, 7, 5, 256, 16, "f32", False), (256, 1, 4, 1, 128, 128, "bf16", False),
]
IDS = ["-".join(map(str, s)) for s in SHAPES]


def _inputs(B, T, H, Hk, d, rot, dtype, seed, pad=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    z = rand(B, T, pad + (H + Hk) * d + 16).to(TYPES[dtype])
    q = z[..., pad:pad + H * d].unflatten(-1, (H, d))
    k = z[..., pad + H * d:pad + (H + Hk) * d].unflatten(-1, (Hk, d))
    position = torch.randint(-1000, 1 << 20, (B, T), generator=g, device="cuda", dtype=torch.int32)
    position[0, 0] = 2 ** 31 - 1
    inv_freq = None if rot == 0 else 1e4 ** (-2 * torch.arange(rot // 2, device="cuda") / rot)
    return q, k, 1 + 0.3 * rand(d), 1 - 0.3 * rand(d), position if rot else None, inv_freq, rand


def _pairs(rot, interleaved):
    return (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))


def _turn(x, position, inv_freq, interleaved, back=False):
    """x [B,T,H,d] turned, and the sum of absolute values of each pair"""
    if inv_freq is None:
        return x, x.abs()
    angle = (position.double()[..., None] * inv_freq.double())[:, :, None]
    c, s = angle.cos(), angle.sin() * (-1 if back else 1)
    one, two = _pairs(2 * inv_freq.numel(), interleaved)
    y, size = x.clone(), x.abs()
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    size[..., one] = size[..., two] = a.abs() + b.abs()
    return y, size


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_matches_the_formula(shape):
    *shape, interleaved = shape
    q, k, wq, wk, position, inv_freq, _ = _inputs(*shape, seed=61)
    say(f"[gpu] qk_norm_rotary {shape} {interleaved}")
    got = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq, eps=EPS, interleaved=interleaved)
    for x, w, y, rstd in ((q, wq, got[0], got[2]), (k, wk, got[1], got[3])):
        assert y.dtype == x.dtype and y.is_contiguous() and y.shape == x.transpose(1, 2).shape
        x = x.double()
        r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        want, size = _turn(x * r * w.double(), position, inv_freq, interleaved)
        tol = 30 * U * size + HALF[y.dtype] * want.abs()
        assert ((y.double().transpose(1, 2) - want).abs() <= tol).all()
        assert ((rstd.double().transpose(1, 2) - r[..., 0]).abs() <= 12 * U * r[..., 0]).all()
    again = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq, eps=EPS, interleaved=interleaved)
    for x, y in zip(got, again):
        assert torch.equal(x, y)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward_matches_the_formula(shape):
    """dn has the rotation's 15 u; xhat and dn w round three times more and the mean is a sum
    as the forward's: 60 u of every term's absolute value for dx.  dw adds rows one after
    the other, at most all of them in one lane, and 300 partial sums."""
    *shape, interleaved = shape
    q, k, wq, wk, position, inv_freq, rand = _inputs(*shape, seed=62)
    B, T, H, Hk, d = shape[:5]
    dy = [rand(B, h, T, d).to(q.dtype) for h in (H, Hk)]
    _, _, *rstd = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq, eps=EPS, interleaved=interleaved)
    say(f"[gpu] qk_norm_rotary_backward {shape} {interleaved}")
    got = kdn.qk_norm_rotary_backward(*dy, q, k, wq, wk, position, inv_freq, *rstd, interleaved=interleaved)
    for i, (x, w) in enumerate(((q, wq), (k, wk))):
        assert got[i].dtype == x.dtype and got[i].shape == x.shape and got[2 + i].dtype == torch.float32
        r, w = rstd[i].double().transpose(1, 2)[..., None], w.double()
        xhat = x.double() * r
        dn, size = _turn(dy[i].double().transpose(1, 2), position, inv_freq, interleaved, back=True)
        want = r * (dn * w - xhat * (dn * w * xhat).mean(-1, keepdim=True))
        most = r * (size * w.abs() + xhat.abs() * (size * w.abs() * xhat.abs()).mean(-1, keepdim=True))
        assert ((got[i].double() - want).abs() <= 60 * U * most + HALF[x.dtype] * want.abs()).all()
        rows = x.shape[0] * x.shape[1] * x.shape[2]
        tol = (rows + 300 + 20) * U * (size * xhat.abs()).sum((0, 1, 2))
        assert ((got[2 + i].double() - (dn * xhat).sum((0, 1, 2))).abs() <= tol).all()
    again = kdn.qk_norm_rotary_backward(*dy, q, k, wq, wk, position, inv_freq, *rstd, interleaved=interleaved)
    for x, y in zip(got, again):
        assert torch.equal(x, y)


def test_far_positions_keep_their_accuracy():
    """Whole turns: inv_freq 2 pi / 64 rounded to float32; position n 64 is off by n 64 times
    that rounding, which 64 bits know and float32 products do not."""
    inv = torch.full((8,), 2 * torch.pi / 64, device="cuda")
    position = torch.tensor([[0, 64, 64 * 12345, 2 ** 31 - 64, -64 * 9999]], dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 5, 1, 16, device="cuda")
    x[..., 0] = 1.0
    w = torch.full((16,), 0.25, device="cuda")
    y = kdn.qk_norm_rotary(x, x, w, w, position, inv, eps=0.0)[0][0, 0].double()
    angle = position[0].double() * inv[0].double()
    assert ((y[:, 0] - angle.cos()).abs() <= 30 * U).all() and ((y[:, 8] - angle.sin()).abs() <= 30 * U).all()


def test_against_differences():
    """Central differences in 64 bits along random directions: 1e-4 of the sum of absolute
    values."""
    q, k, wq, wk, position, inv_freq, rand = _inputs(2, 5, 3, 1, 64, 32, "f32", seed=4)
    dy = [rand(2, h, 5, 64) for h in (3, 1)]
    _, _, *rstd = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq, eps=EPS)
    got = kdn.qk_norm_rotary_backward(*dy, q, k, wq, wk, position, inv_freq, *rstd)

    def loss(q, k, wq, wk):
        total = 0.0
        for x, w, d in ((q, wq, dy[0]), (k, wk, dy[1])):
            n = x * (x.square().mean(-1, keepdim=True) + EPS) ** -0.5 * w
            total = total + (_turn(n, position, inv_freq, False)[0] * d.double().transpose(1, 2)).sum()
        return total

    leaves = (q, k, wq, wk)
    for i in range(4):
        e = rand(*leaves[i].shape).double()
        sides = [loss(*(t.double() + (z * 1e-5 * e if j == i else 0) for j, t in enumerate(leaves))) for z in (1, -1)]
        parts = got[i].double() * e
        assert abs(parts.sum() - (sides[0] - sides[1]) / 2e-5) <= 1e-4 * parts.abs().sum()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_into_the_projections_rows(dtype):
    q, k, wq, wk, position, inv_freq, rand = _inputs(2, 9, 4, 2, 64, 64, dtype, seed=5)
    dy = [rand(2, h, 9, 64).to(q.dtype) for h in (4, 2)]
    _, _, *rstd = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq)
    want = kdn.qk_norm_rotary_backward(*dy, q, k, wq, wk, position, inv_freq, *rstd)
    dz = torch.full((2, 9, 6 * 64 + 40), 7.0, dtype=q.dtype, device="cuda")
    views = dz[..., 16:16 + 4 * 64].unflatten(-1, (4, 64)), dz[..., 16 + 4 * 64:16 + 6 * 64].unflatten(-1, (2, 64))
    got = kdn.qk_norm_rotary_backward(*dy, q, k, wq, wk, position, inv_freq, *rstd, out=views)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert (dz[..., :16] == 7.0).all() and (dz[..., 16 + 6 * 64:] == 7.0).all()
    got = kdn.qk_norm_rotary_backward(*dy, q, k, wq, wk, position, inv_freq, *rstd, out=(q, k))  # over its own inputs
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_other_layouts_of_rows():
    """heads before tokens, batches that share rows, and a batch of one whose stride is odd"""
    q, k, wq, wk, position, inv_freq, _ = _inputs(2, 5, 4, 2, 32, 32, "f32", seed=7)
    want = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    got = kdn.qk_norm_rotary(qt, k.contiguous(), wq, wk, position, inv_freq)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    same = position[:1].expand(3, -1).contiguous()
    got = kdn.qk_norm_rotary(q[:1].expand(3, -1, -1, -1), k[:1].expand(3, -1, -1, -1), wq, wk, same, inv_freq)
    for x, y in zip(got, want):
        assert torch.equal(x, y[:1].expand_as(x))
    flat = torch.empty(5 * 6 * 32 + 1, device="cuda")[:5 * 6 * 32].view(1, 5, 6, 32)
    flat.copy_(torch.cat((q[:1], k[:1]), 2))
    odd = flat.as_strided(flat.shape, (5 * 6 * 32 + 1, 6 * 32, 32, 1))
    got = kdn.qk_norm_rotary(odd[:, :, :4], odd[:, :, 4:], wq, wk, position[:1], inv_freq)
    for x, y in zip(got, want):
        assert torch.equal(x, y[:1])


def test_refuses_what_it_cannot_read():
    q, k, wq, wk, position, inv_freq, _ = _inputs(2, 5, 4, 2, 32, 32, "f32", seed=7, pad=4)
    call = lambda *a: kdn.qk_norm_rotary(*a, wq, wk, position, inv_freq)  # noqa: E731
    z = torch.zeros(2, 5, 6, 36, device="cuda")
    with pytest.raises(kdn.KdnError):  # strides of 36 columns
        call(z[:, :, :4, :32], z[:, :, 4:, :32])
    z = torch.zeros(2, 5, 6, 40, device="cuda")
    with pytest.raises(kdn.KdnError):  # rows that begin 4 bytes off
        call(z[:, :, :4, 1:33], z[:, :, 4:, 1:33])
    with pytest.raises(ValueError):  # columns apart
        call(z[:, :, :4].transpose(2, 3).contiguous().transpose(2, 3)[..., :32], k)
    with pytest.raises(ValueError):
        kdn.qk_norm_rotary(q, k, wq, wk, position, None)
    with pytest.raises(ValueError):
        kdn.qk_norm_rotary(q, k, wq, wk, position.long(), inv_freq)
    with pytest.raises(ValueError):
        kdn.qk_norm_rotary(q, k.to(torch.bfloat16), wq, wk, position, inv_freq)


def test_nothing_to_do():
    w, inv = torch.ones(32, device="cuda"), torch.ones(16, device="cuda")
    for B, T, H, Hk in ((0, 3, 2, 1), (2, 0, 2, 1), (2, 3, 0, 0)):
        q, k = torch.zeros(B, T, H, 32, device="cuda"), torch.zeros(B, T, Hk, 32, device="cuda")
        p = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        out = kdn.qk_norm_rotary(q, k, w, w, p, inv)
        assert out[0].shape == (B, H, T, 32)
        g = kdn.qk_norm_rotary_backward(*out[:2], q, k, w, w, p, inv, *out[2:])
        assert (g[2] == 0).all() and (g[3] == 0).all()
    q, k = torch.randn(1, 3, 2, 32, device="cuda"), torch.zeros(1, 3, 0, 32, device="cuda")
    p = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    out = kdn.qk_norm_rotary(q, k, w, w, p, inv)
    assert torch.isfinite(out[0]).all() and (kdn.qk_norm_rotary_backward(*out[:2], q, k, w, w, p, inv, *out[2:])[3] == 0).all()


def test_what_is_not_finite_stays_in_its_row():
    q, k, wq, wk, position, inv_freq, _ = _inputs(2, 9, 4, 2, 80, 32, "bf16", seed=9)
    want = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq)
    q = q.clone()
    q[1, 3, 2, 70], q[0, 4, 1, 0], q[0, 0] = float("nan"), float("inf"), 0.0
    got = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq)
    assert got[0][1, 2, 3].isnan().all() and (got[0][0, :, 0] == 0).all() and got[0][0, 1, 4, 0].isnan()
    ok = torch.ones(2, 4, 9, dtype=torch.bool, device="cuda")
    ok[1, 2, 3] = ok[0, 1, 4] = False
    ok[0, :, 0] = False
    assert torch.equal(got[0][ok], want[0][ok]) and torch.equal(got[1], want[1])


def test_on_another_stream_and_in_a_graph():
    q, k, wq, wk, position, inv_freq, rand = _inputs(2, 300, 4, 2, 128, 128, "bf16", seed=10)
    dy = [rand(2, h, 300, 128).to(q.dtype) for h in (4, 2)]

    def both():
        out = kdn.qk_norm_rotary(q, k, wq, wk, position, inv_freq)
        return (*out, *kdn.qk_norm_rotary_backward(*dy, q, k, wq, wk, position, inv_freq, *out[2:]))

    eager = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y, z in zip(got, eager, other):
            assert torch.equal(x, y) and torch.equal(y, z)
