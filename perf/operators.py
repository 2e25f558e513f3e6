"""The operators around the KDN recurrence that run in 8 bits or as a plain scan, as cases to be timed and compared.

Each case is one call of one operator:
  norm             s = x + residual, y = s / rms(s) * weight, y in 8 bits with a scale per 128 columns or in x's type
  norm_backward    the gradient of that (dx, dweight) from dy, the kept sum s and the kept 1 / rms
  quantize         x in 8 bits with a scale per 1 x 128 (activations) or 128 x 128 block (weights)
  matmul           C = A B^T of 8-bit operands with those scales
  scan             h_t = a_t h_{t-1} + x_t over [B, H, T, d]
  scan_backward    its gradient (dx, da, dh0) from a, the kept h and dh
  scan_step        one token of it on a cache

`own` chooses between the plain form (elementary torch operations in 32 bits) and the framework's calls.  8 bits are
the e4m3 format without infinities: values up to 448.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
SCALE_MIN = 2.0 ** -126  # smallest scale: an all-zero block has this one
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # decoding: the layer's input norm for 256 sequences, one token each
        {"name": "norm_quant_step", "op": "norm", "rows": 256, "d": 2048, "dtype": "bf16", "out": "fp8", "residual": True},
        # prefill: 8 prompts of 4096 tokens
        {"name": "norm_quant_prompt", "op": "norm", "rows": 32768, "d": 2048, "dtype": "bf16", "out": "fp8", "residual": True},
        # training in 32 bits, a width that is no multiple of 128
        {"name": "norm_f32_ragged", "op": "norm", "rows": 1537, "d": 2056, "dtype": "f32", "out": "same", "residual": True},
        # training: 8 sequences of 4096 tokens
        {"name": "norm_backward", "op": "norm_backward", "rows": 32768, "d": 2048, "dtype": "bf16"},
        # loading a model: the layer's input projection (16 heads of 128, and their gates), once per weight
        {"name": "quantize_weight", "op": "quantize", "rows": 6192, "d": 2048, "dtype": "bf16", "block_rows": 128},
        # activations that no norm produces (the read-out before the output projection), ragged
        {"name": "quantize_rows", "op": "quantize", "rows": 4099, "d": 2056, "dtype": "bf16", "block_rows": 1},
        # decoding one sequence: the input projection of one token
        {"name": "matmul_token", "op": "matmul", "M": 1, "N": 6192, "K": 2048, "out": "bf16"},
        # a ragged mixed batch through an output projection, kept in 32 bits
        {"name": "matmul_ragged", "op": "matmul", "M": 509, "N": 2048, "K": 2064, "out": "f32"},
        # prefill: the input projection of 8 prompts of 4096 tokens
        {"name": "matmul_prompt", "op": "matmul", "M": 32768, "N": 6192, "K": 2048, "out": "bf16"},
        # decoding: 256 sequences of 16 heads, one token each
        {"name": "scan_step", "op": "scan_step", "B": 256, "H": 16, "d": 128, "dtype": "bf16", "gate": "f32"},
        # a long single sequence
        {"name": "scan_long", "op": "scan", "B": 1, "H": 16, "T": 65536, "d": 128, "dtype": "bf16", "gate": "bf16"},
        # training: 8 sequences of 4096 tokens
        {"name": "scan_backward", "op": "scan_backward", "B": 8, "H": 16, "T": 4096, "d": 128, "dtype": "bf16", "gate": "bf16"},
    ]


def _log(rng, low, high, multiple=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(multiple, int(round(v / multiple)) * multiple)


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_backward", "quantize", "matmul", "matmul", "matmul", "scan", "scan",
                     "scan_backward", "scan_step"))
    dtype = rng.choice(("f32", "bf16", "bf16"))
    if op in ("norm", "norm_backward", "quantize"):
        d = _log(rng, 64, 8192, 8)
        rows = _log(rng, 1, min(32768, 2 ** 26 // d))
        c = {"op": op, "rows": rows, "d": d, "dtype": dtype}
        if op == "norm":
            c["out"], c["residual"] = rng.choice(("fp8", "fp8", "same")), rng.random() < 0.8
        if op == "quantize":
            c["block_rows"] = rng.choice((1, 128))
        return c
    if op == "matmul":
        K, N = _log(rng, 64, 8192, 16), _log(rng, 32, 8192)
        M = _log(rng, 1, min(32768, 2 ** 38 // (K * N)))
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(("bf16", "bf16", "f32"))}
    d, gate = rng.choice((32, 64, 128, 128, 200)), rng.choice(("f32", "bf16"))
    if op == "scan_step":
        return {"op": op, "B": _log(rng, 1, 512), "H": rng.choice((4, 8, 16)), "d": d, "dtype": dtype, "gate": gate}
    heads, T = _log(rng, 1, 256), _log(rng, 1, 65536)
    T = min(T, 2 ** 25 // (heads * d))
    return {"op": op, "B": heads, "H": 1, "T": max(1, T), "d": d, "dtype": dtype, "gate": gate}


def _groups(x, block):
    """x [rows, d] -> [rows, ceil(d / block), block], zeros behind the last column."""
    rows, d = x.shape
    n = -(-d // block)
    return torch.nn.functional.pad(x, (0, n * block - d)).view(rows, n, block)


def _quantize(x, block_rows):
    """float32 [rows, d] -> (8-bit [rows, d], float32 scale [ceil(rows / block_rows), ceil(d / 128)])."""
    rows, d = x.shape
    nr = -(-rows // block_rows)
    g = _groups(torch.nn.functional.pad(x, (0, 0, 0, nr * block_rows - rows)), 128)
    g = g.view(nr, block_rows, g.shape[1], 128)
    scale = (g.abs().amax(dim=(1, 3)) / FP8_MAX).clamp_min(SCALE_MIN)
    q = (g / scale[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX)
    return q.reshape(nr * block_rows, -1)[:rows, :d].to(FP8), scale


def _widen(q, scale, block_rows, dtype):
    """The values that 8-bit elements and their scales stand for."""
    rows, d = q.shape
    s = scale.to(dtype).repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :d]
    return q.to(dtype) * s


def _linear(a, x, h0):
    """h_t = a_t h_{t-1} + x_t along dim 2, by doubling: after the step of s each token holds the map of its last 2 s."""
    a, x = a.clone(), x.clone()
    x[:, :, 0] += a[:, :, 0] * h0
    s = 1
    while s < a.shape[2]:
        x[:, :, s:] += a[:, :, s:] * x[:, :, :-s]
        a[:, :, s:] = a[:, :, s:] * a[:, :, :-s]
        s *= 2
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op in ("norm", "norm_backward", "quantize"):
        t, rows, d = TYPES[case["dtype"]], case["rows"], case["d"]
        st = {"case": case, "x": normal(rows, d).to(t)}
        if op != "quantize":
            st["weight"] = 1 + 0.2 * normal(d)
        if op == "norm":
            st["residual"] = (2 * normal(rows, d)).to(t) if case["residual"] else None
        if op == "norm_backward":
            st["s"] = (st.pop("x").float() * 2).to(t)
            st["rstd"] = (st["s"].float().square().mean(1) + EPS).rsqrt()
            st["dy"], st["ds"] = normal(rows, d).to(t), normal(rows, d)
        return st
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        st = {"case": case}
        st["a"], st["a_scale"] = _quantize(normal(M, K), 1)
        st["b"], st["b_scale"] = _quantize(normal(N, K) * K ** -0.5, 128)
        return st
    t, tg = TYPES[case["dtype"]], TYPES[case["gate"]]
    B, H, d = case["B"], case["H"], case["d"]
    if op == "scan_step":
        st = {"case": case, "x": normal(B, H, d).to(t), "a": torch.sigmoid(2 + normal(B, H, d)).to(tg)}
        st["h"] = normal(B, H, d)
        return st
    T = case["T"]
    a = torch.sigmoid((4 if T > 8192 else 2) + normal(B, H, T, d)).to(tg)
    x, h0 = normal(B, H, T, d).to(t), normal(B, H, d)
    if op == "scan":
        return {"case": case, "x": x, "a": a, "h0": h0}
    return {"case": case, "a": a, "h0": h0, "h": _linear(a.float(), x.float(), h0).to(t), "dh": normal(B, H, T, d).to(t),
            "dh_T": normal(B, H, d)}


def _own(st):
    import kalman_filter_memory_amd as kdn

    c = st["case"]
    op = c["op"]
    if op == "norm":
        if c["out"] == "fp8":
            return kdn.rms_norm_quant(st["x"], st["weight"], st["residual"], eps=EPS)
        return kdn.rms_norm(st["x"], st["weight"], st["residual"], eps=EPS)
    if op == "norm_backward":
        return kdn.rms_norm_backward(st["dy"], st["s"], st["weight"], st["rstd"], st["ds"])
    if op == "quantize":
        return kdn.quantize(st["x"], block_rows=c["block_rows"])
    if op == "matmul":
        return kdn.quant_matmul(st["a"], st["a_scale"], st["b"], st["b_scale"], out_dtype=TYPES[c["out"]])
    if op == "scan":
        return kdn.gated_scan(st["x"], st["a"], st["h0"])
    if op == "scan_backward":
        g = kdn.gated_scan_backward(st["a"], st["h"], st["dh"], st["h0"], st["dh_T"])
        return g["dx"], g["da"], g["dh0"]
    return kdn.gated_scan_step(st["x"], st["a"], st["h"]), st["h"]


def run(st):
    if own:
        return _own(st)
    c = st["case"]
    op = c["op"]
    if op == "norm":
        s = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(st["x"].dtype)
        f = s.float()
        rstd = (f.square().mean(1) + EPS).rsqrt()
        y = f * rstd[:, None] * st["weight"]
        if c["out"] == "fp8":
            return (*_quantize(y, 1), s)
        return y.to(s.dtype), s, rstd
    if op == "norm_backward":
        xhat = st["s"].float() * st["rstd"][:, None]
        dy = st["dy"].float()
        dn = dy * st["weight"]
        dx = st["rstd"][:, None] * (dn - xhat * (dn * xhat).mean(1, keepdim=True)) + st["ds"]
        return dx, (dy * xhat).sum(0)
    if op == "quantize":
        return _quantize(st["x"].float(), c["block_rows"])
    if op == "matmul":
        a = _widen(st["a"], st["a_scale"], 1, torch.float32)
        b = _widen(st["b"], st["b_scale"], 128, torch.float32)
        return (a @ b.t()).to(TYPES[c["out"]])
    if op == "scan":
        h = _linear(st["a"].float(), st["x"].float(), st["h0"])
        return h.to(st["x"].dtype), h[:, :, -1].clone()
    if op == "scan_backward":
        # m_t = a_t (dh_t + m_{t+1}), m behind the last token is dh_T; the gradient of h_t is dh_t + m_{t+1}
        a, dh = st["a"].float(), st["dh"].float()
        m = _linear(a.flip(2), (a * dh).flip(2), st["dh_T"]).flip(2)
        dx = dh + torch.cat((m[:, :, 1:], st["dh_T"][:, :, None]), 2)
        before = torch.cat((st["h0"][:, :, None], st["h"][:, :, :-1].float()), 2)
        return dx, dx * before, m[:, :, 0].clone()
    st["h"].copy_(st["a"].float() * st["h"] + st["x"].float())
    return st["h"].to(st["x"].dtype), st["h"]


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "norm":
        s = st["x"].to(f64)
        if st["residual"] is not None:
            s = (s + st["residual"].to(f64)).to(st["x"].dtype).to(f64)
        rstd = 1 / torch.sqrt((s * s).sum(1) / case["d"] + EPS)
        y = torch.einsum("rd,r,d->rd", s, rstd, st["weight"].to(f64))
        if case["out"] == "fp8":
            return (*_exact_quantize(y, 1), s)
        return y, s, rstd
    if op == "norm_backward":
        # y = s r w with r = (mean s^2 + eps)^(-1/2), dr/ds = -r^3 s / d, at the kept r
        s, r, w, dy = (st[n].to(f64) for n in ("s", "rstd", "weight", "dy"))
        along = (dy * w * s).sum(1)
        dx = st["ds"].to(f64) + dy * w * r[:, None] - s * (along * r ** 3 / case["d"])[:, None]
        return dx, torch.einsum("rd,r->d", dy * s, r)
    if op == "quantize":
        return _exact_quantize(st["x"].to(f64), case["block_rows"])
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        c = torch.zeros(M, N, dtype=f64, device="cuda")
        for k in range(0, K, 128):
            p = st["a"][:, k:k + 128].to(f64) @ st["b"][:, k:k + 128].to(f64).t().contiguous()
            p *= st["a_scale"][:, k // 128].to(f64)[:, None]
            p *= st["b_scale"][:, k // 128].to(f64)[torch.arange(N, device="cuda") // 128]
            c += p
        return c
    if op == "scan_step":
        h = st["a"].to(f64) * st["h"].to(f64) + st["x"].to(f64)
        return h, h
    T, h = case["T"], st["h0"].to(f64)
    if op == "scan":
        out = torch.empty(st["x"].shape, dtype=f64, device="cuda")
        for t in range(T):
            h = torch.addcmul(st["x"][:, :, t].to(f64), st["a"][:, :, t].to(f64), h)
            out[:, :, t] = h
        return out, h
    dx, da = (torch.empty(st["a"].shape, dtype=f64, device="cuda") for _ in range(2))
    g = st["dh_T"].to(f64)  # the gradient that reaches h_t from behind
    for t in range(T - 1, -1, -1):
        g = g + st["dh"][:, :, t].to(f64)
        dx[:, :, t] = g
        da[:, :, t] = g * (st["h"][:, :, t - 1].to(f64) if t else h)
        g = g * st["a"][:, :, t].to(f64)
    return dx, da, g


def _exact_quantize(x, block_rows):
    rows, d = x.shape
    scale = torch.empty(-(-rows // block_rows), -(-d // 128), dtype=torch.float64, device=x.device)
    q = torch.empty_like(x)
    if block_rows == 1:
        for j in range(scale.shape[1]):
            part = x[:, 128 * j:128 * (j + 1)]
            scale[:, j] = torch.clamp(part.abs().max(1).values / FP8_MAX, min=SCALE_MIN)
            q[:, 128 * j:128 * (j + 1)] = part / scale[:, j, None]
    else:
        for i in range(scale.shape[0]):
            for j in range(scale.shape[1]):
                part = x[block_rows * i:block_rows * (i + 1), 128 * j:128 * (j + 1)]
                scale[i, j] = torch.clamp(part.abs().max() / FP8_MAX, min=SCALE_MIN)
                q[block_rows * i:block_rows * (i + 1), 128 * j:128 * (j + 1)] = part / scale[i, j]
    return q, scale


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "fp8": 1}
    if op in ("norm", "norm_backward", "quantize"):
        n, e = case["rows"] * case["d"], size[case["dtype"]]
        scales = 4 * -(-case["rows"] // case.get("block_rows", 1)) * -(-case["d"] // 128)
        if op == "quantize":
            return {"bytes": n * (e + 1) + scales, "flops": 2 * n}
        if op == "norm_backward":
            return {"bytes": n * (2 * e + 4 + 4) + 4 * case["rows"] + 8 * case["d"], "flops": 10 * n}
        fp8 = case["out"] == "fp8"
        tail = scales if fp8 else 4 * case["rows"]
        return {"bytes": n * (e * (3 if case["residual"] else 1) + (1 if fp8 else e)) + tail + 4 * case["d"], "flops": 6 * n}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // 128)) + M * N * size[case["out"]], "flops": 2 * M * N * K}
    e, eg, ch = size[case["dtype"]], size[case["gate"]], case["B"] * case["H"] * case["d"]
    if op == "scan_step":
        return {"bytes": ch * (2 * e + eg + 8), "flops": 2 * ch}
    n = ch * case["T"]
    if op == "scan":
        return {"bytes": n * (2 * e + eg) + 8 * ch, "flops": 2 * n}
    return {"bytes": n * (2 * e + eg + 8) + 12 * ch, "flops": 4 * n}
