"""Cases of a layer's operators around its products: the root-mean-square norm with the
residual's addition, the gated activation, and the products of microscaled 4-bit operands
(e2m1 codes with a power-of-two scale for each 32 elements).

Every case runs in two forms on the same inputs: a plain one of elementary torch
operations in 32 bits, and (``own``) this package's operators.  ``exact`` gives the
outputs from the definitions in 64 bits.

The residual stream h = x + residual is held in x's type; the norm is that of the h that
is held, so that a backward pass that starts from h is the gradient of what ran forward.

4-bit operands: a block of 32 elements along K has the scale 2^E, the smallest power of
two with its largest magnitude below 7 * 2^E; the codes are x / 2^E rounded to the nearest
of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code).  Rows: codes (rows, K / 2), two to
a byte, scales (ceil(K / 128), rows, 4) bytes E + 127.  Weights: codes (E, N, K / 2),
scales (E, ceil(N / 128), ceil(K / 128), 32, 4, 4): of row n and block b at
[n // 128, b // 4, n % 32, n % 128 // 32, b % 4].
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
BLOCK = 128          # length of an e4m3 scale's block
MICRO = 32           # of a 4-bit scale's block
E4M3_MAX = 448.0     # the largest e4m3 value
TINY = 2.0 ** -126   # the smallest e4m3 scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step: latency alone
        {"name": "norm_decode", "op": "norm", "T": 64, "H": 7168, "dtype": "bf16", "residual": True, "out": "same", "backward": False},
        # a training step, with the gradient that comes down the residual stream
        {"name": "norm_train", "op": "norm", "T": 8192, "H": 4096, "dtype": "bf16", "residual": True, "out": "same", "backward": True},
        # a prompt on its way to an 8-bit product
        {"name": "norm_e4m3", "op": "norm", "T": 8192, "H": 4096, "dtype": "bf16", "residual": True, "out": "e4m3", "backward": False},
        # a small odd width in 32 bits, first norm of a model (nothing to add)
        {"name": "norm_odd", "op": "norm", "T": 1003, "H": 1401, "dtype": "f32", "residual": False, "out": "same", "backward": True},
        # the activation of a training step
        {"name": "swiglu_train", "op": "swiglu", "T": 8192, "N": 4096, "dtype": "bf16", "out": "same", "backward": True},
        # the same between the two 8-bit products of a decoding step
        {"name": "swiglu_e4m3_decode", "op": "swiglu", "T": 64, "N": 7168, "dtype": "f16", "out": "e4m3", "backward": False},
        # one token through one 4-bit layer (rows are quantised within the call, here and below)
        {"name": "fp4_token", "op": "fp4", "rows": 1, "E": 1, "K": 4096, "N": 4096, "dtype": "bf16"},
        # 4-bit decoding: one large weight matrix for 64 rows
        {"name": "fp4_decode", "op": "fp4", "rows": 64, "E": 1, "K": 16384, "N": 7168, "dtype": "bf16"},
        # 4-bit prompt through one dense layer
        {"name": "fp4_prompt", "op": "fp4", "rows": 8192, "E": 1, "K": 4096, "N": 4096, "dtype": "bf16"},
        # 4-bit decoding over experts: 64 rows hit most of 32 experts
        {"name": "fp4_experts_decode", "op": "fp4", "rows": 64, "E": 32, "K": 4096, "N": 4096, "dtype": "bf16"},
        # 4-bit prompt over experts
        {"name": "fp4_experts", "op": "fp4", "rows": 8192, "E": 32, "K": 4096, "N": 7168, "dtype": "bf16"},
        # a small ragged batch over experts, K no multiple of 128, N none of 64
        {"name": "fp4_odd", "op": "fp4", "rows": 301, "E": 6, "K": 1120, "N": 520, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "swiglu", "fp4", "fp4", "fp4"])
    if op in ("norm", "swiglu"):
        out = rng.choice(["same", "same", "e4m3"])
        width = _log(rng, 64, 8192)
        if out == "e4m3":  # the 8-bit products' rows are multiples of 16
            width = -(-width // 16) * 16
        T = min(_log(rng, 1, 8192), 8192 * 4096 // width)
        dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
        case = {"op": op, "T": T, "H" if op == "norm" else "N": width, "dtype": dtype, "out": out,
                "backward": out == "same" and rng.random() < 0.6}
        if dtype == "f32":
            case["T"] = max(1, T // 2)
        return dict(case, residual=rng.random() < 0.7) if op == "norm" else case
    K, N, E = 32 * _log(rng, 4, 256), 8 * _log(rng, 16, 512), _log(rng, 1, 64)
    while K * N * E > 16 * 4096 * 4096:
        E = max(1, E // 2)
    return {"op": op, "rows": _log(rng, 1, 8192), "E": E, "K": K, "N": N, "dtype": rng.choice(["f16", "bf16"])}


def work(case):
    op, b = case["op"], _SIZE[case["dtype"]]
    if op == "fp4":
        rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
        hit = min(rows, E)
        return {"bytes": rows * K * b + hit * N * (K // 2 + K // MICRO) + rows * N * b, "flops": 2 * rows * K * N}
    T, W = case["T"], case["H"] if op == "norm" else case["N"]
    y = T * W * b if case["out"] == "same" else T * W + T * -(-W // BLOCK) * 4
    if op == "norm":
        n, f = T * W * b + y + W * b, 4 * T * W
        if case["residual"]:
            n += 2 * T * W * b
        if case["backward"]:  # dy in, dx and dw out, and the residual stream's gradient in
            n, f = n + T * W * b * (3 if case["residual"] else 2) + 4 * W, f + 8 * T * W
        return {"bytes": n, "flops": f}
    n, f = 2 * T * W * b + y, 5 * T * W
    if case["backward"]:  # dy in, both gradients out
        n, f = n + 3 * T * W * b, f + 10 * T * W
    return {"bytes": n, "flops": f}


# ------------------------------------------------------------------ inputs
def _group_sizes(rows, E, seed):
    """Ragged group sizes: experts differ in popularity, as a trained router's do."""
    rs = np.random.RandomState(seed % (1 << 31))
    p = np.exp(0.4 * rs.standard_normal(E))
    return rs.multinomial(rows, p / p.sum()).astype(np.int64)


def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], _TYPES[case["dtype"]]
    s = {"case": case}
    if op == "norm":
        T, H = case["T"], case["H"]
        s["x"] = _randn(gen, (T, H), dt)
        s["residual"] = _randn(gen, (T, H), dt, 3.0) if case["residual"] else None  # the stream grows with depth
        s["weight"] = (1.0 + 0.1 * torch.randn((H,), generator=gen, device="cuda")).to(dt)
        if case["backward"]:
            s["dy"] = _randn(gen, (T, H), dt)
            s["dh"] = _randn(gen, (T, H), dt) if case["residual"] else None
        return s
    if op == "swiglu":
        T, N = case["T"], case["N"]
        s["x"] = _randn(gen, (T, 2 * N), dt, 1.5)
        if case["backward"]:
            s["dy"] = _randn(gen, (T, N), dt)
        return s
    rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
    sizes = _group_sizes(rows, E, seed)
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    # what the plain form keeps of the layout: the experts that have rows, and each row's place in a padded batch
    hit = np.nonzero(sizes)[0]
    place = np.concatenate([i * int(sizes.max()) + np.arange(sizes[e]) for i, e in enumerate(hit)])
    s.update(hit=torch.from_numpy(hit).cuda(), place=torch.from_numpy(place).cuda(), longest=int(sizes.max()))
    s["x"] = _randn(gen, (rows, K), dt)
    s["wq"], s["ws"] = _quantize_weights(_randn(gen, (E, N, K), dt, 1 / math.sqrt(K)))
    if own:
        from all_gather_gemm_chunked_gb300 import fp4
        s["plan"] = fp4.Fp4Linear(K, N, n_experts=E)
    return s


def _micro(f):
    """(values of the codes, scale bytes) of float rows (..., K / 32, 32): the scale from the bits of the largest magnitude, whose
    exponent goes up by one from 1.75 on."""
    e = (((f.abs().amax(-1).view(torch.int32) + 0x200000) >> 23) - 2).clamp(min=0)
    v = f * ((254 - e) << 23).view(torch.float32)[..., None]
    a = v.abs()
    half = torch.full_like(a, 0.5)
    step = torch.where(a < 2, half, torch.where(a < 4, 2 * half, 4 * half))
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=6.0), e


def _quantize_weights(w):
    """(E, N, K) weights as a model stores them in 4 bits: codes and scales, laid out as said above."""
    E, N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    q, e = _micro(w.float().view(E, N, K // MICRO, MICRO))
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + (q < 0).to(torch.uint8) * 8).view(E, N, K // 2, 2)
    s = torch.zeros((E, nb * BLOCK, kb * 4), dtype=torch.uint8, device=w.device)
    s[:, :N, :K // MICRO] = e.to(torch.uint8)
    s = s.view(E, nb, 4, 32, kb, 4).permute(0, 1, 4, 3, 2, 5).contiguous()
    return code[..., 0] + code[..., 1] * 16, s.view(torch.float8_e8m0fnu)


def _scale(largest):
    """A block's e4m3 scale from its largest magnitude.  A tensor divides it: by a number, torch would multiply with the number's
    rounded inverse."""
    return (largest / torch.full_like(largest, E4M3_MAX)).clamp(min=TINY)


# ------------------------------------------------------------------ plain forms
def _e4m3_plain(y):
    """(codes, scales (blocks, rows)) of float rows."""
    T, W = y.shape
    kb = -(-W // BLOCK)
    f = torch.zeros((T, kb * BLOCK), dtype=torch.float32, device=y.device)
    f[:, :W] = y
    f = f.view(T, kb, BLOCK)
    s = _scale(f.abs().amax(-1, keepdim=True))
    q = (f * (1.0 / s)).to(torch.float8_e4m3fn).view(T, kb * BLOCK)
    return q.view(torch.uint8)[:, :W].contiguous().view(torch.float8_e4m3fn), s[..., 0].t().contiguous()


def _norm_plain(s):
    case, x, w = s["case"], s["x"], s["weight"].float()
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
    xh = f * rstd
    out = {} if s["residual"] is None else {"h": h}
    if case["out"] == "e4m3":
        out["codes"], out["scales"] = _e4m3_plain(xh * w)
        return out
    out["y"] = (xh * w).to(x.dtype)
    if case["backward"]:
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
        out["dx"] = (dx if s["dh"] is None else dx + s["dh"].float()).to(x.dtype)
        out["dweight"] = (dy * xh).sum(0)
    return out


def _swiglu_plain(s):
    case, x = s["case"], s["x"]
    N = case["N"]
    g, u = x[:, :N].float(), x[:, N:].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    y = g * sg * u
    if case["out"] == "e4m3":
        codes, scales = _e4m3_plain(y)
        return {"codes": codes, "scales": scales}
    out = {"y": y.to(x.dtype)}
    if case["backward"]:
        dy = s["dy"].float()
        out["dx"] = torch.cat([dy * u * sg * (1.0 + g * (1.0 - sg)), dy * g * sg], 1).to(x.dtype)
    return out


def _padded(x, s):
    """Rows to (experts with rows, longest group, columns), zeros behind each group: one batched product takes them all."""
    out = torch.zeros((s["hit"].numel() * s["longest"], x.shape[1]), dtype=torch.float32, device=x.device)
    out[s["place"]] = x
    return out.view(s["hit"].numel(), s["longest"], x.shape[1])


def _fp4_plain(s):
    case, x = s["case"], s["x"]
    rows, K = x.shape
    N, kb, nb = case["N"], -(-K // BLOCK), -(-case["N"] // BLOCK)
    q, e = _micro(x.float().view(rows, K // MICRO, MICRO))
    xd = (q * torch.pow(2.0, e.float() - 127.0)[..., None]).view(rows, K)
    wq, ws = s["wq"][s["hit"]], s["ws"].view(torch.uint8)[s["hit"]]
    E = wq.shape[0]
    code = torch.stack([wq & 15, wq >> 4], -1).view(E, N, K)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    w = torch.cat([values, -values])[code.int()]
    sc = ws.permute(0, 1, 4, 3, 2, 5).reshape(E, nb * BLOCK, kb * 4)[:, :N, :K // MICRO]
    w = (w.view(E, N, K // MICRO, MICRO) * torch.pow(2.0, sc.float() - 127.0)[..., None]).view(E, N, K)
    y = torch.bmm(_padded(xd, s), w.transpose(1, 2))
    return {"y": y.reshape(-1, N)[s["place"]].to(x.dtype)}


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return _norm_plain(s) if op == "norm" else _swiglu_plain(s) if op == "swiglu" else _fp4_plain(s)
    from all_gather_gemm_chunked_gb300 import act, fp4, norm
    if op == "norm":
        out = {}
        if case["out"] == "e4m3":
            codes, scales, h = norm.rms_norm_quantized(s["x"], s["weight"], "e4m3", EPS, residual=s["residual"])
            if s["residual"] is not None:
                out["h"] = h
            out["codes"], out["scales"] = codes, scales
            return out
        r = norm.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
        if s["residual"] is not None:
            out["h"] = r.h
        out["y"] = r.y
        if case["backward"]:
            out["dx"], out["dweight"] = norm.rms_norm_backward(s["dy"], r.h, s["weight"], r.rstd, dh=s["dh"])
        return out
    if op == "swiglu":
        if case["out"] == "e4m3":
            codes, scales = act.swiglu_quantized(s["x"], "e4m3")
            return {"codes": codes, "scales": scales}
        out = {"y": act.swiglu(s["x"])}
        if case["backward"]:
            out["dx"] = act.swiglu_backward(s["dy"], s["x"])
        return out
    xq, xs = fp4.quantize_rows(s["x"])
    return {"y": s["plan"].forward(xq, xs, s["wq"], s["ws"], s["offsets"], out_dtype=s["x"].dtype)}


# ------------------------------------------------------------------ 64 bits
def _exact_e4m3(y):
    """(values of the codes, scales): scale, inverse and quotient are held in 32 bits, as the definition says; the nearest e4m3 value,
    ties to the even code, 3 bits after the leading one, exponents from -6, clipped to +-448."""
    T, W = y.shape
    q, scales = torch.empty_like(y), []
    for b in range(0, W, BLOCK):
        blk = y[:, b:b + BLOCK]
        sc = (blk.abs().amax(1, keepdim=True) / E4M3_MAX).float().clamp(min=TINY)
        v = (blk * (1.0 / sc.double()).float().double()).float().double()
        a = v.abs().cpu().numpy()
        step = torch.from_numpy(np.ldexp(1.0, np.maximum(np.frexp(a)[1] - 1, -6) - 3)).to(y.device)
        q[:, b:b + BLOCK] = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        scales.append(sc[:, 0].double())
    return q, torch.stack(scales)


def _exact_micro(x):
    """Rows as their 4-bit form stands for them: of the eight magnitudes the one between whose neighbours' midpoints a value lies."""
    x = x.double().cpu().numpy()
    b = x.reshape(x.shape[0], -1, MICRO)
    m, e = np.frexp(np.abs(b).max(-1, keepdims=True))  # the largest is m * 2^e, m from 0.5 on
    scale = np.ldexp(1.0, np.where(m >= 0.875, e - 2, e - 3))
    scale = np.where(m > 0, scale, 1.0)
    a = np.abs(b) / scale
    up, down = np.array([0.75, 1.75, 3.5]), np.array([0.25, 1.25, 2.5, 5.0])  # midpoints that round up, and down, to an even code
    code = (a[..., None] >= up).sum(-1) + (a[..., None] > down).sum(-1)
    v = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[code] * scale
    return torch.from_numpy(np.copysign(v, b).reshape(x.shape)).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, w = s["x"].double(), s["weight"].double()
        out = {}
        if s["residual"] is not None:
            held = (x + s["residual"].double()).to(s["x"].dtype)
            out["h"] = held.double()
            x = out["h"]
        r = torch.rsqrt(torch.einsum("th,th->t", x, x) / case["H"] + EPS)
        y = torch.einsum("th,t,h->th", x, r, w)
        if case["out"] == "e4m3":
            out["codes"], out["scales"] = _exact_e4m3(y)
            return out
        out["y"] = y
        if case["backward"]:  # d/dx_i of sum_j dy_j w_j x_j r(x), with dr/dx_i = -x_i r^3 / H
            dy = s["dy"].double()
            dot = torch.einsum("th,h,th->t", dy, w, x)
            out["dx"] = dy * w * r[:, None] - x * (dot * r ** 3 / case["H"])[:, None]
            if s["dh"] is not None:
                out["dx"] = out["dx"] + s["dh"].double()
            out["dweight"] = torch.einsum("th,th,t->h", dy, x, r)
        return out
    if op == "swiglu":
        N = case["N"]
        x = s["x"].double()
        g, u = x[:, :N], x[:, N:]
        p = torch.sigmoid(g)
        if case["out"] == "e4m3":
            out = {}
            out["codes"], out["scales"] = _exact_e4m3(g * p * u)
            return out
        out = {"y": g * p * u}
        if case["backward"]:
            dy = s["dy"].double()
            out["dx"] = torch.cat([dy * u * (p + g * p * (1 - p)), dy * (g * p)], 1)
        return out
    rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
    off = s["offsets"].cpu().tolist()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    n, b = torch.arange(N, device="cuda"), torch.arange(K // MICRO, device="cuda")
    x = _exact_micro(s["x"])
    y = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    for e in range(E):
        if off[e] == off[e + 1]:
            continue
        byte = s["ws"].view(torch.uint8)[e][n[:, None] // 128, b[None] // 4, n[:, None] % 32, n[:, None] % 128 // 32, b[None] % 4]
        w = torch.empty((N, K), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = table[(s["wq"][e] % 16).long()], table[(s["wq"][e] // 16).long()]
        w *= torch.exp2(byte.double() - 127).repeat_interleave(MICRO, 1)
        y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w.t()
    return {"y": y}
