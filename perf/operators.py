"""Cases of the mixture-of-experts operators: the router, the experts' products,
the 8-bit products with a scale for each block of 128, and the combination.

Every case runs in two forms on the same inputs: a plain one of elementary torch
operations in 32 bits, and (``own``) this package's operators.  ``exact`` gives the
outputs from the definitions in 64 bits.

Layout that all of them share: T tokens choose k of E experts each.  The T * k
choices, sorted by expert and within an expert by token, are the rows of the
experts' inputs; ``offsets`` (E + 1 values) says where each expert's rows begin,
``order[row] = token * k + j`` names the choice a row belongs to and ``slots[token, j]``
is its inverse.  A logit of -inf is never chosen: such a choice has expert -1, slot
-1 and weight 0, and no row (the rows from ``offsets[E]`` on are left over, order -1).
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 128          # length of a scale's block
E4M3_MAX = 448.0     # the largest e4m3 value
TINY = 2.0 ** -126   # the smallest scale: keeps 1 / scale finite for a block of zeros


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a small batch: latency alone
        {"name": "route_decode", "op": "route", "T": 64, "E": 64, "k": 4, "dtype": "f32", "masked": 0, "backward": False},
        # a training step's router with its gradient, 16-bit logits (many ties), a few experts masked for some tokens
        {"name": "route_train", "op": "route", "T": 16384, "E": 128, "k": 8, "dtype": "bf16", "masked": 3, "backward": True},
        # the experts' rows back to their tokens: one decoding step
        {"name": "combine_decode", "op": "combine", "T": 33, "E": 32, "k": 4, "H": 4096, "dtype": "f16", "masked": 0, "backward": False},
        # the same for a training step, with the gradients of the rows and of the weights
        {"name": "combine_train", "op": "combine", "T": 8192, "E": 64, "k": 4, "H": 4096, "dtype": "bf16", "masked": 0, "backward": True},
        # a small layer, as a test or a small model has it
        {"name": "experts_small", "op": "experts", "rows": 256, "E": 4, "K": 256, "N": 128, "dtype": "f16", "backward": False},
        # decoding: 16 tokens with 4 experts each read nearly every expert's weights
        {"name": "experts_decode", "op": "experts", "rows": 64, "E": 32, "K": 4096, "N": 4096, "dtype": "bf16", "backward": False},
        # a prompt over many experts of odd width: ragged groups, some far below one tile
        {"name": "experts_prompt_odd", "op": "experts", "rows": 5003, "E": 60, "K": 2056, "N": 1400, "dtype": "f16", "backward": False},
        # a training step of one layer: product, gradient of the input, gradient of the weights
        {"name": "experts_train", "op": "experts", "rows": 16384, "E": 16, "K": 4096, "N": 4096, "dtype": "bf16", "backward": True},
        # 8-bit decoding: one large weight matrix for 64 rows (quantised within the call)
        {"name": "fp8_decode", "op": "fp8", "rows": 64, "E": 1, "K": 16384, "N": 7168, "dtype": "bf16"},
        # 8-bit prompt through one dense layer
        {"name": "fp8_prompt", "op": "fp8", "rows": 8192, "E": 1, "K": 4096, "N": 4096, "dtype": "bf16"},
        # 8-bit prompt over experts
        {"name": "fp8_experts", "op": "fp8", "rows": 8192, "E": 32, "K": 4096, "N": 7168, "dtype": "bf16"},
        # a small ragged batch over experts, K no multiple of 128, N none of 64
        {"name": "fp8_odd", "op": "fp8", "rows": 301, "E": 6, "K": 1104, "N": 520, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "combine", "experts", "experts", "fp8", "fp8"])
    if op == "route":
        E = rng.randint(4, 256)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 8)), "dtype": rng.choice(["f32", "f16", "bf16"]),
                "masked": rng.randint(0, 3), "backward": rng.random() < 0.5}
    if op == "combine":
        E = rng.randint(4, 128)
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(E, 4)), "H": _log(rng, 64, 4096),
                "dtype": rng.choice(["f16", "bf16"]), "masked": 0, "backward": rng.random() < 0.5}
    K, N, E = 16 * _log(rng, 8, 256), 8 * _log(rng, 16, 512), _log(rng, 1, 64)
    while K * N * E > 16 * 4096 * 4096:
        E = max(1, E // 2)
    rows = _log(rng, 1, 8192)
    case = {"op": op, "rows": rows, "E": E, "K": K, "N": N, "dtype": rng.choice(["f16", "bf16"])}
    return dict(case, backward=rng.random() < 0.5) if op == "experts" else case


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, b = case["T"], case["E"], case["k"], _SIZE[case["dtype"]]
        n = T * E * b + T * k * (4 + 4 + 4 + 4) + 4 * (E + 1)
        f = 4 * T * E
        if case["backward"]:  # dweights in, dlogits out (the forward's reads are not repeated)
            n, f = n + T * k * 4 + T * E * b, f + 4 * T * E
        return {"bytes": n, "flops": f}
    if op == "combine":
        T, k, H, b = case["T"], case["k"], case["H"], _SIZE[case["dtype"]]
        n, f = T * k * H * b + T * H * b + T * k * 8, 2 * T * k * H
        if case["backward"]:  # y again only for the weights' gradient: counted once; dout in, dy and dweights out
            n, f = n + T * H * b + T * k * H * b + T * k * 4, f + 3 * T * k * H
        return {"bytes": n, "flops": f}
    rows, E, K, N, b = case["rows"], case["E"], case["K"], case["N"], _SIZE[case["dtype"]]
    hit = min(rows, E)
    f = 2 * rows * K * N
    if op == "fp8":
        return {"bytes": rows * K * b + hit * (K * N + 4 * -(-K // BLOCK) * -(-N // BLOCK)) + rows * N * b, "flops": f}
    n = rows * K * b + hit * K * N * b + rows * N * b
    if case["backward"]:  # dy in; dx out; dw out in 32 bits
        n, f = n + rows * N * b + rows * K * b + E * K * N * 4, 3 * f
    return {"bytes": n, "flops": f}


# ------------------------------------------------------------------ inputs
def _group_sizes(rows, E, seed):
    """Ragged group sizes: experts differ in popularity, as a trained router's do."""
    rs = np.random.RandomState(seed % (1 << 31))
    p = np.exp(0.4 * rs.standard_normal(E))
    return rs.multinomial(rows, p / p.sum()).astype(np.int64)


def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _logits(case, gen):
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=gen, device="cuda") + 0.5 * torch.randn((1, E), generator=gen, device="cuda")
    if case["masked"]:  # some tokens may not use the first experts
        rows = torch.rand((T, 1), generator=gen, device="cuda") < 0.25
        x = x.masked_fill(rows & (torch.arange(E, device="cuda") < min(case["masked"], E - 1))[None], float("-inf"))
    return x.to(_TYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], _TYPES[case["dtype"]]
    s = {"case": case}
    if op == "route":
        s["logits"] = _logits(case, gen)
        s["dweights"] = _randn(gen, (case["T"], case["k"]), torch.float32)
        return s
    if op == "combine":
        T, k, H = case["T"], case["k"], case["H"]
        w, experts, offsets, order, slots = _route_plain(torch.randn((T, case["E"]), generator=gen, device="cuda"), k)
        s.update(weights=w, offsets=offsets, order=order, slots=slots, y=_randn(gen, (T * k, H), dt), dout=_randn(gen, (T, H), dt))
        return s
    rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
    sizes = _group_sizes(rows, E, seed)
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    # what the plain form keeps of the layout: the experts that have rows, and each row's place in a padded batch
    hit = np.nonzero(sizes)[0]
    place = np.concatenate([i * int(sizes.max()) + np.arange(sizes[e]) for i, e in enumerate(hit)])
    s.update(hit=torch.from_numpy(hit).cuda(), place=torch.from_numpy(place).cuda(), longest=int(sizes.max()))
    s["x"] = _randn(gen, (rows, K), dt)
    w = _randn(gen, (E, K, N), dt, 1 / math.sqrt(K))
    if op == "experts":
        s["w"] = w
        if case["backward"]:
            s["dy"] = _randn(gen, (rows, N), dt)
        if own:
            from all_gather_gemm_chunked_gb300 import moe
            s["plan"] = moe.Experts(E, K, N, case["dtype"])
    else:
        s["wq"], s["ws"] = _quantize_weights(w)
        if own:
            from all_gather_gemm_chunked_gb300 import fp8
            s["plan"] = fp8.Fp8Linear(K, N, n_experts=E)
    return s


def _quantize_weights(w):
    """(E, K, N) weights as a model stores them in 8 bits: (E, N, K) codes and one scale for each 128 x 128 block."""
    E, K, N = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    f = torch.zeros((E, nb * BLOCK, kb * BLOCK), dtype=torch.float32, device=w.device)
    f[:, :N, :K] = w.transpose(1, 2)
    f = f.view(E, nb, BLOCK, kb, BLOCK)
    scales = _scale(f.abs().amax((2, 4)))
    q = (f * (1.0 / scales)[:, :, None, :, None]).to(torch.float8_e4m3fn).view(E, nb * BLOCK, kb * BLOCK)
    return q.view(torch.uint8)[:, :N, :K].contiguous().view(torch.float8_e4m3fn), scales


def _scale(largest):
    """A block's scale from its largest magnitude.  A tensor divides it: by a number, torch would multiply with the number's rounded
    inverse, and 16-bit inputs lie on the codes' ties so often that one last bit of the scale moves many codes."""
    return (largest / torch.full_like(largest, E4M3_MAX)).clamp(min=TINY)


# ------------------------------------------------------------------ plain forms
def _route_plain(logits, k):
    """Softmax over the k largest logits of each token (ties: the lowest expert), and the layout of the rows."""
    T, E = logits.shape
    top, experts = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    valid = top != float("-inf")
    e = torch.exp(top - top[:, :1].clamp(min=torch.finfo(torch.float32).min)) * valid
    weights = e / e.sum(1, keepdim=True).clamp(min=TINY)
    flat = torch.where(valid, experts, E).reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=logits.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)[:E]])
    slots = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=logits.device))
    kept = valid.reshape(-1)
    slots = torch.where(kept, slots, -1).reshape(T, k)
    order = torch.where(kept[order], order, -1)
    experts = torch.where(valid, experts, -1)
    return weights, experts.int(), offsets.int(), order.int(), slots.int()


def _route_backward_plain(logits, weights, experts, dweights):
    d = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
    full = torch.zeros((logits.shape[0], logits.shape[1] + 1), dtype=torch.float32, device=logits.device)
    full.scatter_(1, torch.where(experts >= 0, experts, logits.shape[1]).long(), d)
    return full[:, :-1].to(logits.dtype)


def _combine_plain(s):
    y, slots, w = s["y"], s["slots"].long(), s["weights"]
    valid = (slots >= 0)[..., None]
    rows = y.float()[slots.clamp(min=0)] * valid
    out = (rows * w[..., None]).sum(1).to(y.dtype)
    if not s["case"]["backward"]:
        return {"out": out}
    dout = s["dout"].float()[:, None, :]
    dy = torch.zeros((y.shape[0] + 1, y.shape[1]), dtype=y.dtype, device=y.device)
    dy[torch.where(slots >= 0, slots, y.shape[0])] = (w[..., None] * dout).to(y.dtype)
    return {"out": out, "dy": dy[:-1], "dweights": (dout * rows).sum(-1)}


def _padded(x, s):
    """Rows to (experts with rows, longest group, columns), zeros behind each group: one batched product takes them all."""
    out = torch.zeros((s["hit"].numel() * s["longest"], x.shape[1]), dtype=torch.float32, device=x.device)
    out[s["place"]] = x.float()
    return out.view(s["hit"].numel(), s["longest"], x.shape[1])


def _rows(p, s):
    return p.reshape(-1, p.shape[-1])[s["place"]]


def _experts_plain(s):
    x, w = s["x"], s["w"]
    xp, wf = _padded(x, s), w[s["hit"]].float()
    out = {"y": _rows(torch.bmm(xp, wf), s).to(x.dtype)}
    if s["case"]["backward"]:
        dyp = _padded(s["dy"], s)
        out["dx"] = _rows(torch.bmm(dyp, wf.transpose(1, 2)), s).to(x.dtype)
        out["dw"] = torch.zeros(w.shape, dtype=torch.float32, device=w.device)
        out["dw"][s["hit"]] = torch.bmm(xp.transpose(1, 2), dyp)
    return out


def _fp8_plain(s):
    x, wq, ws = s["x"], s["wq"], s["ws"]
    rows, K = x.shape
    N, kb, nb = wq.shape[1], ws.shape[2], ws.shape[1]
    f = torch.zeros((rows, kb * BLOCK), dtype=torch.float32, device=x.device)
    f[:, :K] = x
    f = f.view(rows, kb, BLOCK)
    sx = _scale(f.abs().amax(-1, keepdim=True))
    xd = ((f * (1.0 / sx)).to(torch.float8_e4m3fn).float() * sx).view(rows, kb * BLOCK)[:, :K]
    scales = ws[s["hit"]].repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    wd = wq.view(torch.uint8)[s["hit"]].view(torch.float8_e4m3fn).float() * scales
    return {"y": _rows(torch.bmm(_padded(xd, s), wd.transpose(1, 2)), s).to(x.dtype)}


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "route":
            w, experts, offsets, order, slots = _route_plain(s["logits"], case["k"])
            out = {"weights": w, "experts": experts, "offsets": offsets, "order": order, "slots": slots}
            if case["backward"]:
                out["dlogits"] = _route_backward_plain(s["logits"], w, experts, s["dweights"])
            return out
        return _combine_plain(s) if op == "combine" else _experts_plain(s) if op == "experts" else _fp8_plain(s)
    from all_gather_gemm_chunked_gb300 import fp8, moe
    if op == "route":
        r = moe.route(s["logits"], case["k"])
        out = {"weights": r.weights, "experts": r.experts, "offsets": r.offsets, "order": r.order, "slots": r.slots}
        if case["backward"]:
            out["dlogits"] = moe.route_backward(s["logits"], r, s["dweights"])
        return out
    if op == "combine":
        out = {"out": moe.combine(s["y"], s["slots"], s["weights"])}
        if case["backward"]:
            out["dy"], out["dweights"] = moe.combine_backward(s["dout"], s["y"], s["slots"], s["weights"], s["offsets"])
        return out
    if op == "experts":
        p = s["plan"]
        out = {"y": p.forward(s["x"], s["offsets"], s["w"])}
        if case["backward"]:
            out["dx"] = p.backward_input(s["dy"], s["offsets"], s["w"])
            out["dw"] = p.backward_weight(s["x"], s["dy"], s["offsets"])
        return out
    xq, xs = fp8.quantize_rows(s["x"])
    return {"y": s["plan"].forward(xq, xs, s["wq"], s["ws"], s["offsets"], out_dtype=s["x"].dtype)}


# ------------------------------------------------------------------ 64 bits
def _e4m3(v):
    """The e4m3 value nearest to each v (ties to the even code), clipped to +-448: 3 bits after the leading one, exponents from -6."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20)))
    e = torch.where(torch.pow(2.0, e) > a, e - 1, e)
    step = torch.pow(2.0, e.clamp(min=-6.0) - 3)
    return torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        z = s["logits"].double().cpu().numpy()
        T, k = case["T"], case["k"]
        idx = np.argsort(-z, axis=1, kind="stable")[:, :k]
        t = np.take_along_axis(z, idx, 1)
        p = np.where(np.isneginf(t), 0.0, np.exp(t - np.where(np.isneginf(t[:, :1]), 0.0, t[:, :1])))
        tot = p.sum(1, keepdims=True)
        w = np.divide(p, tot, out=np.zeros_like(p), where=tot > 0)
        out = {"weights": w, "experts": None, "offsets": None, "order": None, "slots": None}
        if case["backward"]:
            g = s["dweights"].double().cpu().numpy()
            d = np.zeros_like(z)
            np.put_along_axis(d, idx, w * (g - (w * g).sum(1, keepdims=True)), 1)
            out["dlogits"] = d
        return out
    if op == "combine":
        slots, w, y = s["slots"].long(), s["weights"].double(), s["y"].double()
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        dy, dw = torch.zeros_like(y), torch.zeros_like(w)
        g = s["dout"].double()
        for j in range(case["k"]):
            at = slots[:, j]
            t = torch.nonzero(at >= 0).flatten()
            r = y[at[t]]
            out[t] += w[t, j, None] * r
            dy[at[t]] = w[t, j, None] * g[t]
            dw[t, j] = torch.einsum("th,th->t", g[t], r)
        return {"out": out, "dy": dy, "dweights": dw} if case["backward"] else {"out": out}
    off = s["offsets"].cpu().tolist()
    x = s["x"].double()
    if op == "fp8":
        K = case["K"]
        for b in range(0, K, BLOCK):  # scale, inverse and quotient are held in 32 bits: their roundings belong to the definition (16-bit inputs often lie on ties)
            blk = x[:, b:b + BLOCK]
            sc = (blk.abs().amax(1, keepdim=True) / E4M3_MAX).float().clamp(min=TINY)
            x[:, b:b + BLOCK] = _e4m3((blk * (1.0 / sc.double()).float().double()).float().double()) * sc.double()
    y = torch.zeros((case["rows"], case["N"]), dtype=torch.float64, device="cuda")
    back = op == "experts" and case["backward"]
    if back:
        g, dx, dw = s["dy"].double(), torch.zeros_like(x), torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if op == "fp8":
            sc = s["ws"][e].double()
            we = s["wq"][e].double()
            n, k = torch.arange(we.shape[0], device="cuda") // BLOCK, torch.arange(we.shape[1], device="cuda") // BLOCK
            we = (we * sc[n][:, k]).t()
        else:
            we = s["w"][e].double()
        y[a:b] = x[a:b] @ we
        if back:
            dx[a:b] = g[a:b] @ we.t()
            dw[e] = x[a:b].t() @ g[a:b]
    return {"y": y, "dx": dx, "dw": dw} if back else {"y": y}
