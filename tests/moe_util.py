"""References in 64 bits and error bounds for the mixture-of-experts tests."""
import numpy as np
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# unit roundoffs above; smallest spacing of the type (a subnormal's rounding error is half of it)
STEP = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def offsets_of(sizes, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def check(got, ref, err, what=""):
    """|got - ref| <= err elementwise; NaN and infinities of ref where got has them."""
    g, r = got.double(), ref.double()
    fine = torch.isfinite(r)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN elsewhere"
    assert torch.equal(g[~fine & ~torch.isnan(r)], r[~fine & ~torch.isnan(r)]), f"{what}: infinities"
    d = (g - r).abs()[fine]
    e = (err if torch.is_tensor(err) else torch.full_like(r, err))[fine]
    if d.numel():
        bad = d > e
        assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {d.numel()} off, worst {float((d - e)[bad].max()):.3e} "
                                     f"beyond its bound (error {float(d[bad].max()):.3e})")


def product_bound(a, b, red, out_dtype):
    """Bound of sum_k a b in 32 bits, any order, each addition off by up to 2^-23 of the
    running sum of magnitudes (truncated additions included), and one rounding."""
    mag = a.abs() @ b.abs()
    ref = (a @ b).abs()
    return (red + 2) * 2.0 ** -23 * mag + U[out_dtype] * ref * 1.01 + STEP[out_dtype]


def route_ref(logits, k, normalize=True):
    """(weights, experts, offsets, order, slots) by the definition, in numpy."""
    z = logits.double().cpu().numpy()
    T, E = z.shape
    w = np.zeros((T, k))
    ex = np.full((T, k), -1, np.int64)
    for t in range(T):
        row = z[t]
        nan = np.isnan(row)
        cand = [e for e in range(E) if not nan[e] and row[e] != -np.inf]
        cand.sort(key=lambda e: (-row[e], e))
        ch = cand[:k]
        ex[t, :len(ch)] = ch
        if not ch:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.exp(row[ch] - row[ch[0]])
            tot = p.sum() if normalize else np.exp(row[~nan] - row[ch[0]]).sum()
            w[t, :len(ch)] = p / tot
        if nan.any():
            w[t, :len(ch)] = np.nan
    flat = ex.reshape(-1)
    rows = [i for e in range(E) for i in np.nonzero(flat == e)[0]]
    order = np.full(T * k, -1, np.int64)
    order[:len(rows)] = rows
    slots = np.full(T * k, -1, np.int64)
    slots[rows] = np.arange(len(rows))
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    return w, ex, offsets, order, slots.reshape(T, k)


def quantize_ref(x, dims):
    """Codes (float64 values) and scales of blocks: `dims` are the block's axes of x, a
    view whose other axes number the blocks.  The roundings to float belong to the
    definition."""
    amax = x.abs().amax(dims, keepdim=True).double()
    s = (amax / 448).float().clamp(min=2.0 ** -126)
    inv = (1.0 / s.double()).float()
    return e4m3((x.double() * inv.double()).float().double()), s


def e4m3(v):
    """Nearest e4m3 value (ties to even, clipped to 448), in 64 bits: a step is 2^-3 of
    the value's power of two, from 2^-6 on.  On the host, where frexp and ldexp are exact."""
    a = v.cpu().numpy()
    step = np.ldexp(1.0, np.maximum(np.frexp(a)[1] - 1, -6) - 3)
    return torch.from_numpy(np.clip(np.rint(a / step) * step, -448.0, 448.0)).to(v.device)
