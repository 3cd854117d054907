"""Router, gather and combine, with their gradients, against the definitions in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import moe  # noqa: E402
from moe_util import STEP, U, check, randn, rng, route_ref  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _same_layout(r, ref):
    _, ex, off, order, slots = ref
    for name, got, want in (("experts", r.experts, ex), ("offsets", r.offsets, off), ("order", r.order, order),
                            ("slots", r.slots, slots)):
        assert np.array_equal(got.cpu().numpy(), want), name


def _weights_bound(logits, k, E):
    """exp within 2 ulp of its rounded argument, a sum of up to E terms, a quotient."""
    spread = logits.float().nan_to_num(0, 0, 0).abs().amax() * 2
    return float((spread + E + 8) * 2.0 ** -23)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (5, 7, 3), (64, 64, 4), (127, 33, 5), (128, 256, 8),
                                   (129, 16, 2), (700, 60, 6), (1000, 512, 32), (300, 1024, 4), (5000, 3, 3)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("normalize", [True, False])
def test_route(T, E, k, dtype, normalize):
    logits = randn(rng(T + E), (T, E), dtype)
    r = moe.route(logits, k, normalize)
    ref = route_ref(logits, k, normalize)
    _same_layout(r, ref)
    check(r.weights, torch.from_numpy(ref[0]).cuda(), _weights_bound(logits, k, E), "weights")


@pytest.mark.parametrize("T", [40, 400])
def test_route_ties_and_masks(T):
    g = rng(3)
    z = torch.randint(-2, 3, (T, 24), generator=g, device="cuda").float() / 2  # many ties
    z = z.masked_fill(torch.rand((T, 24), generator=g, device="cuda") < 0.7, float("-inf"))
    z[0] = float("-inf")                       # nothing left
    z[1] = float("-inf")
    z[1, 7] = 1.0                              # one left
    z[2] = 0.0
    z[2, ::2] = -0.0                           # -0 ties with +0
    z[3] = torch.finfo(torch.float32).min      # the lowest value is no mask
    z[4] = float("-inf")
    z[4, 3] = torch.finfo(torch.float32).min
    for normalize in (True, False):
        r = moe.route(z, 6, normalize)
        ref = route_ref(z, 6, normalize)
        _same_layout(r, ref)
        check(r.weights, torch.from_numpy(ref[0]).cuda(), 40 * 2.0 ** -23)
        assert int(r.offsets[-1]) < T * 6 and r.experts[0].tolist() == [-1] * 6
        assert bool((r.weights[0] == 0).all())


def test_route_nan_and_infinity():
    z = randn(rng(4), (70, 20))
    z[5, 2] = float("nan")
    z[6] = float("nan")
    z[7, 3] = float("inf")
    r, ref = moe.route(z, 4), route_ref(z, 4)
    _same_layout(r, ref)
    check(r.weights, torch.from_numpy(ref[0]).cuda(), 40 * 2.0 ** -23)
    assert bool(torch.isnan(r.weights[5]).all()) and r.experts[6].tolist() == [-1] * 4


def test_route_pitched_and_empty():
    wide = randn(rng(5), (200, 50), torch.bfloat16)
    _same_layout(moe.route(wide[:, 10:43], 3), route_ref(wide[:, 10:43], 3))
    r = moe.route(torch.empty((0, 9), device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 10 and r.weights.shape == (0, 2)
    assert moe.route_backward(torch.empty((0, 9), device="cuda"), r, r.weights).shape == (0, 9)


def _dlogits_ref(logits, ref, dw, normalize):
    z = logits.double().cpu().numpy()
    w, ex = ref[0], ref[1]
    g = dw.double().cpu().numpy()
    g = np.where(ex >= 0, g, 0)
    dot = (w * g).sum(1, keepdims=True)
    out = np.zeros_like(z)
    for t in range(z.shape[0]):
        if not normalize and (z[t] != -np.inf).any():
            p = np.exp(z[t] - z[t].max())
            out[t] = -p / p.sum() * dot[t]
        for j in range(w.shape[1]):
            if ex[t, j] >= 0:
                out[t, ex[t, j]] = w[t, j] * (g[t, j] - dot[t, 0])
    return torch.from_numpy(out).cuda()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (6, 9, 4), (130, 40, 8), (50, 700, 32), (3000, 64, 2)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("normalize", [True, False])
def test_route_backward(T, E, k, dtype, normalize):
    g = rng(T * 3 + E)
    logits = randn(g, (T, E), dtype)
    if E > 2 * k:
        logits[:, 1] = float("-inf")
    if T > 4 and k > 1:
        logits[2] = float("-inf")
        logits[3, 1:] = float("-inf")
    dw = randn(g, (T, k))
    r = moe.route(logits, k, normalize)
    d = moe.route_backward(logits, r, dw)
    ref = _dlogits_ref(logits, route_ref(logits, k, normalize), dw, normalize)
    # products and sums of k terms of weights that are off by _weights_bound
    mag = float(dw.abs().max()) * 3
    finite = logits.masked_fill(logits == float("-inf"), 0)
    err = mag * (2 * _weights_bound(finite, k, E) + (k + 4) * 2.0 ** -23)
    check(d, ref, err + 1.01 * U[dtype] * ref.abs() + STEP[dtype], "dlogits")


@pytest.mark.parametrize("normalize", [True, False])
def test_route_backward_is_the_difference(normalize):
    """Central differences of <dweights, weights>, with logits far enough apart that a
    step changes no choice.  Step h: truncation error about h^2 |f'''| / 6 <= h^2 |dw|,
    rounding of the weights 2^-22 |dw| k / h."""
    g = rng(17)
    T, E, k, h = 12, 10, 3, 2.0 ** -7
    z = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i)) for i in range(T)]).float().cuda() * 0.5
    dw = randn(g, (T, k))
    r = moe.route(z, k, normalize)
    d = moe.route_backward(z, r, dw)
    tol = float(dw.abs().max()) * (h * h + 2.0 ** -22 * k / h)
    for e in range(E):
        step = torch.zeros_like(z)
        step[:, e] = h
        a, b = moe.route(z + step, k, normalize), moe.route(z - step, k, normalize)
        diff = ((a.weights - b.weights).double() * dw).sum(1) / (2 * h)
        assert float((diff - d[:, e]).abs().max()) <= tol


ROWS = [(1, 1, 8), (3, 2, 1), (9, 4, 7), (33, 5, 72), (40, 8, 4096), (17, 3, 2056), (5, 32, 130), (300, 2, 1000)]


@pytest.mark.parametrize("T,k,H", ROWS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("masked", [False, True])
def test_gather_and_combine(T, k, H, dtype, masked):
    g = rng(T + k + H)
    E = max(k, 6)
    logits = randn(g, (T, E))
    if masked:
        logits = logits.masked_fill(torch.rand((T, E), generator=g, device="cuda") < 0.5, float("-inf"))
    r = moe.route(logits, k)
    x, y, dout = randn(g, (T, H), dtype), randn(g, (T * k, H), dtype), randn(g, (T, H), dtype)
    used, order = int(r.offsets[-1]), r.order.long()
    rows = moe.gather(x, r)
    assert torch.equal(rows[:used], x[order[:used] // k]) and not bool(rows[used:].any())
    if masked:
        y[used:] = float("nan")  # rows in nobody's use are not read
    out, plain = moe.combine(y, r.slots, r.weights), moe.combine(y, r.slots)
    dy, dw = moe.combine_backward(dout, y, r.slots, r.weights, r.offsets)
    valid, s = (r.slots >= 0)[..., None], r.slots.long().clamp(min=0)
    yr = torch.where(valid, y.double()[s], 0.0)
    w = r.weights.double()[..., None]
    for got, ref, mag in ((out, (w * yr).sum(1), (w * yr).abs().sum(1)), (plain, yr.sum(1), yr.abs().sum(1))):
        check(got, ref, (k + 1) * 2.0 ** -24 * mag + 1.01 * U[dtype] * ref.abs() + STEP[dtype])
    t, j = order[:used] // k, order[:used] % k
    ref = r.weights.double()[t, j][:, None] * dout.double()[t]
    check(dy[:used], ref, 1.01 * U[dtype] * ref.abs() + STEP[dtype] + 2.0 ** -24 * ref.abs())
    assert not bool(dy[used:].any())
    g_ = dout.double()[:, None]
    check(dw, (g_ * yr).sum(-1), (H + 1) * 2.0 ** -24 * (g_ * yr).abs().sum(-1) + 1e-30)


# rows that share a block, pieces that the end of a row cuts, rows beyond the last block's
@pytest.mark.parametrize("T,k,H", [(13, 3, 118), (7, 2, 255), (9, 2, 257), (11, 4, 1025), (5, 3, 2191), (6, 5, 520), (19, 1, 2048)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_any_length(T, k, H, dtype):
    test_gather_and_combine(T, k, H, dtype, True)


def test_combine_without_offsets_and_pitched():
    g = rng(23)
    T, k, H = 21, 4, 64
    r = moe.route(randn(g, (T, 8)), k)
    yw, dw_ = randn(g, (T * k, H + 32), torch.float16), randn(g, (T, H + 8), torch.float16)
    y, dout = yw[:, 32:], dw_[:, 3:H + 3]  # 6 bytes off: single elements
    a = moe.combine_backward(dout, y, r.slots, r.weights)
    b = moe.combine_backward(dout.contiguous(), y.contiguous(), r.slots, r.weights, r.offsets)
    assert torch.equal(a[0], b[0])
    check(a[1], b[1], float((H + 1) * 2.0 ** -23 * (dout.double().abs().max() * y.double().abs().max() * H)))
    assert torch.equal(moe.combine(y, r.slots, r.weights), moe.combine(y.contiguous(), r.slots, r.weights))
    assert torch.equal(moe.gather(dout, r), moe.gather(dout.contiguous(), r))


def test_combine_gradients_are_the_differences():
    """combine is linear in y and in the weights: with small whole numbers (weights in
    eighths) the differences are exact."""
    g = rng(24)
    T, k, H = 9, 3, 24
    r = moe.route(randn(g, (T, 7)), k)

    def ints(shape):
        return torch.randint(-4, 5, shape, generator=g, device="cuda").float()

    y, v, dout, w, u = ints((T * k, H)), ints((T * k, H)), ints((T, H)), ints((T, k)) / 8, ints((T, k)) / 8
    dy, dw = moe.combine_backward(dout, y, r.slots, w, r.offsets)
    d = (moe.combine(y + v, r.slots, w) - moe.combine(y - v, r.slots, w)) / 2
    assert float((dout * d).double().sum()) == float((dy * v).double().sum())
    d = (moe.combine(y, r.slots, w + u) - moe.combine(y, r.slots, w - u)) / 2
    assert float((dout * d).double().sum()) == float((dw * u).double().sum())
    x, vx, dr = ints((T, H)), ints((T, H)), ints((T * k, H))
    d = (moe.gather(x + vx, r) - moe.gather(x - vx, r)) / 2
    assert float((dr * d).double().sum()) == float((moe.combine(dr, r.slots) * vx).double().sum())


def test_slots_and_order_out_of_range_are_left_out():
    T, k, H = 4, 2, 16
    r = moe.route(randn(rng(25), (T, 4)), k)
    slots, order = r.slots.clone(), r.order.clone()
    slots[1, 0], slots[2, 1], order[3] = T * k, -7, T * k + 5
    y = torch.ones((T * k, H), device="cuda")
    out = moe.combine(y, slots)
    assert out[:, 0].tolist() == [2, 1, 1, 2]
    rows = moe.gather(torch.ones((T, H), device="cuda"), r._replace(order=order))
    assert rows[3].abs().sum() == 0 and bool((rows[[0, 1, 2, 4]] == 1).all())
    dy, dw = moe.combine_backward(torch.ones((T, H), device="cuda"), y, slots, r.weights, r.offsets)
    assert float(dw[1, 0]) == 0 and float(dw[2, 1]) == 0 and float(dw[0, 0]) == H


def test_stream_argument():
    z = randn(rng(26), (500, 32))
    want = moe.route(z, 4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = moe.route(z, 4, stream=s)
    s.synchronize()
    for a, b in zip(got[:5], want[:5]):
        assert torch.equal(a, b)


def test_refusals():
    z = torch.zeros((4, 8), device="cuda")
    r = moe.route(z, 2)
    for bad_k in (0, 9, 33, -1):
        with pytest.raises(B_.AgGemmError) as e:
            moe.route(z, bad_k)
        assert e.value.code == B_.ERR_INVALID
    with pytest.raises(B_.AgGemmError):
        moe.route(torch.zeros((2, 1025), device="cuda"), 2)
    for bad in (z.cpu(), z.double(), z.t(), z[0], "z"):
        with pytest.raises((TypeError, ValueError)):
            moe.route(bad, 2)
    y = torch.zeros((8, 16), device="cuda")
    with pytest.raises(ValueError):
        moe.combine(y[:7], r.slots)
    with pytest.raises(TypeError):
        moe.combine(y, r.slots.long())
    with pytest.raises(TypeError):
        moe.combine(y, r.slots, r.weights.half())
    with pytest.raises(TypeError):
        moe.combine_backward(torch.zeros((4, 16), dtype=torch.float16, device="cuda"), y, r.slots, r.weights)
    with pytest.raises(ValueError):
        moe.combine_backward(torch.zeros((3, 16), device="cuda"), y, r.slots, r.weights)
    with pytest.raises(ValueError):
        moe.route_backward(z, r, torch.zeros((4, 3), device="cuda"))
    with pytest.raises(ValueError):
        moe.gather(torch.zeros((5, 16), device="cuda"), r)
    lib = B_.library_handle()
    assert lib.ag_moe_route(4, 8, 2, 7, None, 8, 1, None, None, None, None, None, None, None) == B_.ERR_INVALID
    assert lib.ag_moe_route(4, 8, 2, 0, None, 8, 1, None, None, None, None, None, None, None) == B_.ERR_INVALID
    assert lib.ag_moe_route_workspace(1 << 29, 8, 2) == B_.ERR_UNSUPPORTED
