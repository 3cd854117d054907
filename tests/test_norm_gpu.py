"""The root-mean-square norm, its gradient and its outputs as codes, against the definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp4, fp8, norm  # noqa: E402
from layer_util import row_values  # noqa: E402
from moe_util import STEP, U, check, randn, rng  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
F = 2.0 ** -24  # a rounding to float
# lengths: one element, odd ones, a warp's, a block's, two and four pieces a thread, beyond what registers hold
SHAPES = [(1, 1), (3, 7), (5, 64), (2, 118), (70, 256), (33, 1401), (9, 2048), (400, 2056), (64, 7168), (310, 4096),
          (6, 9001), (305, 8192), (3, 16384), (2, 32768), (4, 40000), (0, 64)]


def forward_ref(x, res, w, eps):
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    d = h.double()
    rstd = 1 / torch.sqrt((d * d).mean(1) + eps)
    return h, rstd, d * rstd[:, None] * w.double()


def forward_error(H):
    """Of y before its rounding, relative: the squares' sum (at most 32 terms in a thread, or H / 1024, and ten steps of
    a tree), whose root halves it, and eight more roundings."""
    return ((48 + H / 1024) / 2 + 8) * F


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual,w32", [(False, False), (True, True)])
def test_forward(T, H, dtype, residual, w32):
    g = rng(T + H)
    x, w = randn(g, (T, H), dtype), (1 + randn(g, (H,), scale=0.2)).to(torch.float32 if w32 else dtype)
    res = randn(g, (T, H), dtype, 3.0) if residual else None
    r = norm.rms_norm(x, w, 1e-5, res)
    h, rstd, y = forward_ref(x, res, w, 1e-5)
    assert torch.equal(r.h, h) and (residual or r.h.data_ptr() == x.data_ptr())
    check(r.rstd, rstd, forward_error(H) * rstd, "rstd")
    check(r.y, y, (forward_error(H) + 1.01 * U[dtype]) * y.abs() + STEP[dtype], "y")


@pytest.mark.parametrize("H", [64, 4096, 4097])
def test_column_blocks_and_alignment(H):
    """x and the residual as column blocks: 16-byte aligned, and one element off."""
    g = rng(H)
    w = randn(g, (H,), torch.bfloat16)
    for first in (8, 1):
        x, res = (randn(g, (20, H + 24), torch.bfloat16)[:, first:first + H] for _ in range(2))
        r = norm.rms_norm(x, w, residual=res)
        h, rstd, y = forward_ref(x, res, w, 1e-6)
        assert torch.equal(r.h, h)
        check(r.y, y, (forward_error(H) + 1.01 * U[x.dtype]) * y.abs(), "y")
        dy, dh = (randn(g, (20, H + 24), torch.bfloat16)[:, first:first + H] for _ in range(2))
        dx, dw = norm.rms_norm_backward(dy, r.h, w, r.rstd, dh)
        cx, cw = norm.rms_norm_backward(dy.contiguous(), r.h, w, r.rstd, dh.contiguous())
        backward_check(dx, dw, dy, r.h, w, r.rstd, dh)
        if first == 8:
            assert torch.equal(dx, cx) and torch.equal(dw, cw)


def test_special_values():
    x = randn(rng(1), (6, 512))
    x[0] = 0
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    x[3] *= 1e-30                                 # squares below the smallest float: eps alone counts
    x[4] = 1e18                                   # large, squares still finite
    w = torch.ones(512, device="cuda")
    r = norm.rms_norm(x, w, 1e-6)
    assert not bool(r.y[0].any()) and float(r.rstd[0]) == pytest.approx(1000.0, rel=1e-6)
    assert bool(torch.isnan(r.y[1]).all())
    assert float(r.rstd[2]) == 0 and bool(torch.isnan(r.y[2, 7])) and int(torch.isnan(r.y[2]).sum()) == 1
    check(r.y[3], x[3].double() * 1000.0, 1e-6 * x[3].abs().double() * 1000, "tiny")  # (1e-6 as a float is off by 2^-25 or so)
    check(r.y[4], torch.ones_like(r.y[4]), 64 * F, "large")
    assert bool(torch.isfinite(r.y[5]).all())
    zero = norm.rms_norm(x[:1], w, 0.0)           # 1 / 0, and zero times that
    assert float(zero.rstd[0]) == float("inf") and bool(torch.isnan(zero.y).all())


def test_sums_past_the_largest_float():
    """Rows of large elements beside others, several teams in a block and rows that are read twice: no row's squares spill
    over into another's."""
    for T, H in ((50, 64), (40, 512), (310, 2048), (3, 40000)):
        x, w = randn(rng(H), (T, H)), torch.ones(H, device="cuda")
        x[::3] *= 1e25
        r = norm.rms_norm(x, w, 1e-6)
        _, rstd, y = forward_ref(x, None, w, 1e-6)
        check(r.rstd, rstd, forward_error(H) * rstd, "rstd")
        check(r.y, y, (forward_error(H) + 1.01 * F) * y.abs(), "y")
        dy = randn(rng(H + 1), (T, H))
        dx, dw = norm.rms_norm_backward(dy, r.h, w, r.rstd)
        backward_check(dx, dw, dy, r.h, w, r.rstd, None)


def backward_check(dx, dw, dy, h, w, rstd, dh):
    T, H = dy.shape
    g, xh = dy.double() * w.double(), h.double() * rstd.double()[:, None]
    rs = rstd.double()[:, None]
    dot, mag = (g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    add = 0 if dh is None else dh.double()
    ref = rs * (g - xh * dot) + add
    d = 48 + H / 512  # additions behind one another in the row's sum
    err = F * rs * (8 * (g.abs() + (xh * dot).abs()) + (d + 8) * xh.abs() * mag) + 2 * F * abs(add)
    check(dx, ref, err + 1.01 * U[dy.dtype] * ref.abs() + STEP[dy.dtype], "dx")
    # a thread's rows, the teams of a block, every 16th of at most 304 parts, the 16 sums
    terms = dy.double() * xh
    check(dw, terms.sum(0), (T / 300 + 64 + 8) * F * terms.abs().sum(0) + 1e-300, "dweight")


@pytest.mark.parametrize("T,H", SHAPES + [(1500, 128), (2000, 1401), (3001, 96)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("more,w32", [(False, True), (True, False)])
def test_backward(T, H, dtype, more, w32):
    g = rng(2 * T + H)
    x, w = randn(g, (T, H), dtype), (1 + randn(g, (H,), scale=0.2)).to(torch.float32 if w32 else dtype)
    r = norm.rms_norm(x, w)
    dy, dh = randn(g, (T, H), dtype), randn(g, (T, H), dtype) if more else None
    dx, dw = norm.rms_norm_backward(dy, r.h, w, r.rstd, dh)
    assert dx.dtype == dtype and dw.dtype == torch.float32
    backward_check(dx, dw, dy, r.h, w, r.rstd, dh)
    again = norm.rms_norm_backward(dy, r.h, w, r.rstd, dh)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_backward_is_the_slope():
    """Differences of the formula in 64 bits along random directions."""
    g = rng(11)
    T, H, step = 7, 384, 1e-5
    x, w, dy = randn(g, (T, H)), 1 + randn(g, (H,), scale=0.2), randn(g, (T, H))
    r = norm.rms_norm(x, w)
    dx, dw = norm.rms_norm_backward(dy, r.h, w, r.rstd)

    def f(x, w):
        return (forward_ref(x.double(), None, w, 1e-6)[2] * dy.double()).sum()

    for seed in range(3):
        v, u = randn(rng(seed), (T, H)).double(), randn(rng(50 + seed), (H,)).double()
        # (the difference is off by its third derivative's share, of the order of step^2, and by 2^-53 / step)
        by_x = (f(x.double() + step * v, w) - f(x.double() - step * v, w)) / (2 * step)
        by_w = (f(x, w.double() + step * u) - f(x, w.double() - step * u)) / (2 * step)
        size = dx.double().norm() * v.norm() + dw.double().norm() * u.norm()
        assert abs((dx.double() * v).sum() - by_x) < 1e-6 * size
        assert abs((dw.double() * u).sum() - by_w) < 1e-6 * size


@pytest.mark.parametrize("T,H", [(1, 32), (5, 160), (40, 4096), (310, 1056), (3, 16416), (2, 40000), (0, 64)])
@pytest.mark.parametrize("codes", ["e4m3", "mxfp4"])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_of_floats(T, H, codes, residual):
    """With float rows the unrounded y can be had: its codes and scales, bit for bit."""
    g = rng(T + H)
    x, w = randn(g, (T, H)), 1 + randn(g, (H,), scale=0.2)
    x[:, :32] *= 1e-3
    res = randn(g, (T, H)) if residual else None
    q, s, h = norm.rms_norm_quantized(x, w, codes, residual=res)
    r = norm.rms_norm(x, w, residual=res)
    wq, ws = (fp8 if codes == "e4m3" else fp4).quantize_rows(r.y)
    assert q.dtype == wq.dtype and s.dtype == ws.dtype and torch.equal(h, r.h)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s.view(torch.uint8), ws.view(torch.uint8))


@pytest.mark.parametrize("T,H", [(1, 32), (5, 160), (40, 4096), (310, 1056), (64, 7168), (3, 40000)])
@pytest.mark.parametrize("dtype", TYPES[1:])
def test_codes_of_halves(T, H, dtype):
    """16-bit rows: what the codes stand for is off by at most half a step, beside the float's own error."""
    g = rng(T + H + 1)
    x, res, w = randn(g, (T, H), dtype), randn(g, (T, H), dtype), (1 + randn(g, (H,), scale=0.2)).to(dtype)
    h, rstd, y = forward_ref(x, res, w, 1e-6)
    err = forward_error(H) * y.abs()
    q, s, got = norm.rms_norm_quantized(x, w, "e4m3", residual=res)
    assert torch.equal(got, h)
    kb = -(-H // 128)
    pad = torch.zeros((T, kb * 128), dtype=torch.float64, device="cuda")
    pad[:, :H] = y
    scale = (pad.view(T, kb, 128).abs().amax(2) / 448).clamp(min=2.0 ** -126)
    check(s.t(), scale, (forward_error(H) + 2 * F) * scale, "e4m3 scales")
    unit = s.double().t().repeat_interleave(128, 1)[:, :H]
    a = y.abs() / unit
    half = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))) / 16
    # (the quotient's two roundings; a value next to a power of two may be rounded with the step above it)
    check(q.double() * unit, y, (half * 1.001 + 4 * F * a) * unit + 2 * err, "e4m3")
    q, s, _ = norm.rms_norm_quantized(x, w, "mxfp4", residual=res)
    byte = s.view(torch.uint8).permute(1, 0, 2).flatten(1)[:, :H // 32].double()
    most = y.view(T, H // 32, 32).abs().amax(2) / torch.exp2(byte - 127)
    assert bool((most < 7 * (1 + forward_error(H))).all()) and bool((most >= 3.5 * (1 - forward_error(H))).all())
    unit = torch.exp2(byte - 127).repeat_interleave(32, 1)
    a = y.abs() / unit
    half = torch.where(a < 2 * 1.001, 0.25, torch.where(a < 4 * 1.001, 0.5, 1.0))
    half = torch.where(a > 1.999, torch.where(a > 3.999, 1.0, 0.5), half)
    check(row_values(q, s), y, half * unit + 2 * err, "mxfp4")


def test_streams():
    g = rng(5)
    x, w = randn(g, (64, 4096), torch.bfloat16), randn(g, (4096,), torch.bfloat16)
    want = norm.rms_norm(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = norm.rms_norm(x, w, stream=s)
    back = norm.rms_norm_backward(x, got.h, w, got.rstd, stream=s)
    codes = norm.rms_norm_quantized(x, w, "e4m3", stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(want.y, got.y) and torch.equal(want.rstd, got.rstd)
    for a, b in zip(back, norm.rms_norm_backward(x, want.h, w, want.rstd)):
        assert torch.equal(a, b)
    assert torch.equal(codes[0].view(torch.uint8), norm.rms_norm_quantized(x, w, "e4m3")[0].view(torch.uint8))


def test_captured_and_replayed():
    g = rng(6)
    x, res, w, dy = (randn(g, s, torch.bfloat16) for s in ((300, 2048), (300, 2048), (2048,), (300, 2048)))

    def step():
        r = norm.rms_norm(x, w, residual=res)
        return (*r, *norm.rms_norm_backward(dy, r.h, w, r.rstd, dh=dy))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(2):
        x.copy_(randn(rng(seed), x.shape, x.dtype))
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_refusals():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    rstd = torch.ones(4, device="cuda")
    for bad in (dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(w=w[:32]), dict(w=w.half()), dict(w=w.cpu()),
                dict(res=x[:2]), dict(res=x.float()), dict(x=x.cpu())):
        with pytest.raises((TypeError, ValueError)):
            norm.rms_norm(bad.get("x", x), bad.get("w", w), residual=bad.get("res"))
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(B_.AgGemmError):
            norm.rms_norm(x, w, eps)
    with pytest.raises(TypeError):
        norm.rms_norm(x, w, "small")
    for bad in (dict(dy=x.float()), dict(h=x[:3]), dict(rstd=rstd[:3]), dict(rstd=rstd.double()), dict(dh=x.float()), dict(dh=x[:, :32])):
        with pytest.raises((TypeError, ValueError)):
            norm.rms_norm_backward(bad.get("dy", x), bad.get("h", x), w, bad.get("rstd", rstd), bad.get("dh"))
    with pytest.raises(ValueError):
        norm.rms_norm_quantized(x, w, "e5m2")
    with pytest.raises(B_.AgGemmError):
        norm.rms_norm_quantized(x[:, :24].contiguous(), w[:24].contiguous(), "e4m3")
    with pytest.raises(B_.AgGemmError):
        norm.rms_norm_quantized(x[:, :48].contiguous(), w[:48].contiguous(), "mxfp4")
    with pytest.raises(B_.AgGemmError):
        norm.rms_norm_quantized(torch.zeros((4, 72), dtype=torch.bfloat16, device="cuda")[:, 4:68], w, "e4m3")
