"""Norms of rows and eps at the ends of the range of floats, against the definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import fp4, norm  # noqa: E402
from moe_util import STEP, U, check, randn, rng  # noqa: E402
from test_norm_gpu import forward_error, forward_ref  # noqa: E402

MAX = float(torch.finfo(torch.float32).max)


def held(eps):
    """eps as the float that the norm takes."""
    return float(torch.tensor(eps, dtype=torch.float32))


# teams of a warp and of several, frames, rows that are read twice
SHAPES = [(7, 1), (50, 64), (40, 517), (310, 2048), (700, 1001), (3, 40000)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("scale,eps", [(1e18, 1e36), (1e20, MAX), (1e22, 1e38), (1.0, MAX), (3e18, MAX), (1e30, 1e-6)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_eps(T, H, scale, eps, dtype):
    """eps beside mean squares that pass the largest float, or with which it does."""
    g = rng(T + H)
    x, w = randn(g, (T, H), dtype), (1 + randn(g, (H,), scale=0.2)).to(dtype)
    x[::3] *= scale  # (rows of ordinary size beside them)
    r = norm.rms_norm(x, w, eps)
    _, rstd, y = forward_ref(x, None, w, held(eps))
    check(r.rstd, rstd, forward_error(H) * rstd, "rstd")
    check(r.y, y, (forward_error(H) + 1.01 * U[dtype]) * y.abs() + STEP[dtype], "y")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("scale", [1e-16, 1e-19, 1e-22, 1e-25, 1e-37])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_rows(T, H, scale, eps, dtype):
    """Rows whose squares are below the smallest float, beside rows of ordinary size, with no eps or a small one."""
    g = rng(T + H + 1)
    x, w = randn(g, (T, H), dtype), (1 + randn(g, (H,), scale=0.2)).to(dtype)
    x[x == 0] = 1.0
    x[::3] *= scale
    x[1::3, : H // 2] *= scale  # (whole warps of small elements in an ordinary row)
    r = norm.rms_norm(x, w, eps)
    _, rstd, y = forward_ref(x, None, w, held(eps))
    check(r.rstd, rstd, forward_error(H) * rstd, "rstd")
    check(r.y, y, (forward_error(H) + 1.01 * U[dtype]) * y.abs() + STEP[dtype], "y")


@pytest.mark.parametrize("T,H", [(40, 512), (310, 2048), (3, 40000)])
def test_small_rows_to_codes(T, H):
    """Of floats, with the residual's addition: the codes of the unrounded y, bit for bit."""
    g = rng(T)
    x, res, w = randn(g, (T, H), scale=1e-24), randn(g, (T, H), scale=1e-24), randn(g, (H,))
    r = norm.rms_norm(x, w, 0.0, res)
    assert torch.equal(r.h, x + res) and bool(torch.isfinite(r.y).all())
    q, s, h = norm.rms_norm_quantized(x, w, "mxfp4", 0.0, res)
    wq, ws = fp4.quantize_rows(r.y)
    assert torch.equal(h, r.h) and torch.equal(q, wq) and torch.equal(s.view(torch.uint8), ws.view(torch.uint8))


def test_zeros_and_not_finite_values_without_eps():
    """Zeros stay 0 / 0; an infinity or NaN stays in its row, beside small ones."""
    x = randn(rng(4), (700, 256), scale=1e-24)
    x[0], x[1, 3], x[2, 4] = 0, float("inf"), float("nan")
    x[5, 1:] = 0
    w = torch.ones(256, device="cuda")
    r = norm.rms_norm(x, w, 0.0)
    assert float(r.rstd[0]) == float("inf") and bool(r.y[0].isnan().all())
    assert float(r.rstd[1]) == 0 and bool(r.y[1, 3].isnan()) and int(r.y[1].isnan().sum()) == 1
    assert bool(r.y[2].isnan().all())
    _, rstd, y = forward_ref(x[3:], None, w, 0.0)
    check(r.rstd[3:], rstd, forward_error(256) * rstd, "rstd")
    check(r.y[3:], y, (forward_error(256) + 1.01 * U[x.dtype]) * y.abs(), "y")


@pytest.mark.parametrize("T,H", [(4000, 64), (900, 2048), (700, 16384), (64, 32768)])
def test_rstd_is_rounded_once(T, H):
    """Whole numbers whose squares' sum is a float in any order, and a mean that is one: rstd is the nearest float or, within
    2^-10 of a tie, its neighbour."""
    x = torch.randint(-16, 17, (T, H), generator=rng(H), device="cuda").float()  # sums of H squares: below 2^8 H <= 2^23
    x[:, 0] = torch.randint(1, 17, (T,), generator=rng(T), device="cuda").float()
    w = torch.ones(H, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        got = norm.rms_norm(x.to(dtype), w.to(dtype), 0.0).rstd.double()
        want = 1 / torch.sqrt((x.double() ** 2).sum(1) / H)
        step = torch.exp2(torch.floor(torch.log2(want)) - 23)
        assert float(((got - want).abs() / step).max()) <= 0.5 + 2.0 ** -10
