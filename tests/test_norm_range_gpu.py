"""Norms of rows and eps at the ends of the range of floats, against the definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import norm  # noqa: E402
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
