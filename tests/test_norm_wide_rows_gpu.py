"""Gradients of the norm at widths around the widest that a team of threads holds: aligned rows, rows that begin
anywhere alike in all operands, and narrower accesses."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import norm  # noqa: E402
from moe_util import randn, rng  # noqa: E402
from test_norm_gpu import backward_check  # noqa: E402


@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("dtype,H", [(t, H) for t in (torch.bfloat16, torch.float16) for H in (8185, 8187, 16375, 16376, 16377, 16378,
                                     16379, 16380, 16382, 16383, 16384, 16385, 16386, 16388, 16392)] +
                                    [(torch.float32, H) for H in (4093, 8188, 8189, 8190, 8191, 8192, 8193, 8194, 8196)])
def test_widths(rows, dtype, H):
    g = rng(rows + H)
    dy, h, dh = (randn(g, (rows, H), dtype) for _ in range(3))
    w, rstd = randn(g, (H,), torch.float32 if H % 3 else dtype), torch.rand(rows, generator=g, device="cuda") + 0.5
    dx, dw = norm.rms_norm_backward(dy, h, w, rstd, dh)
    backward_check(dx, dw, dy, h, w, rstd, dh)
    dx, dw = norm.rms_norm_backward(dy, h, w, rstd)
    backward_check(dx, dw, dy, h, w, rstd, None)
