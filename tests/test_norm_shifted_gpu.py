"""Gradients of rows that begin anywhere but alike in all operands, by raw pointers: every operand and dx off an aligned
address by the same elements, pitched rows with values that are not finite between them, several rows a block."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from moe_util import randn, rng  # noqa: E402
from test_norm_gpu import backward_check  # noqa: E402

DTYPE = {torch.float16: B_.F16, torch.bfloat16: B_.BF16, torch.float32: B_.F32}


def rows_at(g, T, H, dtype, first, pitch):
    """(T, H) rows `pitch` apart, the first `first` elements behind an aligned address; all else NaN."""
    flat = torch.full((first + T * pitch + 64,), float("nan"), dtype=dtype, device="cuda")
    rows = flat[first:first + T * pitch].view(T, pitch)[:, :H]
    rows.copy_(randn(g, (T, H), dtype))
    return rows


@pytest.mark.parametrize("T,H", [(700, 1001), (3000, 130), (609, 9), (3, 4101), (640, 4099), (3000, 2050), (300, 16377)])
@pytest.mark.parametrize("more", [0, 1, 3])  # 16-byte pieces between rows
@pytest.mark.parametrize("off", [0, 1, -1])
@pytest.mark.parametrize("dtype", DTYPE)
def test_alike(T, H, more, off, dtype):
    V = 16 // torch.empty(0, dtype=dtype).element_size()
    if dtype == torch.float32 and H > 8188:
        H = 8189
    first, pitch = off % V, H + V * more
    g = rng(T + H + first)
    dy, h, dh = (rows_at(g, T, H, dtype, first, p) for p in (pitch, pitch + V, H))
    w, rstd = randn(g, (H,), dtype), torch.rand(T, generator=g, device="cuda") + 0.5
    out = torch.full((first + T * H + 64,), -7.0, dtype=dtype, device="cuda")
    dw = torch.empty(H, device="cuda")
    ws = torch.empty(B_.ag_norm_rms_backward_workspace(T, H), dtype=torch.uint8, device="cuda")
    for gh in (dh, None):
        B_.ag_norm_rms_backward(T, H, DTYPE[dtype], dy.data_ptr(), dy.stride(0), h.data_ptr(), h.stride(0), w.data_ptr(), DTYPE[dtype],
                                rstd.data_ptr(), None if gh is None else gh.data_ptr(), H, out[first:].data_ptr(), dw.data_ptr(),
                                ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        backward_check(out[first:first + T * H].view(T, H), dw, dy, h, w, rstd, gh)
        assert bool((out[:first] == -7).all()) and bool((out[first + T * H:] == -7).all())
