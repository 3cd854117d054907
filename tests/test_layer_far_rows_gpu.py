"""A layer's operators on matrices of more than 2^31 elements, one at a time, each with the memory that it needs itself."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import act, fp4, norm  # noqa: E402
from moe_util import rng  # noqa: E402

T, H, FEW = 262_400, 8192, 1001  # 2^31 elements and 2 097 152 more; as many rows at each end are compared
GB = 1 << 30


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def first_norm(x, w):
    return norm.rms_norm(x, w, residual=x)


def gradient(x, w):
    return norm.rms_norm_backward(x, x, w, norm.rms_norm(x, w).rstd, dh=x)[:1]


# outputs with rows in dimension 0 or 1; GB beside x's 4.0: the outputs, and copies of what is compared
CALLS = {
    "norm": (first_norm, (0, 0, 0), 8.1),
    "norm to e4m3": (lambda x, w: norm.rms_norm_quantized(x, w, "e4m3")[:2], (0, 1), 2.2),
    "norm to 4 bits": (lambda x, w: norm.rms_norm_quantized(x, w, "mxfp4")[:2], (0, 1), 1.2),
    "gradient": (gradient, (0,), 8.2),
    "gated": (lambda x, w: (act.swiglu(x),), (0,), 2.1),
    "gated to 4 bits": (lambda x, w: act.swiglu_quantized(x, "mxfp4"), (0, 1), 0.7),
    "gated gradient": (lambda x, w: (act.swiglu_backward(x[:, : H // 2], x),), (0,), 4.1),
    "rows to 4 bits": (lambda x, w: fp4.quantize_rows(x), (0, 1), 1.2),
}


@pytest.mark.parametrize("name", CALLS)
def test_ends(name):
    """The first and last rows give what they give alone."""
    call, dims, gb = CALLS[name]
    torch.cuda.empty_cache()
    need = int((4.0 + gb + 1.0) * GB)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need / GB:.1f} GB of free device memory")
    g = rng(2)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    x[FEW:T - FEW] = 1.5
    for rows in (slice(0, FEW), slice(T - FEW, T)):
        x[rows] = torch.randn((FEW, H), generator=g, device="cuda").bfloat16()
    w = torch.randn(H, generator=g, device="cuda").bfloat16()
    whole = call(x, w)
    for rows in (slice(0, FEW), slice(T - FEW, T)):
        for dim, a, b in zip(dims, whole, call(x[rows], w)):
            assert same(a[:, rows] if dim else a[rows], b), name
    del x, whole, a, b
    torch.cuda.empty_cache()
