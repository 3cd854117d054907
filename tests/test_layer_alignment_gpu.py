"""What outputs as codes ask of their inputs' alignment, and that the plain outputs ask nothing."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import act, fp4, norm  # noqa: E402
from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from moe_util import U, check, randn, rng  # noqa: E402
from test_norm_gpu import forward_error  # noqa: E402

T, H = 5, 64


@pytest.mark.parametrize("codes", ["e4m3", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", ["x", "residual", "weight"])
def test_norm(codes, dtype, which):
    g = rng(1)
    a = {"x": randn(g, (T, H), dtype), "residual": randn(g, (T, H), dtype), "weight": randn(g, (H,), dtype)}
    want, whole = norm.rms_norm(**a), norm.rms_norm_quantized(codes=codes, **a)
    off = torch.empty(a[which].numel() + 1, dtype=dtype, device="cuda")[1:].view(a[which].shape)
    off.copy_(a[which])
    got = norm.rms_norm(**{**a, which: off})
    assert torch.equal(got.h, want.h)
    # (the sums' order may be another: both are within this of the value in 64 bits)
    check(got.y, want.y, 2.01 * (forward_error(H) + 1.01 * U[dtype]) * want.y.double().abs(), "y")
    with pytest.raises(B_.AgGemmError, match="16-byte aligned") as e:
        norm.rms_norm_quantized(codes=codes, **{**a, which: off})
    assert e.value.code == B_.ERR_INVALID
    again = norm.rms_norm_quantized(codes=codes, **a)  # (an aligned call behind the refusal)
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(whole, again))


@pytest.mark.parametrize("codes", ["e4m3", "mxfp4"])
def test_gated_and_rows(codes):
    x = randn(rng(2), (T, 2 * H + 4), torch.float16)
    assert torch.equal(act.swiglu(x[:, 4:]), act.swiglu(x[:, 4:].contiguous()))
    for bad in (x[:, 4:], x[:, : 2 * H]):  # a base and a pitch of 8 bytes
        with pytest.raises(B_.AgGemmError, match="16"):
            act.swiglu_quantized(bad, codes)
        with pytest.raises(B_.AgGemmError, match="16"):
            fp4.quantize_rows(bad)
    with pytest.raises(B_.AgGemmError, match="16-byte aligned"):
        fp4.quantize_weights(torch.zeros(H * 8 + 1, dtype=torch.float16, device="cuda")[1:].view(H, 8))
