"""Tensors of one call on different devices, or on another than the plan's, are refused before
anything is allocated or launched.  (The tensors are torch's fake ones: they have a device and a
shape, and no memory, so that no second GPU is needed.)"""
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("torch._subclasses.fake_tensor")

from all_gather_gemm_chunked_gb300 import build as _build  # noqa: E402
from test_moe_devices import _fake  # noqa: E402

T, H, N, E = 4, 64, 32, 3
F32, BF16, U8, E8 = torch.float32, torch.bfloat16, torch.uint8, torch.float8_e8m0fnu
ROW, HALF, W = ((T, H), BF16), ((T, H // 2), BF16), ((H,), BF16)


@pytest.fixture(scope="module")
def M():
    _build.build()
    from all_gather_gemm_chunked_gb300 import act, fp4, norm
    return norm, act, fp4


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_quantized", "rms_norm_backward", "swiglu_backward"])
def test_tensors_on_two_devices_are_refused(M, name):
    norm, act, _ = M
    specs, call = {
        "rms_norm": ([ROW, W, ROW], lambda x, w, r: norm.rms_norm(x, w, residual=r)),
        "rms_norm_quantized": ([ROW, W, ROW], lambda x, w, r: norm.rms_norm_quantized(x, w, "e4m3", residual=r)),
        "rms_norm_backward": ([ROW, ROW, W, ((T,), F32), ROW], norm.rms_norm_backward),
        "swiglu_backward": ([HALF, ROW], act.swiglu_backward),
    }[name]
    on = _fake(*specs)
    for other in range(len(specs)):
        with pytest.raises(ValueError, match="device"):
            call(*on(other))


@pytest.mark.gpu
def test_4_bit_products_on_two_devices_are_refused(M):
    fp4 = M[2]
    specs = (((T, H // 2), U8), ((1, T, 4), E8), ((E, N, H // 2), U8), ((E, 1, 1, 32, 4, 4), E8), ((E + 1,), torch.int32), ((T, N), BF16))
    with fp4.Fp4Linear(H, N, n_experts=E) as p:
        on = _fake(*specs)
        for other in range(6):
            with pytest.raises(ValueError, match="device"):
                p.forward(*on(other))
        with pytest.raises(ValueError, match="device"):  # all on one, the plan on another
            p.forward(*[_fake(s)(0)[0] for s in specs])


@pytest.mark.gpu
def test_a_stream_of_another_device_is_refused(M):
    x, w = _fake(ROW, W)(0)[0], torch.ones(H, dtype=BF16, device="cuda")
    for call in (lambda s: M[0].rms_norm(x, w, stream=s), lambda s: M[1].swiglu(x, stream=s), lambda s: M[2].quantize_rows(x, stream=s)):
        with pytest.raises(ValueError, match="device"):
            call(torch.cuda.Stream())
