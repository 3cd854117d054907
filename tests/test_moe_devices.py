"""Tensors of one call on different devices, or on another than the plan's, are refused
before anything is allocated or launched.  (The tensors are torch's fake ones: they have a
device and a shape, and no memory, so that no second GPU is needed.)"""
from unittest import mock

import pytest

torch = pytest.importorskip("torch")
FakeTensorMode = pytest.importorskip("torch._subclasses.fake_tensor").FakeTensorMode

from all_gather_gemm_chunked_gb300 import build as _build  # noqa: E402

T, K, H, E, N = 4, 2, 32, 8, 64


@pytest.fixture(scope="module")
def M():
    _build.build()
    from all_gather_gemm_chunked_gb300 import fp8, moe
    return moe, fp8


def _fake(*specs):
    """Tensors of (shape, type) on cuda:0, and a function that moves one of them."""
    def make(shape, dtype, index):
        # (left in, it would allocate on the device)
        with mock.patch("torch._subclasses.fake_tensor.init_gpu_context", lambda *a: None, create=True), FakeTensorMode():
            return torch.empty(shape, dtype=dtype, device="cuda:%d" % index)

    def on(other):
        return [make(s, d, 1 if i == other else 0) for i, (s, d) in enumerate(specs)]
    return on


F32, I32, BF16 = torch.float32, torch.int32, torch.bfloat16
ROUTE = [((T, K), F32), ((T, K), I32), ((E + 1,), I32), ((T * K,), I32), ((T, K), I32)]


def _calls(moe, fp8):
    def routing(t):
        return moe.Routing(*t, True)

    return {
        "route_backward": ([((T, E), F32), ((T, K), F32)] + ROUTE, [1, 2, 3],
                           lambda z, dw, *r: moe.route_backward(z, routing(r), dw)),
        "gather": ([((T, H), BF16)] + ROUTE, [4, 5], lambda x, *r: moe.gather(x, routing(r))),
        "combine": ([((T * K, H), BF16), ((T, K), I32), ((T, K), F32)], [1, 2], moe.combine),
        "combine_backward": ([((T, H), BF16), ((T * K, H), BF16), ((T, K), I32), ((T, K), F32), ((E + 1,), I32)],
                             [0, 1, 2, 3, 4], moe.combine_backward),
        "quantize_rows": ([((T, H), BF16)] + ROUTE, [4, 5], lambda x, *r: fp8.quantize_rows(x, routing(r))),
    }


@pytest.mark.parametrize("name", ["route_backward", "gather", "combine", "combine_backward", "quantize_rows"])
def test_tensors_on_two_devices_are_refused(M, name):
    specs, others, call = _calls(*M)[name]
    on = _fake(*specs)
    for other in others:
        with pytest.raises(ValueError, match="device"):
            call(*on(other))


@pytest.mark.gpu
def test_products_on_two_devices_are_refused(M):
    moe, fp8 = M
    rows = T * K
    x, dy, off, w, out = ((rows, H), BF16), ((rows, N), BF16), ((E + 1,), I32), ((E, H, N), BF16), ((rows, N), BF16)
    dx, dw = ((rows, H), BF16), ((E, H, N), F32)
    with moe.Experts(E, H, N) as p:
        for specs, call in (((x, off, w, out), p.forward), ((dy, off, w, dx), p.backward_input),
                            ((x, dy, off, dw), p.backward_weight)):
            on = _fake(*specs)
            for other in range(4):
                with pytest.raises(ValueError, match="device"):
                    call(*on(other))
            with pytest.raises(ValueError, match="device"):  # all on one, the plan on another
                call(*[_fake(s)(0)[0] for s in specs])
    e4 = torch.float8_e4m3fn
    specs = (((rows, H), e4), ((1, rows), F32), ((E, N, H), e4), ((E, 1, 1), F32), off, out)
    with fp8.Fp8Linear(H, N, n_experts=E) as p:
        on = _fake(*specs)
        for other in range(6):
            with pytest.raises(ValueError, match="device"):
                p.forward(*on(other))
        with pytest.raises(ValueError, match="device"):
            p.forward(*[_fake(s)(0)[0] for s in specs])


@pytest.mark.gpu
def test_a_stream_of_another_device_is_refused(M):
    z = _fake(((T, E), F32))(0)[0]
    with pytest.raises(ValueError, match="device"):
        M[0].route(z, K, stream=torch.cuda.Stream())


@pytest.mark.gpu
def test_a_call_leaves_the_current_device():
    from all_gather_gemm_chunked_gb300 import moe
    r = moe.route(torch.randn((5, E), device="cuda"), K)
    assert r.weights.device == torch.device("cuda", torch.cuda.current_device())


def test_plan_device_of_no_plan(M):
    from all_gather_gemm_chunked_gb300 import binding as B_
    assert B_.library_handle().ag_moe_plan_device(None) == B_.ERR_INVALID
