"""Every function of include/ag_layer.h through the binding's wrappers, with raw pointers, against
the torch front end's results."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import act, fp4, moe, norm  # noqa: E402
from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from moe_util import randn, rng  # noqa: E402


def like(*ts):
    out = [torch.empty_like(t) for t in ts]
    for t in out:
        t.view(torch.uint8).fill_(77)
    return out


def p(t):
    return t.data_ptr()


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.fixture
def s():
    return torch.cuda.current_stream().cuda_stream


def test_norm(s):
    g = rng(1)
    T, H, bf = 37, 256, torch.bfloat16
    x, res, dy, dh = (randn(g, (T, H), bf) for _ in range(4))
    w = randn(g, (H,))
    n = norm.rms_norm(x, w, 1e-5, res)
    y, h, rstd = like(*n)
    B_.ag_norm_rms(T, H, B_.BF16, p(x), H, p(res), H, p(w), B_.F32, 1e-5, p(y), p(h), p(rstd), s)
    assert same(y, n.y) and same(h, n.h) and same(rstd, n.rstd)
    B_.ag_norm_rms(T, H, B_.BF16, p(x), H, None, 0, p(w), B_.F32, 1e-5, p(y), None, None, s)
    assert same(y, norm.rms_norm(x, w, 1e-5).y)
    want = norm.rms_norm_backward(dy, n.h, w, n.rstd, dh)
    dx, dw = like(*want)
    ws = torch.empty(B_.ag_norm_rms_backward_workspace(T, H), dtype=torch.uint8, device="cuda")
    B_.ag_norm_rms_backward(T, H, B_.BF16, p(dy), H, p(n.h), H, p(w), B_.F32, p(n.rstd), p(dh), H, p(dx), p(dw), p(ws), s)
    assert same(dx, want[0]) and same(dw, want[1])
    B_.ag_norm_rms_backward(0, H, B_.BF16, None, H, None, H, None, B_.F32, None, None, H, None, p(dw), None, s)
    assert not bool(dw.any())
    for name, code in (("e4m3", B_.E4M3), ("mxfp4", B_.E2M1)):
        want = norm.rms_norm_quantized(x, w, name, 1e-5, res)
        q, sc, h = like(*want)
        B_.ag_norm_rms_quantized(T, H, B_.BF16, p(x), H, p(res), H, p(w), B_.F32, 1e-5, code, p(q), p(sc), p(h), s)
        assert same(q, want[0]) and same(sc, want[1]) and same(h, want[2])


def test_activation(s):
    g = rng(2)
    T, N, f16 = 21, 96, torch.float16
    x, dy = randn(g, (T, 2 * N), f16), randn(g, (T, N), f16)
    want = act.swiglu(x)
    y, = like(want)
    B_.ag_act_swiglu(T, N, B_.F16, p(x), 2 * N, p(y), s)
    assert same(y, want)
    want = act.swiglu_backward(dy, x)
    dx, = like(want)
    B_.ag_act_swiglu_backward(T, N, B_.F16, p(dy), N, p(x), 2 * N, p(dx), s)
    assert same(dx, want)
    for name, code in (("e4m3", B_.E4M3), ("mxfp4", B_.E2M1)):
        want = act.swiglu_quantized(x, name)
        q, sc = like(*want)
        B_.ag_act_swiglu_quantized(T, N, B_.F16, p(x), 2 * N, code, p(q), p(sc), s)
        assert same(q, want[0]) and same(sc, want[1])


def test_4_bit(s):
    g = rng(3)
    T, E, k, K, N, bf = 37, 5, 2, 160, 48, torch.bfloat16
    x, w, r = randn(g, (T, K), bf), randn(g, (E, K, N), bf), moe.route(randn(g, (T, E)), k)
    (xq, xs), (wq, ws) = fp4.quantize_rows(x, r), fp4.quantize_weights(w)
    q, sc = like(xq, xs)
    B_.ag_fp4_quantize_rows(T * k, K, B_.BF16, p(x), K, T, p(r.order), k, p(q), p(sc), s)
    assert same(q, xq) and same(sc, xs)
    q, sc = like(wq, ws)
    B_.ag_fp4_quantize_weights(E, K, N, B_.BF16, p(w), p(q), p(sc), s)
    assert same(q, wq) and same(sc, ws)
    h = B_.ag_moe_plan_create(E, K, N, B_.E2M1)
    try:
        assert B_.ag_moe_plan_tile_rows(h, 30, 0) == 64 and B_.ag_moe_plan_tile_rows(h, 1 << 20, 0) == 224
        with pytest.raises(B_.AgGemmError):
            B_.ag_moe_plan_tile_rows(h, 30, 1)  # no input gradient
        with fp4.Fp4Linear(K, N, n_experts=E) as plan:
            want = plan.forward(xq, xs, wq, ws, r.offsets)
        y, = like(want)
        B_.ag_fp4_forward(h, T * k, p(xq), p(xs), p(r.offsets), p(wq), p(ws), p(y), N, B_.BF16, s)
        assert same(y, want) and B_.ag_moe_plan_status(h) == B_.OK
        for bad in (dict(xq=p(xq) + 8), dict(xs=p(xs) + 4), dict(wq=p(wq) + 4), dict(ws=p(ws) + 8), dict(xs=None), dict(ws=None),
                    dict(ld=N + 4), dict(ld=N - 8), dict(t=B_.E4M3), dict(off=None), dict(rows=-1)):
            a = dict(rows=T * k, xq=p(xq), xs=p(xs), off=p(r.offsets), wq=p(wq), ws=p(ws), ld=N, t=B_.BF16)
            a.update(bad)
            with pytest.raises(B_.AgGemmError) as e:
                B_.ag_fp4_forward(h, a["rows"], a["xq"], a["xs"], a["off"], a["wq"], a["ws"], p(y), a["ld"], a["t"], s)
            assert e.value.code == B_.ERR_INVALID, bad
        # a plan of one type takes no other's product
        with pytest.raises(B_.AgGemmError):
            B_.ag_fp8_forward(h, T * k, p(xq), p(xs), p(r.offsets), p(wq), p(ws), p(y), N, B_.BF16, s)
        with pytest.raises(B_.AgGemmError):
            B_.ag_moe_forward(h, T * k, p(x), K, p(r.offsets), p(w), N, K * N, p(y), N, B_.BF16, s)
    finally:
        B_.ag_moe_plan_destroy(h)
    with moe.Experts(E, K, N) as plan, pytest.raises(B_.AgGemmError):
        B_.ag_fp4_forward(plan.handle, T * k, p(xq), p(xs), p(r.offsets), p(wq), p(ws), p(y), N, B_.BF16, s)
