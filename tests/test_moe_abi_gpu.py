"""Every function of include/ag_moe.h through the binding's wrappers, with raw pointers,
against the torch front end's results."""
import pytest

torch = pytest.importorskip("torch")

from all_gather_gemm_chunked_gb300 import build as _build  # noqa: E402


def test_binding_has_every_header_function():
    _build.build()
    from all_gather_gemm_chunked_gb300 import binding as B_
    for name in B_.header_functions(B_.HEADER_MOE):
        assert callable(getattr(B_, name)), name


gpu = pytest.mark.gpu


@pytest.fixture
def layer():
    """T tokens, their routing, rows, weights and gradients of a small layer."""
    from all_gather_gemm_chunked_gb300 import moe
    from moe_util import randn, rng
    g = rng(3)
    T, E, k, K, N = 37, 5, 2, 64, 48
    logits = randn(g, (T, E))
    r = moe.route(logits, k)
    return dict(T=T, E=E, k=k, K=K, N=N, logits=logits, r=r, x=randn(g, (T, K), torch.bfloat16),
                w=randn(g, (E, K, N), torch.bfloat16), dout=randn(g, (T, N), torch.bfloat16), stream=torch.cuda.current_stream().cuda_stream)


def _like(*ts):
    return [torch.full_like(t, 77) if t.dtype != torch.float8_e4m3fn else torch.zeros_like(t) for t in ts]


def _p(t):
    return t.data_ptr()


@gpu
def test_router(layer):
    from all_gather_gemm_chunked_gb300 import binding as B_, moe
    T, E, k, z, r, s = (layer[n] for n in ("T", "E", "k", "logits", "r", "stream"))
    assert B_.ag_moe_route_workspace(T, E, k) == 0
    out = _like(*r[:5])
    B_.ag_moe_route(T, E, k, B_.F32, _p(z), E, 1, *map(_p, out), None, s)
    assert all(torch.equal(a, b) for a, b in zip(out, r[:5]))
    big = torch.randn((3000, E), device="cuda")  # two kernels, with a workspace
    ws = torch.empty(B_.ag_moe_route_workspace(3000, E, k), dtype=torch.uint8, device="cuda")
    want = moe.route(big, k)
    out = _like(*want[:5])
    B_.ag_moe_route(3000, E, k, B_.F32, _p(big), E, 1, *map(_p, out), _p(ws), s)
    assert all(torch.equal(a, b) for a, b in zip(out, want[:5]))
    dw = torch.randn((T, k), device="cuda")
    dz = torch.empty_like(z)
    B_.ag_moe_route_backward(T, E, k, B_.F32, _p(z), E, 1, _p(r.weights), _p(r.experts), _p(dw), _p(dz), s)
    assert torch.equal(dz, moe.route_backward(z, r, dw))


@gpu
def test_rows_and_products(layer):
    from all_gather_gemm_chunked_gb300 import binding as B_, moe
    T, E, k, K, N, r, x, w, dout, s = (layer[n] for n in ("T", "E", "k", "K", "N", "r", "x", "w", "dout", "stream"))
    S, bf = T * k, B_.BF16
    rows, = _like(moe.gather(x, r))
    B_.ag_moe_gather(T, k, K, bf, _p(x), K, _p(r.order), _p(rows), s)
    assert torch.equal(rows, moe.gather(x, r))
    h = B_.ag_moe_plan_create(E, K, N, bf)
    try:
        assert B_.ag_moe_plan_device(h) == torch.cuda.current_device() and B_.ag_moe_plan_tile_rows(h, S, 0) == 64
        B_.ag_moe_plan_set_timeout_ns(h, 3_000_000_000)
        with pytest.raises(B_.AgGemmError) as e:
            B_.ag_moe_plan_set_timeout_ns(h, 0)
        assert e.value.code == B_.ERR_INVALID
        with moe.Experts(E, K, N) as p:
            y = p.forward(rows, r.offsets, w)
            got, = _like(y)
            B_.ag_moe_forward(h, S, _p(rows), K, _p(r.offsets), _p(w), N, K * N, _p(got), N, bf, s)
            assert torch.equal(got, y)
            dy, dweights = moe.combine_backward(dout, y, r.slots, r.weights, r.offsets)
            a, b = _like(dy, dweights)
            B_.ag_moe_combine_backward(T, k, N, bf, _p(dout), N, _p(y), N, _p(r.slots), _p(r.weights), _p(r.offsets) + 4 * E,
                                       _p(a), _p(b), s)
            assert torch.equal(a, dy) and torch.equal(b, dweights)
            out, = _like(moe.combine(y, r.slots, r.weights))
            B_.ag_moe_combine(T, k, N, bf, _p(y), N, _p(r.slots), _p(r.weights), _p(out), s)
            assert torch.equal(out, moe.combine(y, r.slots, r.weights))
            dx, dw = p.backward_input(dy, r.offsets, w), p.backward_weight(rows, dy, r.offsets)
            a, b = _like(dx, dw)
            B_.ag_moe_backward_input(h, S, _p(dy), N, _p(r.offsets), _p(w), N, K * N, _p(a), K, bf, s)
            B_.ag_moe_backward_weight(h, S, _p(rows), K, _p(dy), N, _p(r.offsets), _p(b), B_.F32, s)
            assert torch.equal(a, dx) and torch.equal(b, dw)
        assert B_.ag_moe_plan_status(h) == B_.OK and B_.ag_moe_plan_status_word(h) == 0
        B_.ag_moe_plan_reset(h, s)
        assert B_.ag_moe_plan_status(h) == B_.OK
    finally:
        B_.ag_moe_plan_destroy(h)


@gpu
def test_8_bit(layer):
    from all_gather_gemm_chunked_gb300 import binding as B_, fp8
    T, E, k, K, N, r, x, w, s = (layer[n] for n in ("T", "E", "k", "K", "N", "r", "x", "w", "stream"))
    S, bf = T * k, B_.BF16
    (xq, xs), (wq, ws) = fp8.quantize_rows(x, r), fp8.quantize_weights(w)
    q, sc = _like(xq, xs)
    B_.ag_fp8_quantize_rows(S, K, bf, _p(x), K, T, _p(r.order), k, _p(q), _p(sc), s)
    assert torch.equal(q.view(torch.uint8), xq.view(torch.uint8)) and torch.equal(sc, xs)
    q, sc = _like(wq, ws)
    B_.ag_fp8_quantize_weights(E, K, N, bf, _p(w), _p(q), _p(sc), s)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(sc, ws)
    with fp8.Fp8Linear(K, N, n_experts=E) as p:
        y = p.forward(xq, xs, wq, ws, r.offsets)
        got, = _like(y)
        B_.ag_fp8_forward(p.handle, S, _p(xq), _p(xs), _p(r.offsets), _p(wq), _p(ws), _p(got), N, bf, s)
        assert torch.equal(got, y) and p.status() == B_.OK
