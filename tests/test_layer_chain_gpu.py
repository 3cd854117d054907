"""A layer's operators launched one behind the other: each may start while the one before it is
still writing its inputs (a product may ask for its weights even earlier), and has to wait for them."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import act, fp4, fp8, moe, norm  # noqa: E402
from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from moe_util import randn, rng  # noqa: E402


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T,E,k,K,N", [(24, 6, 2, 256, 320), (1500, 12, 4, 512, 256), (300, 8, 3, 544, 1120)])
def test_calls_in_a_row_give_what_separate_calls_give(T, E, k, K, N):
    g = rng(T + K)
    bf = torch.bfloat16
    w_up, w_down = randn(g, (E, K, 2 * N), bf, K ** -0.5), randn(g, (E, N, K), bf, N ** -0.5)
    wn, dout, dh = randn(g, (K,), bf), randn(g, (T, K), bf), randn(g, (T, K), bf)
    inputs = [(randn(g, (T, K), bf, 2.0 ** i), randn(g, (T, K), bf), randn(g, (T, E), bf)) for i in range(4)]

    def step(x, res, logits, plans, between):
        up, down, up4, down4, dense = plans
        out = []

        def keep(*ts):
            out.extend(ts)
            between()
            return ts if len(ts) > 1 else ts[0]

        y, h, rstd = keep(*norm.rms_norm(x, wn, residual=res))
        r = moe.route(logits, k)
        keep(*r[:5])
        rows = keep(moe.gather(y, r))
        gu = keep(up.forward(rows, r.offsets, w_up))
        a = keep(act.swiglu(gu))
        z = keep(down.forward(a, r.offsets, w_down))
        dz, _ = keep(*moe.combine_backward(dout, z, r.slots, r.weights, r.offsets))
        da = keep(down.backward_input(dz, r.offsets, w_down))
        dgu = keep(act.swiglu_backward(da, gu))
        dx = keep(moe.combine(keep(up.backward_input(dgu, r.offsets, w_up)), r.slots))
        keep(*norm.rms_norm_backward(dx, h, wn, rstd, dh))
        # weights that are made right before their product
        uq = keep(*fp4.quantize_weights(w_up * (1 + x[0, 0].abs())))
        dq = keep(*fp4.quantize_weights(w_down * (1 + x[0, 1].abs())))
        g4 = keep(up4.forward(*keep(*fp4.quantize_rows(y, r)), *uq, r.offsets))
        z4 = keep(down4.forward(*keep(*act.swiglu_quantized(g4, "mxfp4")), *dq, r.offsets))
        xq, xs, h2 = keep(*norm.rms_norm_quantized(keep(moe.combine(z4, r.slots, r.weights)), wn, "mxfp4", residual=h))
        wq, ws = keep(*fp4.quantize_weights(w_up[0] * (1 + x[0, 2].abs())))
        keep(dense.forward(xq, xs, wq, ws))
        keep(*norm.rms_norm_quantized(h2, wn, "e4m3"))
        keep(*act.swiglu_quantized(gu, "e4m3"))
        return out

    with moe.Experts(E, K, 2 * N) as a, moe.Experts(E, N, K) as b, fp4.Fp4Linear(K, 2 * N, E) as c, fp4.Fp4Linear(N, K, E) as d, \
            fp4.Fp4Linear(K, 2 * N) as e:
        plans = (a, b, c, d, e)
        want = [step(*i, plans, torch.cuda.synchronize) for i in inputs]
        for _ in range(8):
            got = [step(*i, plans, lambda: None) for i in inputs]
            torch.cuda.synchronize()
            for s, t in zip(want, got):
                for n, (p, q) in enumerate(zip(s, t)):
                    assert same(p, q), n
            del got
        assert all(p.status() == B_.OK for p in plans)


@pytest.mark.parametrize("rows,K,N", [(1, 4096, 1024), (64, 8192, 2560), (20, 1120, 24320)])
def test_weights_written_right_before_their_product(rows, K, N):
    """One expert and few rows: the kernel asks for its first weights before it waits."""
    g = rng(rows)
    x = randn(g, (rows, K), torch.bfloat16)
    xq, xs = fp4.quantize_rows(x)
    forms = [fp4.quantize_weights(randn(g, (K, N), torch.bfloat16)) for _ in range(3)]
    wq, ws = torch.empty_like(forms[0][0]), torch.empty_like(forms[0][1])
    with fp4.Fp4Linear(K, N) as p:
        want = [p.forward(xq, xs, *f) for f in forms]
        torch.cuda.synchronize()
        got = []
        for i in range(30):
            wq.copy_(forms[i % 3][0])
            ws.view(torch.uint8).copy_(forms[i % 3][1].view(torch.uint8))
            got.append(p.forward(xq, xs, wq, ws))
        assert p.status() == B_.OK
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3])


def test_products_on_streams_and_in_graphs():
    """A plan whose sums are cut between pairs, on two streams, captured, and replayed."""
    g = rng(4)
    K, N, bf = 8192, 1024, torch.bfloat16
    xs = [fp4.quantize_rows(randn(g, (48, K), bf)) for _ in range(2)]
    w = fp4.quantize_weights(randn(g, (K, N), bf))
    streams = [torch.cuda.Stream() for _ in range(2)]
    with fp4.Fp4Linear(K, N) as p:
        want = [p.forward(*x, *w) for x in xs]
        torch.cuda.synchronize()
        got = [p.forward(*xs[i % 2], *w, stream=streams[i % 2]) for i in range(20)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # two branches that share the plan's workspace
            fork = torch.cuda.current_stream()
            side = torch.cuda.Stream()
            side.wait_stream(fork)
            a = p.forward(*xs[0], *w)
            b = p.forward(*xs[1], *w, stream=side)
            fork.wait_stream(side)
        for _ in range(5):
            a.zero_()
            b.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        assert p.status() == B_.OK


def test_norm_and_product_in_8_bits():
    """The codes a norm makes are what the product of quantised rows reads."""
    g = rng(9)
    T, H, N, bf = 70, 1040, 264, torch.bfloat16
    x, w = randn(g, (T, H)), randn(g, (H,))
    wq, ws = fp8.quantize_weights(randn(g, (H, N), bf))
    with fp8.Fp8Linear(H, N) as p:
        q, s, _ = norm.rms_norm_quantized(x, w, "e4m3")
        assert torch.equal(p.forward(q, s, wq, ws), p.forward(*fp8.quantize_rows(norm.rms_norm(x, w).y), wq, ws))
