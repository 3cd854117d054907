"""Operators launched one behind the other: each may start while the one before it is still
writing its inputs, and has to wait for them."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp8, moe  # noqa: E402
from moe_util import randn, rng  # noqa: E402


@pytest.mark.parametrize("T,E,k,K,N", [(24, 6, 2, 256, 320), (1500, 12, 4, 512, 264), (300, 8, 3, 520, 1104)])
def test_calls_in_a_row_give_what_separate_calls_give(T, E, k, K, N):
    g = rng(T + K)
    w, dout = randn(g, (E, K, N), torch.bfloat16, K ** -0.5), randn(g, (T, N), torch.bfloat16)
    inputs = [(randn(g, (T, K), torch.bfloat16, 2.0 ** i), randn(g, (T, E), torch.bfloat16)) for i in range(4)]
    low = K % 16 == 0

    def step(x, logits, p, q, between):
        out = []

        def keep(*ts):
            out.extend(ts)
            between()
            return ts if len(ts) > 1 else ts[0]

        r = moe.route(logits, k)
        keep(*r[:5])
        rows = keep(moe.gather(x, r))
        y = keep(p.forward(rows, r.offsets, w))
        keep(moe.combine(y, r.slots, r.weights))
        dy, dweights = keep(*moe.combine_backward(dout, y, r.slots, r.weights, r.offsets))
        keep(moe.route_backward(logits, r, dweights))
        dx = keep(p.backward_input(dy, r.offsets, w))
        keep(p.backward_weight(rows, dy, r.offsets))
        keep(moe.combine(dx, r.slots))
        if low:
            wq, ws = fp8.quantize_weights(w * (1 + x[0, 0].abs()))
            between()
            xq, xs = fp8.quantize_rows(x, r)
            between()
            keep(moe.combine(keep(q.forward(xq, xs, wq, ws, r.offsets)), r.slots, r.weights))
        return out

    with moe.Experts(E, K, N) as p, fp8.Fp8Linear(K if low else 16, N, n_experts=E) as q:
        want = [step(x, z, p, q, torch.cuda.synchronize) for x, z in inputs]
        for _ in range(10):
            got = [step(x, z, p, q, lambda: None) for x, z in inputs]
            torch.cuda.synchronize()
            for a, b in zip(want, got):
                for s, t in zip(a, b):
                    assert torch.equal(s, t)
            del got
        assert p.status() == B_.OK and q.status() == B_.OK
