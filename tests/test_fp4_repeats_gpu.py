"""4-bit products over and over: the same bits and no wait that runs out, beside work that delays their warps."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import fp4  # noqa: E402
from layer_util import row_values, weight_values  # noqa: E402
from moe_util import STEP, U, check, randn, rng  # noqa: E402


# long row tiles of one and of many experts, of few and of many stages, and short ones in shares
@pytest.mark.parametrize("rows,E,K,N,times", [(8192, 32, 4096, 2048, 400), (4000, 7, 1184, 3000, 400), (2500, 1, 8192, 4096, 400),
                                              (3000, 16, 480, 5000, 400), (64, 1, 8192, 4096, 1500), (64, 32, 1024, 2048, 1500)])
def test_repeats(rows, E, K, N, times):
    g = rng(rows + K)
    sizes = torch.bincount(torch.randint(0, E, (rows,), generator=g, device="cuda"), minlength=E)
    off = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).int()
    x = randn(g, (rows, K), torch.bfloat16)
    wq, ws = fp4.quantize_weights(randn(g, (E, K, N), torch.bfloat16, K ** -0.5))
    with fp4.Fp4Linear(K, N, n_experts=E) as p:
        xq, xs = fp4.quantize_rows(x)
        first = p.forward(xq, xs, wq, ws, off)
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")
        side = torch.cuda.Stream()
        other = torch.zeros(1 << 26, device="cuda")
        for i in range(times):
            if i % 4 == 0:
                with torch.cuda.stream(side):
                    other.add_(1.0)  # memory traffic beside the products
            y = p.forward(xq, xs, wq, ws, off)
            wrong += (y != first).any()
        torch.cuda.synchronize()
        assert p.status() == 0 and int(wrong) == 0
    xd, at = row_values(xq, xs), 0
    for e, n in enumerate(sizes.tolist()):  # the first rows of each expert: what the repeats repeat is right
        n_ref = min(n, 3)
        a, b = xd[at:at + n_ref], weight_values(wq[e:e + 1], ws[e:e + 1])[0].t()
        ref, mag = a @ b, a.abs() @ b.abs()
        check(first[at:at + n_ref], ref, (K + 8) * 2.0 ** -23 * mag + 1.01 * U[torch.bfloat16] * ref.abs() + STEP[torch.bfloat16],
              f"expert {e}")
        at += n
