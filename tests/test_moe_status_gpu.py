"""A plan's status and the runs around a bad one."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp8, moe  # noqa: E402
from moe_util import check, offsets_of, product_bound, randn, rng  # noqa: E402


@pytest.mark.parametrize("rows,K,N", [(700, 16384, 2048), (40, 8192, 256)])
def test_runs_after_bad_offsets_are_whole(rows, K, N):
    """Bad offsets concern their own run: later ones, whose waits last longer than 20 us
    (the epilogue's for a sum of 256 k-blocks), give what they give otherwise."""
    g = rng(K)
    x, w = randn(g, (rows, K), torch.bfloat16), randn(g, (2, K, N), torch.bfloat16, K ** -0.5)
    good, bad = offsets_of([rows - 9, 9]), torch.tensor([0, rows + 1, rows], dtype=torch.int32, device="cuda")
    with moe.Experts(2, K, N) as p:
        want = p.forward(x, good, w)
        assert p.status() == B_.OK
        out = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device="cuda")
        p.forward(x, bad, w, out=out)
        got = [p.forward(x, good, w) for _ in range(4)]
        assert p.status() == B_.ERR_INVALID and p.status_word() & 0xFF == 16
        assert bool((out == 3).all()) and all(torch.equal(y, want) for y in got)
        assert p.status() == B_.ERR_INVALID  # until the reset
        p.reset()
        assert torch.equal(p.forward(x, good, w), want) and p.status() == B_.OK
    a, b = x[:200].double(), w[0].double()
    n = min(200, rows - 9)
    check(want[:n], (a @ b)[:n], product_bound(a, b, K, torch.bfloat16)[:n])


def test_e4m3_runs_after_bad_offsets_are_whole():
    g = rng(4)
    rows, K, N = 700, 8192, 2048
    x, w = randn(g, (rows, K), torch.bfloat16), randn(g, (2, K, N), torch.bfloat16)
    q, wq = fp8.quantize_rows(x), fp8.quantize_weights(w)
    good, bad = offsets_of([300, 400]), torch.tensor([0, 5, rows + 1], dtype=torch.int32, device="cuda")
    with fp8.Fp8Linear(K, N, n_experts=2) as p:
        want = p.forward(*q, *wq, good)
        p.forward(*q, *wq, bad)
        got = [p.forward(*q, *wq, good) for _ in range(4)]
        assert p.status() == B_.ERR_INVALID and all(torch.equal(y, want) for y in got)
