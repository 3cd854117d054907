"""Products at the documented limit of rows."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp8, moe  # noqa: E402
from moe_util import rng  # noqa: E402

LIMIT = 2 ** 31 - 256


def test_rows_beyond_the_limit_are_refused():
    lib = B_.library_handle()
    a = torch.zeros(64, dtype=torch.float16, device="cuda").data_ptr()
    with moe.Experts(1, 8, 8, "f16") as p, fp8.Fp8Linear(16, 8) as q:
        for rows in (LIMIT + 1, 2 ** 31 - 1, 2 ** 31, -1):
            assert lib.ag_moe_forward(p.handle, rows, a, 8, None, a, 8, 64, a, 8, 0, None) == B_.ERR_INVALID
            assert lib.ag_moe_backward_input(p.handle, rows, a, 8, None, a, 8, 64, a, 8, 0, None) == B_.ERR_INVALID
            assert lib.ag_moe_backward_weight(p.handle, rows, a, 8, a, 8, None, a, 0, None) == B_.ERR_INVALID
            assert lib.ag_fp8_forward(q.handle, rows, a, a, None, a, a, a, 8, 0, None) == B_.ERR_INVALID


@pytest.mark.skipif(torch.cuda.mem_get_info()[0] < 150 << 30, reason="needs 110 GB of free device memory")
@pytest.mark.parametrize("rows", [2_140_000_000, LIMIT])
def test_one_group_of_very_many_rows(rows):
    """Small whole numbers: every sum is exact."""
    P, K, N = (1 << 22) + 5, 8, 8  # the rows repeat after P
    g = rng(1)

    def ints(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").half()

    base, w = ints(P, K), ints(1, K, N)
    x = torch.empty((rows, K), dtype=torch.float16, device="cuda")
    for a in range(0, rows, P):
        x[a:a + P] = base[:rows - a]
    dy = torch.zeros((rows, N), dtype=torch.float16, device="cuda")
    ends = torch.tensor([0, 1, P, rows // 2, 2_139_127_000, rows - 300, rows - 2, rows - 1], device="cuda")
    dy[ends] = ints(len(ends), N)
    want = (base.double() @ w[0].double()).half()
    with moe.Experts(1, K, N, "f16") as p:
        y = p.forward(x, None, w)
        dw = p.backward_weight(x, dy, None)
        assert p.status() == B_.OK
    assert all(torch.equal(y[a:a + P], want[:rows - a]) for a in range(0, rows, P))
    assert torch.equal(dw[0].double(), x[ends].double().t() @ dy[ends].double())
    del x, y, dy
    torch.cuda.empty_cache()
