"""Sums of very many terms in 16-bit outputs: the error stays near the output's rounding."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import moe  # noqa: E402
from moe_util import STEP, U, check, rng  # noqa: E402

# An accumulator takes at most 128 k-blocks of four additions, each off by at most 2^-23 of
# the running sum (all terms are positive here); the sums of up to 1024 accumulators are
# added in 32 bits, to nearest.
SUM = (512 + 1024 / 2) * 2.0 ** -23


def _positive(g, shape, scale, dtype):
    return (torch.rand(shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype,name", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
@pytest.mark.parametrize("rows,K,N", [(1 << 22, 256, 128), (500_000, 1664, 1536)])
def test_weight_gradient(rows, K, N, dtype, name):
    g = rng(1)
    x, dy = _positive(g, (rows, K), 2.0 ** -6, dtype), _positive(g, (rows, N), 2.0 ** -5, dtype)
    ref = torch.zeros((K, N), dtype=torch.float64, device="cuda")
    for a in range(0, rows, 1 << 17):
        ref += x[a:a + (1 << 17)].double().t() @ dy[a:a + (1 << 17)].double()
    with moe.Experts(1, K, N, name) as p:
        dw = p.backward_weight(x, dy, None, out_dtype=dtype)
        assert p.status() == B_.OK
    check(dw[0], ref, (SUM + 1.01 * U[dtype]) * ref + STEP[dtype])


@pytest.mark.parametrize("K,rows", [(1 << 22, 48), (1 << 20, 700)])
def test_forward(K, rows):
    g = rng(2)
    N, dt = 256, torch.float16
    x, w = _positive(g, (rows, K), 2.0 ** -6, dt), _positive(g, (1, K, N), 2.0 ** -6, dt)
    ref = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    for a in range(0, K, 1 << 16):
        ref += x[:, a:a + (1 << 16)].double() @ w[0, a:a + (1 << 16)].double()
    with moe.Experts(1, K, N, "f16") as p:
        y = p.forward(x, None, w)
        assert p.status() == B_.OK
    check(y, ref, (SUM + 1.01 * U[dt]) * ref + STEP[dt])
