"""Scales whose product leaves the floats' normal range."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import fp8  # noqa: E402
from moe_util import STEP, U, check, rng  # noqa: E402

# rows and N of short row tiles and of long ones (rows on the MMA's M side)
SHAPES = [(40, 64), (600, 2056)]


def _operands(rows, K, N, seed):
    g = rng(seed)
    q = torch.randn((rows, K), generator=g, device="cuda").mul(50).to(fp8.E4M3)
    w = torch.randn((N, K), generator=g, device="cuda").mul(50).to(fp8.E4M3)
    return q, torch.ones((-(-K // 128), rows), device="cuda"), w, torch.ones((-(-N // 128), -(-K // 128)), device="cuda")


def _exact(q, xs, w, ws):
    K, N = q.shape[1], w.shape[0]
    a = q.double() * xs.double().t().repeat_interleave(128, 1)[:, :K]
    b = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return a @ b.t(), a.abs() @ b.abs().t()


@pytest.mark.parametrize("rows,N", SHAPES)
def test_a_block_of_zeros_stays_zero_under_large_scales(rows, N):
    K = 384
    q, xs, w, ws = _operands(rows, K, N, 1)
    z = q.view(torch.uint8)
    z[:, 128:256] = 0
    xs[1], ws[:, 1] = 1e30, 1e30  # their product is no float
    with fp8.Fp8Linear(K, N) as p:
        y = p.forward(q, xs, w, ws, out_dtype=torch.float32)
    ref, mag = _exact(q, xs, w, ws)
    check(y, ref, (K + 8) * 2.0 ** -23 * mag + 1.01 * U[torch.float32] * ref.abs() + STEP[torch.float32])


@pytest.mark.parametrize("rows,N", SHAPES)
def test_small_scales(rows, N):
    """A product of scales below 2^-126 is off by at most 2^-150, a block's sum is at most
    448 * 448 * 128 < 2^24.7: 2^-125 a block beside the usual roundings."""
    K = 384
    q, xs, w, ws = _operands(rows, K, N, 2)
    xs[0], ws[:, 0] = 1e-30, 1e-12
    xs[1:], ws[:, 1:] = 1e-19, 1e-19
    with fp8.Fp8Linear(K, N) as p:
        y = p.forward(q, xs, w, ws, out_dtype=torch.float32)
    ref, mag = _exact(q, xs, w, ws)
    check(y, ref, (K + 8) * 2.0 ** -23 * mag + 3 * 2.0 ** -125 + 1.01 * U[torch.float32] * ref.abs() + STEP[torch.float32])


@pytest.mark.parametrize("rows,N", SHAPES)
def test_infinite_and_nan_scales_are_kept(rows, N):
    K = 256
    q, xs, w, ws = _operands(rows, K, N, 3)
    xs[0, 3], xs[1, 5] = float("inf"), float("nan")
    with fp8.Fp8Linear(K, N) as p:
        y = p.forward(q, xs, w, ws, out_dtype=torch.float32)
    assert not bool(torch.isfinite(y[3]).any()) and bool(torch.isnan(y[5]).all())
    keep = [i for i in range(rows) if i not in (3, 5)]
    assert bool(torch.isfinite(y[keep]).all())
