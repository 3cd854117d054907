"""e4m3 operands with block scales, and their product, against the definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp8, moe  # noqa: E402
from moe_util import STEP, U, check, offsets_of, quantize_ref, randn, rng  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _pad(x, rows, cols):
    out = torch.zeros(x.shape[:-2] + (rows, cols), dtype=x.dtype, device=x.device)
    out[..., :x.shape[-2], :x.shape[-1]] = x
    return out


def _rows_ref(x):
    """(codes as values, scales (KB, rows))"""
    n, K = x.shape
    kb = -(-K // 128)
    q, s = quantize_ref(_pad(x, n, kb * 128).view(n, kb, 128), (2,))
    return q.reshape(n, -1)[:, :K], s[:, :, 0].t()


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 128), (8, 144), (77, 1104), (64, 4096), (9, 5008), (130, 256)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_rows(rows, K, dtype):
    x = randn(rng(rows + K), (rows, K), dtype)
    if rows > 2:
        x[1] = 0
        x[2] *= 1e-4 if dtype == torch.float16 else 1e-39  # subnormals
    q, s = fp8.quantize_rows(x)
    rq, rs = _rows_ref(x)
    assert torch.equal(s, rs)
    assert torch.equal(q.double(), rq)


def test_quantize_rows_not_finite():
    x = randn(rng(1), (4, 256))
    x[0, 3], x[1, 130], x[2, 0] = float("inf"), float("nan"), float("-inf")
    q, s = fp8.quantize_rows(x)
    v = q.float()
    assert bool(torch.isnan(v[0, 3])) and bool(torch.isnan(v[1, 130])) and bool(torch.isnan(v[2, 0]))
    assert float(s[0, 0]) == float("inf") and bool(torch.isfinite(s[1]).all())
    assert int(torch.isnan(v).sum()) == 3 and bool(torch.isfinite(v[3]).all())


@pytest.mark.parametrize("T,k,K", [(5, 2, 32), (40, 4, 1040)])
def test_quantize_gathers_the_experts_rows(T, k, K):
    g = rng(2)
    logits = randn(g, (T, 8)).masked_fill(torch.rand((T, 8), generator=g, device="cuda") < 0.6, float("-inf"))
    r = moe.route(logits, k)
    wide = randn(g, (T, K + 8), torch.bfloat16)
    x = wide[:, 8:]
    q, s = fp8.quantize_rows(x, r)
    gq, gs = fp8.quantize_rows(moe.gather(x, r))
    assert torch.equal(q.view(torch.uint8), gq.view(torch.uint8)) and torch.equal(s, gs)


def _weights_ref(w):
    E, K, N = w.shape
    kb, nb = -(-K // 128), -(-N // 128)
    t = _pad(w.transpose(1, 2), nb * 128, kb * 128).view(E, nb, 128, kb, 128)
    q, s = quantize_ref(t, (2, 4))
    return q.reshape(E, nb * 128, kb * 128)[:, :N, :K], s[:, :, 0, :, 0]


@pytest.mark.parametrize("E,K,N", [(1, 16, 8), (2, 128, 128), (3, 272, 200), (1, 1024, 264)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_weights(E, K, N, dtype):
    w = randn(rng(E + K + N), (E, K, N), dtype)
    w[0, :8] *= 300 if dtype == torch.float16 else 1e6
    q, s = fp8.quantize_weights(w)
    rq, rs = _weights_ref(w)
    assert torch.equal(s, rs) and torch.equal(q.double(), rq)
    q2, s2 = fp8.quantize_weights(w[0])
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])


SHAPES = [
    ([1], 16, 8),
    ([0, 1, 0], 128, 40),
    ([3, 0, 17, 31, 32, 33, 0], 256, 256),
    ([64, 65, 63], 400, 264),
    ([300, 1, 255, 256, 257], 528, 520),
    ([7], 4096, 512),
    ([60, 0, 30], 2064, 1024),
    ([700], 640, 136),
    ([16] * 33, 144, 328),
]


@pytest.mark.parametrize("sizes,K,N", SHAPES)
@pytest.mark.parametrize("out_dtype", TYPES)
def test_product(sizes, K, N, out_dtype):
    g = rng(K + N)
    rows, E = sum(sizes), len(sizes)
    x, w, off = randn(g, (rows, K), torch.bfloat16), randn(g, (E, K, N), torch.bfloat16, K ** -0.5), offsets_of(sizes)
    x[: rows // 2] *= 30  # scales that differ between rows and blocks
    w[:, : K // 2] *= 0.01
    (xq, xs), (wq, ws) = fp8.quantize_rows(x), fp8.quantize_weights(w)
    with fp8.Fp8Linear(K, N, n_experts=E) as p:
        y = p.forward(xq, xs, wq, ws, off, out_dtype=out_dtype)
        assert p.status() == B_.OK
    xd = xq.double() * xs.double().t().repeat_interleave(128, 1)[:, :K]
    wd = wq.double() * ws.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    at = 0
    for e, n in enumerate(sizes):
        a, b = xd[at:at + n], wd[e].t()
        ref, mag = a @ b, a.abs() @ b.abs()
        # a block's sum in the tensor core, its scale, the sum over blocks, the rounding
        check(y[at:at + n], ref, (K + 8) * 2.0 ** -23 * mag + 1.01 * U[out_dtype] * ref.abs() + STEP[out_dtype], f"expert {e}")
        at += n


def test_whole_numbers_are_exact():
    """Codes that are small whole numbers and scales that are powers of two: every sum is exact."""
    g = rng(5)
    K, N, rows = 1024, 384, 200
    q = torch.randint(-8, 9, (rows, K), generator=g, device="cuda").float()
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float()
    xs = 2.0 ** torch.randint(-3, 4, (K // 128, rows), generator=g, device="cuda").float()
    ws = 2.0 ** torch.randint(-3, 4, (N // 128, K // 128), generator=g, device="cuda").float()
    with fp8.Fp8Linear(K, N) as p:
        y = p.forward(q.to(fp8.E4M3), xs, w.to(fp8.E4M3), ws, out_dtype=torch.float32)
    a = q.double() * xs.double().t().repeat_interleave(128, 1)
    b = w.double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    assert torch.equal(y.double(), a @ b.t())


def test_rows_of_nan_stay_alone():
    g = rng(6)
    sizes, K, N = [10, 20, 5], 256, 128
    x, w, off = randn(g, (35, K), torch.bfloat16), randn(g, (3, K, N), torch.bfloat16), offsets_of(sizes)
    (xq, xs), (wq, ws) = fp8.quantize_rows(x), fp8.quantize_weights(w)
    x[10:30] = float("nan")
    bq, bs = fp8.quantize_rows(x)
    with fp8.Fp8Linear(K, N, n_experts=3) as p:
        want, got = p.forward(xq, xs, wq, ws, off), p.forward(bq, bs, wq, ws, off)
    assert torch.equal(want[:10], got[:10]) and torch.equal(want[30:], got[30:])
    assert bool(torch.isnan(got[10:30]).all())


def test_runs_repeat_bit_for_bit():
    g = rng(7)
    x, w = randn(g, (64, 8192), torch.bfloat16), randn(g, (8192, 512), torch.bfloat16)
    (xq, xs), (wq, ws) = fp8.quantize_rows(x), fp8.quantize_weights(w)
    with fp8.Fp8Linear(8192, 512) as p:
        first = p.forward(xq, xs, wq, ws).clone()
        for _ in range(5):
            assert torch.equal(first, p.forward(xq, xs, wq, ws))


def test_no_rows_and_refusals():
    K, N = 256, 64
    w = torch.zeros((K, N), dtype=torch.float16, device="cuda")
    wq, ws = fp8.quantize_weights(w)
    x = torch.zeros((8, K), dtype=torch.float16, device="cuda")
    xq, xs = fp8.quantize_rows(x)
    e = fp8.quantize_rows(x[:0])
    with fp8.Fp8Linear(K, N) as p:
        assert p.forward(*e, wq, ws).shape == (0, N)
        assert not bool(p.forward(xq, xs, wq, ws).any())
        for bad in ((x, xs, wq, ws), (xq, xs.t(), wq, ws), (xq, xs, wq.t(), ws), (xq, xs, wq, ws[:, :1]), (xq[:, :128], xs, wq, ws)):
            with pytest.raises((TypeError, ValueError)):
                p.forward(*bad)
        with pytest.raises(B_.AgGemmError):
            p.forward(xq, xs, wq, ws, out_dtype=torch.float64)
        with pytest.raises(ValueError):
            p.forward(xq, xs, wq, ws, offsets_of([4, 4]).repeat(2))
    with pytest.raises(B_.AgGemmError):
        fp8.quantize_rows(x[:, :40])            # K % 16
    with pytest.raises(B_.AgGemmError):
        fp8.quantize_rows(torch.zeros((4, 72), dtype=torch.float16, device="cuda")[:, 4:68])  # 8-byte aligned
    with pytest.raises(ValueError):
        fp8.quantize_weights(w.t())
    with pytest.raises(B_.AgGemmError):
        fp8.Fp8Linear(200, 64)                  # K % 16
    with pytest.raises(B_.AgGemmError):
        fp8.quantize_weights(torch.zeros((256, 12), device="cuda"))  # N % 8
