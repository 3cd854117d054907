"""A layer's operators at the documented limit of rows, and on matrices of more than 2^32 bytes and 2^31 elements."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import act, fp4, norm  # noqa: E402
from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from layer_util import code_values  # noqa: E402
from moe_util import rng  # noqa: E402

LIMIT = 2 ** 31 - 256
large = pytest.mark.skipif(torch.cuda.mem_get_info()[0] < 150 << 30, reason="needs 110 GB of free device memory")


def test_4_bit_rows_beyond_the_limit_are_refused():
    lib = B_.library_handle()
    a = torch.zeros(64, device="cuda").data_ptr()
    with fp4.Fp4Linear(32, 8) as p:
        for rows in (LIMIT + 1, 2 ** 31 - 1, 2 ** 31, -1):
            assert lib.ag_fp4_forward(p.handle, rows, a, a, None, a, a, a, 8, 0, None) == B_.ERR_INVALID


@large
def test_one_group_of_very_many_4_bit_rows():
    """Scales of 1 and sums of 32 codes: every sum is exact."""
    rows, P, K, N = LIMIT, (1 << 22) + 5, 32, 8  # the rows repeat after P
    g = rng(1)
    base, w = (torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, generator=g, device="cuda") for n in (P, N))
    x = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    for a in range(0, rows, P):
        x[a:a + P] = base[:rows - a]
    xs = torch.full((1, rows, 4), 127, dtype=torch.uint8, device="cuda").view(fp4.E8M0)
    ws = torch.full((1, 1, 32, 4, 4), 127, dtype=torch.uint8, device="cuda").view(fp4.E8M0)
    want = (code_values(base) @ code_values(w).t()).bfloat16()
    with fp4.Fp4Linear(K, N) as p:
        y = p.forward(x, xs, w, ws)
        assert p.status() == B_.OK
    assert all(torch.equal(y[a:a + P], want[:rows - a]) for a in range(0, rows, P))
    del x, xs, y
    torch.cuda.empty_cache()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@large
def test_rows_beyond_2_to_the_31_elements():
    """The last rows of a large matrix give what they give in one of fewer (but many) rows."""
    T, H, few, bf = 290_001, 8192, 1001, torch.bfloat16
    g = rng(2)
    x = torch.empty((T, H), dtype=bf, device="cuda")
    for a in range(0, T, 50_000):
        x[a:a + 50_000] = torch.randn((min(50_000, T - a), H), generator=g, device="cuda").to(bf)
    w = torch.randn(H, generator=g, device="cuda").to(bf)
    ends = (slice(0, few), slice(T - few, T))
    for call, parts in ((lambda t: norm.rms_norm(t, w, residual=t), (0, 0, 0)), (lambda t: norm.rms_norm_quantized(t, w, "e4m3"), (0, 1)),
                        (lambda t: norm.rms_norm_quantized(t, w, "mxfp4"), (0, 1)), (lambda t: (act.swiglu(t),), (0,)),
                        (lambda t: act.swiglu_quantized(t, "mxfp4"), (0, 1)), (lambda t: (act.swiglu_backward(t[:, :H // 2], t),), (0,)),
                        (fp4.quantize_rows, (0, 1))):
        whole = call(x)
        for rows in ends:
            for part, (a, b) in zip(parts, zip(whole, call(x[rows]))):
                assert same(a[:, rows] if part else a[rows], b)
        del whole, a, b
    r = norm.rms_norm(x, w)
    dx, dw = norm.rms_norm_backward(x, r.h, w, r.rstd, dh=x)
    for rows in ends:
        assert same(dx[rows], norm.rms_norm_backward(x[rows], r.h[rows], w, r.rstd[rows], dh=x[rows])[0])
    # (dx of x itself: sums of many products of one sign, so 32-bit sums are off by little)
    want = torch.zeros(H, dtype=torch.float64, device="cuda")
    for a in range(0, T, 50_000):
        want += (x[a:a + 50_000].double() ** 2 * r.rstd[a:a + 50_000].double()[:, None]).sum(0)
    assert bool(((dw.double() - want).abs() <= (T / 300 + 72) * 2.0 ** -24 * want).all())
    del x, r, dx
    torch.cuda.empty_cache()


@large
def test_very_many_short_rows():
    T = 2 ** 31 - 1
    x = torch.full((T, 1), 2.0, dtype=torch.float16, device="cuda")
    x[-1], x[T // 2] = -3.0, 0.0
    r = norm.rms_norm(x, torch.ones(1, dtype=torch.float16, device="cuda"), 0.25)
    want = torch.tensor([2.0, 0.0, -3.0], dtype=torch.float64)
    got = r.y[[0, T // 2, T - 1], 0].double().cpu()
    assert bool(((got - want / torch.sqrt(want * want + 0.25)).abs() <= 2.0 ** -11).all())
    assert int((r.y == r.y[0]).sum()) == T - 2
    del x, r
    q = torch.full((T // 16, 32), 2.0, dtype=torch.float16, device="cuda")
    assert bool((act.swiglu(q)[-1] == act.swiglu(q[:1])[0]).all())
    torch.cuda.empty_cache()
