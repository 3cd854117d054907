"""Products whose groups take tiles of 256 rows, against 64 bits: ragged last tiles in both
directions, split sums, outputs whose rows start 16 bytes off 32."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp8, moe  # noqa: E402
from moe_util import STEP, U, check, offsets_of, product_bound, randn, rng  # noqa: E402

LONG = 256


def _groups(sizes):
    at = 0
    for e, n in enumerate(sizes):
        yield e, at, at + n
        at += n


# sizes, K, N: whole sums of few k-blocks, split sums of many, wide tiles that end inside
# 32 columns and inside 8
ROWS = [
    ([300, 257, 1, 700], 528, 2056),
    ([1, 0, 255, 900, 64], 208, 3000),
    ([600], 8192, 2056),
    ([600], 4096, 2304),
]


@pytest.mark.parametrize("sizes,K,N", ROWS)
@pytest.mark.parametrize("out_f32", [False, True])
def test_forward_and_input_gradient(sizes, K, N, out_f32):
    dt = torch.bfloat16
    od = torch.float32 if out_f32 else dt
    g = rng(K + N)
    rows, E, off = sum(sizes), len(sizes), offsets_of(sizes)
    x, w = randn(g, (rows, K), dt), randn(g, (E, K, N), dt, K ** -0.5)
    # the gradient's product runs the other way: over K, N columns wide
    v = randn(g, (E, N, K), dt, K ** -0.5)
    with moe.Experts(E, K, N) as p, moe.Experts(E, N, K) as back:
        assert p.tile_rows(rows) == back.tile_rows(rows, input_gradient=True) == LONG
        y, dx = p.forward(x, off, w, out_dtype=od), back.backward_input(x, off, v, out_dtype=od)
        for _ in range(3):
            assert torch.equal(y, p.forward(x, off, w, out_dtype=od))
            assert torch.equal(dx, back.backward_input(x, off, v, out_dtype=od))
        assert p.status() == B_.OK and back.status() == B_.OK
    for e, a, b in _groups(sizes):
        xd = x[a:b].double()
        for got, m in ((y, w[e].double()), (dx, v[e].double().t())):
            check(got[a:b], xd @ m, product_bound(xd, m, K, od), f"expert {e}")


def _scaled(sizes, K, N, seed):
    g = rng(seed)
    rows, E = sum(sizes), len(sizes)
    x, w = randn(g, (rows, K), torch.bfloat16), randn(g, (E, K, N), torch.bfloat16, K ** -0.5)
    x[: rows // 2] *= 30
    w[:, : K // 2] *= 0.01
    (xq, xs), (wq, ws) = fp8.quantize_rows(x), fp8.quantize_weights(w)
    xd = xq.double() * xs.double().t().repeat_interleave(128, 1)[:, :K]
    wd = wq.double() * ws.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return xq, xs, wq, ws, xd, wd


@pytest.mark.parametrize("sizes,K,N", ROWS + [([500, 0, 80], 144, 2600)])
@pytest.mark.parametrize("out_dtype,shift", [(torch.float32, 0), (torch.float16, 0), (torch.bfloat16, 0), (torch.bfloat16, 8)])
def test_e4m3(sizes, K, N, out_dtype, shift):
    xq, xs, wq, ws, xd, wd = _scaled(sizes, K, N, K + N)
    rows, off = sum(sizes), offsets_of(sizes)
    # `shift` elements of 2 bytes: rows 16 bytes off a multiple of 32
    wide = torch.full((rows, N + 2 * shift + (-N % 16 if shift else 0)), 7.0, dtype=out_dtype, device="cuda")
    out = wide[:, shift:shift + N]
    with fp8.Fp8Linear(K, N, n_experts=len(sizes)) as p:
        assert p.tile_rows(rows) == LONG
        y = p.forward(xq, xs, wq, ws, off, out=out, out_dtype=out_dtype).clone()
        for _ in range(3):
            assert torch.equal(y, p.forward(xq, xs, wq, ws, off, out_dtype=out_dtype))
        assert p.status() == B_.OK
    assert bool((wide[:, :shift] == 7).all()) and bool((wide[:, shift + N:] == 7).all())
    for e, a, b in _groups(sizes):
        m = wd[e].t()
        ref, mag = xd[a:b] @ m, xd[a:b].abs() @ m.abs()
        check(y[a:b], ref, (K + 8) * 2.0 ** -23 * mag + 1.01 * U[out_dtype] * ref.abs() + STEP[out_dtype], f"expert {e}")


def test_groups_next_to_nan_rows():
    """A tile of 256 rows of one group covers rows of NaN of the next."""
    sizes, K, N = [300, 290, 270], 256, 2048
    xq, xs, wq, ws, xd, wd = _scaled(sizes, K, N, 9)
    xs[:, 300:590] = float("nan")
    g = rng(10)
    x, w = randn(g, (860, K), torch.bfloat16), randn(g, (3, K, N), torch.bfloat16, K ** -0.5)
    x[300:590] = float("nan")
    off = offsets_of(sizes)
    with fp8.Fp8Linear(K, N, n_experts=3) as low, moe.Experts(3, K, N) as p:
        assert low.tile_rows(860) == p.tile_rows(860) == LONG
        y, z = low.forward(xq, xs, wq, ws, off, out_dtype=torch.float32), p.forward(x, off, w)
    assert bool(torch.isnan(y[300:590]).all()) and bool(torch.isnan(z[300:590]).all())
    for e, a, b in ((0, 0, 300), (2, 590, 860)):
        m = wd[e].t()
        ref, mag = xd[a:b] @ m, xd[a:b].abs() @ m.abs()
        check(y[a:b], ref, (K + 8) * 2.0 ** -23 * mag + 1.01 * 2.0 ** -24 * ref.abs() + STEP[torch.float32])
        check(z[a:b], x[a:b].double() @ w[e].double(), product_bound(x[a:b].double(), w[e].double(), K, torch.bfloat16))


def test_tile_rows():
    with moe.Experts(2, 64, 2048) as p, fp8.Fp8Linear(64, 2048, n_experts=2) as q:
        # 64 and 96 rows a group on average, or all short tiles at once
        assert p.tile_rows(0) == p.tile_rows(128) == q.tile_rows(192) == 64
        assert p.tile_rows(100000) == q.tile_rows(100000) == 256
        assert p.tile_rows(600, input_gradient=True) == 64 and p.tile_rows(600) == 256
        for bad in (lambda: p.tile_rows(-1), lambda: p.tile_rows(1 << 31), lambda: q.tile_rows(5, input_gradient=True)):
            with pytest.raises(B_.AgGemmError) as e:
                bad()
            assert e.value.code == B_.ERR_INVALID
    assert B_.library_handle().ag_moe_plan_tile_rows(None, 1, 0) == B_.ERR_INVALID


# more half tiles than pairs: whole ones, of 256 rows of dw; groups before poisoned ones; a
# long group whose sums are split all the same
@pytest.mark.parametrize("sizes,bad,K,N", [([300, 1, 0, 64, 70, 16, 5], [1, 4, 6], 520, 776), ([90, 33, 100], [1], 1160, 1304),
                                           ([11993], [], 1664, 1536)])
@pytest.mark.parametrize("out_f32", [False, True])
def test_weight_gradient_in_whole_tiles(sizes, bad, K, N, out_f32):
    dt = torch.float16
    od = torch.float32 if out_f32 else dt
    g = rng(K + N)
    rows, E, off = sum(sizes), len(sizes), offsets_of(sizes)
    x, dy = randn(g, (rows, K), dt), randn(g, (rows, N), dt)
    for e, a, b in _groups(sizes):
        if e in bad:
            x[a:b], dy[a:b] = float("inf"), float("nan")
    with moe.Experts(E, K, N, "f16") as p:
        dw = p.backward_weight(x, dy, off, out_dtype=od)
        for _ in range(3):
            assert torch.equal(dw.nan_to_num(), p.backward_weight(x, dy, off, out_dtype=od).nan_to_num())
        assert p.status() == B_.OK
    for e, a, b in _groups(sizes):
        if e not in bad:
            xd, gd = x[a:b].double().t(), dy[a:b].double()
            check(dw[e], xd @ gd, product_bound(xd, gd, b - a, od), f"dw of {e}")
