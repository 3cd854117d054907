"""Microscaled 4-bit operands and their product against the definitions in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp4, moe  # noqa: E402
from layer_util import micro_ref, packed, row_values, row_words, weight_pieces, weight_values  # noqa: E402
from moe_util import STEP, U, check, offsets_of, randn, rng  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 128), (8, 160), (77, 1120), (64, 4096), (9, 5024), (130, 256)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_rows(rows, K, dtype):
    x = randn(rng(rows + K), (rows, K), dtype)
    if rows > 4:
        x[1] = 0
        x[2] *= 1e-4 if dtype == torch.float16 else 1e-39  # subnormals
        x[3] *= 1e4 if dtype == torch.float16 else 1e37
        # every tie and every border of the scales
        x[4, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, device="cuda", dtype=dtype)
        x[5, :64] = torch.tensor([7.0, 6.99, -7.0, 1.75] * 16, device="cuda", dtype=dtype)
    q, s = fp4.quantize_rows(x)
    assert s.dtype == torch.float8_e8m0fnu and q.dtype == torch.uint8
    code, byte = micro_ref(x)
    assert np.array_equal(bytes_of(s), row_words(byte))
    assert np.array_equal(q.cpu().numpy(), packed(code))


def test_largest_and_smallest_magnitudes():
    """Blocks at the ends of the range of floats: the scale's byte ends at 0 and at 253."""
    x = torch.zeros((6, 64), device="cuda")
    x[0, 3] = torch.finfo(torch.float32).max
    x[1, 3], x[1, 40] = 2.0 ** -149, -2.0 ** -126
    x[2, 3], x[2, 4] = 1.75 * 2.0 ** 127, -2.0 ** 125
    x[3, 3] = 2.0 ** -125
    x[4, 63] = 7 * 2.0 ** -127
    q, s = fp4.quantize_rows(x)
    code, byte = micro_ref(x)
    assert byte.max() == 253 and byte.min() == 0
    assert np.array_equal(bytes_of(s), row_words(byte)) and np.array_equal(q.cpu().numpy(), packed(code))


def test_an_error_is_at_most_half_a_step():
    x = randn(rng(3), (200, 512))
    q, s = fp4.quantize_rows(x)
    byte = s.view(torch.uint8).permute(1, 0, 2).flatten(1).double()
    unit = torch.exp2(byte - 127).repeat_interleave(32, 1)
    a = x.double().abs() / unit
    half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0))
    assert bool(((row_values(q, s) - x.double()).abs() <= half * unit).all())


def test_not_finite_blocks_are_nan():
    x = randn(rng(1), (4, 256))
    x[0, 3], x[1, 130], x[2, 255] = float("inf"), float("nan"), float("-inf")
    q, s = fp4.quantize_rows(x)
    nan = torch.isnan(row_values(q, s))
    want = torch.zeros_like(nan)
    want[0, :32] = want[1, 128:160] = want[2, 224:] = True
    assert torch.equal(nan, want)
    assert bool(torch.isnan(s.float()).sum() == 3)


@pytest.mark.parametrize("T,k,K", [(5, 2, 32), (40, 4, 1056)])
def test_quantize_gathers_the_experts_rows(T, k, K):
    g = rng(2)
    logits = randn(g, (T, 8)).masked_fill(torch.rand((T, 8), generator=g, device="cuda") < 0.6, float("-inf"))
    r = moe.route(logits, k)
    wide = randn(g, (T, K + 8), torch.bfloat16)
    x = wide[:, 8:]
    q, s = fp4.quantize_rows(x, r)
    gq, gs = fp4.quantize_rows(moe.gather(x, r))
    assert torch.equal(q, gq) and torch.equal(s.view(torch.uint8), gs.view(torch.uint8))


@pytest.mark.parametrize("E,K,N", [(1, 32, 8), (2, 128, 128), (3, 288, 200), (1, 1024, 264)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_weights(E, K, N, dtype):
    w = randn(rng(E + K + N), (E, K, N), dtype)
    w[0, :8] *= 300 if dtype == torch.float16 else 1e6
    q, s = fp4.quantize_weights(w)
    code, byte = micro_ref(w.transpose(1, 2).reshape(E * N, K))
    assert np.array_equal(q.cpu().numpy(), packed(code).reshape(E, N, K // 2))
    assert np.array_equal(bytes_of(s), weight_pieces(byte.reshape(E, N, K // 32)))
    q2, s2 = fp4.quantize_weights(w[0])
    assert torch.equal(q2, q[0]) and torch.equal(s2.view(torch.uint8), s[0].view(torch.uint8))


SHAPES = [
    ([1], 32, 8),
    ([1], 256, 256),
    ([0, 1, 0], 128, 40),
    ([3, 0, 17, 31, 32, 33, 0], 256, 256),
    ([64, 65, 63], 416, 264),
    ([300, 1, 255, 256, 257], 544, 520),
    ([223, 224, 225, 100, 129, 130], 320, 392),
    ([7], 4096, 512),
    ([60, 0, 30], 2080, 1024),
    ([700], 640, 136),
    ([16] * 33, 160, 328),
    ([5], 16384, 640),
    ([64], 8192, 4096),               # sums cut between pairs, across tiles too
    ([1] * 5, 4096, 768),
    ([10, 0, 40, 65], 16384, 520),
    ([17] * 9, 4640, 2560),           # more tiles than pairs, less than twice as many
    ([2000], 1088, 2312),
]


@pytest.mark.parametrize("sizes,K,N", SHAPES)
@pytest.mark.parametrize("out_dtype", TYPES)
def test_product(sizes, K, N, out_dtype):
    g = rng(K + N)
    rows, E = sum(sizes), len(sizes)
    x, w, off = randn(g, (rows, K), torch.bfloat16), randn(g, (E, K, N), torch.bfloat16, K ** -0.5), offsets_of(sizes)
    x[: rows // 2] *= 30  # scales that differ between rows and blocks
    x[:, ::64] *= 8
    w[:, : K // 2] *= 0.01
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_weights(w)
    with fp4.Fp4Linear(K, N, n_experts=E) as p:
        y = p.forward(xq, xs, wq, ws, off, out_dtype=out_dtype)
        assert p.status() == B_.OK
    xd, wd = row_values(xq, xs), weight_values(wq, ws)
    at = 0
    for e, n in enumerate(sizes):
        a, b = xd[at:at + n], wd[e].t()
        ref, mag = a @ b, a.abs() @ b.abs()
        check(y[at:at + n], ref, (K + 8) * 2.0 ** -23 * mag + 1.01 * U[out_dtype] * ref.abs() + STEP[out_dtype], f"expert {e}")
        at += n


@pytest.mark.parametrize("rows", [1, 33, 64, 200, 700])
def test_whole_numbers_are_exact(rows):
    """Random codes, scales from 1/2 to 2: a sum is a multiple of 2^-4 below 2^18, and exact in any order."""
    g = rng(5)
    K, N = 1024, 384

    def operand(n):
        return (torch.randint(0, 256, (n, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                torch.randint(126, 129, (n, K // 32), generator=g, device="cuda", dtype=torch.uint8))

    (xq, xb), (wq, wb) = operand(rows), operand(N)
    xs = torch.from_numpy(row_words(xb.cpu().numpy())).cuda().view(fp4.E8M0)
    ws = torch.from_numpy(weight_pieces(wb.cpu().numpy()[None]))[0].cuda().view(fp4.E8M0)
    with fp4.Fp4Linear(K, N) as p:
        y = p.forward(xq, xs, wq, ws, out_dtype=torch.float32)
        assert p.status() == B_.OK
    assert torch.equal(y.double(), row_values(xq, xs) @ weight_values(wq[None], ws[None])[0].t())


@pytest.mark.parametrize("K,rows", [(1 << 21, 5), (1 << 19, 300)])
def test_long_sums(K, rows):
    """Positive terms into 16-bit outputs: an accumulator takes at most 128 k-blocks of four additions, each off by up to
    2^-23 of the running sum; the sums of up to 64 accumulators are added to nearest."""
    g = rng(2)
    N = 264
    x, w = (torch.rand((rows, K), generator=g, device="cuda") + 0.1).half(), torch.rand((K, N), generator=g, device="cuda").half()
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_weights(w)
    del x, w
    with fp4.Fp4Linear(K, N) as p:
        y = p.forward(xq, xs, wq, ws, out_dtype=torch.bfloat16)
        assert p.status() == B_.OK
    ref = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    for a in range(0, K, 1 << 15):
        b = a + (1 << 15)
        xd = row_values(xq[:, a // 2:b // 2], xs[a // 128:b // 128])
        ref += xd @ weight_values(wq[None, :, a // 2:b // 2], ws[None, :, a // 128:b // 128])[0].t()
    check(y, ref, ((512 + 64) * 2.0 ** -23 + 1.01 * U[torch.bfloat16]) * ref)


def test_far_scales():
    """Scales of 2^-90 and 2^80 beside one another: a product of values is their product."""
    K, N, rows = 64, 8, 40
    x, w = torch.zeros((rows, K), device="cuda"), torch.zeros((K, N), device="cuda")
    x[:, 0], x[:, 40] = 3 * 2.0 ** 80, 2.0 ** -60
    w[0], w[40] = 2.0 ** -90, 1.5 * 2.0 ** -20
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_weights(w)
    with fp4.Fp4Linear(K, N) as p:
        y = p.forward(xq, xs, wq, ws, out_dtype=torch.float32)
    assert bool((y == 3 * 2.0 ** -10).all())  # (the other term is below its last bit)


def test_rows_of_nan_stay_alone():
    g = rng(6)
    sizes, K, N = [10, 20, 5], 256, 128
    x, w, off = randn(g, (35, K), torch.bfloat16), randn(g, (3, K, N), torch.bfloat16), offsets_of(sizes)
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_weights(w)
    x[10:30] = float("nan")
    bq, bs = fp4.quantize_rows(x)
    w[1, 3, 5] = float("inf")
    vq, vs = fp4.quantize_weights(w)
    with fp4.Fp4Linear(K, N, n_experts=3) as p:
        want, got = p.forward(xq, xs, wq, ws, off), p.forward(bq, bs, wq, ws, off)
        column = p.forward(xq, xs, vq, vs, off)
    assert torch.equal(want[:10], got[:10]) and torch.equal(want[30:], got[30:])
    assert bool(torch.isnan(got[10:30]).all())
    bad = torch.isnan(column)
    assert bool(bad[10:30, 5].all()) and int(bad.sum()) == 20
    assert torch.equal(column[~bad], want[~bad])


def test_rows_outside_the_groups_are_left():
    g = rng(8)
    K, N = 160, 72
    x, w = randn(g, (50, K), torch.bfloat16), randn(g, (2, K, N), torch.bfloat16)
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_weights(w)
    off = torch.tensor([4, 20, 45], dtype=torch.int32, device="cuda")
    wide = torch.full((50, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    with fp4.Fp4Linear(K, N, n_experts=2) as p:
        p.forward(xq, xs, wq, ws, off, out=wide[:, 8:8 + N])
        assert p.status() == B_.OK
    xd, wd = row_values(xq, xs), weight_values(wq, ws)
    assert bool((wide[:4] == 7).all()) and bool((wide[45:] == 7).all())
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + N:] == 7).all())
    for e, (a, b) in enumerate([(4, 20), (20, 45)]):
        ref, mag = xd[a:b] @ wd[e].t(), xd[a:b].abs() @ wd[e].abs().t()
        check(wide[a:b, 8:8 + N], ref, (K + 8) * 2.0 ** -23 * mag + 1.01 * U[torch.bfloat16] * ref.abs(), f"expert {e}")


@pytest.mark.parametrize("K,N", [(128, 40), (8192, 2560)])
@pytest.mark.parametrize("first,last", [(0, 50), (4, 45), (0, 0), (50, 50), (49, 50), (0, 51), (3, 2), (-1, 50)])
def test_offsets_of_one_expert(K, N, first, last):
    """Its rows need not be all of them, and offsets that are none leave everything as it was."""
    g = rng(K + first)
    x, w = randn(g, (50, K), torch.bfloat16), randn(g, (K, N), torch.bfloat16)
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_weights(w)
    off = torch.tensor([first, last], dtype=torch.int32, device="cuda")
    with fp4.Fp4Linear(K, N) as p:
        want = p.forward(xq, xs, wq, ws, out_dtype=torch.float32)
        out = torch.full_like(want, 7.0)
        p.forward(xq, xs, wq, ws, off, out=out, out_dtype=torch.float32)
        good = 0 <= first <= last <= 50
        assert p.status() == (B_.OK if good else B_.ERR_INVALID)
        if not good:
            assert bool((out == 7).all())
            p.reset()
            assert torch.equal(p.forward(xq, xs, wq, ws, out_dtype=torch.float32), want) and p.status() == B_.OK
            return
    assert bool((out[:first] == 7).all()) and bool((out[last:] == 7).all())
    mag = row_values(xq, xs).abs() @ weight_values(wq[None], ws[None])[0].abs().t()
    check(out[first:last], want[first:last], 2 * (K + 8) * 2.0 ** -23 * mag[first:last])  # (tiles of other rows may add in another order)


def test_runs_repeat_bit_for_bit():
    g = rng(7)
    x, w = randn(g, (64, 16384), torch.bfloat16), randn(g, (16384, 512), torch.bfloat16)
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_weights(w)
    with fp4.Fp4Linear(16384, 512) as p:
        first = p.forward(xq, xs, wq, ws).clone()
        for _ in range(5):
            assert torch.equal(first, p.forward(xq, xs, wq, ws))


def test_no_rows_and_refusals():
    K, N = 256, 64
    w = torch.zeros((K, N), dtype=torch.float16, device="cuda")
    wq, ws = fp4.quantize_weights(w)
    x = torch.zeros((8, K), dtype=torch.float16, device="cuda")
    xq, xs = fp4.quantize_rows(x)
    e = fp4.quantize_rows(x[:0])
    with fp4.Fp4Linear(K, N) as p:
        assert p.forward(*e, wq, ws).shape == (0, N)
        assert not bool(p.forward(xq, xs, wq, ws).any())
        for bad in ((x, xs, wq, ws), (xq, xs.view(torch.uint8), wq, ws), (xq, xs[:1], wq, ws), (xq, xs, wq.t(), ws),
                    (xq, xs, wq, ws[:, :1]), (xq[:, :64], xs, wq, ws), (xq[:7], xs, wq, ws)):
            with pytest.raises((TypeError, ValueError)):
                p.forward(*bad)
        with pytest.raises(B_.AgGemmError):
            p.forward(xq, xs, wq, ws, out_dtype=torch.float64)
        with pytest.raises(ValueError):
            p.forward(xq, xs, wq, ws, offsets_of([4, 4]).repeat(2))
        off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
        p.forward(xq, xs, wq, ws, off)
        assert p.status() == B_.ERR_INVALID
        p.reset()
        assert p.status() == B_.OK
    with pytest.raises(B_.AgGemmError):
        fp4.quantize_rows(x[:, :48])            # K % 32
    with pytest.raises(B_.AgGemmError):
        fp4.quantize_rows(torch.zeros((4, 72), dtype=torch.float16, device="cuda")[:, 4:68])  # 8-byte aligned
    with pytest.raises(ValueError):
        fp4.quantize_weights(w.t())
    with pytest.raises(B_.AgGemmError):
        fp4.Fp4Linear(208, 64)                  # K % 32
    with pytest.raises(B_.AgGemmError):
        fp4.quantize_weights(torch.zeros((256, 12), device="cuda"))  # N % 8
