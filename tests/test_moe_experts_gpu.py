"""Products grouped by expert and their gradients against 64-bit products."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import moe  # noqa: E402
from moe_util import check, offsets_of, product_bound, randn, rng  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16}

# sizes of the groups, K, N: empty groups, one row, tile edges, sizes that are no
# multiple of a tile, of 64 or of 16, several tiles, and few tiles (split sums)
SHAPES = [
    ([1], 64, 64),
    ([0, 1, 0], 72, 40),
    ([3, 0, 17, 31, 32, 33, 0], 128, 256),
    ([64, 65, 63], 200, 264),
    ([300, 1, 255, 256, 257], 264, 520),
    ([0, 0, 700], 512, 128),
    ([5], 4096, 512),
    ([40, 0, 0, 30], 2048, 1024),
    ([16] * 33, 64, 328),
    ([129] * 3, 8, 8),
]


def _case(sizes, K, N, dt, seed, E=None):
    g = rng(seed)
    rows, E = sum(sizes), len(sizes)
    return (randn(g, (rows, K), dt), randn(g, (E, K, N), dt, K ** -0.5), randn(g, (rows, N), dt),
            offsets_of(sizes))


def _per_expert(sizes, fn):
    at, out = 0, []
    for e, n in enumerate(sizes):
        out.append(fn(e, at, at + n))
        at += n
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("sizes,K,N", SHAPES)
def test_products_match_64_bits(sizes, K, N, dtype, out_f32):
    dt = DT[dtype]
    x, w, dy, off = _case(sizes, K, N, dt, 1000 + K + N)
    od = torch.float32 if out_f32 else dt
    with moe.Experts(len(sizes), K, N, dtype) as p:
        y = p.forward(x, off, w, out_dtype=od)
        dx = p.backward_input(dy, off, w, out_dtype=od)
        dw = p.backward_weight(x, dy, off, out_dtype=od)
        assert p.status() == B_.OK
    xd, wd, gd = x.double(), w.double(), dy.double()
    for e, (a, b) in enumerate(_per_expert(sizes, lambda e, a, b: (a, b))):
        check(y[a:b], xd[a:b] @ wd[e], product_bound(xd[a:b], wd[e], K, od), f"y of {e}")
        check(dx[a:b], gd[a:b] @ wd[e].t(), product_bound(gd[a:b], wd[e].t(), N, od), f"dx of {e}")
        check(dw[e], xd[a:b].t() @ gd[a:b], product_bound(xd[a:b].t(), gd[a:b], b - a, od), f"dw of {e}")
        if a == b:
            assert not bool(dw[e].any())


def test_neighbours_with_infinities_and_nan_stay_out():
    """Rows next to a group's end hold infinities and NaN: they must not reach the group."""
    sizes, K, N = [5, 70, 1, 0, 64, 9], 136, 72
    x, w, dy, off = _case(sizes, K, N, torch.float16, 5)
    bad = [1, 4]  # experts whose rows are poisoned
    at = 0
    for e, n in enumerate(sizes):
        if e in bad:
            x[at:at + n] = float("inf")
            dy[at:at + n] = float("nan")
        at += n
    with moe.Experts(len(sizes), K, N, "f16") as p:
        y, dx, dw = p.forward(x, off, w), p.backward_input(dy, off, w), p.backward_weight(x, dy, off)
        assert p.status() == B_.OK
    for e, (a, b) in enumerate(_per_expert(sizes, lambda e, a, b: (a, b))):
        if e in bad:
            continue
        xd, wd, gd = x[a:b].double(), w[e].double(), dy[a:b].double()
        check(y[a:b], xd @ wd, product_bound(xd, wd, K, torch.float16), f"y of {e}")
        check(dx[a:b], gd @ wd.t(), product_bound(gd, wd.t(), N, torch.float16), f"dx of {e}")
        check(dw[e], xd.t() @ gd, product_bound(xd.t(), gd, b - a, torch.float32), f"dw of {e}")


@pytest.mark.parametrize("sizes,bad", [([16, 7, 48, 5, 96, 3, 64], [1, 3, 5]), ([80, 300, 112], [1]), ([33, 0, 16, 9], [0, 3])])
def test_groups_that_end_with_a_step_next_to_poison(sizes, bad):
    """Groups of whole steps of 16 rows, and an empty one, before rows of NaN."""
    K, N = 264, 136
    x, _, dy, off = _case(sizes, K, N, torch.bfloat16, 31)
    at = 0
    for e, n in enumerate(sizes):
        if e in bad:
            x[at:at + n] = float("nan")
            dy[at:at + n] = float("inf")
        at += n
    with moe.Experts(len(sizes), K, N) as p:
        dw = p.backward_weight(x, dy, off)
        assert p.status() == B_.OK
    for e, (a, b) in enumerate(_per_expert(sizes, lambda e, a, b: (a, b))):
        if e not in bad:
            xd, gd = x[a:b].double(), dy[a:b].double()
            check(dw[e], xd.t() @ gd, product_bound(xd.t(), gd, b - a, torch.float32), f"dw of {e}")
            assert a < b or not bool(dw[e].any())


def test_gradients_are_the_differences_of_the_product():
    """The product is linear: with small whole numbers every value is exact, and
    <dy, y(x + v) - y(x - v)> / 2 = <dx, v>, the same for the weights."""
    sizes, K, N = [7, 0, 40, 129], 96, 80
    g = rng(6)
    rows = sum(sizes)

    def ints(shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(torch.float16)

    x, v, dy, w, u, off = ints((rows, K)), ints((rows, K)), ints((rows, N)), ints((4, K, N)), ints((4, K, N)), offsets_of(sizes)
    f32 = torch.float32
    with moe.Experts(4, K, N, "f16") as p:
        dx = p.backward_input(dy, off, w, out_dtype=f32).double()
        dw = p.backward_weight(x, dy, off).double()
        d = (p.forward(x + v, off, w, out_dtype=f32).double() - p.forward(x - v, off, w, out_dtype=f32).double()) / 2
        dv = (p.forward(x, off, w + u, out_dtype=f32).double() - p.forward(x, off, w - u, out_dtype=f32).double()) / 2
    assert float((dy.double() * d).sum()) == float((dx * v.double()).sum())
    assert float((dy.double() * dv).sum()) == float((dw * u.double()).sum())


def test_rows_outside_the_groups_keep_their_values():
    sizes, K, N = [4, 30], 64, 128
    g = rng(7)
    x, w = randn(g, (50, K), torch.bfloat16), randn(g, (2, K, N), torch.bfloat16)
    off = offsets_of(sizes, start=3)
    out = torch.full((50, N), 7.0, dtype=torch.bfloat16, device="cuda")
    with moe.Experts(2, K, N) as p:
        p.forward(x, off, w, out=out)
        assert p.status() == B_.OK
    assert bool((out[:3] == 7).all()) and bool((out[37:] == 7).all())
    for e, (a, b) in enumerate([(3, 7), (7, 37)]):
        check(out[a:b], x[a:b].double() @ w[e].double(),
              product_bound(x[a:b].double(), w[e].double(), K, torch.bfloat16))


def test_column_blocks_and_pitched_weights():
    """x, dy, outputs and weights as blocks of wider tensors."""
    sizes, K, N = [20, 100, 3], 128, 192
    g = rng(8)
    rows = sum(sizes)
    xw, dyw = randn(g, (rows, K + 64), torch.float16), randn(g, (rows, N + 8), torch.float16)
    ww = randn(g, (3, K, 2 * N), torch.float16, K ** -0.5)
    x, dy, w, off = xw[:, 64:], dyw[:, :N], ww[:, :, N:], offsets_of(sizes)
    yw = torch.full((rows, 2 * N), 5.0, dtype=torch.float16, device="cuda")
    with moe.Experts(3, K, N, "f16") as p:
        p.forward(x, off, w, out=yw[:, :N])
        dx = p.backward_input(dy, off, w)
        dw = p.backward_weight(x, dy, off)
        a = p.forward(x.contiguous(), off, w.contiguous())
        b = p.backward_input(dy.contiguous(), off, w.contiguous())
        c = p.backward_weight(x.contiguous(), dy.contiguous(), off)
    assert torch.equal(yw[:, :N], a) and bool((yw[:, N:] == 5).all())
    assert torch.equal(dx, b) and torch.equal(dw, c)


def test_no_rows():
    w = randn(rng(9), (2, 64, 64), torch.float16)
    off = offsets_of([0, 0])
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    with moe.Experts(2, 64, 64, "f16") as p:
        assert p.forward(x, off, w).shape == (0, 64)
        assert p.backward_input(x, off, w).shape == (0, 64)
        assert not bool(p.backward_weight(x, x, off).any())


def test_one_expert_without_offsets():
    g = rng(10)
    x, w = randn(g, (77, 128), torch.bfloat16), randn(g, (1, 128, 96), torch.bfloat16)
    with moe.Experts(1, 128, 96) as p:
        y = p.forward(x, None, w)
    check(y, x.double() @ w[0].double(), product_bound(x.double(), w[0].double(), 128, torch.bfloat16))


@pytest.mark.parametrize("sizes,K,N", [([60], 8192, 512), ([20, 0, 44], 4096, 256), ([600], 2048, 256)])
def test_runs_repeat_bit_for_bit(sizes, K, N):
    """Split sums are added in the order of their parts, whoever arrives last."""
    x, w, dy, off = _case(sizes, K, N, torch.bfloat16, 11)
    with moe.Experts(len(sizes), K, N) as p:
        first = [t.clone() for t in (p.forward(x, off, w), p.backward_input(dy, off, w), p.backward_weight(x, dy, off))]
        for _ in range(5):
            for a, b in zip(first, (p.forward(x, off, w), p.backward_input(dy, off, w), p.backward_weight(x, dy, off))):
                assert torch.equal(a, b)


@pytest.mark.parametrize("sizes,K,N", [([3754], 608, 376), ([1000, 0, 1, 2049], 264, 72), ([511, 512, 513, 65], 256, 520)])
@pytest.mark.parametrize("out_f32", [False, True])
def test_long_groups_of_small_weights(sizes, K, N, out_f32):
    """The sums over a group's rows are split between pairs: each part, the ragged last
    one, parts without rows, and infinities in the rows behind the last group."""
    dt = torch.bfloat16
    x, _, dy, off = _case(sizes + [9], K, N, dt, 21)
    rows, od = sum(sizes), torch.float32 if out_f32 else dt
    x[rows:], dy[rows:] = float("inf"), float("nan")
    with moe.Experts(len(sizes), K, N) as p:
        dw = p.backward_weight(x, dy, off[:-1].contiguous(), out_dtype=od)
        for _ in range(4):
            assert torch.equal(dw, p.backward_weight(x, dy, off[:-1].contiguous(), out_dtype=od))
        assert p.status() == B_.OK
    xd, gd = x.double(), dy.double()
    for e, (a, b) in enumerate(_per_expert(sizes, lambda e, a, b: (a, b))):
        check(dw[e], xd[a:b].t() @ gd[a:b], product_bound(xd[a:b].t(), gd[a:b], b - a, od), f"dw of {e}")


def test_runs_on_two_streams_do_not_meet():
    """One plan's runs share its workspace: a run on another stream waits for the last."""
    g = rng(12)
    xs = [randn(g, (48, 4096), torch.bfloat16) for _ in range(2)]
    w = randn(g, (1, 4096, 512), torch.bfloat16, 1 / 64)
    with moe.Experts(1, 4096, 512) as p:
        want = [p.forward(x, None, w) for x in xs]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [p.forward(xs[i % 2], None, w, stream=streams[i % 2]) for i in range(8)]
        torch.cuda.synchronize()
        assert p.status() == B_.OK
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("off", [[0, 10, 5, 20], [0, 5, 10, 21], [-1, 5, 10, 20], [0, 30, 10, 20]])
def test_bad_offsets_write_nothing_and_are_reported(off):
    x = randn(rng(13), (20, 64), torch.float16)
    w = randn(rng(14), (3, 64, 64), torch.float16)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    with moe.Experts(3, 64, 64, "f16") as p:
        out = torch.full((20, 64), 3.0, dtype=torch.float16, device="cuda")
        p.forward(x, o, w, out=out)
        assert p.status() == B_.ERR_INVALID and bool((out == 3).all())
        dw = torch.full((3, 64, 64), 3.0, dtype=torch.float32, device="cuda")
        p.backward_weight(x, x, o, out=dw)
        assert p.status() == B_.ERR_INVALID and bool((dw == 3).all())
        p.reset()
        y = p.forward(x, offsets_of([10, 5, 5]), w)
        assert p.status() == B_.OK
    check(y[:10], x[:10].double() @ w[0].double(), product_bound(x[:10].double(), w[0].double(), 64, torch.float16))


def test_many_experts():
    sizes = [(i * 7) % 5 for i in range(1024)]
    K, N = 64, 64
    x, w, dy, off = _case(sizes, K, N, torch.bfloat16, 15)
    with moe.Experts(1024, K, N) as p:
        y = p.forward(x, off, w)
        dw = p.backward_weight(x, dy, off)
        assert p.status() == B_.OK
    e = torch.repeat_interleave(torch.arange(1024, device="cuda"), torch.tensor(sizes, device="cuda"))
    ref = torch.bmm(x.double()[:, None], w.double()[e])[:, 0]
    mag = torch.bmm(x.double().abs()[:, None], w.double()[e].abs())[:, 0]
    check(y, ref, (K + 2) * 2.0 ** -23 * mag + 2.0 ** -8 * 1.01 * ref.abs() + 1e-30)
    dref = torch.zeros((1024, K, N), dtype=torch.float64, device="cuda")
    dref.index_add_(0, e, x.double()[:, :, None] * dy.double()[:, None, :])
    check(dw, dref, 8 * 2.0 ** -23 * 64.0)


def test_refusals():
    x = torch.zeros((8, 64), dtype=torch.float16, device="cuda")
    w = torch.zeros((2, 64, 64), dtype=torch.float16, device="cuda")
    off = offsets_of([4, 4])
    for args in [(0, 64, 64), (1025, 64, 64), (2, 60, 64), (2, 64, 12), (2, 0, 64)]:
        with pytest.raises(B_.AgGemmError) as e:
            moe.Experts(*args, "f16")
        assert e.value.code == B_.ERR_INVALID
    with pytest.raises(ValueError):
        moe.Experts(2, 64, 64, "f32")
    with moe.Experts(2, 64, 64, "f16") as p:
        for bad in (x.float(), x.bfloat16(), x.cpu(), x[:, :32], x.t(), "x"):
            with pytest.raises((TypeError, ValueError)):
                p.forward(bad, off, w)
        for bad in (w[:1], w.float(), w.transpose(1, 2)):
            with pytest.raises((TypeError, ValueError)):
                p.forward(x, off, bad)
        for bad in (off.long(), off[:2], off.cpu()):
            with pytest.raises((TypeError, ValueError)):
                p.forward(x, bad, w)
        with pytest.raises(B_.AgGemmError):
            p.forward(x, None, w)           # two experts need offsets
        with pytest.raises(B_.AgGemmError):
            p.forward(x, off, w, out_dtype=torch.bfloat16)
        with pytest.raises(ValueError):
            p.forward(x, off, w, out=torch.empty((8, 32), dtype=torch.float16, device="cuda"))
        with pytest.raises(ValueError):
            p.backward_weight(x, x[:4], off)
        wide = torch.zeros((8, 68), dtype=torch.float16, device="cuda")
        with pytest.raises(B_.AgGemmError):  # rows 136 bytes apart
            p.forward(wide[:, :64], off, w)
        big = torch.zeros(8 * 64 + 8, dtype=torch.float16, device="cuda")
        with pytest.raises(B_.AgGemmError):  # 2-byte aligned
            p.forward(big[1:513].view(8, 64), off, w)
        lib = B_.library_handle()
        assert lib.ag_moe_forward(None, 1, None, 0, None, None, 0, 0, None, 0, 0, None) == B_.ERR_INVALID
        assert lib.ag_fp8_forward(p.handle, 1, None, None, None, None, None, None, 0, 0, None) == B_.ERR_INVALID


def test_runs_in_a_cuda_graph():
    """A plan's runs can be captured, whatever stream ran before, and replayed on new inputs."""
    from all_gather_gemm_chunked_gb300 import fp8
    g = rng(31)
    T, E, k, K, N = 24, 6, 2, 256, 320
    x, logits = randn(g, (T, K), torch.bfloat16), randn(g, (T, E))
    w = randn(g, (E, K, N), torch.bfloat16, K ** -0.5)
    wq, ws = fp8.quantize_weights(w)

    def step():
        r = moe.route(logits, k)
        y = up.forward(moe.gather(x, r), r.offsets, w)
        z = low.forward(*fp8.quantize_rows(x, r), wq, ws, r.offsets)
        return moe.combine(y, r.slots, r.weights), moe.combine(z, r.slots, r.weights)

    with moe.Experts(E, K, N) as up, fp8.Fp8Linear(K, N, n_experts=E) as low:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for seed in (32, 33):
            x.copy_(randn(rng(seed), (T, K), torch.bfloat16))
            logits.copy_(randn(rng(seed + 5), (T, E)))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            for a, b in zip(got, step()):
                assert torch.equal(a, b)
        assert up.status() == B_.OK and low.status() == B_.OK


def test_rows_counts_around_the_tile_heights():
    """Short and long row tiles, chosen by the mean rows of a group, agree with 64 bits at
    the change-over (64 rows a group) and at tile edges."""
    K, N, E = 128, 64, 2
    g = rng(41)
    w = randn(g, (E, K, N), torch.float16, K ** -0.5)
    for sizes in ([64, 64], [65, 64], [0, 128], [129, 0], [1, 255], [257, 1], [512, 31]):
        x, off = randn(g, (sum(sizes), K), torch.float16), offsets_of(sizes)
        with moe.Experts(E, K, N, "f16") as p:
            y = p.forward(x, off, w)
        at = 0
        for e, n in enumerate(sizes):
            a, b = x[at:at + n].double(), w[e].double()
            check(y[at:at + n], a @ b, product_bound(a, b, K, torch.float16), f"{sizes} {e}")
            at += n
