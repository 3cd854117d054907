"""Long sums of 4-bit products: those that are cut between pairs or split, whole numbers that are exact in any order, and
sums in which a term too small for the running sum is kept, because the sum leaves the tensor core in segments."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import fp4  # noqa: E402
from layer_util import row_values, row_words, weight_pieces, weight_values  # noqa: E402
from moe_util import offsets_of, rng  # noqa: E402


def operands(g, rows, E, K, N):
    """Random codes, and scales of 1/2, 1 and 2: values are multiples of 1/4."""
    def codes(*shape):
        return torch.randint(0, 256, shape + (K // 2,), generator=g, device="cuda", dtype=torch.uint8)

    def scales(*shape):
        return torch.randint(126, 129, shape + (K // 32,), generator=g, device="cuda", dtype=torch.uint8).cpu().numpy()

    return (codes(rows), torch.from_numpy(row_words(scales(rows))).cuda().view(fp4.E8M0),
            codes(E, N), torch.from_numpy(weight_pieces(scales(E, N))).cuda().view(fp4.E8M0))


@pytest.mark.parametrize("sizes,K,N", [
    ([1], 16384, 256), ([5], 16384, 640), ([64], 16384, 2056),  # short tiles of one expert, each cut among several pairs
    ([1], 4096, 4096), ([64], 8192, 4096), ([33], 4640, 16384),
    ([10, 0, 40, 65], 16384, 520), ([1] * 5, 4096, 768),        # of several
    ([17] * 9, 4640, 2560), ([64] * 80, 1056, 264),             # more tiles than pairs
    ([700], 16384, 136), ([300, 0, 250], 8192, 264),            # long tiles in parts
    ([225] * 7, 2080, 2056), ([2000], 8224, 2312),              # and whole ones
])
def test_whole_numbers_are_exact(sizes, K, N):
    """A sum of products is a multiple of 2^-4, and any part of it at most the sum of magnitudes: below 2^20, so that every
    partial sum is a float, whatever the order.  16-bit outputs are that, rounded once."""
    rows, E = sum(sizes), len(sizes)
    xq, xs, wq, ws = operands(rng(rows + K), rows, E, K, N)
    ref, at = [], 0
    xd, wd = row_values(xq, xs), weight_values(wq, ws)
    for e, n in enumerate(sizes):
        a, b = xd[at:at + n], wd[e].t()
        assert n == 0 or float((a.abs() @ b.abs()).max()) < 2.0 ** 20
        ref.append(a @ b)
        at += n
    ref = torch.cat(ref)
    with fp4.Fp4Linear(K, N, n_experts=E) as p:
        for t in (torch.float32, torch.bfloat16, torch.float16):
            y = p.forward(xq, xs, wq, ws, offsets_of(sizes), out_dtype=t)
            assert p.status() == B_.OK
            # (every value is a float, so that its way to 16 bits rounds it once)
            assert torch.equal(y, ref.float().to(t)), t


def spiked(n, K, first, rest):
    """(n, K): `first` at 0, `rest` at every 64th element behind it, zeros: at most one term for each step of the tensor core."""
    x = torch.zeros((n, K), device="cuda")
    x[:, 64::64] = rest
    x[:, 0] = first
    return x


@pytest.mark.parametrize("rows,K,N", [(3, 1 << 15, 264), (64, 1 << 16, 1024), (300, 1 << 15, 264), (2000, 1 << 14, 2312)])
def test_segments_of_float_outputs(rows, K, N):
    """2^24 and then halves, one a step of 64 elements: a float from 2^24 on has steps of 2, so a half added to it alone is lost.
    A segment is 8 k-blocks of 256, or ends earlier by whole pairs of k-blocks: behind the first, its halves make
    16 (or a multiple of 4), which the 32-bit sums take exactly.  Of the first segment's 15.5 all may be lost."""
    xq, xs = fp4.quantize_rows(spiked(rows, K, 4096.0, 0.5))
    wq, ws = fp4.quantize_weights(spiked(N, K, 4096.0, 1.0).t().contiguous())
    with fp4.Fp4Linear(K, N) as p:
        y = p.forward(xq, xs, wq, ws, out_dtype=torch.float32)
        assert p.status() == B_.OK
    segments = K // 2048
    assert bool((y >= 2.0 ** 24 + 16 * (segments - 1)).all()) and bool((y <= 2.0 ** 24 + 16 * segments).all())


@pytest.mark.parametrize("rows", [3, 300])
def test_segments_of_half_outputs(rows):
    """The same where the output has 16 bits and a segment 128 k-blocks: 2^15 and then 2^-10 a step, a quarter of a float's
    step there, but 1/2 a segment.  128 segments make 63.5 to 64 of them (those of the first may be lost), two steps of
    fp16."""
    K, N = 1 << 22, 8
    xq, xs = fp4.quantize_rows(spiked(rows, K, 256.0, 2.0 ** -5))
    wq, ws = fp4.quantize_weights(spiked(N, K, 128.0, 2.0 ** -5).t().contiguous())
    with fp4.Fp4Linear(K, N) as p:
        y = p.forward(xq, xs, wq, ws, out_dtype=torch.float16)
        assert p.status() == B_.OK
    assert bool((y == 32768 + 64).all())
