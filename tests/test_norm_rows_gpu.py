"""Norms of rows that begin anywhere: odd widths and pitches, bases and outputs off by single elements."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import norm  # noqa: E402
from moe_util import STEP, U, check, randn, rng  # noqa: E402
from test_norm_gpu import TYPES, backward_check, forward_error, forward_ref  # noqa: E402

DTYPE = {torch.float16: B_.F16, torch.bfloat16: B_.BF16, torch.float32: B_.F32}


def rows_at(g, T, H, dtype, first, pitch, scale=1.0):
    """(T, H), its first element `first` elements behind an aligned address."""
    flat = randn(g, (first + T * pitch + 64,), dtype, scale)
    return flat[first:first + T * pitch].view(T, pitch)[:, :H]


# widths around those of a warp's lanes (31 of them, 16 bytes each), of a block's warps, with one, two and four
# pieces a lane, and beyond; T on both sides of the rules on rows
@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (700, 97), (400, 129), (1, 241), (400, 247), (305, 249), (304, 497), (700, 991),
                                 (609, 993), (20, 1985), (700, 4099), (5, 7937), (305, 9001), (3, 15873), (2, 31739), (2, 31745)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_any_row(T, H, dtype, residual):
    g = rng(3 * T + H)
    w = randn(g, (H,), torch.float32 if T % 2 else dtype)
    x = rows_at(g, T, H, dtype, 1, H + 3)
    res = rows_at(g, T, H, dtype, 3, H + 6, 3.0) if residual else None
    r = norm.rms_norm(x, w, 1e-5, res)
    h, rstd, y = forward_ref(x, res, w, 1e-5)
    assert torch.equal(r.h, h)
    check(r.rstd, rstd, forward_error(H) * rstd, "rstd")
    check(r.y, y, (forward_error(H) + 1.01 * U[dtype]) * y.abs() + STEP[dtype], "y")
    if T >= 5:
        dy, dh = rows_at(g, T, H, dtype, 1, H + 1), rows_at(g, T, H, dtype, 2, H + 5)
        dx, dw = norm.rms_norm_backward(dy, r.h, w, r.rstd, dh)
        backward_check(dx, dw, dy, r.h, w, r.rstd, dh)


@pytest.mark.parametrize("first_y,first_h", [(0, 0), (1, 1), (1, 4), (7, 2)])
@pytest.mark.parametrize("T,H", [(2, 3), (400, 131), (33, 1401), (700, 1001)])
@pytest.mark.parametrize("dtype", TYPES)
def test_outputs_anywhere(first_y, first_h, T, H, dtype):
    """By raw pointers: y and h off by different elements, and nothing written beside them."""
    g = rng(T + H + first_y)
    x, res, w = randn(g, (T, H), dtype), randn(g, (T, H), dtype), randn(g, (H,), dtype)
    y, h = (torch.full((first + T * H + 16,), -7.0, dtype=dtype, device="cuda") for first in (first_y, first_h))
    rstd = torch.empty(T, device="cuda")
    B_.ag_norm_rms(T, H, DTYPE[dtype], x.data_ptr(), H, res.data_ptr(), H, w.data_ptr(), DTYPE[dtype], 1e-5,
                   y[first_y:].data_ptr(), h[first_h:].data_ptr(), rstd.data_ptr(), torch.cuda.current_stream().cuda_stream)
    want_h, _, want = forward_ref(x, res, w, 1e-5)
    assert torch.equal(h[first_h:first_h + T * H].view(T, H), want_h)
    check(y[first_y:first_y + T * H].view(T, H), want, (forward_error(H) + 1.01 * U[dtype]) * want.abs() + STEP[dtype], "y")
    for t, first in ((y, first_y), (h, first_h)):
        assert bool((t[:first] == -7).all()) and bool((t[first + T * H:] == -7).all())


def test_any_row_special_values():
    """Infinities and NaN stay in their rows; squares past the largest float are summed anew."""
    x = randn(rng(9), (700, 1001), torch.bfloat16)
    x[1, 5], x[3, 0], x[5, 1000] = float("nan"), float("inf"), 1e30
    x[7] = 0
    w = torch.ones(1001, device="cuda", dtype=torch.bfloat16)
    r = norm.rms_norm(x, w)
    clean = [i for i in range(12) if i not in (1, 3)]
    h, rstd, y = forward_ref(x[clean], None, w, 1e-6)
    check(r.y[clean], y, (forward_error(1001) + 1.01 * U[torch.bfloat16]) * y.abs() + STEP[torch.bfloat16], "y")
    assert bool(r.y[1].isnan().all()) and bool(r.y[3, 0].isnan()) and bool((r.y[3, 1:] == 0).all())


@pytest.mark.parametrize("T,H,dtype", [(700, 4096, torch.bfloat16), (700, 1001, torch.float16), (310, 4099, torch.bfloat16),
                                       (400, 1401, torch.float32), (40, 100, torch.bfloat16)])
def test_captured(T, H, dtype):
    """Forward and gradient in a graph (kernels that ask for more shared memory among them), replayed on other inputs."""
    g = rng(T * H)
    x, res, dy, dh = (randn(g, (T, H), dtype) for _ in range(4))
    w = randn(g, (H,), dtype)

    def step():
        n = norm.rms_norm(x, w, residual=res)
        return (n.y, n.h, n.rstd, *norm.rms_norm_backward(dy, n.h, w, n.rstd, dh))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        for t in (x, res, dy, dh):
            t.copy_(randn(g, (T, H), dtype))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_gradients_on_two_streams():
    """Two gradients at once: each has its own workspace."""
    g = rng(77)
    T, H = 3000, 2056
    sets = [[randn(g, (T, H), torch.bfloat16) for _ in range(2)] for _ in range(2)]
    w, rstd = randn(g, (H,), torch.bfloat16), torch.rand(T, generator=g, device="cuda")
    want = [norm.rms_norm_backward(dy, h, w, rstd) for dy, h in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for (dy, h), s in zip(sets, streams):
            with torch.cuda.stream(s):
                got.append(norm.rms_norm_backward(dy, h, w, rstd))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,H,dtype", [(700, 1001, torch.bfloat16), (700, 1002, torch.float16), (610, 9, torch.bfloat16),
                                       (3, 4101, torch.bfloat16), (700, 501, torch.float32), (1300, 4099, torch.bfloat16)])
def test_gradient_of_a_row_stays_apart(T, H, dtype):
    """Pieces at a row's ends hold elements of its neighbours: not finite ones there change nothing else."""
    g = rng(T + 7 * H)
    dy, h, dh = (randn(g, (T, H), dtype) for _ in range(3))
    w, rstd = randn(g, (H,), dtype), torch.rand(T, generator=g, device="cuda") + 0.5
    want, dw = norm.rms_norm_backward(dy, h, w, rstd, dh)
    backward_check(want, dw, dy, h, w, rstd, dh)
    bad = list(range(1, T, 2))
    dy[bad[0::3]], h[bad[1::3]], dh[bad[2::3]] = float("nan"), float("inf"), float("nan")
    got = norm.rms_norm_backward(dy, h, w, rstd, dh)[0]
    assert torch.equal(got[0::2], want[0::2])
