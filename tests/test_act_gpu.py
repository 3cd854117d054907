"""The gated activation, its gradient and its outputs as codes, against the definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import act, fp4, fp8  # noqa: E402
from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from layer_util import row_values  # noqa: E402
from moe_util import STEP, U, check, randn, rng  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
F = 2.0 ** -24  # a rounding to float
SHAPES = [(1, 1), (3, 7), (5, 64), (2, 118), (70, 256), (33, 1401), (64, 7168), (310, 4096), (2, 20000), (0, 64)]


def parts(x):
    d = x.double()
    g, u = d[:, :x.shape[1] // 2], d[:, x.shape[1] // 2:]
    return g, u, torch.sigmoid(g)


# exp is off by at most 2 ulps (2^-22) of itself, so s by 2^-22 (1 - s) and three roundings more: 8 F in all
S_ERROR = 8 * F


@pytest.mark.parametrize("T,N", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(T, N, dtype):
    x = randn(rng(T + N), (T, 2 * N), dtype, 3.0)
    g, u, s = parts(x)
    y = g * s * u
    check(act.swiglu(x), y, (S_ERROR + 2 * F + 1.01 * U[dtype]) * y.abs() + STEP[dtype], "y")


@pytest.mark.parametrize("T,N", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(T, N, dtype):
    gen = rng(T + 2 * N)
    x, dy = randn(gen, (T, 2 * N), dtype, 3.0), randn(gen, (T, N), dtype)
    backward_check(act.swiglu_backward(dy, x), dy, x)


def backward_check(dx, dy, x):
    g, u, s = parts(x)
    N, d = dy.shape[1], dy.double()
    t = 1 + g * (1 - s)
    ref = torch.cat([d * u * s * t, d * g * s], 1)
    # 1 - s is off by s's error, which g carries into t
    err_g = (d * u * s).abs() * ((S_ERROR + 4 * F) * t.abs() + (S_ERROR + 2 * F) * g.abs() + F)
    err = torch.cat([err_g, (S_ERROR + 3 * F) * (d * g * s).abs()], 1)
    check(dx, ref, err + 1.01 * U[dy.dtype] * ref.abs() + STEP[dy.dtype], "dx")


@pytest.mark.parametrize("N", [64, 2048, 2049])
def test_column_blocks_and_alignment(N):
    gen = rng(N)
    for first in (8, 1):
        x, dy = randn(gen, (20, 2 * N + 24), torch.bfloat16)[:, first:first + 2 * N], randn(gen, (20, N + 16), torch.bfloat16)[:, first:first + N]
        assert torch.equal(act.swiglu(x), act.swiglu(x.contiguous()))
        assert torch.equal(act.swiglu_backward(dy, x), act.swiglu_backward(dy.contiguous(), x.contiguous()))


def test_special_values():
    big = torch.finfo(torch.float32).max
    nan, inf = float("nan"), float("inf")
    x = torch.tensor([[0.0, -100.0, 100.0, -big, big, nan, 1.0, inf, 0.0], [3.0, 2.0, 2.0, 1.0, 1.0, 1.0, inf, 1.0, nan]], device="cuda").reshape(1, 18)
    y = act.swiglu(x)[0].tolist()
    # s(-100) = 3.72e-44 lies among floats 2^-149 = 1.4e-45 apart, and exp is off by at most 2 of these steps, the
    # rounding by half of one: 3.5e-45, times what s is multiplied with (200, 198, 100)
    assert y[:5] == [0.0, pytest.approx(-7.44e-42, abs=7.1e-43), 200.0, 0.0, big]
    assert y[5] != y[5] and y[6] == inf and y[7] == inf and y[8] != y[8]
    dx = act.swiglu_backward(torch.ones((1, 9), device="cuda"), x)[0]
    assert dx[:3].tolist() == [1.5, pytest.approx(-7.366e-42, abs=7e-43), 2.0]
    assert dx[3:5].tolist() == [0.0, 1.0] and dx[9:14].tolist() == [0.0, pytest.approx(-3.72e-42, abs=3.6e-43), 100.0, 0.0, big]
    assert bool(torch.isnan(dx[5]))


@pytest.mark.parametrize("dtype", TYPES)
def test_far_gates(dtype):
    """Gates from -110 to 110, where the exponential leaves the range of floats."""
    n = 4096
    x = torch.cat([torch.linspace(-110, 110, n, device="cuda"), randn(rng(3), (n,))]).to(dtype)[None]
    dy = randn(rng(4), (1, n), dtype)
    g, u, s = parts(x)
    # beside the error near zero: the approximate exponential's |g| 2^-24, and where s lies among floats 2^-149
    # apart (or is flushed to them), three and a half of those steps
    y, grain = g * s * u, 3.5 * 2.0 ** -149 * (1 + g.abs())
    check(act.swiglu(x), y, (S_ERROR + (4 + g.abs()) * F + 1.01 * U[dtype]) * y.abs() + grain * u.abs() + STEP[dtype], "y")
    d, t = dy.double(), 1 + g * (1 - s)
    ref = torch.cat([d * u * s * t, d * g * s], 1)
    rel = S_ERROR + (6 + g.abs()) * F
    err = torch.cat([(d * u).abs() * (s * (rel * t.abs() + rel * g.abs() * (1 - s)) + grain * t.abs()), (d * g).abs() * (rel * s) + grain * d.abs()], 1)
    # products below 2^-126 are rounded to 2^-149, by half of it: dy s, which u t (or g) multiplies, and that times u, which t does
    err = err + 2.0 ** -150 * torch.cat([(u * t).abs() + t.abs() + 1, g.abs() + 1], 1)
    check(act.swiglu_backward(dy, x), ref, err + 1.01 * U[dtype] * ref.abs() + STEP[dtype], "dx")


def test_backward_is_the_slope():
    """Differences of the formula in 64 bits along random directions."""
    gen = rng(12)
    x, dy, step = randn(gen, (6, 400), scale=2.0), randn(gen, (6, 200)), 1e-5
    dx = act.swiglu_backward(dy, x).double()

    def f(x):
        g, u, s = parts(x)
        return (g * s * u * dy.double()).sum()

    for seed in range(3):
        v = randn(rng(seed), x.shape).double()
        slope = (f(x.double() + step * v) - f(x.double() - step * v)) / (2 * step)
        assert abs((dx * v).sum() - slope) < 1e-6 * dx.norm() * v.norm()


@pytest.mark.parametrize("T,N", [(1, 32), (5, 160), (40, 4096), (310, 1056), (2, 20000), (0, 64)])
@pytest.mark.parametrize("codes", ["e4m3", "mxfp4"])
def test_codes_of_floats(T, N, codes):
    """With float rows the unrounded y can be had: its codes and scales, bit for bit."""
    x = randn(rng(T + N), (T, 2 * N), scale=2.0)
    q, s = act.swiglu_quantized(x, codes)
    wq, ws = (fp8 if codes == "e4m3" else fp4).quantize_rows(act.swiglu(x))
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s.view(torch.uint8), ws.view(torch.uint8))


@pytest.mark.parametrize("T,N", [(1, 32), (5, 160), (40, 4096), (310, 1056)])
@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("codes", ["e4m3", "mxfp4"])
def test_codes_of_halves(T, N, dtype, codes):
    """The unrounded y of 16-bit rows is that of the same rows as floats."""
    x = randn(rng(T + N + 1), (T, 2 * N), dtype, 2.0)
    q, s = act.swiglu_quantized(x, codes)
    wq, ws = act.swiglu_quantized(x.float(), codes)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s.view(torch.uint8), ws.view(torch.uint8))


def test_streams_and_capture():
    gen = rng(5)
    x, dy = randn(gen, (64, 4096), torch.bfloat16), randn(gen, (64, 2048), torch.bfloat16)

    def step(stream=None):
        return act.swiglu(x, stream=stream), act.swiglu_backward(dy, x, stream=stream), *act.swiglu_quantized(x, "mxfp4", stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.current_stream().wait_stream(s)
    want = step()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(randn(rng(9), x.shape, x.dtype))
    graph.replay()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, step()))


def test_refusals():
    x, dy = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    for bad in (x[:, :63], x[:, :0], x[0], x.double(), x.t(), x.cpu()):
        with pytest.raises((TypeError, ValueError)):
            act.swiglu(bad)
    for bad in (dy.float(), dy[:3], x, dy.t()):
        with pytest.raises((TypeError, ValueError)):
            act.swiglu_backward(bad, x)
    with pytest.raises(ValueError):
        act.swiglu_quantized(x, "int4")
    with pytest.raises(B_.AgGemmError):
        act.swiglu_quantized(torch.zeros((4, 48), dtype=torch.bfloat16, device="cuda"), "e4m3")
    with pytest.raises(B_.AgGemmError):
        act.swiglu_quantized(torch.zeros((4, 96), dtype=torch.bfloat16, device="cuda"), "mxfp4")
    with pytest.raises(B_.AgGemmError):
        act.swiglu_quantized(torch.zeros((4, 72), dtype=torch.bfloat16, device="cuda")[:, 4:68], "mxfp4")
