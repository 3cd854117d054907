"""The workspace of split sums: a plan has none before a run that may split."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import moe  # noqa: E402
from moe_util import randn, rng  # noqa: E402

MIB = 1 << 20


def _free():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


def test_plans_that_never_split_hold_little():
    x, w = randn(rng(1), (64, 64), torch.bfloat16), randn(rng(2), (1, 64, 64), torch.bfloat16)
    with moe.Experts(1, 64, 64) as p:
        out = p.forward(x, None, w)  # (kernels loaded)
    before = _free()
    plans = [moe.Experts(1, 64, 64) for _ in range(16)]
    for p in plans:
        p.forward(x, None, w, out=out)
        assert p.status() == B_.OK
    assert before - _free() <= 64 * MIB  # 16 workspaces would be 640
    for p in plans:
        p.close()


def test_first_split_run():
    x, w = randn(rng(3), (48, 4096), torch.bfloat16), randn(rng(4), (1, 4096, 512), torch.bfloat16, 1 / 64)
    with moe.Experts(1, 4096, 512) as p:
        want = p.forward(x, None, w)
        before = _free()
        assert torch.equal(p.forward(x, None, w), want) and before - _free() <= 2 * MIB
    out = torch.empty_like(want)
    with moe.Experts(1, 4096, 512) as p:  # its first run is captured
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.forward(x, None, w, out=out)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert torch.equal(p.forward(x, None, w), want) and p.status() == B_.OK
