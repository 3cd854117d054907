"""Plans and streams: a new plan's cleared workspace, runs from several threads' default
streams, branches of one captured graph."""
import threading
import time

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300 import moe  # noqa: E402
from moe_util import randn, rng  # noqa: E402

CYCLES_PER_MS = 2_000_000  # at about 2 GHz


def test_a_new_plan_is_clean_on_any_stream():
    """Work waits on the default stream while a plan is made and used on a stream that does
    not wait for it: what the plan clears at its start must not come after its first run."""
    x, w = randn(rng(1), (20, 64), torch.float16), randn(rng(2), (3, 64, 64), torch.float16)
    bad = torch.tensor([0, 10, 5, 20], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    for wait_ms in (0, 300):  # (the first time loads the kernels, which waits for the device)
        torch.cuda.synchronize()
        torch.cuda._sleep(wait_ms * CYCLES_PER_MS)
        with moe.Experts(3, 64, 64, "f16") as p:
            p.forward(x, bad, w, stream=s)  # leaves a status
            s.synchronize()
            torch.cuda.synchronize()
            assert p.status() == B_.ERR_INVALID
