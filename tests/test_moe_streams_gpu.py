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
PER_THREAD = 2             # the handle of a host thread's own default stream


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


def _split_product():
    """One expert whose sums are split, and its operands."""
    g = rng(3)
    return randn(g, (48, 4096), torch.bfloat16), randn(g, (1, 4096, 512), torch.bfloat16, 1 / 64)


def test_runs_on_two_threads_default_streams_are_ordered():
    """The per-thread default stream has one handle in every thread, but is not one stream:
    a run that shares the workspace with one of another thread waits for it."""
    x, w = _split_product()
    s = torch.cuda.ExternalStream(PER_THREAD)
    queued, over = threading.Event(), threading.Event()
    with moe.Experts(1, 4096, 512) as p:
        want = p.forward(x, None, w)
        p.forward(x, None, w, stream=s)
        with torch.cuda.stream(s):
            torch.cuda._sleep(0)
        torch.cuda.synchronize()

        def first():
            with torch.cuda.stream(s):
                torch.cuda._sleep(400 * CYCLES_PER_MS)
                p.forward(x, None, w)
            queued.set()
            over.wait()  # (a thread's stream ends with it)

        t = threading.Thread(target=first)
        t.start()
        queued.wait()
        try:
            got = p.forward(x, None, w, stream=s)
            done = torch.cuda.Event()
            done.record(s)
            time.sleep(0.05)
            early = done.query()
            torch.cuda.synchronize()
        finally:
            over.set()
            t.join()
        assert not early
        assert torch.equal(got, want) and p.status() == B_.OK


def test_a_run_behind_its_own_stream_and_a_reset():
    x, w = _split_product()
    s = torch.cuda.Stream()
    with moe.Experts(1, 4096, 512) as p:
        want = p.forward(x, None, w)
        for stream in (s, None, s):
            p.reset(stream)
            got = [p.forward(x, None, w, stream=s) for _ in range(3)] + [p.forward(x, None, w)]
            torch.cuda.synchronize()
            assert p.status() == B_.OK and all(torch.equal(g, want) for g in got)


def test_branches_of_a_captured_graph_are_ordered():
    """Two streams of one capture run products that share the plan's workspace."""
    x, w = _split_product()
    xs = [x, x * 2, x * 3, x * 4]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with moe.Experts(1, 4096, 512) as p:
        want = [p.forward(t, None, w) for t in xs]
        torch.cuda.synchronize()
        for _ in range(2):  # (a second capture knows nothing of the first one's events)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=a):
                b.wait_stream(a)
                got = [p.forward(t, None, w, stream=s) for t, s in zip(xs, (a, b, a, b))]
                a.wait_stream(b)
            for _ in range(20):
                for t in got:
                    t.zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(g, t) for g, t in zip(got, want))
        assert all(torch.equal(p.forward(t, None, w), y) for t, y in zip(xs, want))
        assert p.status() == B_.OK


def test_a_reset_comes_before_later_runs_on_any_stream():
    x, w = randn(rng(1), (20, 64), torch.float16), randn(rng(2), (3, 64, 64), torch.float16)
    bad = torch.tensor([0, 10, 5, 20], dtype=torch.int32, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with moe.Experts(3, 64, 64, "f16") as p:
        for wait_ms in (0, 300):
            p.reset()
            assert p.status() == B_.OK
            with torch.cuda.stream(a):
                torch.cuda._sleep(wait_ms * CYCLES_PER_MS)
            p.reset(a)
            p.forward(x, bad, w, stream=b)  # this run's status is newer than the reset
            torch.cuda.synchronize()
            assert p.status() == B_.ERR_INVALID
