"""AllGather+GEMM plans and streams: a new plan's cleared counters, runs from several
threads' default streams."""
import threading
import time

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import binding as B_  # noqa: E402
from all_gather_gemm_chunked_gb300.plan import Plan  # noqa: E402

CYCLES_PER_MS = 2_000_000  # at about 2 GHz
PER_THREAD = 2             # the handle of a host thread's own default stream


def _problem(M=512, K=256, N=256):
    g = torch.Generator(device="cuda").manual_seed(5)
    a = torch.randint(-3, 4, (M, K), generator=g, device="cuda").half()  # exact sums
    b = torch.randint(-3, 4, (K, N), generator=g, device="cuda").half()
    return list(a.chunk(2)), b, (a.double() @ b.double()).float()


def test_a_new_plan_is_clean_on_any_stream():
    """Work waits on the default stream while a plan is made and used on a stream that does
    not wait for it: the counters are clear before the first run, and stay after it."""
    shards, b, want = _problem()
    s = torch.cuda.Stream()
    for wait_ms in (0, 300):  # (the first time loads the kernels, which waits for the device)
        torch.cuda.synchronize()
        torch.cuda._sleep(wait_ms * CYCLES_PER_MS)
        with Plan(2, 512, 256, 256) as p, torch.cuda.stream(s):
            first = p.run(shards, b)
            s.synchronize()
            torch.cuda.synchronize()
            second = p.run(shards, b)
            s.synchronize()
            assert p.status() == B_.OK
        assert torch.equal(first, want) and torch.equal(second, want)


def test_runs_on_two_threads_default_streams_are_ordered():
    """The per-thread default stream has one handle in every thread, but is not one stream."""
    shards, b, want = _problem()
    s = torch.cuda.ExternalStream(PER_THREAD)
    queued, over = threading.Event(), threading.Event()
    with Plan(2, 512, 256, 256) as p:
        with torch.cuda.stream(s):
            p.run(shards, b)
            torch.cuda._sleep(0)
        torch.cuda.synchronize()
        got = []

        def first():
            with torch.cuda.stream(s):
                torch.cuda._sleep(400 * CYCLES_PER_MS)
                got.append(p.run(shards, b))
            queued.set()
            over.wait()  # (a thread's stream ends with it)

        t = threading.Thread(target=first)
        t.start()
        queued.wait()
        try:
            with torch.cuda.stream(s):
                got.append(p.run(shards, b))
                done = torch.cuda.Event()
                done.record(s)
            time.sleep(0.05)
            early = done.query()
            torch.cuda.synchronize()
        finally:
            over.set()
            t.join()
        assert not early and p.status() == B_.OK
        assert all(torch.equal(c, want) for c in got)


def test_a_run_in_a_cuda_graph():
    """A run behind another on the capturing stream, captured and replayed once."""
    shards, b, want = _problem()
    s = torch.cuda.Stream()
    out = torch.empty_like(want)
    for mode in (B_.MODE_PIPELINED, B_.MODE_COMPUTE_ONLY):
        with Plan(2, 512, 256, 256) as p:
            with torch.cuda.stream(s):
                p.run(shards, b, out)
            torch.cuda.synchronize()
            p.set_mode(mode)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                p.run(shards, b, out)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
