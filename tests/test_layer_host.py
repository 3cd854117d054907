"""ag_layer.h without a GPU: exports, argument checks that come before any CUDA call."""
import subprocess

import pytest

from all_gather_gemm_chunked_gb300 import build as _build


@pytest.fixture(scope="module")
def B():
    _build.build()
    from all_gather_gemm_chunked_gb300 import binding
    return binding


def test_library_exports_every_header_function(B):
    names = B.header_functions(B.HEADER_LAYER)
    assert len(names) >= 3
    out = subprocess.run(["nm", "-D", "--defined-only", _build.LIB], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported
    for name in names:
        assert callable(getattr(B, name)), name


@pytest.mark.parametrize("args", [(2, 48, 64, 5), (2, 0, 64, 5), (2, 64, 60, 5), (0, 64, 64, 5), (1, 1 << 25, 64, 5), (2, 64, 64, 6)])
def test_fp4_plan_refused(B, args):
    with pytest.raises(B.AgGemmError) as e:
        B.ag_moe_plan_create(*args)
    assert e.value.code == B.ERR_INVALID


def test_fp4_calls_refused(B):
    lib, p = B.library_handle(), 1 << 20  # (a pointer that is checked and not followed)
    rows = lambda rows=4, K=64, dtype=0, x=p, ld=64, src=4, order=None, k=1, q=p, s=p: (  # noqa: E731
        lib.ag_fp4_quantize_rows(rows, K, dtype, x, ld, src, order, k, q, s, None))
    for bad in (dict(dtype=1), dict(dtype=4), dict(rows=-1), dict(rows=1 << 31), dict(src=3), dict(K=48), dict(K=0), dict(x=None),
                dict(ld=63), dict(ld=60), dict(x=p + 8), dict(q=None), dict(s=None), dict(q=p + 8), dict(s=p + 4),
                dict(order=p, k=0), dict(order=p, k=33)):
        assert rows(**bad) == B.ERR_INVALID, bad
    assert rows(rows=0, x=None) == B.OK
    weights = lambda E=1, K=64, N=8, dtype=0, w=p, q=p, s=p: lib.ag_fp4_quantize_weights(E, K, N, dtype, w, q, s, None)  # noqa: E731
    for bad in (dict(E=0), dict(E=1025), dict(K=48), dict(N=12), dict(dtype=1), dict(w=None), dict(q=None), dict(s=None),
                dict(w=p + 4), dict(q=p + 8), dict(s=p + 8)):
        assert weights(**bad) == B.ERR_INVALID, bad
    assert weights(E=1024, K=1 << 24, N=1 << 24) == B.ERR_UNSUPPORTED
    assert lib.ag_fp4_forward(None, 1, p, p, None, p, p, p, 8, 0, None) == B.ERR_INVALID
