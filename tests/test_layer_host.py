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
    assert len(names) >= 10
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


def test_norm_calls_refused(B):
    lib, p = B.library_handle(), 1 << 20

    def forward(rows=4, H=64, dtype=0, x=p, ld=64, res=None, ldr=64, w=p, wt=0, eps=1e-6, y=p, h=None, rstd=None):
        return lib.ag_norm_rms(rows, H, dtype, x, ld, res, ldr, w, wt, eps, y, h, rstd, None)

    for bad in (dict(dtype=1), dict(dtype=4), dict(rows=-1), dict(H=0), dict(x=None), dict(w=None), dict(y=None), dict(ld=63),
                dict(res=p), dict(res=p, h=p, ldr=63), dict(wt=2), dict(wt=1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(rows=0, eps=-1.0)):
        assert forward(**bad) == B.ERR_INVALID, bad
    assert forward(rows=1 << 31) == forward(H=(1 << 24) + 1, ld=1 << 25) == forward(ld=1 << 36) == B.ERR_UNSUPPORTED
    assert forward(rows=0, x=None, y=None) == B.OK

    def codes(rows=4, H=64, dtype=0, x=p, ld=64, res=None, ldr=64, w=p, wt=0, eps=1e-6, code=4, q=p, s=p, h=None):
        return lib.ag_norm_rms_quantized(rows, H, dtype, x, ld, res, ldr, w, wt, eps, code, q, s, h, None)

    for bad in (dict(code=0), dict(code=3), dict(code=6), dict(H=24, ld=24), dict(H=48, ld=48, code=5), dict(q=None), dict(s=None),
                dict(q=p + 8), dict(s=p + 4), dict(x=p + 8), dict(ld=68), dict(w=p + 8), dict(res=p, h=p + 8), dict(res=p + 8, h=p),
                dict(res=p, h=p, ldr=68)):
        assert codes(**bad) == B.ERR_INVALID, bad
    assert codes(rows=0, x=None) == B.OK

    def backward(rows=4, H=64, dtype=0, dy=p, lddy=64, h=p, ldh=64, w=p, wt=0, rstd=p, dh=None, lddh=64, dx=p, dw=p, ws=p):
        return lib.ag_norm_rms_backward(rows, H, dtype, dy, lddy, h, ldh, w, wt, rstd, dh, lddh, dx, dw, ws, None)

    for bad in (dict(dtype=1), dict(rows=-1), dict(H=0), dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(dx=None),
                dict(dw=None), dict(ws=None), dict(ws=p + 4), dict(lddy=63), dict(ldh=63), dict(dh=p, lddh=63), dict(wt=2)):
        assert backward(**bad) == B.ERR_INVALID, bad
    assert B.ag_norm_rms_backward_workspace(0, 64) == 0
    assert B.ag_norm_rms_backward_workspace(5, 64) == 5 * 64 * 4
    assert B.ag_norm_rms_backward_workspace(1 << 20, 4096) == 304 * 4096 * 4
    assert lib.ag_norm_rms_backward_workspace(-1, 64) == B.ERR_INVALID


def test_activation_calls_refused(B):
    lib, p = B.library_handle(), 1 << 20
    forward = lambda rows=4, N=32, dtype=0, x=p, ld=64, y=p: lib.ag_act_swiglu(rows, N, dtype, x, ld, y, None)  # noqa: E731
    for bad in (dict(dtype=1), dict(rows=-1), dict(N=0), dict(x=None), dict(y=None), dict(ld=63)):
        assert forward(**bad) == B.ERR_INVALID, bad
    assert forward(rows=1 << 31) == forward(N=(1 << 24) + 1, ld=1 << 26) == B.ERR_UNSUPPORTED
    assert forward(rows=0, x=None) == B.OK
    codes = lambda rows=4, N=32, dtype=0, x=p, ld=64, code=4, q=p, s=p: (  # noqa: E731
        lib.ag_act_swiglu_quantized(rows, N, dtype, x, ld, code, q, s, None))
    for bad in (dict(code=3), dict(N=24), dict(N=48, ld=96, code=5), dict(q=None), dict(s=p + 4), dict(x=p + 8), dict(ld=68), dict(ld=56)):
        assert codes(**bad) == B.ERR_INVALID, bad
    backward = lambda rows=4, N=32, dtype=0, dy=p, lddy=32, x=p, ld=64, dx=p: (  # noqa: E731
        lib.ag_act_swiglu_backward(rows, N, dtype, dy, lddy, x, ld, dx, None))
    for bad in (dict(dtype=1), dict(dy=None), dict(x=None), dict(dx=None), dict(lddy=31), dict(ld=63), dict(N=0)):
        assert backward(**bad) == B.ERR_INVALID, bad
    assert backward(rows=0, dy=None) == B.OK
