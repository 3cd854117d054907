"""ag_moe.h without a GPU: exports, argument checks that come before any CUDA call."""
import subprocess

import pytest

from all_gather_gemm_chunked_gb300 import build as _build


@pytest.fixture(scope="module")
def B():
    _build.build()
    from all_gather_gemm_chunked_gb300 import binding
    return binding


def test_library_exports_every_header_function(B):
    names = B.header_functions(B.HEADER_MOE)
    assert len(names) >= 18
    out = subprocess.run(["nm", "-D", "--defined-only", _build.LIB], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported


@pytest.mark.parametrize("T,E,k,code", [(4, 0, 1, -1), (4, 1025, 1, -1), (4, 8, 0, -1), (4, 8, 9, -1), (4, 64, 33, -1),
                                        (-1, 8, 2, -1), ((1 << 28) + 1, 8, 2, -2), (1 << 27, 64, 16, -2)])
def test_route_sizes_refused(B, T, E, k, code):
    with pytest.raises(B.AgGemmError) as e:
        B.ag_moe_route_workspace(T, E, k)
    assert e.value.code == code and e.value.message


def test_route_workspace(B):
    assert B.ag_moe_route_workspace(0, 8, 2) == 0
    assert B.ag_moe_route_workspace(1 << 20, 64, 2) == 152 * 64 * 4


@pytest.mark.parametrize("args", [(0, 64, 64, 0), (1025, 64, 64, 0), (2, 60, 64, 0), (2, 64, 60, 2), (2, 24, 64, 4),
                                  (2, 64, 64, 1), (2, 64, 64, 3), (1, 1 << 25, 64, 0)])
def test_plan_refused(B, args):
    with pytest.raises(B.AgGemmError) as e:
        B.ag_moe_plan_create(*args)
    assert e.value.code == B.ERR_INVALID


def test_null_plan_is_rejected(B):
    lib = B.library_handle()
    assert lib.ag_moe_plan_status(None) == B.ERR_INVALID
    assert lib.ag_moe_plan_reset(None, None) == B.ERR_INVALID
    assert lib.ag_moe_forward(None, 1, None, 0, None, None, 0, 0, None, 0, 0, None) == B.ERR_INVALID
    assert lib.ag_moe_backward_weight(None, 1, None, 0, None, 0, None, None, 0, None) == B.ERR_INVALID
    assert lib.ag_fp8_forward(None, 1, None, None, None, None, None, None, 0, 0, None) == B.ERR_INVALID
    lib.ag_moe_plan_destroy(None)


def test_null_pointers_are_rejected(B):
    lib = B.library_handle()
    assert lib.ag_moe_gather(4, 2, 16, 0, None, 16, None, None, None) == B.ERR_INVALID
    assert lib.ag_moe_combine(4, 2, 16, 0, None, 16, None, None, None, None) == B.ERR_INVALID
    assert lib.ag_fp8_quantize_rows(4, 16, 0, None, 16, 4, None, 1, None, None, None) == B.ERR_INVALID
    assert lib.ag_fp8_quantize_weights(1, 16, 8, 0, None, None, None, None) == B.ERR_INVALID
    assert lib.ag_fp8_quantize_weights(1, 24, 8, 0, None, None, None, None) == B.ERR_INVALID
