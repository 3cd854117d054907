// checks.h -- argument checks that the host sides of ag_moe.h and ag_layer.h share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ag_gemm.h"
#include "ag_moe.h"
#include "host.h"

namespace agg {

constexpr int64_t kMaxRowLen = 1LL << 24;  // columns of a row (grid limit)

inline bool float_type(int dtype) {
  return dtype == AG_GEMM_F16 || dtype == AG_GEMM_BF16 || dtype == AG_MOE_F32;
}
inline int esize(int dtype) { return dtype == AG_MOE_F32 ? 4 : dtype == AG_MOE_E4M3 ? 1 : 2; }

inline int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? AG_GEMM_OK : cuda_fail(e, what);
}

// A matrix that is read or written in pieces of 16 bytes.
inline int check_matrix(const char* name, const void* p, int64_t ld, int64_t cols, int dtype) {
  if (!p) return fail(AG_GEMM_ERR_INVALID, "%s is NULL", name);
  if (!aligned16(p)) return fail(AG_GEMM_ERR_INVALID, "%s must be 16-byte aligned", name);
  if (ld < cols || ld * esize(dtype) % 16 != 0)
    return fail(AG_GEMM_ERR_INVALID, "%s: row pitch %lld must be at least %lld and a multiple of 16 bytes",
                name, (long long)ld, (long long)cols);
  if (ld >= (1LL << 36)) return fail(AG_GEMM_ERR_UNSUPPORTED, "%s: row pitch too large", name);
  return AG_GEMM_OK;
}

}  // namespace agg
