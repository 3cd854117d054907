// host.cu -- the thread's last error, the log and TMA descriptor encoding.
#include "host.h"

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "ag_gemm.h"

namespace {
thread_local int g_last_error = AG_GEMM_OK;
thread_local char g_last_msg[512] = "";

void log_line(int level, const char* fmt, va_list ap) {
  if (agg::log_level() < level) return;
  char buf[640];
  vsnprintf(buf, sizeof(buf), fmt, ap);
  std::fprintf(stderr, "[ag_gemm] %s\n", buf);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}
}  // namespace

namespace agg {

int log_level() {
  static const int level = [] {
    const char* v = std::getenv("AG_GEMM_LOG");
    if (!v || !*v) return 0;
    const int l = std::atoi(v);
    return l < 0 ? 0 : (l > 3 ? 3 : l);
  }();
  return level;
}

void log_msg(int level, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  log_line(level, fmt, ap);
  va_end(ap);
}

int fail(int code, const char* fmt, ...) {
  g_last_error = code;
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_msg, sizeof(g_last_msg), fmt, ap);
  va_end(ap);
  log_msg(1, "error %d: %s", code, g_last_msg);
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(e == cudaErrorMemoryAllocation ? AG_GEMM_ERR_OOM : AG_GEMM_ERR_CUDA, "%s: %s",
              what, cudaGetErrorString(e));
}

int last_error() { return g_last_error; }
const char* last_error_message() { return g_last_msg; }

int encode_tiled(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank,
                 const cuuint64_t* dims, const cuuint64_t* strides_bytes, const cuuint32_t* box,
                 CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(AG_GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, type, static_cast<cuuint32_t>(rank),
                  const_cast<void*>(base), dims, strides_bytes, box, estride,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(AG_GEMM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return AG_GEMM_OK;
}

}  // namespace agg
