// host.h -- what the host sides of the library share: the thread's last error,
// the log, TMA descriptor encoding and the current-device guard (host.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace agg {

int log_level();  // AG_GEMM_LOG=0..3 (read once): 1 errors, 2 plans, 3 runs
void log_msg(int level, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Records the thread's last error and returns its code.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int cuda_fail(cudaError_t e, const char* what);
int last_error();
const char* last_error_message();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Tensor of rank 2 to 5, innermost dimension first; zero fill out of bounds.
int encode_tiled(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank,
                 const cuuint64_t* dims, const cuuint64_t* strides_bytes, const cuuint32_t* box,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// Clears a new plan's memory on a stream of its own and waits for that: a memset on the
// default stream would come behind that stream's work, and so perhaps behind (or into) the
// plan's first run on a stream that does not wait for the default one.
class Clearer {
 public:
  Clearer() : e_(cudaStreamCreateWithFlags(&stream_, cudaStreamNonBlocking)) {}
  ~Clearer() {
    if (stream_) cudaStreamDestroy(stream_);
  }
  Clearer(const Clearer&) = delete;
  Clearer& operator=(const Clearer&) = delete;
  cudaError_t clear(void* p, size_t bytes) {
    if (e_ == cudaSuccess && bytes > 0) e_ = cudaMemsetAsync(p, 0, bytes, stream_);
    return e_;
  }
  cudaError_t finish() {
    if (e_ == cudaSuccess) e_ = cudaStreamSynchronize(stream_);
    return e_;
  }

 private:
  cudaStream_t stream_ = nullptr;
  cudaError_t e_;
};

// A stream by the number that no other stream has: one handle stands for every thread's
// own default stream, and a destroyed stream's may be given to a new one while its work is
// pending.  While the stream is captured the number is 0 (to ask for it would end the
// capture), and handles are compared.
struct StreamId {
  cudaStream_t handle = nullptr;
  unsigned long long number = 0;  // plus 1
  StreamId() = default;
  StreamId(cudaStream_t stream, bool captured) : handle(stream) {
    unsigned long long n = 0;
    if (!captured && cudaStreamGetId(stream, &n) == cudaSuccess) number = n + 1;
  }
  bool operator!=(const StreamId& o) const {
    return number && o.number ? number != o.number : handle != o.handle;
  }
};
inline bool is_captured(cudaStream_t stream) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  return cudaStreamIsCapturing(stream, &capture) != cudaSuccess || capture != cudaStreamCaptureStatusNone;
}

// Makes `dev` current; restores the caller's current device on scope exit.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

}  // namespace agg
