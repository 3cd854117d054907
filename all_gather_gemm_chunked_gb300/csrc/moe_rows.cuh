// moe_rows.cuh -- launchers of the router and of the kernels that move rows
// between tokens and experts (moe_rows.cu), and of the 8-bit quantisation
// (fp8_quant.cu).  Arguments as in ag_moe.h, checked by the caller.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace agg {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kScaleBlock = 128;
enum ElemType : int { kTypeF16 = 0, kTypeBf16 = 2, kTypeF32 = 3, kTypeE4m3 = 4 };

// Programmatic dependent launch: a kernel of this library may start while the kernel
// before it in the stream is still running (launch latency and set-up overlap it) and
// waits for that one's end, and its writes, before it touches global memory.  Inputs may
// be what that kernel writes, so they are read with plain loads: __ldg, or __restrict__ on
// an input, would promise the compiler that they do not change while the kernel runs, and
// let it move loads to before the wait.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// First in every kernel that touches global memory at once.
__device__ __forceinline__ void pdl_enter() {
  pdl_trigger();
  pdl_wait();
}

// A launch with that attribute.  Its own error is returned (cudaGetLastError would also
// return an earlier one's).
inline cudaError_t launch_args(const void* kernel, dim3 grid, int threads, size_t smem,
                               cudaStream_t stream, void** args, int cluster = 1) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  return [&](P... p) {
    void* list[] = {static_cast<void*>(&p)...};
    return launch_args(reinterpret_cast<const void*>(kernel), grid, threads, 0, stream, list);
  }(static_cast<P>(args)...);
}

struct RouteArgs {
  const void* logits;
  int64_t T, ld;
  int E, k, dtype, normalize;
  float* weights;
  int32_t* experts;
  int32_t* offsets;
  int32_t* order;
  int32_t* slots;
  int32_t* counts;  // [blocks][E], of more than one block
};
int route_blocks(int64_t T, int k);
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteArgs& a, const float* dweights, void* dlogits,
                                  cudaStream_t stream);

cudaError_t launch_gather(int64_t T, int k, int64_t H, int dtype, const void* x, int64_t ldx,
                          const int32_t* order, void* out, cudaStream_t stream);
cudaError_t launch_combine(int64_t T, int k, int64_t H, int dtype, const void* y, int64_t ldy,
                           const int32_t* slots, const float* weights, void* out,
                           cudaStream_t stream);
cudaError_t launch_combine_backward(int64_t T, int k, int64_t H, int dtype, const void* dout,
                                    int64_t ldd, const void* y, int64_t ldy, const int32_t* slots,
                                    const float* weights, const int32_t* offsets_end, void* dy,
                                    float* dweights, cudaStream_t stream);

cudaError_t launch_quantize_rows(int64_t rows, int64_t K, int dtype, const void* x, int64_t ldx,
                                 int64_t src_rows, const int32_t* order, int k, void* q,
                                 float* scales, cudaStream_t stream);
cudaError_t launch_quantize_weights(int E, int64_t K, int64_t N, int dtype, const void* w,
                                    void* q, float* scales, cudaStream_t stream);

}  // namespace agg
