// fp8_quant.cu -- e4m3 operands with one scale per 128 elements (rows) or per
// 128 x 128 block (weights):  s = max(amax / 448, 2^-126),  q = e4m3(x * (1 / s)),
// each of the three rounded to float.  The floor 2^-126 keeps 1 / s finite, so a
// block of zeros gets codes 0; an infinity makes its own code NaN (inf * 0) and a
// NaN stays NaN.

#include "moe_rows.cuh"
#include "moe_types.cuh"

namespace agg {

namespace {
// Bound by memory (2 bytes in, 1 out per element).  A warp takes 256 elements of
// a row per step, 8 per lane: 16 lanes make one scale block, whose maximum takes
// four shuffles.  All of a lane's loads are issued before the first use.  The
// eight warps of a block take eight neighbouring rows, so that the scales they
// write ([K block][row]) fill 32-byte sectors.  (32768 rows of 4096, bf16: 69 us,
// 5.9 TB/s; 64 rows of 16384: 2.3 us.)
constexpr int kQuantSteps = 4;
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(int64_t rows, int64_t K,
                                                            const T* x, int64_t ldx,
                                                            int64_t src_rows,
                                                            const int32_t* order,
                                                            int k, uint8_t* __restrict__ q,
                                                            float* __restrict__ scales) {
  pdl_enter();
  constexpr int V = Elem<T>::kVec;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  if (r >= rows) return;
  int64_t src = r;
  bool in = true;
  if (order) {
    const int32_t o = order[r];
    src = o / k;
    in = o >= 0;
  }
  in = in && src < src_rows;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (256 * kQuantSteps) + lane * 8;
  float f[kQuantSteps][8 / V][V];
#pragma unroll
  for (int i = 0; i < kQuantSteps; ++i) {
    const int64_t c = c0 + i * 256;  // (K % 16 == 0: a lane's 8 elements are all in or all out)
#pragma unroll
    for (int h = 0; h < 8 / V; ++h) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[i][h][v] = 0.0f;
      if (in && c < K) load_elems<T, V>(x + src * ldx + c + h * V, f[i][h]);
    }
  }
#pragma unroll
  for (int i = 0; i < kQuantSteps; ++i) {
    const int64_t c = c0 + i * 256;
    float amax = 0.0f;
#pragma unroll
    for (int h = 0; h < 8 / V; ++h)
#pragma unroll
      for (int v = 0; v < V; ++v) amax = fmaxf(amax, fabsf(f[i][h][v]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = block_scale(amax), inv = __frcp_rn(s);
    if (c < K) {
      uint32_t w[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float a0 = f[i][(4 * b) / V][(4 * b) % V], a1 = f[i][(4 * b + 1) / V][(4 * b + 1) % V];
        const float a2 = f[i][(4 * b + 2) / V][(4 * b + 2) % V], a3 = f[i][(4 * b + 3) / V][(4 * b + 3) % V];
        w[b] = e4m3x2(__fmul_rn(a0, inv), __fmul_rn(a1, inv)) |
               (e4m3x2(__fmul_rn(a2, inv), __fmul_rn(a3, inv)) << 16);
      }
      *reinterpret_cast<uint2*>(q + r * K + c) = make_uint2(w[0], w[1]);
      if ((lane & 15) == 0) scales[(c / kScaleBlock) * rows + r] = s;
    }
  }
}

// Two neighbouring elements, and as floats.
template <typename T>
struct Two {
  uint32_t u;
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ float2 get() const {
    const T* v = reinterpret_cast<const T*>(&u);
    return make_float2(Elem<T>::get(v[0]), Elem<T>::get(v[1]));
  }
};
template <>
struct Two<float> {
  float2 u;
  __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ float2 get() const { return u; }
};

// One block per 128 x 128 block of an expert's weights (done once per model): a thread
// holds two columns of 32 rows in registers, all its loads in flight; maximum, then the
// codes transposed through shared memory.  Bound by memory
// (16 x 4096 x 4096 bf16: 201 us, 4.0 TB/s).
constexpr int kTilePitch = kScaleBlock + 4;
template <typename T>
__global__ void __launch_bounds__(256) quantize_weights_kernel(int64_t K, int64_t N,
                                                               const T* w,
                                                               uint8_t* __restrict__ q,
                                                               float* __restrict__ scales) {
  pdl_enter();
  __shared__ __align__(16) uint8_t tile[kScaleBlock][kTilePitch];
  __shared__ float red[8];
  const int64_t KB = (K + kScaleBlock - 1) / kScaleBlock, NB = (N + kScaleBlock - 1) / kScaleBlock;
  const int64_t kb = blockIdx.x % KB, nb = (blockIdx.x / KB) % NB, e = blockIdx.x / (KB * NB);
  const int col = (threadIdx.x & 63) * 2, row0 = (threadIdx.x >> 6) * 32;
  const int64_t n = nb * kScaleBlock + col;  // (N is even: both columns are there, or none)
  const T* src = w + (e * K + kb * kScaleBlock + row0) * N + n;
  const int rows = static_cast<int>(K - kb * kScaleBlock < kScaleBlock ? K - kb * kScaleBlock : kScaleBlock);
  Two<T> v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = Two<T>{};
    if (n < N && row0 + i < rows) v[i].load(src + i * N);
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float2 f = v[i].get();
    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, red[i]);
  const float s = block_scale(amax), inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    float2 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = v[i + j].get();
      f[j].x = __fmul_rn(f[j].x, inv);
      f[j].y = __fmul_rn(f[j].y, inv);
    }
    *reinterpret_cast<uint32_t*>(&tile[col][row0 + i]) = e4m3x2(f[0].x, f[1].x) | (e4m3x2(f[2].x, f[3].x) << 16);
    *reinterpret_cast<uint32_t*>(&tile[col + 1][row0 + i]) = e4m3x2(f[0].y, f[1].y) | (e4m3x2(f[2].y, f[3].y) << 16);
  }
  if (threadIdx.x == 0) scales[(e * NB + nb) * KB + kb] = s;
  __syncthreads();
  // rows n of q: 128 codes along K, 4 per thread and step
#pragma unroll
  for (int i = threadIdx.x; i < kScaleBlock * (kScaleBlock / 4); i += 256) {
    const int row = i >> 5, c = (i & 31) * 4;
    const int64_t nn = nb * kScaleBlock + row;
    if (nn < N && c < rows)
      *reinterpret_cast<uint32_t*>(q + (e * N + nn) * K + kb * kScaleBlock + c) =
          *reinterpret_cast<const uint32_t*>(&tile[row][c]);
  }
}
}  // namespace

cudaError_t launch_quantize_rows(int64_t rows, int64_t K, int dtype, const void* x, int64_t ldx,
                                 int64_t src_rows, const int32_t* order, int k, void* q,
                                 float* scales, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8),
                  static_cast<unsigned>((K + 256 * kQuantSteps - 1) / (256 * kQuantSteps)));
  uint8_t* out = static_cast<uint8_t*>(q);
  if (dtype == kTypeF32)
    return launch(quantize_rows_kernel<float>, dim3(grid), 256, stream, 
        rows, K, static_cast<const float*>(x), ldx, src_rows, order, k, out, scales);
  else if (dtype == kTypeF16)
    return launch(quantize_rows_kernel<__half>, dim3(grid), 256, stream, 
        rows, K, static_cast<const __half*>(x), ldx, src_rows, order, k, out, scales);
  else
    return launch(quantize_rows_kernel<__nv_bfloat16>, dim3(grid), 256, stream, 
        rows, K, static_cast<const __nv_bfloat16*>(x), ldx, src_rows, order, k, out, scales);
}

cudaError_t launch_quantize_weights(int E, int64_t K, int64_t N, int dtype, const void* w,
                                    void* q, float* scales, cudaStream_t stream) {
  const int64_t blocks = E * ((K + kScaleBlock - 1) / kScaleBlock) * ((N + kScaleBlock - 1) / kScaleBlock);
  uint8_t* out = static_cast<uint8_t*>(q);
  const unsigned grid = static_cast<unsigned>(blocks);
  if (dtype == kTypeF32)
    return launch(quantize_weights_kernel<float>, dim3(grid), 256, stream, K, N, static_cast<const float*>(w), out, scales);
  else if (dtype == kTypeF16)
    return launch(quantize_weights_kernel<__half>, dim3(grid), 256, stream, K, N, static_cast<const __half*>(w), out, scales);
  else
    return launch(quantize_weights_kernel<__nv_bfloat16>, dim3(grid), 256, stream, 
        K, N, static_cast<const __nv_bfloat16*>(w), out, scales);
}

}  // namespace agg
