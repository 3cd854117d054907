// fp4_quant.cu -- microscaled e2m1 operands (fp4_codes.cuh) of rows and of weights.

#include "fp4_codes.cuh"
#include "layer_rows.cuh"

namespace agg {

namespace {
// The largest magnitude's bits as a float; of 16-bit elements two at a time, whose bits
// order as the magnitudes do.
template <typename T, int V>
__device__ __forceinline__ uint32_t largest_of(const Piece<T, V>& p) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) m = max(m, p.w[v] & 0x7fffffffu);
    return m;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < Piece<T, V>::kWords; ++i) m = __vmaxu2(m, p.w[i] & 0x7fff7fffu);
    const uint16_t one = static_cast<uint16_t>(max(m & 0xffffu, m >> 16));
    return __float_as_uint(Elem<T>::get(reinterpret_cast<const T&>(one)));
  }
}

// Bound by memory (2 bytes in, a little above half a byte out per element).  A warp takes
// 256 elements of a row per step, 8 per lane: 4 lanes make one block, whose maximum takes
// two shuffles, and 16 lanes the word of four scales.  All of a lane's loads are issued
// before the first use.  The eight warps of a block take eight neighbouring rows, so that
// the words they write ([K / 128][row]) fill 32-byte sectors.  (8192 x 4096 bf16: 13.5 us, 6.3 TB/s.)
template <typename T, int kSteps>
__global__ void __launch_bounds__(256) quantize_rows4_kernel(int64_t rows, int64_t K, const T* x, int64_t ldx,
                                                             int64_t src_rows, const int32_t* order, int k,
                                                             uint8_t* __restrict__ q, uint32_t* __restrict__ scales) {
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
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (256 * kSteps) + lane * 8;
  const int left = static_cast<int>(K - c0);  // (K % 32 == 0: a lane's 8 elements are all in or all out)
  const T* from = x + src * ldx + c0;
  Piece<T, V> p[kSteps][8 / V];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
#pragma unroll
    for (int h = 0; h < 8 / V; ++h) {
      p[i][h] = Piece<T, V>{};
      if (in && i * 256 < left) p[i][h].load(from + i * 256 + h * V);
    }
  }
  uint32_t* const codes = reinterpret_cast<uint32_t*>(q + (r * K + c0) / 2);
  uint32_t* words = scales + (c0 / kScaleBlock) * rows + r;
#pragma unroll
  for (int i = 0; i < kSteps; ++i, words += 2 * rows) {
    if (i * 256 >= left + lane * 8) break;  // (all of the warp)
    float g[8];
    uint32_t largest = 0;
#pragma unroll
    for (int h = 0; h < 8 / V; ++h) {
      float f[V];
      p[i][h].get(f);
#pragma unroll
      for (int v = 0; v < V; ++v) g[h * V + v] = f[v];
      largest = max(largest, largest_of(p[i][h]));
    }
    largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
    largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
    const uint32_t s = micro_scale(largest);
    const float inv = micro_inverse(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= inv;
    uint32_t word = s << ((lane >> 2 & 3) * 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (i * 256 < left) {
      codes[i * 32] = e2m1x8(g);
      if ((lane & 15) == 0) *words = word;
    }
  }
}

// Two neighbouring elements as floats.
template <typename T>
__device__ __forceinline__ float2 load_two(const T* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  const T* v = reinterpret_cast<const T*>(&u);
  return make_float2(Elem<T>::get(v[0]), Elem<T>::get(v[1]));
}
template <>
__device__ __forceinline__ float2 load_two<float>(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}

// One block per 128 x 128 block of an expert's weights (done once per model): a thread
// holds one block of 32 along K of two columns, all its loads in flight, and writes their
// 16 bytes of codes each; the four threads of a column write 64 neighbouring bytes.  (32 x
// 4096 x 4096 bf16 275 us, 4.9 TB/s; 16384 x 7168 69; 4096 x 4096 17, of floats 23: a block's stores
// lie K / 2 bytes apart, column by column.)
template <typename T>
__global__ void __launch_bounds__(256) quantize_weights4_kernel(int64_t K, int64_t N, const T* w,
                                                                uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  pdl_enter();
  const int64_t KB = (K + kScaleBlock - 1) / kScaleBlock, NB = (N + kScaleBlock - 1) / kScaleBlock;
  const int64_t kb = blockIdx.x % KB, nb = (blockIdx.x / KB) % NB, e = blockIdx.x / (KB * NB);
  const int col = (threadIdx.x & 63) * 2, part = threadIdx.x >> 6;
  const int64_t n = nb * kScaleBlock + col, k0 = kb * kScaleBlock + part * kMicroBlock;
  const bool in = n < N && k0 < K;  // (N is even, K a multiple of 32: all of both columns' blocks, or nothing)
  float v[2][kMicroBlock];
#pragma unroll
  for (int i = 0; i < kMicroBlock; ++i) {
    float2 f = make_float2(0.0f, 0.0f);
    if (in) f = load_two(w + (e * K + k0 + i) * N + n);
    v[0][i] = f.x;
    v[1][i] = f.y;
  }
  uint8_t* piece = scales + ((e * NB + nb) * KB + kb) * 512 + part;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t largest = 0;
#pragma unroll
    for (int i = 0; i < kMicroBlock; ++i) largest = max(largest, magnitude_bits(v[h][i]));
    const uint32_t s = micro_scale(largest);
    const float inv = micro_inverse(s);
    uint32_t word[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = v[h][8 * j + i] * inv;
      word[j] = e2m1x8(g);
    }
    if (in) *reinterpret_cast<uint4*>(q + ((e * N + n + h) * K + k0) / 2) = make_uint4(word[0], word[1], word[2], word[3]);
    const int c = col + h;
    piece[(c & 31) * 16 + (c >> 5) * 4] = static_cast<uint8_t>(s);
  }
}
}  // namespace

cudaError_t launch_quantize_rows4(int64_t rows, int64_t K, int dtype, const void* x, int64_t ldx,
                                  int64_t src_rows, const int32_t* order, int k, void* q,
                                  void* scales, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  // Eight steps of 256 elements a warp where that leaves work for every SM, else one.  (bf16, one
  // step and eight: 1024 x 4096 3.5 us and 4.5, 2048 x 4096 6.2 and 6.2, 8192 x 1024 6.1 and 5.4,
  // 8192 x 4096 18.7 and 13.5.)
  const int steps = rows * K >= int64_t{152} * 8 * 6144 && K >= 1024 ? 8 : 1;
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8), static_cast<unsigned>((K + 256 * steps - 1) / (256 * steps)));
  auto go = [&](auto t) {
    using T = decltype(t);
    return launch(steps == 8 ? quantize_rows4_kernel<T, 8> : quantize_rows4_kernel<T, 1>, grid, 256, stream, rows, K,
                  static_cast<const T*>(x), ldx, src_rows, order, k, static_cast<uint8_t*>(q),
                  static_cast<uint32_t*>(scales));
  };
  return dtype == kTypeF32 ? go(float{}) : dtype == kTypeF16 ? go(__half{}) : go(__nv_bfloat16{});
}

cudaError_t launch_quantize_weights4(int E, int64_t K, int64_t N, int dtype, const void* w, void* q,
                                     void* scales, cudaStream_t stream) {
  const int64_t blocks = E * ((K + kScaleBlock - 1) / kScaleBlock) * ((N + kScaleBlock - 1) / kScaleBlock);
  const unsigned grid = static_cast<unsigned>(blocks);
  uint8_t *out = static_cast<uint8_t*>(q), *bytes = static_cast<uint8_t*>(scales);
  if (dtype == kTypeF32)
    return launch(quantize_weights4_kernel<float>, dim3(grid), 256, stream, K, N, static_cast<const float*>(w), out, bytes);
  if (dtype == kTypeF16)
    return launch(quantize_weights4_kernel<__half>, dim3(grid), 256, stream, K, N, static_cast<const __half*>(w), out, bytes);
  return launch(quantize_weights4_kernel<__nv_bfloat16>, dim3(grid), 256, stream, K, N,
                static_cast<const __nv_bfloat16*>(w), out, bytes);
}

}  // namespace agg
