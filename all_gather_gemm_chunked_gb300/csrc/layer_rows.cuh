// layer_rows.cuh -- launchers of the norm (norm.cu) and of the gated activation (act.cu),
// and what their kernels share: a row's threads, and outputs as codes with scales.
// Arguments as in ag_layer.h, checked by the caller.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4_codes.cuh"
#include "moe_rows.cuh"
#include "moe_types.cuh"

namespace agg {

struct NormArgs {
  int64_t rows, H;
  const void* x;
  int64_t ldx;
  const void* residual;  // or null
  int64_t ldr;
  const void* weight;
  int weight_f32;        // weights are floats (otherwise the rows' type)
  float eps;
  float inv_H;           // (made by the launcher)
  void* out;             // y, or codes
  void* scales;          // of the codes
  void* h;               // with a residual
  float* rstd;           // or null
};
// out_type: dtype itself, kTypeE4m3 or kTypeE2m1.
cudaError_t launch_norm(NormArgs a, int dtype, int out_type, cudaStream_t stream);

struct NormBackwardArgs {
  int64_t rows, H;
  const void* dy;
  int64_t lddy;
  const void* h;
  int64_t ldh;
  const void* weight;
  int weight_f32;
  const float* rstd;
  const void* dh;  // or null
  int64_t lddh;
  void* dx;
  float* dweight;
  float* parts;    // [norm_parts][H]
};
// Sums of the weight's gradient that are made first and then added.
int64_t norm_parts(int64_t rows);
cudaError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, cudaStream_t stream);

struct GateArgs {
  int64_t rows, N;
  const void* x;   // gate, and N columns on the other factor
  int64_t ldx;
  const void* dy;  // backward
  int64_t lddy;
  void* out;       // y, codes, or the gradient of x
  void* scales;
};
cudaError_t launch_swiglu(const GateArgs& a, int dtype, int out_type, cudaStream_t stream);
cudaError_t launch_swiglu_backward(const GateArgs& a, int dtype, cudaStream_t stream);

#ifdef __CUDACC__
// V neighbouring elements as they lie in memory, 16, 4 or 2 bytes.  (Loads are volatile: in
// the order of the source, behind a launch's wait, and none sinks to its use.)
template <typename T, int V>
struct Piece {
  static constexpr int kBytes = V * static_cast<int>(sizeof(T)), kWords = kBytes < 4 ? 1 : kBytes / 4;
  static_assert(kBytes == 16 || kBytes == 4 || kBytes == 2, "one access");
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 16) {
      asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    } else if constexpr (kBytes == 4) {
      asm volatile("ld.global.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    } else {
      uint16_t h;
      asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p));
      w[0] = h;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 16)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = __uint_as_float(w[v]);
    } else if constexpr (V == 1) {
      const uint16_t h = static_cast<uint16_t>(w[0]);
      f[0] = Elem<T>::get(reinterpret_cast<const T&>(h));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const float2 p = Elem<T>::unpair(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = __float_as_uint(f[v]);
    } else if constexpr (V == 1) {
      const T h = Elem<T>::put(f[0]);
      w[0] = reinterpret_cast<const uint16_t&>(h);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = Elem<T>::pair(f[2 * i], f[2 * i + 1]);
    }
  }
};
template <typename T, int V>
__device__ __forceinline__ void store_floats(T* p, const float (&f)[V]) {
  Piece<T, V> r;
  r.put(f);
  r.store(p);
}

// Places of a row's codes and scales from column c on (their addresses are made once a
// thread: at each piece, in 64 bits, they cost a tenth of the time).
template <int OUT>
struct CodePlace {
  uint8_t* q;
  uint32_t* s;     // of c's 128 elements: an e4m3 scale, or four e2m1 ones
  int64_t blocks;  // from one 128 elements' to the next
  __device__ __forceinline__ CodePlace(void* codes, void* scales, int64_t rows, int64_t H, int64_t row, int64_t c)
      : q(static_cast<uint8_t*>(codes) + (OUT == kTypeE4m3 ? row * H + c : (row * H + c) / 2)),
        s(static_cast<uint32_t*>(scales) + (c / kScaleBlock) * rows + row), blocks(rows) {}
  // n elements on, a multiple of 128
  __device__ __forceinline__ void advance(int n) {
    q += OUT == kTypeE4m3 ? n : n / 2;
    s += n / kScaleBlock * blocks;
  }
};

// V neighbouring elements of a row as codes, by the lanes of a whole warp, which hold V
// elements each, the next lane the next V; past the row (`in` false) they are zeros.  The
// same codes and scales as quantising the floats.
template <int OUT, int V>
__device__ __forceinline__ void put_codes(const CodePlace<OUT>& at, bool in, float (&f)[V]) {
  static_assert(V == 8 || V == 4, "16 bytes of the rows' type");
  const int lane = threadIdx.x & 31;
  constexpr int kLanes = kScaleBlock / V;  // of 128 elements
  if constexpr (OUT == kTypeE4m3) {
    float amax = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) amax = fmaxf(amax, fabsf(f[v]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = block_scale(amax), inv = __frcp_rn(s);
    uint32_t w[V / 4];
#pragma unroll
    for (int b = 0; b < V / 4; ++b)
      w[b] = e4m3x2(__fmul_rn(f[4 * b], inv), __fmul_rn(f[4 * b + 1], inv)) |
             (e4m3x2(__fmul_rn(f[4 * b + 2], inv), __fmul_rn(f[4 * b + 3], inv)) << 16);
    if (!in) return;
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(at.q) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(at.q) = w[0];
    if ((lane & (kLanes - 1)) == 0) *at.s = __float_as_uint(s);
  } else {
    uint32_t largest = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) largest = max(largest, magnitude_bits(f[v]));
#pragma unroll
    for (int o = kMicroBlock / V / 2; o > 0; o >>= 1)
      largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    const uint32_t s = micro_scale(largest);
    const float inv = micro_inverse(s);
    float g[8] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = f[v] * inv;
    const uint32_t code = e2m1x8(g);
    uint32_t word = s << ((lane / (kMicroBlock / V) & 3) * 8);
#pragma unroll
    for (int o = kMicroBlock / V; o < kLanes; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    if (!in) return;
    if constexpr (V == 8)
      *reinterpret_cast<uint32_t*>(at.q) = code;
    else
      *reinterpret_cast<uint16_t*>(at.q) = static_cast<uint16_t>(code);
    if ((lane & (kLanes - 1)) == 0) *at.s = word;
  }
}

// Rows that begin anywhere.  A frame is 16 bytes' worth of elements, V of them; frames lie so
// that those of the output are aligned, and lanes 0 to 30 of a warp have 31 neighbouring ones.
// An operand's elements of a frame lie in two aligned 16-byte pieces: the lane's own, and the
// next lane's (lane 31 has no frame, only a piece).  Pieces that are not all of the row are
// read, and frames written, element by element.
constexpr int kFrames = 31;
// A frame's elements out of two neighbouring pieces, from the d-th on (the same d in all lanes).
template <typename T>
__device__ __forceinline__ Piece<T, 16 / sizeof(T)> from_pieces(uint32_t (&w)[8], int d) {
  const int words = d * static_cast<int>(sizeof(T)) / 4;
  if (words & 2)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (words & 1)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  Piece<T, 16 / sizeof(T)> p;
#pragma unroll
  for (int i = 0; i < 4; ++i) p.w[i] = sizeof(T) == 2 ? __funnelshift_r(w[i], w[i + 1], (d & 1) * 16) : w[i];
  return p;
}
template <typename T>
struct Anywhere {
  static constexpr int V = 16 / sizeof(T);
  const T* row;
  int H, d;  // elements of the row; of a frame's start past an aligned address
  __device__ __forceinline__ Anywhere(const T* row_, int64_t H_, int c)
      : row(row_), H(static_cast<int>(H_)),
        d(static_cast<int>((reinterpret_cast<uintptr_t>(row_ + c) & 15) / sizeof(T))) {}
  // The piece of the frame at column c: all of the row, or made of what is, and zeros.
  __device__ __forceinline__ bool whole(int c) const { return c - d >= 0 && c - d + V <= H; }
  __device__ __forceinline__ Piece<T, V> part(int c) const {
    Piece<T, V> p{};
    const int a = c - d;
    if (a < H && a + V > 0) {
      T e[V];
#pragma unroll
      for (int v = 0; v < V; ++v) e[v] = a + v >= 0 && a + v < H ? row[a + v] : T(0.0f);
      __builtin_memcpy(p.w, e, 16);
    }
    return p;
  }
  __device__ __forceinline__ Piece<T, V> ask(int c) const {
    if (!whole(c)) return part(c);
    Piece<T, V> p;
    p.load(row + c - d);
    return p;
  }
  // The frame of the pieces (all lanes of the warp).
  __device__ __forceinline__ Piece<T, V> frame(const Piece<T, V>& own) const {
    if (d == 0) return own;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = own.w[i];
      w[4 + i] = __shfl_down_sync(0xffffffffu, own.w[i], 1);
    }
    return from_pieces<T>(w, d);
  }
};
// A frame at column c of a row of H elements, from lanes that have one.
template <typename T, int V>
__device__ __forceinline__ void store_frame(T* row, int H, int c, const Piece<T, V>& p) {
  if ((reinterpret_cast<uintptr_t>(row + c) & 15) == 0 && c >= 0 && c + V <= H) {
    p.store(row + c);
    return;
  }
  T e[V];
  __builtin_memcpy(e, p.w, 16);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (c + v >= 0 && c + v < H) row[c + v] = e[v];
}

// The sum over a team's threads (whole warps, `first` of the block's on, or 8 or 16 lanes of
// one; `part` has a float for each warp of the block), the same in every thread and every call.
__device__ __forceinline__ float team_sum(float v, int team, int first, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < team) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (team <= 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < team >> 5 ? part[first + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
#endif

// The bytes of an access that all of some rows allow: 16, 4, or one element's.
struct Access {
  uint64_t bits = 0;
  Access& rows(const void* p, int64_t ld, int size) {  // (null: not there)
    if (p) bits |= reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(ld * size);
    return *this;
  }
  bool by(int bytes) const { return (bits & static_cast<uint64_t>(bytes - 1)) == 0; }
};

}  // namespace agg
