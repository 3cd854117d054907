// moe_types.cuh -- element types of the mixture-of-experts kernels: loads of 16
// bytes to floats, stores of floats to 16 bytes, single elements, e4m3 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace agg {

// kVec elements make 16 bytes.
template <typename T>
struct Elem;

template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr uint32_t kNegInf = 0;  // (16-bit types only)
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xfc00u;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpair(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpair(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
};

template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xff80u;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bfloat16 is the upper half of a float
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
};

// V consecutive elements: one 16-byte access where V is the type's kVec, single
// elements (V = 1) where rows are not 16-byte aligned.
template <typename T, int V>
__device__ __forceinline__ void load_elems(const T* p, float (&f)[V]) {
  if constexpr (V == 1)
    f[0] = Elem<T>::get(*p);
  else
    Elem<T>::unpack(*reinterpret_cast<const uint4*>(p), f);
}
template <typename T, int V>
__device__ __forceinline__ void store_elems(T* p, const float (&f)[V]) {
  if constexpr (V == 1)
    *p = Elem<T>::put(f[0]);
  else
    *reinterpret_cast<uint4*>(p) = Elem<T>::pack(f);
}

// The same as it is loaded, in half (16-bit types) of the registers of its floats:
// for loads that wait in flight.
template <typename T, int V>
struct Raw {
  uint4 u;
  // (volatile: in the order of the source, behind a launch's wait, and none sinks to its
  // use; as ordinary loads combine took 54 us instead of 51)
  __device__ __forceinline__ void load(const T* p) {
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  }
  __device__ __forceinline__ void get(float (&f)[V]) const { Elem<T>::unpack(u, f); }
};
template <typename T>
struct Raw<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T* p) { u = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = Elem<T>::get(u); }
};

// Two floats to e4m3 codes (nearest, ties to even, clipped to +-448; NaN stays
// NaN), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace agg
