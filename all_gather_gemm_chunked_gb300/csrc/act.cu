// act.cu -- gated activation: y = g s u with s = 1 / (1 + exp(-g)), for rows that hold the
// gate g and the other factor u side by side, and its gradient
//
//   dg = dy u s (1 + g (1 - s)),   du = dy g s
//
// Bound by memory: every element is read once, in 16-byte accesses where rows are aligned,
// with all of a thread's loads in flight before the first is used.  A team of 2^log
// threads takes 2^log * P pieces of a row.  (8192 x 2 x 2048 bf16: 14.8 us, 6.8 TB/s; backward
// 25.4, 6.6 TB/s; to e4m3 17.1, to 4 bits 17.4, 4.9 and 4.4 TB/s.)

#include "layer_rows.cuh"

namespace agg {

namespace {
constexpr int kThreads = 256;

__device__ __forceinline__ float reciprocal(float d) {  // of 1 and on; within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}
// exp(x) for |x| <= 100, within 2 ulps (zero from -87.3 down): with t = x / ln 2 rounded, exp(x) = 2^t exp(x - t ln 2), whose
// second factor is 1 + (x - t ln 2) but for its square, below 2^-33.  ln 2 in two parts, after Cody
// and Waite.
__device__ __forceinline__ float exp_near(float x) {
  const float t = x * 1.44269504f;
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return fmaf(e, fmaf(t, 1.90465429e-9f, fmaf(-t, 0.693147182f, x)), e);
}

// s = 1 / (1 + exp(-g)) and 1 - s = exp(-g) s.  Below -80 s is exp(g): exp(-g) passes the largest
// float from -88.7 on, but g s lies within floats to -103.  (Looked for once for all V.)
//
// kExact (floats, and codes, whose ties a last bit of y decides): to about an ulp, the reciprocal
// after one step of Newton's iteration.  Otherwise (y rounded to 16 bits) by the approximate
// exponential, off by |g| 2^-24 and 2 ulps.  To codes the kernels are bound by instructions: 8192 x 2 x
// 4096 bf16 to e4m3 took 42 us with expf and __fdividef, now 33, its loads and stores 25.
template <bool kExact, int V>
__device__ __forceinline__ void sigmoid(const float (&g)[V], float (&s)[V], float (&rest)[V]) {
  float least = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float e = kExact ? exp_near(fmaxf(-g[v], -100.0f)) : __expf(-g[v]), d = 1.0f + e, r = reciprocal(d);
    s[v] = kExact ? fmaf(r, fmaf(-d, r, 1.0f), r) : r;
    rest[v] = e * s[v];
    least = fminf(least, g[v]);
  }
  if (least < -80.0f) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (g[v] < -80.0f) {
        s[v] = expf(g[v]);
        rest[v] = 1.0f;
      }
  }
}

template <typename T, int V, int P, int OUT>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const GateArgs a, int log) {
  pdl_enter();
  const int team = 1 << log, thread = threadIdx.x & (team - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads >> log) + (threadIdx.x >> log);
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (team * P * V) + thread * V;
  const int left = row < a.rows ? static_cast<int>(a.N - c0) : 0;  // elements of the row from c0 on
  const T *x = static_cast<const T*>(a.x) + row * a.ldx + c0, *y = x + a.N;
  Piece<T, V> g[P], u[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    g[i] = u[i] = Piece<T, V>{};
    if (i * team * V < left) {
      g[i].load(x + i * team * V);
      u[i].load(y + i * team * V);
    }
  }
  constexpr bool kCodes = OUT == kTypeE4m3 || OUT == kTypeE2m1;
  [[maybe_unused]] T* const out = static_cast<T*>(a.out) + row * a.N + c0;
  [[maybe_unused]] CodePlace<OUT> place(a.out, a.scales, a.rows, a.N, row, c0);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const bool in = i * team * V < left;
    if (!__any_sync(0xffffffffu, in)) break;
    float f[V], v[V], s[V], rest[V];
    g[i].get(f);
    u[i].get(v);
    sigmoid<sizeof(T) == 4 || kCodes>(f, s, rest);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = f[j] * s[j] * v[j];
    if constexpr (kCodes) {
      put_codes<OUT, V>(place, in, f);
      place.advance(team * V);
    } else {
      if (in) store_floats(out + i * team * V, f);
    }
  }
}

template <typename T, int V, int P>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(const GateArgs a, int log) {
  pdl_enter();
  const int team = 1 << log, thread = threadIdx.x & (team - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads >> log) + (threadIdx.x >> log);
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (team * P * V) + thread * V;
  if (row >= a.rows) return;
  const int left = static_cast<int>(a.N - c0);
  const T *x = static_cast<const T*>(a.x) + row * a.ldx + c0, *y = x + a.N,
          *dy = static_cast<const T*>(a.dy) + row * a.lddy + c0;
  T *dg = static_cast<T*>(a.out) + row * 2 * a.N + c0, *du = dg + a.N;
  Piece<T, V> g[P], u[P], d[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (i * team * V < left) {
      g[i].load(x + i * team * V);
      u[i].load(y + i * team * V);
      d[i].load(dy + i * team * V);
    }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (i * team * V >= left) break;
    float f[V], v[V], e[V], s[V], rest[V];
    g[i].get(f);
    u[i].get(v);
    d[i].get(e);
    sigmoid<sizeof(T) == 4>(f, s, rest);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float es = e[j] * s[j];
      v[j] = es * v[j] * fmaf(f[j], rest[j], 1.0f);
      e[j] = es * f[j];
    }
    store_floats(dg + i * team * V, v);
    store_floats(du + i * team * V, e);
  }
}

// A team's log, and the grid: rows, and pieces of them.
struct Shape {
  int log;
  dim3 grid;
};
Shape shape_of(int64_t rows, int64_t N, int V, int P) {
  const int64_t pieces = (N + V - 1) / V;
  int log = 5;
  while (log < 8 && (P << log) < pieces) ++log;
  const int64_t per = kThreads >> log, cols = static_cast<int64_t>(P) << log;
  return {log, dim3(static_cast<unsigned>((rows + per - 1) / per), static_cast<unsigned>((pieces + cols - 1) / cols))};
}

template <typename F>
cudaError_t with_type(int dtype, const F& f) {
  return dtype == kTypeF32 ? f(float{}) : dtype == kTypeF16 ? f(__half{}) : f(__nv_bfloat16{});
}

// Pieces a thread: more in flight where there is enough to do for all SMs.  (bf16, one piece and
// four: 1024 x 2 x 2048 2.6 us and 3.6, 2048 rows 5.0 and 5.5, 4096 rows 8.1 and 7.8, 8192 rows to
// e4m3 19.3 and 17.2; backward, one and two: 2048 rows 7.1 and 7.3, 8192 rows 26.7 and 25.5; rows of
// 512 14.8 and 15.8.)
bool plenty(const GateArgs& a, int V) { return a.rows * ((a.N + V - 1) / V) >= 152 * 4096 && a.N >= 32 * 4 * V; }
template <typename T, int V, int OUT>
cudaError_t forward(const GateArgs& a, cudaStream_t stream) {
  constexpr int kFew = V * sizeof(T) == 16 ? 1 : 4, kMost = V * sizeof(T) == 16 ? 4 : 8;
  const bool most = plenty(a, V);
  const Shape s = shape_of(a.rows, a.N, V, most ? kMost : kFew);
  return most ? launch(swiglu_kernel<T, V, kMost, OUT>, s.grid, kThreads, stream, a, s.log)
              : launch(swiglu_kernel<T, V, kFew, OUT>, s.grid, kThreads, stream, a, s.log);
}
template <typename T, int V>
cudaError_t backward(const GateArgs& a, cudaStream_t stream) {
  constexpr int kFew = V * sizeof(T) == 16 ? 1 : 4, kMost = V * sizeof(T) == 16 ? 2 : 8;
  const bool most = plenty(a, V);
  const Shape s = shape_of(a.rows, a.N, V, most ? kMost : kFew);
  return most ? launch(swiglu_backward_kernel<T, V, kMost>, s.grid, kThreads, stream, a, s.log)
              : launch(swiglu_backward_kernel<T, V, kFew>, s.grid, kThreads, stream, a, s.log);
}
}  // namespace

cudaError_t launch_swiglu(const GateArgs& a, int dtype, int out_type, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const int size = dtype == kTypeF32 ? 4 : 2;
  Access at;  // (N too: the other factor begins N elements behind the gate)
  at.rows(a.x, a.ldx, size).rows(a.out, a.N, out_type == dtype ? size : 16);
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    constexpr int V = Elem<T>::kVec, V4 = 4 / sizeof(T);
    if (out_type == kTypeE4m3) return forward<T, V, kTypeE4m3>(a, stream);
    if (out_type == kTypeE2m1) return forward<T, V, kTypeE2m1>(a, stream);
    if (at.by(16)) return forward<T, V, kTypeF32>(a, stream);
    return at.by(4) ? forward<T, V4, kTypeF32>(a, stream) : forward<T, 1, kTypeF32>(a, stream);
  });
}

cudaError_t launch_swiglu_backward(const GateArgs& a, int dtype, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const int size = dtype == kTypeF32 ? 4 : 2;
  Access at;
  at.rows(a.x, a.ldx, size).rows(a.dy, a.lddy, size).rows(a.out, a.N, size);
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    constexpr int V = Elem<T>::kVec, V4 = 4 / sizeof(T);
    if (at.by(16)) return backward<T, V>(a, stream);
    return at.by(4) ? backward<T, V4>(a, stream) : backward<T, 1>(a, stream);
  });
}

}  // namespace agg
