// norm.cu -- root-mean-square norm with the residual's addition, and its gradient.
//
//   h = x + residual (rounded to the rows' type: that is the residual stream),
//   rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//
// The norm is that of the rounded h: the backward pass, which starts from the stored h,
// is then the gradient of what ran forward.  With g = dy w and xh = h rstd,
//
//   dx = rstd (g - xh mean(g xh)) + dh   (of x and of the residual),  dw = sum over rows of dy xh
//
// Bound by memory: each row is read once and held in registers (as it was loaded: in half
// of its floats' registers) while its sum goes through the team of threads that shares it;
// sums and everything between the loads and the stores are floats.  y is rounded once, to
// the rows' type or to codes (put_codes).

#include <type_traits>

#include "layer_rows.cuh"

namespace agg {

namespace {
constexpr int kSms = 152;

// V weights, as they are loaded; floats or the rows' type.
template <typename W, int V>
struct Weights {
  static constexpr int kV = V * sizeof(W) > 16 ? 16 / sizeof(W) : V == 2 && sizeof(W) == 4 ? 1 : V, kN = V / kV;
  Piece<W, kV> r[kN];
  __device__ __forceinline__ void load(const W* p) {
#pragma unroll
    for (int i = 0; i < kN; ++i) r[i].load(p + i * kV);
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float g[kV];
      r[i].get(g);
#pragma unroll
      for (int v = 0; v < kV; ++v) f[i * kV + v] = g[v];
    }
  }
};

// h, rounded, in the place of x.  (Pairs of 16-bit elements are added as such: their sum in
// floats is exact, or so far from a tie that rounding it once more gives the same.)
template <typename T, int V>
__device__ __forceinline__ void add_residual(Piece<T, V>& x, const Piece<T, V>& r) {
  if constexpr (sizeof(T) == 2 && V > 1) {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
#pragma unroll
    for (int i = 0; i < Piece<T, V>::kWords; ++i) {
      const T2 s = __hadd2(reinterpret_cast<const T2&>(x.w[i]), reinterpret_cast<const T2&>(r.w[i]));
      x.w[i] = reinterpret_cast<const uint32_t&>(s);
    }
  } else {
    float a[V], b[V];
    x.get(a);
    r.get(b);
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] += b[v];
    x.put(a);
  }
}
template <typename T, int V>
__device__ __forceinline__ float squares(const Piece<T, V>& r, float scale, float sum) {
  float f[V];
  r.get(f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f[v] *= scale;
    sum = fmaf(f[v], f[v], sum);
  }
  return sum;
}
// rstd of a row from its team's sums of squares; squares(scale) is a thread's sum of those
// of its elements times scale.  Where elements from 10^18 on make the sum pass the largest
// float, it is made anew of elements times 2^-80 (all threads of the block or, with teams of
// one warp, of the warp take that way together).
template <typename F>
__device__ __forceinline__ float team_rstd(const NormArgs& a, int team_warps, int first, float (*part)[32], const F& squares) {
  constexpr float kSmall = 0x1p-80f, kLarge = 1e37f;  // (32 warps' sums up to that are finite)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;  // first: of the team's warps
  auto over_warp = [](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  float sum = over_warp(squares(1.0f));
  bool large = !(sum <= kLarge);
  if (team_warps > 1) {
    if (lane == 0) part[0][warp] = sum;
    large = __syncthreads_or(large);
    sum = over_warp(lane < team_warps ? part[0][first + lane] : 0.0f);
  }
  float scale = 1.0f, eps = a.eps;
  if (large) {
    float s = over_warp(squares(kSmall));
    if (team_warps > 1) {
      if (lane == 0) part[1][warp] = s;
      __syncthreads();
      s = over_warp(lane < team_warps ? part[1][first + lane] : 0.0f);
    }
    if (!(sum <= kLarge)) {
      sum = s;
      scale = kSmall;
      eps = 0.0f;  // (eps 2^-160)
    }
  }
  return scale * rsqrtf(fmaf(sum, a.inv_H, eps));
}

// Where a thread's piece of y goes, and the next, n elements on, a multiple of 128 where y
// becomes codes.
template <int OUT, typename T, int V>
struct RowPlace {
  static constexpr bool kCodes = OUT == kTypeE4m3 || OUT == kTypeE2m1;
  T* y;
  CodePlace<OUT> codes;
  __device__ __forceinline__ RowPlace(const NormArgs& a, int64_t row, int64_t c)
      : y(static_cast<T*>(a.out) + row * a.H + c), codes(a.out, a.scales, a.rows, a.H, row, c) {}
  __device__ __forceinline__ void put(bool in, const Piece<T, V>& h, float rstd, const float (&w)[V], int n) {
    float f[V];
    h.get(f);
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = f[v] * rstd * w[v];
    if constexpr (kCodes) {
      if (!in)
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.0f;
      put_codes<OUT, V>(codes, in, f);
      codes.advance(n);
    } else {
      if (in) store_floats(y, f);
      y += n;
    }
  }
};

// A team of threads has a row, P pieces of V elements a thread: a block's threads (log 10), or
// 2^log of them, several teams a block.
template <typename T, typename W, int V, int P, int OUT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a, int team, int log) {
  pdl_enter();
  __shared__ float part[2][32];
  const int thread = threadIdx.x & ((1 << log) - 1), number = threadIdx.x >> log;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (log == 10 ? 1 : blockDim.x >> log) + number;
  const int c0 = thread * V, left = row < a.rows ? static_cast<int>(a.H) - c0 : 0;  // elements of the row from c0 on
  const T* x = static_cast<const T*>(a.x) + row * a.ldx + c0;
  Piece<T, V> h[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    h[i] = Piece<T, V>{};
    if (i * team * V < left) h[i].load(x + i * team * V);
  }
  if (a.residual) {
    const T* const res = static_cast<const T*>(a.residual) + row * a.ldr + c0;
    T* const held = static_cast<T*>(a.h) + row * a.H + c0;
    Piece<T, V> r[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      r[i] = Piece<T, V>{};
      if (i * team * V < left) r[i].load(res + i * team * V);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      add_residual(h[i], r[i]);
      if (i * team * V < left) h[i].store(held + i * team * V);
    }
  }
  const float rstd = team_rstd(a, team >> 5, number << (log - 5), part, [&](float scale) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) sum = squares(h[i], scale, sum);
    return sum;
  });
  if (a.rstd && thread == 0 && left > 0) a.rstd[row] = rstd;
  RowPlace<OUT, T, V> place(a, row, c0);
  const W* const weight = static_cast<const W*>(a.weight) + c0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const bool in = i * team * V < left;
    if (!__any_sync(0xffffffffu, in)) break;
    Weights<W, V> w{};
    if (in) w.load(weight + i * team * V);
    float f[V];
    w.get(f);
    place.put(in, h[i], rstd, f, team * V);
  }
}

// A block has a row of any length, which it reads twice.
template <typename T, typename W, int V, int OUT>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float part[2][32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* h = static_cast<T*>(a.h) + row * a.H;
  const float rstd = team_rstd(a, 32, 0, part, [&](float scale) {
    float sum = 0.0f;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.H; c += 1024 * V) {
      Piece<T, V> v, r;
      v.load(x + c);
      if (a.residual) {
        r.load(static_cast<const T*>(a.residual) + row * a.ldr + c);
        add_residual(v, r);
        v.store(h + c);
      }
      sum = squares(v, scale, sum);
    }
    return sum;
  });
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  const T* from = a.residual ? h : x;  // (each thread reads what it wrote itself)
  RowPlace<OUT, T, V> place(a, row, static_cast<int64_t>(threadIdx.x) * V);
  const int64_t end = (a.H + 1024 * V - 1) / (1024 * V) * (1024 * V);  // (the lanes of a warp stay together)
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < end; c += 1024 * V) {
    const bool in = c < a.H;
    Piece<T, V> v{};
    Weights<W, V> w{};
    float f[V];
    if (in) {
      v.load(from + c);
      w.load(static_cast<const W*>(a.weight) + c);
    }
    w.get(f);
    place.put(in, v, rstd, f, 1024 * V);
  }
}

// ------------------------------------------------------------------ gradient
// Rows whose pieces fit a team, P a thread.  A thread keeps its columns from row to row,
// and their share of the weight's gradient in registers; a block adds its teams' and
// stores one part.
template <typename T, typename W, int V, int P, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 1024 ? 1 : 2) norm_backward_kernel(const NormBackwardArgs a, int log) {
  pdl_enter();
  // The next row's loads ahead of this one's sum, where registers allow.
  constexpr bool kAhead = P * Piece<T, V>::kWords <= 4;
  __shared__ float part[2][32];
  __shared__ float sums[THREADS == 1024 ? 1 : THREADS * V * P];
  const int team = 1 << log, thread = threadIdx.x & (team - 1), teams = THREADS >> log;
  const int c0 = thread * V;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  const T *dy = static_cast<const T*>(a.dy) + c0, *h = static_cast<const T*>(a.h) + c0,
          *dh = static_cast<const T*>(a.dh) + c0;
  float dw[P][V] = {};
  Weights<W, V> rw[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    rw[i] = Weights<W, V>{};
    if (c0 + i * team * V < a.H) rw[i].load(static_cast<const W*>(a.weight) + c0 + i * team * V);
  }
  const float inv = 1.0f / static_cast<float>(a.H);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * teams;
  int64_t row = first + (threadIdx.x >> log);
  Piece<T, V> rg[P], rh[P], rd[P];
  float rstd = 0.0f;
  auto load = [&] {
    const bool valid = row < a.rows;
    if (valid) rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = i * team * V;
      rg[i] = rh[i] = rd[i] = Piece<T, V>{};
      if (valid && c0 + c < a.H) {
        rg[i].load(dy + row * a.lddy + c);
        rh[i].load(h + row * a.ldh + c);
        if (a.dh) rd[i].load(dh + row * a.lddh + c);
      }
    }
  };
  if (kAhead) load();
  int turn = 0;
  for (int64_t base = first; base < a.rows; base += step, turn ^= 1) {  // (all teams: they share a barrier)
    if (!kAhead) load();
    Piece<T, V> pg[P], ph[P], pd[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      pg[i] = rg[i];
      ph[i] = rh[i];
      pd[i] = rd[i];
    }
    const float rs = rstd;
    const int64_t at = row;
    const bool valid = at < a.rows;
    row += step;
    if (kAhead) load();
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float g[V], x[V], w[V];
      pg[i].get(g);
      ph[i].get(x);
      rw[i].get(w);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[v] *= rs;
        if (valid) dw[i][v] = fmaf(g[v], x[v], dw[i][v]);
        dot = fmaf(g[v] * w[v], x[v], dot);
      }
    }
    dot = team_sum(dot, team >> 5, part[turn]) * inv;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = i * team * V;
      if (!valid || c0 + c >= a.H) continue;
      float g[V], x[V], w[V], d[V];
      pg[i].get(g);
      ph[i].get(x);
      rw[i].get(w);
      pd[i].get(d);
#pragma unroll
      for (int v = 0; v < V; ++v) g[v] = fmaf(rs, fmaf(-x[v] * rs, dot, g[v] * w[v]), a.dh ? d[v] : 0.0f);
      store_floats(static_cast<T*>(a.dx) + at * a.H + c0 + c, g);
    }
  }
  float* to = a.parts + static_cast<int64_t>(blockIdx.x) * a.H;
  if constexpr (THREADS != 1024) {
    if (teams > 1) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
          sums[(threadIdx.x >> log) * (team * P * V) + i * team * V + c0 + v] = dw[i][v];
      __syncthreads();
      for (int c = threadIdx.x; c < a.H; c += THREADS) {
        float s = 0.0f;
        for (int t = 0; t < teams; ++t) s += sums[t * (team * P * V) + c];
        to[c] = s;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = c0 + i * team * V;
    if (c >= a.H) continue;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int v = 0; v < V; v += 4)
        *reinterpret_cast<float4*>(to + c + v) = make_float4(dw[i][v], dw[i][v + 1], dw[i][v + 2], dw[i][v + 3]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) to[c + v] = dw[i][v];
    }
  }
}

// Rows of any length: a block has a row, which it reads twice ...
template <typename T, typename W, int V>
__global__ void __launch_bounds__(512) norm_backward_long_kernel(const NormBackwardArgs a) {
  pdl_enter();
  __shared__ float part[32];
  const int64_t row = blockIdx.x;
  const T *dy = static_cast<const T*>(a.dy) + row * a.lddy, *h = static_cast<const T*>(a.h) + row * a.ldh;
  const float rs = a.rstd[row];
  float dot = 0.0f;
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.H; c += 512 * V) {
    Piece<T, V> rg, rh;
    Weights<W, V> rw;
    rg.load(dy + c);
    rh.load(h + c);
    rw.load(static_cast<const W*>(a.weight) + c);
    float g[V], x[V], w[V];
    rg.get(g);
    rh.get(x);
    rw.get(w);
#pragma unroll
    for (int v = 0; v < V; ++v) dot = fmaf(g[v] * w[v], x[v] * rs, dot);
  }
  dot = team_sum(dot, 16, part) / static_cast<float>(a.H);
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.H; c += 512 * V) {
    Piece<T, V> rg, rh, rd{};
    Weights<W, V> rw;
    rg.load(dy + c);
    rh.load(h + c);
    rw.load(static_cast<const W*>(a.weight) + c);
    if (a.dh) rd.load(static_cast<const T*>(a.dh) + row * a.lddh + c);
    float g[V], x[V], w[V], d[V];
    rg.get(g);
    rh.get(x);
    rw.get(w);
    rd.get(d);
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = fmaf(rs, fmaf(-x[v] * rs, dot, g[v] * w[v]), a.dh ? d[v] : 0.0f);
    store_floats(static_cast<T*>(a.dx) + row * a.H + c, g);
  }
}
// ... and the weight's gradient comes by columns, a thread for each, over a part of the rows.
constexpr int kColumnThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kColumnThreads) norm_columns_kernel(const NormBackwardArgs a, int64_t part_rows) {
  pdl_enter();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kColumnThreads + threadIdx.x;
  if (c >= a.H) return;
  const int64_t r0 = blockIdx.y * part_rows, r1 = r0 + part_rows < a.rows ? r0 + part_rows : a.rows;
  const T *dy = static_cast<const T*>(a.dy) + c, *h = static_cast<const T*>(a.h) + c;
  float sum = 0.0f;
#pragma unroll 4
  for (int64_t r = r0; r < r1; ++r)
    sum = fmaf(Elem<T>::get(dy[r * a.lddy]), Elem<T>::get(h[r * a.ldh]) * a.rstd[r], sum);
  a.parts[blockIdx.y * a.H + c] = sum;
}

// The sum of the parts, 32 columns a block: each warp adds every 16th part, then the warps'
// sums are added in their order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps) norm_sum_kernel(const float* parts, int64_t n, int64_t H, float* dweight) {
  pdl_enter();
  __shared__ float sums[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < H)
#pragma unroll 8
    for (int64_t i = warp; i < n; i += kSumWarps) s += parts[i * H + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < H) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) s += sums[i][lane];
    dweight[c] = s;
  }
}

int team_log(int64_t threads) {
  int log = 5;
  while ((1LL << log) < threads) ++log;
  return log;
}

constexpr int kMaxParts = 2 * kSms;

template <typename F>
cudaError_t with_types(int dtype, int weight_f32, const F& f) {
  if (dtype == kTypeF32) return f(float{}, float{});
  if (dtype == kTypeF16) return weight_f32 ? f(__half{}, float{}) : f(__half{}, __half{});
  return weight_f32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}
int size_of(int dtype) { return dtype == kTypeF32 ? 4 : 2; }

template <typename T, typename W, int V, int P, int OUT>
cudaError_t launch_norm_p(const NormArgs& a, int64_t pieces, cudaStream_t stream) {
  // (teams of more than 64 threads: no more warps than the row needs)
  const int64_t need = (pieces + P - 1) / P;
  const int log = need > 64 ? 10 : team_log(need), team = log == 10 ? static_cast<int>((need + 31) / 32 * 32) : 1 << log;
  const int threads = log == 10 ? team : 128, per = threads / team;
  const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per));
  return launch(norm_kernel<T, W, V, P, OUT>, grid, threads, stream, a, team, log);
}
template <typename T, typename W, int V, int OUT>
cudaError_t launch_norm_v(const NormArgs& a, cudaStream_t stream) {
  constexpr bool kVec = V * sizeof(T) == 16;
  constexpr int kFew = kVec ? 1 : 4, kMost = kVec ? 4 : 8;
  const int64_t pieces = (a.H + V - 1) / V;
  if (pieces > 1024 * kMost)
    return launch(norm_long_kernel<T, W, V, OUT>, dim3(static_cast<unsigned>(a.rows)), 1024, stream, a);
  // Few rows are spread over more threads; of many, more of a row is in flight in a thread
  // (8192 x 4096 bf16: 40.0 us with four pieces, 40.9 with two, without a residual 21.7 and
  // 30.3; 64 x 7168 2.6 with one, 3.1 with two).  Rows of a few pieces have no more.
  if (pieces > 1024 * kFew || (a.rows > 2 * kSms && pieces >= 32 * kMost)) return launch_norm_p<T, W, V, kMost, OUT>(a, pieces, stream);
  return launch_norm_p<T, W, V, kFew, OUT>(a, pieces, stream);
}

// kWide: teams of 1024 threads (log 10) alone.
template <typename T, typename W, int V, int P, bool kWide>
cudaError_t launch_backward_p(const NormBackwardArgs& a, int log, int64_t& parts, cudaStream_t stream) {
  const int64_t per = log == 10 ? 1 : 512 >> log, blocks = (a.rows + per - 1) / per;
  const int64_t most = log == 10 ? kSms : kMaxParts;
  parts = blocks < most ? blocks : most;
  const dim3 grid(static_cast<unsigned>(parts));
  if constexpr (!kWide)
    if (log < 10) return launch(norm_backward_kernel<T, W, V, P, 512>, grid, 512, stream, a, log);
  return launch(norm_backward_kernel<T, W, V, P, 1024>, grid, 1024, stream, a, log);
}
template <typename T, typename W, int V>
cudaError_t launch_backward_v(const NormBackwardArgs& a, int64_t& parts, cudaStream_t stream) {
  constexpr bool kVec = V * sizeof(T) == 16;
  constexpr int kFew = kVec ? 1 : 4, kMost = kVec ? 2 : 8;
  const int64_t pieces = (a.H + V - 1) / V;
  if (pieces <= 1024 * kFew)
    return launch_backward_p<T, W, V, kFew, false>(a, team_log((pieces + kFew - 1) / kFew), parts, stream);
  if (pieces <= 1024 * kMost) return launch_backward_p<T, W, V, kMost, true>(a, 10, parts, stream);
  cudaError_t e = launch(norm_backward_long_kernel<T, W, V>, dim3(static_cast<unsigned>(a.rows)), 512, stream, a);
  if (e != cudaSuccess) return e;
  parts = norm_parts(a.rows, a.H);
  const int64_t part_rows = (a.rows + parts - 1) / parts;
  const dim3 grid(static_cast<unsigned>((a.H + kColumnThreads - 1) / kColumnThreads), static_cast<unsigned>(parts));
  return launch(norm_columns_kernel<T>, grid, kColumnThreads, stream, a, part_rows);
}
}  // namespace

cudaError_t launch_norm(NormArgs a, int dtype, int out_type, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  a.inv_H = 1.0f / static_cast<float>(a.H);
  const int size = size_of(dtype);
  Access at;
  at.rows(a.x, a.ldx, size).rows(a.weight, a.H, size).rows(a.out, a.H, out_type == dtype ? size : 16);
  if (a.residual) at.rows(a.residual, a.ldr, size).rows(a.h, a.H, size);
  return with_types(dtype, a.weight_f32, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int V = Elem<T>::kVec, V4 = 4 / sizeof(T);
    if (out_type == kTypeE4m3) return launch_norm_v<T, W, V, kTypeE4m3>(a, stream);
    if (out_type == kTypeE2m1) return launch_norm_v<T, W, V, kTypeE2m1>(a, stream);
    if (at.by(16)) return launch_norm_v<T, W, V, kTypeF32>(a, stream);
    return at.by(4) ? launch_norm_v<T, W, V4, kTypeF32>(a, stream) : launch_norm_v<T, W, 1, kTypeF32>(a, stream);
  });
}

int64_t norm_parts(int64_t rows, int64_t) { return rows < kMaxParts ? rows : kMaxParts; }

cudaError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, cudaStream_t stream) {
  if (a.rows == 0) return cudaMemsetAsync(a.dweight, 0, static_cast<size_t>(a.H) * 4, stream);
  const int size = size_of(dtype);
  Access at;
  at.rows(a.dy, a.lddy, size).rows(a.h, a.ldh, size).rows(a.weight, a.H, size).rows(a.dx, a.H, size).rows(a.dh, a.lddh, size);
  int64_t parts = 0;
  const cudaError_t e = with_types(dtype, a.weight_f32, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int V = Elem<T>::kVec, V4 = 4 / sizeof(T);
    if (at.by(16)) return launch_backward_v<T, W, V>(a, parts, stream);
    return at.by(4) ? launch_backward_v<T, W, V4>(a, parts, stream) : launch_backward_v<T, W, 1>(a, parts, stream);
  });
  if (e != cudaSuccess) return e;
  return launch(norm_sum_kernel, dim3(static_cast<unsigned>((a.H + 31) / 32)), 32 * kSumWarps, stream, a.parts, parts,
                a.H, a.dweight);
}

}  // namespace agg
