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
//
// Measured, 8192 x 4096 bf16: with the residual 40.1 us (6.7 TB/s), without 22.2 (6.1), with it and
// to e4m3 37.1 (6.4), to 4 bits 34.3 (6.4); gradient 47.0 (5.7 TB/s: its second launch and the end
// of the first take 5 us).  64 x 7168 with the residual 2.7 us.

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
// 1 / sqrt(m), to the nearest but for about 2^-40: the approximate root (2 ulps) after one step of
// Newton's iteration, r + r (1 - m r^2) / 2, with m r in two parts.  It is every element's factor: by
// the approximate root alone floats of y were off by a twelfth more, and e4m3 codes next to ties a
// little oftener; with an exact root and division 8192 x 4096 bf16 took 41.3 us, so 40.8.  (Zero and
// infinite m have no step.)
__device__ __forceinline__ float inverse_root(float m) {
  const float r = rsqrtf(m), p = m * r, rest = fmaf(m, r, -p);
  const float better = fmaf(0.5f * r, fmaf(-rest, r, fmaf(-p, r, 1.0f)), r);
  return better == better ? better : r;
}
// rstd of a row from its team's sums of squares; squares(scale) is a thread's sum of those
// of its elements times scale.  Where the squares, or eps, pass the largest float (elements from
// 10^18 on), or where squares below the smallest normal one lose bits that eps does not hide
// (elements below 10^-15, eps below 2^-80), the sum is made anew of scaled elements, eps times the
// scale's square: of all threads of the block or, with teams of one warp, of the warp together.
// (A sum from 2^-100 on has lost at most 2^24 halves of 2^-149, a quarter of its last bit.)
template <typename F>
__device__ __forceinline__ float team_rstd(const NormArgs& a, int team_warps, int first, float (*part)[32], const F& squares) {
  constexpr float kMost = 1e37f, kDown = 0x1p-80f;  // (32 warps' sums up to that are finite)
  constexpr float kLeast = 0x1p-100f, kLeastEps = 0x1p-80f, kUp = 0x1p100f;  // (2^24 squares then stay below 2^124)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;  // first: of the team's warps
  auto over_warp = [](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  auto scale_of = [&](float sum) {
    return !(sum <= kMost) || a.eps > kMost ? kDown : sum < kLeast && a.eps < kLeastEps ? kUp : 1.0f;
  };
  float sum = over_warp(squares(1.0f));
  bool again = scale_of(sum) != 1.0f;  // (of a warp's share: where a row's sum is small, all its warps' are)
  if (team_warps > 1) {
    if (lane == 0) part[0][warp] = sum;
    again = __syncthreads_or(again);
    sum = over_warp(lane < team_warps ? part[0][first + lane] : 0.0f);
  }
  float scale = 1.0f, m = fmaf(sum, a.inv_H, a.eps);
  if (again) {
    scale = scale_of(sum);
    sum = over_warp(squares(scale));
    if (team_warps > 1) {
      if (lane == 0) part[1][warp] = sum;
      __syncthreads();
      sum = over_warp(lane < team_warps ? part[1][first + lane] : 0.0f);
    }
    m = fmaf(sum, a.inv_H, a.eps * scale * scale);
  }
  return scale * inverse_root(m);
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

// Rows of any alignment, by frames: a team of whole warps has a row, P frames a lane, several
// teams a block.  (8192 x 4099 bf16 with the residual 59 us: memory 48 % busy, issue slots 57 %; 27 warps an SM,
// as 64 registers of five-warp blocks allow, wait for loads and at the sum's barrier.)
template <typename T, typename W, int P>
__global__ void __launch_bounds__(1024) norm_frames_kernel(const NormArgs a, int team_warps) {
  constexpr int V = 16 / sizeof(T);
  pdl_enter();
  __shared__ float part[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, number = warp / team_warps, first = number * team_warps;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ((blockDim.x >> 5) / team_warps) + number;
  const bool valid = row < a.rows;
  const int H = valid ? static_cast<int>(a.H) : 0, step = team_warps * kFrames * V;
  T* const y = static_cast<T*>(a.out) + row * a.H;
  const int c0 = ((warp - first) * kFrames + lane) * V - static_cast<int>((reinterpret_cast<uintptr_t>(y) & 15) / sizeof(T));
  const Anywhere<T> x(static_cast<const T*>(a.x) + row * a.ldx, H, c0);
  Piece<T, V> h[P];
#pragma unroll
  for (int i = 0; i < P; ++i) h[i] = x.ask(c0 + i * step);
  if (a.residual) {
    const Anywhere<T> res(static_cast<const T*>(a.residual) + row * a.ldr, H, c0);
    Piece<T, V> r[P];
#pragma unroll
    for (int i = 0; i < P; ++i) r[i] = res.ask(c0 + i * step);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      h[i] = x.frame(h[i]);
      add_residual(h[i], res.frame(r[i]));
      if (lane < kFrames) store_frame(static_cast<T*>(a.h) + row * a.H, H, c0 + i * step, h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) h[i] = x.frame(h[i]);
  }
  // (what lies outside the row is zero; lane 31's frames are the next warp's)
  const float rstd = team_rstd(a, team_warps, first, part, [&](float scale) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) sum = squares(h[i], scale, sum);
    return lane < kFrames ? sum : 0.0f;
  });
  if (a.rstd && threadIdx.x == first * 32 && valid) a.rstd[row] = rstd;
  if (lane >= kFrames) return;
  const W* const weight = static_cast<const W*>(a.weight);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = c0 + i * step;
    if (c >= H) break;
    float f[V], w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = c + v >= 0 && c + v < H ? Elem<W>::get(weight[c + v]) : 0.0f;
    h[i].get(f);
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = f[v] * rstd * w[v];
    Piece<T, V> p;
    p.put(f);
    store_frame(y, H, c, p);
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
// stores one part.  The rows to come are copied to shared memory, two ahead, each piece by
// the thread that reads it, twice: registers for what is in flight would leave room for
// fewer columns and threads.  (8192 x 8192 bf16 83 us, with rows in registers 97; 8192 x
// 5120 55 and 68.  Single 16-bit elements, which no such copy takes, stay in registers.)
//
// kShifted: rows that begin anywhere, but all operands' at the same distance from an aligned
// address.  The rows of a team are a multiple of V apart, so that distance is the team's, and
// its columns begin that much before the row: all pieces are aligned, and those at the row's
// ends are written element by element.  (8192 x 4099 bf16 63 us; by single elements, with rows
// read twice, 140.)
constexpr int kSlots = 2;
template <typename T, int V, int P, bool kCopied = (V * sizeof(T) >= 4)>
struct Ring {
  static constexpr int kBytes = 3 * P * kSlots * V * static_cast<int>(sizeof(T));  // of a thread
  using Word = std::conditional_t<V * sizeof(T) == 16, uint4, uint32_t>;
  Word* mine;
  int n;
  __device__ __forceinline__ explicit Ring(uint8_t* bytes)
      : mine(reinterpret_cast<Word*>(bytes) + threadIdx.x), n(static_cast<int>(blockDim.x)) {}
  __device__ __forceinline__ Word* at(int slot, int operand, int i) const { return mine + ((slot * 3 + operand) * P + i) * n; }
  __device__ __forceinline__ void clear(int slot, int operand, int i) { *at(slot, operand, i) = Word{}; }
  __device__ __forceinline__ void put(int slot, int operand, int i, int v, T x) {  // one element
    reinterpret_cast<T*>(at(slot, operand, i))[v] = x;
  }
  __device__ __forceinline__ void ask(int slot, int operand, int i, const T* from) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(at(slot, operand, i)));
    if constexpr (sizeof(Word) == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
  }
  __device__ __forceinline__ void get(int slot, int operand, int i, float (&f)[V]) const {
    Piece<T, V> p;
    const Word w = *at(slot, operand, i);
    __builtin_memcpy(p.w, &w, sizeof(p.w));
    p.get(f);
  }
};
template <typename T, int V, int P>
struct Ring<T, V, P, false> {
  static constexpr int kBytes = P * V * 4;  // (its columns' sums)
  Piece<T, V> r[kSlots][3][P];
  __device__ __forceinline__ explicit Ring(uint8_t*) {}
  __device__ __forceinline__ void clear(int slot, int operand, int i) { r[slot][operand][i] = Piece<T, V>{}; }
  __device__ __forceinline__ void ask(int slot, int operand, int i, const T* from) { r[slot][operand][i].load(from); }
  __device__ __forceinline__ void get(int slot, int operand, int i, float (&f)[V]) const { r[slot][operand][i].get(f); }
};
template <typename T, typename W, int V, int P, bool kShifted>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormBackwardArgs a, int team, int teams) {
  pdl_enter();
  using R = Ring<T, V, P>;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  __shared__ float part[2][32];
  R ring(ring_bytes);
  const int number = threadIdx.x / team, thread = threadIdx.x - number * team, H = static_cast<int>(a.H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams, first = static_cast<int64_t>(blockIdx.x) * teams;
  // of a row of dx: elements from an aligned address to its start
  auto shift_of = [&](int64_t r) {
    return kShifted ? static_cast<int>((reinterpret_cast<uintptr_t>(static_cast<T*>(a.dx) + r * a.H) & 15) / sizeof(T)) : 0;
  };
  const int c0 = thread * V - shift_of(first + number);
  auto inside = [&](int c) { return c < H && (!kShifted || c + V > 0); };  // at least one element
  auto whole = [&](int c) { return !kShifted || (c >= 0 && c + V <= H); };
  float dw[P][V] = {};
  Weights<W, V> rw[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = c0 + i * team * V;
    rw[i] = Weights<W, V>{};
    if (!inside(c)) continue;
    if (whole(c) && !kShifted) {
      rw[i].load(static_cast<const W*>(a.weight) + c);
    } else {
      W w[V];
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = c + v >= 0 && c + v < H ? static_cast<const W*>(a.weight)[c + v] : W(0.0f);
      __builtin_memcpy(&rw[i], w, sizeof(w));
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int s = 0; s < kSlots; ++s)  // what no copy fills
#pragma unroll
      for (int o = 0; o < 3; ++o)
        if (!inside(c0 + i * team * V) || (o == 2 && !a.dh)) ring.clear(s, o, i);
  const float inv = 1.0f / static_cast<float>(a.H);
  int64_t row = first + number, next = row;  // next: the row to ask for
  float rstd[kSlots];
  auto ask = [&](int slot) {
    if (next < a.rows) {
      const T *dy = static_cast<const T*>(a.dy) + next * a.lddy + c0, *h = static_cast<const T*>(a.h) + next * a.ldh + c0,
              *dh = static_cast<const T*>(a.dh) + next * a.lddh + c0;
      rstd[slot] = a.rstd[next];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int n = i * team * V, c = c0 + n;
        if (!inside(c)) continue;
        // (all of the operands, if not of the row)
        if (whole(c) || ((next > 0 || c >= 0) && (next + 1 < a.rows || c + V <= H))) {
          ring.ask(slot, 0, i, dy + n);
          ring.ask(slot, 1, i, h + n);
          if (a.dh) ring.ask(slot, 2, i, dh + n);
        } else if constexpr (kShifted) {
#pragma unroll 1
          for (int v = 0; v < V; ++v) {
            if (c + v < 0 || c + v >= H) continue;
            ring.put(slot, 0, i, v, dy[n + v]);
            ring.put(slot, 1, i, v, h[n + v]);
            if (a.dh) ring.put(slot, 2, i, v, dh[n + v]);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next += step;
  };
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    rstd[s] = 0.0f;
    ask(s);
  }
  for (int64_t base = first; base < a.rows;) {  // (all teams: they share a barrier)
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      if (base >= a.rows) break;
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
      const float rs = rstd[s];
      const bool valid = row < a.rows;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float g[V], x[V], w[V];
        ring.get(s, 0, i, g);
        ring.get(s, 1, i, x);
        rw[i].get(w);
        if (kShifted && !whole(c0 + i * team * V))  // (what is not of the row may be anything)
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (static_cast<unsigned>(c0 + i * team * V + v) >= static_cast<unsigned>(H)) g[v] = x[v] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          x[v] *= rs;
          if (valid) dw[i][v] = fmaf(g[v], x[v], dw[i][v]);
          dot = fmaf(g[v] * w[v], x[v], dot);
        }
      }
      dot = team_sum(dot, team, number * (team >> 5), part[s]) * inv;
      T* dx = static_cast<T*>(a.dx) + row * a.H + c0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = c0 + i * team * V;
        if (!valid || !inside(c)) continue;
        float g[V], x[V], w[V], d[V];
        ring.get(s, 0, i, g);
        ring.get(s, 1, i, x);
        ring.get(s, 2, i, d);
        rw[i].get(w);
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = fmaf(rs, fmaf(-x[v] * rs, dot, g[v] * w[v]), d[v]);
        if (whole(c)) {
          store_floats(dx + i * team * V, g);
        } else if constexpr (kShifted) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (c + v >= 0 && c + v < H) dx[i * team * V + v] = Elem<T>::put(g[v]);
        }
      }
      ask(s);
      row += step;
      base += step;
    }
  }
  float* to = a.parts + static_cast<int64_t>(blockIdx.x) * a.H;
  if (kShifted || teams > 1) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* sums = reinterpret_cast<float*>(ring_bytes);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) sums[number * (team * P * V) + (i * team + thread) * V + v] = dw[i][v];
    __syncthreads();
    const int shift = shift_of(first);  // of the block's first team; a row on it is H more, modulo V
    for (int c = threadIdx.x; c < a.H; c += teams * team) {
      float s = 0.0f;
#pragma unroll 4
      for (int t = 0; t < teams; ++t) s += sums[t * (team * P * V) + c + (kShifted ? (shift + t * H) & (V - 1) : 0)];
      to[c] = s;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = i * team * V;
    if (c0 + c >= H) continue;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int v = 0; v < V; v += 4)
        *reinterpret_cast<float4*>(to + c0 + c + v) = make_float4(dw[i][v], dw[i][v + 1], dw[i][v + 2], dw[i][v + 3]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) to[c0 + c + v] = dw[i][v];
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
  dot = team_sum(dot, 512, 0, part) / static_cast<float>(a.H);
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
  if constexpr (V > 1) {  // (single elements: narrow rows alone)
    if (pieces > 1024 * kMost)
      return launch(norm_long_kernel<T, W, V, OUT>, dim3(static_cast<unsigned>(a.rows)), 1024, stream, a);
    // Few rows are spread over more threads; of many, more of a row is in flight in a thread
    // (8192 x 4096 bf16: 40.0 us with four pieces, 40.9 with two, without a residual 21.7 and
    // 30.3; 64 x 7168 2.6 with one, 3.1 with two).  Rows of a few pieces have no more.
    if (pieces > 1024 * kFew || (a.rows > 2 * kSms && pieces >= 32 * kMost))
      return launch_norm_p<T, W, V, kMost, OUT>(a, pieces, stream);
  }
  return launch_norm_p<T, W, V, kFew, OUT>(a, pieces, stream);
}

template <typename T, typename W>
cudaError_t launch_norm_frames(const NormArgs& a, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T), kWarp = kFrames * V;
  const int64_t warps = (a.H + V - 1 + kWarp - 1) / kWarp;  // of one frame a lane
  if (warps > 32 * 4)
    return launch(norm_long_kernel<T, W, 1, kTypeF32>, dim3(static_cast<unsigned>(a.rows)), 1024, stream, a);
  auto go = [&](auto kernel, int64_t P) {
    const int team = static_cast<int>((warps + P - 1) / P), teams = team < 4 ? 4 / team : 1;
    return launch(kernel, dim3(static_cast<unsigned>((a.rows + teams - 1) / teams)), 32 * team * teams, stream, a, team);
  };
  // (frames a lane, one, two, four: 8192 x 4099 bf16 94 us, 76, 57; 500 x 1001 4.0, 3.7, 5.5; 64 x
  // 7001 3.7, 4.3, 4.4)
  if (warps > 64 || (warps >= 4 && a.rows > 4 * kSms)) return go(norm_frames_kernel<T, W, 4>, 4);
  if (warps > 32 || (warps >= 2 && a.rows > 2 * kSms)) return go(norm_frames_kernel<T, W, 2>, 2);
  return go(norm_frames_kernel<T, W, 1>, 1);
}

// A team's threads: as many warps as a row needs, or 8 or 16 lanes.
int backward_team(int64_t H, int per_thread) {
  const int64_t need = (H + per_thread - 1) / per_thread;
  return need <= 8 ? 8 : need <= 16 ? 16 : static_cast<int>((need + 31) / 32 * 32);
}
// A block an SM, of as many teams as 1024 threads hold (of few rows no more than that each has one).
template <typename T, typename W, int V, int P, bool kShifted>
cudaError_t launch_backward_p(const NormBackwardArgs& a, int64_t& parts, cudaStream_t stream) {
  const int team = backward_team(kShifted ? a.H + V - 1 : a.H, V * P);
  const int64_t most = 1024 / team, each = (a.rows + kSms - 1) / kSms;
  const int whole = team < 32 ? 32 / team : 1;  // teams of a warp
  const int teams = each < most ? static_cast<int>(each + whole - 1) / whole * whole : static_cast<int>(most);
  const int threads = team * teams;
  const int64_t blocks = (a.rows + teams - 1) / teams;
  parts = blocks < kSms ? blocks : kSms;
  using R = Ring<T, V, P>;
  const void* kernel = reinterpret_cast<const void*>(norm_backward_kernel<T, W, V, P, kShifted>);
  const size_t smem = static_cast<size_t>(threads) * R::kBytes;
  if (smem > 47 * 1024) {  // (with the kernel's own 256 bytes: what needs no leave)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 * R::kBytes);
    if (e != cudaSuccess) return e;
  }
  void* args[] = {const_cast<NormBackwardArgs*>(&a), const_cast<int*>(&team), const_cast<int*>(&teams)};
  return launch_args(kernel, dim3(static_cast<unsigned>(parts)), threads, smem, stream, args);
}
template <typename T, typename W, int V, bool kShifted = false>
cudaError_t launch_backward_v(const NormBackwardArgs& a, int64_t& parts, cudaStream_t stream) {
  constexpr int kBytes = V * static_cast<int>(sizeof(T)), kFew = kBytes == 16 ? 1 : 4, kMost = 2 * kFew;
  // The fewer pieces a thread where their teams fill the SM or rows are few; else the more, of
  // smaller teams (8192 x 4096 bf16: 45.7 us with one piece, 46.1 with two, 8192 x 6144 68.9 and
  // 64.1, 512 x 8192 12.0 and 13.0).  Rows in registers have room for no more (5000 x 777 19.1 and 31.6,
  // 8192 x 4099 304 and, read twice, 140).
  const int64_t H = kShifted ? a.H + V - 1 : a.H;
  const int team = backward_team(H, V * kFew);
  const bool few = kBytes < 4 || a.rows <= 8 * kSms || 1024 / team * team >= 960;
  if (team <= 1024 && few) return launch_backward_p<T, W, V, kFew, kShifted>(a, parts, stream);
  if constexpr (kShifted) {  // (where shifted_fits)
    return launch_backward_p<T, W, V, kMost, true>(a, parts, stream);
  } else {
    if constexpr (kBytes >= 4)
      if (backward_team(H, V * kMost) <= 1024) return launch_backward_p<T, W, V, kMost, false>(a, parts, stream);
    cudaError_t e = launch(norm_backward_long_kernel<T, W, V>, dim3(static_cast<unsigned>(a.rows)), 512, stream, a);
    if (e != cudaSuccess) return e;
    parts = norm_parts(a.rows);
    const int64_t part_rows = (a.rows + parts - 1) / parts;
    const dim3 grid(static_cast<unsigned>((a.H + kColumnThreads - 1) / kColumnThreads), static_cast<unsigned>(parts));
    return launch(norm_columns_kernel<T>, grid, kColumnThreads, stream, a, part_rows);
  }
}
// Whether a row's shifted pieces of V elements fit a team.
bool shifted_fits(int64_t H, int V) { return backward_team(H + V - 1, 2 * V) <= 1024; }
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
    constexpr int V = Elem<T>::kVec;
    if (out_type == kTypeE4m3) return launch_norm_v<T, W, V, kTypeE4m3>(a, stream);
    if (out_type == kTypeE2m1) return launch_norm_v<T, W, V, kTypeE2m1>(a, stream);
    if (at.by(16)) return launch_norm_v<T, W, V, kTypeF32>(a, stream);
    // Many rows of 16-bit elements that 4-byte accesses can take, or that are narrow, one by one; the
    // others by frames.  (8192 rows with the residual: of 4100 49 us and, by frames, 55, of 101 4.2 and
    // 6.3, of 4099 105 and 59; 64 of 7001 4.6 and 3.8; floats, 4096 x 4099 59 and 43.)
    if constexpr (sizeof(T) == 2)
      if (a.rows > 2 * kSms && (at.by(4) || a.H <= 128))
        return at.by(4) ? launch_norm_v<T, W, 2, kTypeF32>(a, stream) : launch_norm_v<T, W, 1, kTypeF32>(a, stream);
    return launch_norm_frames<T, W>(a, stream);
  });
}

int64_t norm_parts(int64_t rows) { return rows < kMaxParts ? rows : kMaxParts; }

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
    // Rows at the same distance from an aligned address in all operands (and no shorter than a
    // piece, which then reaches no further than the next row), where there are many or they are
    // wide, and a team holds them; others by narrower accesses.  (bf16, shifted and narrow: 8192 x
    // 1001 20.4 us and 31.2, 8192 x 2050 38.5 and 47.1, 64 x 7001 7.8 and 11.7, but 500 x 251 6.4 and
    // 5.4, 100 x 4001 8.9 and 7.2.  2000 x 16380, which no team holds shifted: read twice by single
    // elements 165, by 4 bytes 87.)
    auto like_dx = [&](const void* p, int64_t ld) {
      return !p || (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(a.dx)) & 15) == 0 && (ld - a.H) % V == 0);
    };
    if (a.H >= V && (a.rows > 4 * kSms || a.H > 4096) && shifted_fits(a.H, V) && like_dx(a.dy, a.lddy) && like_dx(a.h, a.ldh) &&
        like_dx(a.dh, a.lddh))
      return launch_backward_v<T, W, V, true>(a, parts, stream);
    return at.by(4) ? launch_backward_v<T, W, V4>(a, parts, stream) : launch_backward_v<T, W, 1>(a, parts, stream);
  });
  if (e != cudaSuccess) return e;
  return launch(norm_sum_kernel, dim3(static_cast<unsigned>((a.H + 31) / 32)), 32 * kSumWarps, stream, a.parts, parts,
                a.H, a.dweight);
}

}  // namespace agg
