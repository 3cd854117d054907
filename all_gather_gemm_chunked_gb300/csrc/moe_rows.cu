// moe_rows.cu -- the router (top-k, softmax, expert-sorted layout) and the moves
// of rows between tokens and experts, with their gradients.
//
// All of it is bound by memory, or by latency where the batch is small, so each
// kernel reads its inputs once, with 16-byte accesses where rows are aligned, and
// keeps sums in 32-bit registers.  No atomic decides an order: the layout comes
// from counts and prefix sums, and every sum has a fixed order.

#include <math_constants.h>

#include "moe_rows.cuh"
#include "moe_types.cuh"

namespace agg {

namespace {
constexpr uint32_t kAll = 0xffffffffu;

// ------------------------------------------------------------------ router
// Logits as unsigned keys in the same order; 0 for what is not there.  -0 counts
// as +0.  Keys up to kKeyNegInf are never chosen.
constexpr uint32_t kKeyNegInf = 0x007fffffu;
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Keys of 16-bit logits: the value's bits in the same order above, 0xffff - expert below,
// so that one reduction finds the largest logit's lowest expert.  -0 counts as +0.
template <typename T>
__host__ __device__ constexpr uint32_t packed_neg_inf() {
  return (sizeof(T) == 2 && Elem<T>::kNegInf != 0 ? (0xffffu ^ Elem<T>::kNegInf) << 16 : 0u) | 0xffffu;
}
template <typename T>
__device__ __forceinline__ uint32_t pack_key(T v, int expert) {
  uint32_t b = 0;
  if constexpr (sizeof(T) == 2) b = *reinterpret_cast<const uint16_t*>(&v);
  if (b == 0x8000u) b = 0;
  return ((b ^ ((b >> 15) ? 0xffffu : 0x8000u)) << 16) | (0xffffu - static_cast<uint32_t>(expert));
}
template <typename T>
__device__ __forceinline__ float packed_logit(uint32_t key) {
  const uint32_t k = key >> 16;
  const uint16_t b = static_cast<uint16_t>(k ^ ((k >> 15) ? 0x8000u : 0xffffu));
  if constexpr (sizeof(T) == 2)
    return Elem<T>::get(*reinterpret_cast<const T*>(&b));
  else
    return 0.0f;
}
__device__ __forceinline__ int packed_expert(uint32_t key) {
  return static_cast<int>(0xffffu - (key & 0xffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Sorts a lane's keys, largest first (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = j; i < j + k; ++i)
          if (i + k < N && i / (2 * p) == (i + k) / (2 * p)) {
            const uint32_t hi = max(key[i], key[i + k]);
            key[i + k] = min(key[i], key[i + k]);
            key[i] = hi;
          }
}

// Two tokens by one warp (side by side: a token's rounds are a chain of warp
// reductions, and two chains take little longer than one): lane holds experts lane,
// lane + 32, ...; each of the k rounds takes the largest key left (one reduction) and
// the lowest expert that has it (a second one).  Writes the choices and their weights;
// `chosen` gets, in lane j < k, the j-th choice's expert (-1: none).  A token from
// `end` on is left out.
__host__ __device__ constexpr int tokens_of(int VPL) { return VPL <= 8 ? 2 : 1; }
template <typename T, int VPL>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t t0, int64_t end, int lane,
                                       int (&chosen)[tokens_of(VPL)]) {
  constexpr int kTokens = tokens_of(VPL);
  // 16-bit logits: value and expert in one key (16 bits of either), so that a round is
  // one reduction: the largest key is the largest logit's lowest expert.
  constexpr bool kPacked = sizeof(T) == 2;
  // Such a lane's keys are sorted first: a round then looks at its largest alone (16384
  // tokens of 256 experts, k 8: 18.3 us, 20.7 with all keys in each round; 128 experts,
  // k 1: 11.3 and 11.1).
  constexpr bool kSorted = kPacked && VPL <= 8;
  uint32_t key[kTokens][VPL];
  bool nan[kTokens];
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    const T* row = static_cast<const T*>(a.logits) + (t0 + n) * a.ld;
    T v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      v[i] = e < a.E && t0 + n < end ? row[e] : Elem<T>::put(-CUDART_INF_F);
    }
    nan[n] = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float f = Elem<T>::get(v[i]);
      const bool is_nan = f != f;
      nan[n] |= is_nan;
      key[n][i] = kPacked ? pack_key<T>(v[i], i * 32 + lane) : logit_key(f);
      if (i * 32 + lane >= a.E || is_nan) key[n][i] = 0u;
    }
  }
  float all[kTokens] = {};  // sum of exp(logit - largest) over all experts
  uint32_t mine[kTokens] = {};
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    if constexpr (kSorted) sort_keys(key[n]);
    nan[n] = __any_sync(kAll, nan[n]);
    chosen[n] = -1;
  }
  for (int j = 0; j < a.k; ++j) {
    uint32_t best[kTokens], top[kTokens];
    int bi[kTokens];
    bool any = false;
#pragma unroll
    for (int n = 0; n < kTokens; ++n) {
      best[n] = key[n][0];
      bi[n] = lane;
#pragma unroll
      for (int i = 1; i < (kSorted ? 1 : VPL); ++i) {
        if (kPacked) {
          best[n] = max(best[n], key[n][i]);
        } else if (key[n][i] > best[n]) {
          best[n] = key[n][i];
          bi[n] = i * 32 + lane;
        }
      }
      top[n] = __reduce_max_sync(kAll, best[n]);
      any |= top[n] > (kPacked ? packed_neg_inf<T>() : kKeyNegInf);
    }
    if (!any) break;
    if (j == 0 && !a.normalize) {
#pragma unroll
      for (int n = 0; n < kTokens; ++n) {
        const float m = kPacked ? packed_logit<T>(top[n]) : key_logit(top[n]);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (key[n][i] != 0u)
            all[n] += expf((kPacked ? packed_logit<T>(key[n][i]) : key_logit(key[n][i])) - m);
        all[n] = warp_sum(all[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < kTokens; ++n) {
      const bool real = top[n] > (kPacked ? packed_neg_inf<T>() : kKeyNegInf);
      int e;
      if (kPacked) {
        e = real ? packed_expert(top[n]) : -1;
        if constexpr (kSorted) {
          const bool taken = key[n][0] == top[n];
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (taken) key[n][i] = i + 1 < VPL ? key[n][i + 1] : 0u;
        } else {
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (key[n][i] == top[n]) key[n][i] = 0u;
        }
      } else {
        e = static_cast<int>(__reduce_min_sync(
            kAll, real && best[n] == top[n] ? static_cast<uint32_t>(bi[n]) : 0xffffffffu));
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (i * 32 + lane == e) key[n][i] = 0u;
      }
      if (lane == j && real) {
        mine[n] = top[n];
        chosen[n] = e;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    const float l = kPacked ? packed_logit<T>(mine[n]) : key_logit(mine[n]);
    const float m = __shfl_sync(kAll, l, 0);
    const float p = chosen[n] >= 0 ? expf(l - m) : 0.0f;
    const float sum = a.normalize ? warp_sum(p) : all[n];
    float w = chosen[n] >= 0 ? p / sum : 0.0f;
    if (nan[n] && chosen[n] >= 0) w = CUDART_NAN_F;
    if (lane < a.k && t0 + n < end) {
      a.weights[(t0 + n) * a.k + lane] = w;
      a.experts[(t0 + n) * a.k + lane] = chosen[n];
    }
  }
}

// The tokens of block b and of its warps: contiguous, in order.
struct Share {
  int64_t t0, t1;
};
__device__ __forceinline__ Share share_of(int64_t first, int64_t end, int64_t part, int64_t parts) {
  const int64_t n = end - first, per = (n + parts - 1) / parts;
  const int64_t a = first + part * per, b = a + per;
  return {a < end ? a : end, b < end ? b : end};
}

constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
// Tokens of a block: place() holds prefixes of its choices of an expert in 16 bits (in 32
// bits 1024 experts would take 128 KB of shared memory instead of 64).
constexpr int64_t kBlockTokens = 65535;

// Sum over the block's threads before this one (value of thread e at e).
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sums, int warp,
                                                    int lane) {
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(kAll, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const uint32_t own = warp_sums[lane];
    uint32_t w = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(kAll, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w - own;
  }
  __syncthreads();
  return warp_sums[warp] + s - v;
}

// Place a block's choices c0 .. c1 - 1 (token * k + j), 32 a warp at a time.  A row's
// place is its expert's first row, plus the expert's choices in earlier blocks, in
// earlier warps of this block, in this warp's earlier steps and in earlier lanes (a
// match of the experts over the warp): counts and prefix sums alone, so the order
// within an expert is the tokens' (a token chooses an expert at most once).
// smem: [kRouteWarps][E] uint16 counts and, later, counts of this block's earlier choices
// (a block has at most kBlockTokens tokens, see route_blocks), then E uint32 first rows, 32 warp sums, the number of rows in use, E counts of
// earlier blocks.  `blocks`: blocks that place, with their counts if more than one.
__device__ void place(const RouteArgs& a, int64_t c0, int64_t c1, int blocks, uint8_t* smem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint16_t* cnt = reinterpret_cast<uint16_t*>(smem);
  uint32_t* base = reinterpret_cast<uint32_t*>(smem + ((kRouteWarps * a.E * 2 + 15) & ~15));
  uint32_t* sums = base + a.E;
  // this warp's choices: a multiple of 32, the first 64 of them held in registers
  const int64_t per = ((c1 - c0 + kRouteThreads - 1) / kRouteThreads) * 32;
  const int64_t w0 = c0 + warp * per, w1 = w0 + per < c1 ? w0 + per : c1;
  auto load = [&](int64_t c) { return c < w1 ? __ldcg(a.experts + c) : -1; };
  const int held0 = load(w0 + lane), held1 = load(w0 + 32 + lane);
  auto expert_at = [&](int64_t c) { return c == w0 ? held0 : c == w0 + 32 ? held1 : load(c + lane); };
  for (int i = threadIdx.x; i < kRouteWarps * a.E / 2; i += kRouteThreads)
    reinterpret_cast<uint32_t*>(cnt)[i] = 0;
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) base[e] = sums[33 + e] = 0;
  __syncthreads();
  uint16_t* mine = cnt + warp * a.E;
  uint32_t match0 = 0, match1 = 0;  // held too: a match takes a step for each distinct expert
  for (int64_t c = w0; c < w1; c += 32) {
    const int x = expert_at(c);
    const uint32_t same = __match_any_sync(kAll, x);
    if (c == w0) match0 = same;
    if (c == w0 + 32) match1 = same;
    if (x >= 0 && lane == __ffs(same) - 1) mine[x] = static_cast<uint16_t>(mine[x] + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  const int e = threadIdx.x;
  uint32_t total = 0, before = 0;
  if (blocks == 1) {
    if (e < a.E)
#pragma unroll 16
      for (int w = 0; w < kRouteWarps; ++w) total += cnt[w * a.E + e];
  } else {
    // groups of E threads read the blocks' counts side by side
    uint32_t* early = sums + 33;  // the earlier blocks' part (base holds the totals)
    const int groups = kRouteThreads / a.E;
    const int g = e / a.E, x = e - g * a.E;
    uint32_t all = 0, own = 0;
    if (g < groups)
      for (int b0 = g; b0 < blocks; b0 += 8 * groups) {
        uint32_t c[8];  // eight loads in flight, whatever is left
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int b = b0 + i * groups;
          c[i] = b < blocks ? static_cast<uint32_t>(__ldcg(a.counts + b * a.E + x)) : 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          all += c[i];
          if (b0 + i * groups < static_cast<int>(blockIdx.x)) own += c[i];
        }
      }
    // integer additions: the same in any order
    if (all) atomicAdd(&base[x], all);
    if (own) atomicAdd(&early[x], own);
    __syncthreads();
    if (e < a.E) {
      total = base[e];
      before = early[e];
    }
    __syncthreads();
  }
  const uint32_t first = block_exclusive(e < a.E ? total : 0u, sums, warp, lane);
  if (e < a.E) {
    base[e] = first + before;
    if (blockIdx.x == 0) a.offsets[e + 1] = static_cast<int32_t>(first + total);
    if (blockIdx.x == 0 && e == 0) a.offsets[0] = 0;
    uint32_t run = 0;  // counts to the counts of earlier warps
#pragma unroll
    for (int v0 = 0; v0 < kRouteWarps; v0 += 8) {
      uint32_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = cnt[(v0 + w) * a.E + e];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        cnt[(v0 + w) * a.E + e] = static_cast<uint16_t>(run);
        run += c[w];
      }
    }
    if (e == a.E - 1) sums[32] = first + total;  // rows in use
  }
  __syncthreads();
  for (int64_t c = w0; c < w1; c += 32) {
    const int x = expert_at(c);
    const uint32_t same = c == w0 ? match0 : c == w0 + 32 ? match1 : __match_any_sync(kAll, x);
    int32_t row = -1;
    if (x >= 0) {
      row = static_cast<int32_t>(base[x] + mine[x] + __popc(same & ((1u << lane) - 1u)));
      a.order[row] = static_cast<int32_t>(c + lane);
    }
    __syncwarp();
    if (x >= 0 && lane == __ffs(same) - 1) mine[x] = static_cast<uint16_t>(mine[x] + __popc(same));
    if (c + lane < w1) a.slots[c + lane] = row;
    __syncwarp();
  }
  for (int64_t s = sums[32] + static_cast<int64_t>(blocks == 1 ? 0 : blockIdx.x) * kRouteThreads + threadIdx.x;
       s < a.T * a.k; s += static_cast<int64_t>(blocks) * kRouteThreads)
    a.order[s] = -1;
}

size_t place_smem(int E) {
  return ((static_cast<size_t>(kRouteWarps) * E * 2 + 15) & ~size_t{15}) + 2 * E * 4 + 33 * 4;
}

// Few tokens: a cluster of blocks chooses, its first block places, one launch.
// (Choosing is bound by instructions: 75 tokens of 182 experts on one SM took 8 us.)
template <typename T, int VPL>
__global__ void __launch_bounds__(kRouteThreads) route_one_kernel(const RouteArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31;
  constexpr int kTokens = tokens_of(VPL);
  // tokens go round the blocks, so that a block's warps are few where tokens are
  for (int64_t t = (static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x) * kTokens; t < a.T;
       t += static_cast<int64_t>(kRouteWarps) * gridDim.x * kTokens) {
    int chosen[kTokens];
    choose<T, VPL>(a, t, a.T, lane, chosen);
  }
  // the choices of all blocks are written
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x == 0) place(a, 0, a.T * a.k, 1, smem);
}

// More: one kernel chooses and counts the choices of each block's tokens, the
// next places them.  Warps take tokens in pairs (one each cost as much as two).
// (2048 tokens of 64 experts, k 4: 6.9 us; 16384 of 256, k 8: 18.3 us.)
template <typename T, int VPL>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const RouteArgs a) {
  pdl_wait();
  __shared__ uint32_t cnt[kMaxExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) cnt[e] = 0;
  __syncthreads();
  const Share blk = share_of(0, a.T, blockIdx.x, gridDim.x);
  constexpr int kTokens = tokens_of(VPL);
  for (int64_t t = blk.t0 + warp * kTokens; t < blk.t1; t += kRouteWarps * kTokens) {
    int chosen[kTokens];
    choose<T, VPL>(a, t, blk.t1, lane, chosen);
#pragma unroll
    for (int n = 0; n < kTokens; ++n)
      if (chosen[n] >= 0) atomicAdd(&cnt[chosen[n]], 1u);  // (integer counts: any order)
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = static_cast<int32_t>(cnt[e]);
}

__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const RouteArgs a) {
  pdl_wait();
  extern __shared__ __align__(16) uint8_t smem[];
  const Share blk = share_of(0, a.T, blockIdx.x, gridDim.x);
  place(a, blk.t0 * a.k, blk.t1 * a.k, static_cast<int>(gridDim.x), smem);
}

// Gradient of the logits, one warp per token.  normalize: w_j (dw_j - sum w dw) at the
// chosen experts, 0 elsewhere.  Otherwise p_e ([e chosen] dw - sum w dw) with the softmax
// p over all experts, which is computed again from the logits.  The row is written as
// for experts that were not chosen first, then, behind a warp barrier, the k choices.
// (16384 x 128, k 8, bf16: 3.2 us, over all experts 6.5.)
template <typename T>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteArgs a,
                                                             const float* dweights,
                                                             T* dlogits) {
  pdl_enter();
  constexpr int V = Elem<T>::kVec;
  const int lane = threadIdx.x & 31;
  const bool vec = a.E % V == 0 && (reinterpret_cast<uintptr_t>(dlogits) & 15u) == 0;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
       t < a.T; t += warps) {
    float w = 0.0f, dw = 0.0f;
    int expert = -1;
    if (lane < a.k) {
      w = a.weights[t * a.k + lane];
      expert = a.experts[t * a.k + lane];
      dw = dweights[t * a.k + lane];
    }
    T* out = dlogits + t * a.E;
    const bool chosen = expert >= 0 && expert < a.E;
    const float dot = warp_sum(chosen ? w * dw : 0.0f);
    if (a.normalize) {
      if (vec) {
        for (int e = lane * V; e < a.E; e += 32 * V)
          *reinterpret_cast<uint4*>(out + e) = make_uint4(0, 0, 0, 0);
      } else {
        for (int e = lane; e < a.E; e += 32) out[e] = Elem<T>::put(0.0f);
      }
    } else {
      const T* row = static_cast<const T*>(a.logits) + t * a.ld;
      float m = -CUDART_INF_F, s = 0.0f;
      for (int e = lane; e < a.E; e += 32) m = fmaxf(m, Elem<T>::get(row[e]));
      m = warp_max(m);
      // (a token with no finite logit has no choices: its gradient is zero)
      const bool some = m != -CUDART_INF_F;
      if (some)
        for (int e = lane; e < a.E; e += 32) s += expf(Elem<T>::get(row[e]) - m);
      const float scale = some ? -dot / warp_sum(s) : 0.0f;
      for (int e = lane; e < a.E; e += 32)
        out[e] = Elem<T>::put(some ? expf(Elem<T>::get(row[e]) - m) * scale : 0.0f);
    }
    __syncwarp();
    if (chosen) out[expert] = Elem<T>::put(w * (dw - dot));
  }
}

// ------------------------------------------------------------------ rows
constexpr int kRowLog = 8, kRowThreads = 1 << kRowLog;

// A thread moves pieces of V elements, a row's threads apart: of 16 bytes, or where rows
// are not 16-byte aligned single elements, several of them, so that as many bytes are in
// flight.  (8192 tokens, k 4, H 4096, bf16: aligned rows combine in 52 us, their gradient
// takes 90, gather 65; with odd pitches 80, 120 and 91, one element a thread 182, 220 and
// 528.)
constexpr int kPieces = 4;
constexpr int kGatherPieces = 8, kGatherVec = 4;  // (gather with one 16-byte piece 80 us)
// Short rows share a block, each with the warps that it fills: a block a row is bound by
// the time a block lives.  (5317 tokens, k 3, H 118: combine 3.8 us against 6.7, gradient
// 6.4 and 12.6, gather 5.5 and 17.0; 8192 tokens, k 8, H 1000: gradient 50 and 66.  Rows
// that fill a block keep their number of threads as a constant: as a variable it cost
// combine registers, 60 us against 52 for 8192 tokens, k 4, H 4096.)
struct RowShape {
  int log;       // threads of a row, a power of two from 32 on
  unsigned x, y; // blocks over the rows, blocks over a row
};
RowShape row_shape(int64_t rows, int64_t H, int per_thread) {
  RowShape s{kRowLog, 0, 0};
  while (s.log > 5 && (H + per_thread - 1) / per_thread <= (1 << (s.log - 1))) --s.log;
  const int64_t per = kRowThreads >> s.log, span = static_cast<int64_t>(per_thread) << s.log;
  s.x = static_cast<unsigned>((rows + per - 1) / per);
  s.y = static_cast<unsigned>((H + span - 1) / span);
  return s;
}

// 2^log threads per row of out and as many times V * N columns.  (32768 rows of 4096: 66 us,
// 5.1 TB/s of reads and writes.)
template <typename T, int V, int N, bool kShort>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(int64_t T_, int k, int64_t H, int log_,
                                                             const T* x, int64_t ldx,
                                                             const int32_t* order,
                                                             T* __restrict__ out) {
  pdl_enter();
  const int log = kShort ? log_ : kRowLog, step = V << log;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * (kRowThreads >> log) + (threadIdx.x >> log);
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * step * N + (threadIdx.x & ((1 << log) - 1)) * V;
  if (c0 >= H || s >= T_ * k) return;
  const int32_t o = order[s];
  const int64_t t = o / k;
  const bool in = o >= 0 && t < T_;
  Raw<T, V> r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t c = c0 + i * step;
    if (in && c < H) r[i].load(x + t * ldx + c);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t c = c0 + i * step;
    float f[V] = {};
    if (in) r[i].get(f);
    if (c < H) store_elems<T, V>(out + s * H + c, f);
  }
}

// 2^log threads per token and as many times V * N columns: the k rows are read with four
// loads a piece in flight per thread and summed in registers in the order of j.  Bound by
// the bytes in flight (a token's slots come first, then its rows): the loads wait as they
// came and six blocks share an SM (8192 tokens, k 4, H 4096: 51 us, 6.6 TB/s; as floats,
// four blocks, 92).
template <typename T, int V, int N, bool kShort>
__global__ void __launch_bounds__(kRowThreads, kShort ? 5 : 6) combine_kernel(int64_t T_, int k, int64_t H, int log_,
                                                                 const T* y, int64_t ldy,
                                                                 const int32_t* slots,
                                                                 const float* weights,
                                                                 T* __restrict__ out) {
  pdl_enter();
  const int log = kShort ? log_ : kRowLog, step = V << log;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads >> log) + (threadIdx.x >> log);
  const int S = static_cast<int>(T_ * k);
  const int64_t c = static_cast<int64_t>(blockIdx.y) * step * N + (threadIdx.x & ((1 << log) - 1)) * V;
  if (c >= H || t >= T_) return;
  const int64_t left = H - c;  // pieces from there on are outside
  float acc[N][V] = {};
  slots += t * k;
  if (weights) weights += t * k;
  for (int j0 = 0; j0 < k; j0 += 4) {
    Raw<T, V> r[4][N];
    int s[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      s[u] = j0 + u < k ? slots[j0 + u] : -1;
      if (s[u] >= S) s[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s[u] >= 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i * step < left) r[u][i].load(y + s[u] * ldy + c + i * step);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s[u] >= 0) {
        const float w = weights ? weights[j0 + u] : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float f[V];
          r[u][i].get(f);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[i][v] = fmaf(w, f[v], acc[i][v]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * step < left) store_elems<T, V>(out + t * H + c + i * step, acc[i]);
}

// 2^log threads per token: dy rows and, over the whole row, the dot products.  Four
// choices at a time; dout is read again for the next four.  (8192 tokens, k 4, H 4096:
// 90 us, 6.7 TB/s.)
template <typename T, int V, int N, bool kShort>
__global__ void __launch_bounds__(kRowThreads, 4) combine_backward_kernel(
    int64_t T_, int k, int64_t H, int log_, const T* dout, int64_t ldd,
    const T* y, int64_t ldy, const int32_t* slots,
    const float* weights, const int32_t* offsets_end,
    T* __restrict__ dy, float* __restrict__ dweights) {
  pdl_enter();
  __shared__ float part[kRowThreads / 32][4];
  const int log = kShort ? log_ : kRowLog, step = V << log;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int thread = threadIdx.x & ((1 << log) - 1);  // of the token
  const int64_t per = kRowThreads >> log, S = T_ * k;
  const int64_t t = blockIdx.x * per + (threadIdx.x >> log);
  for (int j0 = 0; j0 < k; j0 += 4) {
    int64_t s[4];
    float w[4], dot[4] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u;
      s[u] = j < k && t < T_ ? slots[t * k + j] : -1;
      if (s[u] >= S) s[u] = -1;
      w[u] = s[u] >= 0 ? weights[t * k + j] : 0.0f;
    }
    for (int64_t c = thread * V; c < H && t < T_; c += step * N) {
      Raw<T, V> r[4][N], rg[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * step < H - c) rg[i].load(dout + t * ldd + c + i * step);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (s[u] >= 0)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (i * step < H - c) r[u][i].load(y + s[u] * ldy + c + i * step);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i * step >= H - c) break;
        float g[V];
        rg[i].get(g);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (s[u] >= 0) {
            float d[V], f[V];
            r[u][i].get(f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
              dot[u] = fmaf(g[v], f[v], dot[u]);
              d[v] = w[u] * g[v];
            }
            store_elems<T, V>(dy + s[u] * H + c + i * step, d);
          }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      dot[u] = warp_sum(dot[u]);
      if (lane == 0) part[warp][u] = dot[u];
    }
    __syncthreads();
    if (thread < 4 && j0 + thread < k && t < T_) {
      float sum = 0.0f;
      for (int i = 0; i < (1 << log) / 32; ++i) sum += part[warp + i][thread];
      dweights[t * k + j0 + thread] = sum;
    }
    __syncthreads();
  }
  if (offsets_end) {  // rows that belong to no choice
    const int64_t end = *offsets_end;
    const float zero[V] = {};
    for (int64_t r = (end < 0 ? 0 : end) + t; r < S; r += gridDim.x * per)
      for (int64_t c = thread * V; c < H; c += step)
        store_elems<T, V>(dy + r * H + c, zero);
  }
}

bool aligned(const void* p, int64_t ld, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * esize) % 16 == 0;
}

template <typename T>
const void* route_one_fn(int vpl) {
  switch (vpl) {
    case 1: return reinterpret_cast<const void*>(&route_one_kernel<T, 1>);
    case 2: return reinterpret_cast<const void*>(&route_one_kernel<T, 2>);
    case 4: return reinterpret_cast<const void*>(&route_one_kernel<T, 4>);
    case 8: return reinterpret_cast<const void*>(&route_one_kernel<T, 8>);
    case 16: return reinterpret_cast<const void*>(&route_one_kernel<T, 16>);
    default: return reinterpret_cast<const void*>(&route_one_kernel<T, 32>);
  }
}
template <typename T>
const void* route_choose_fn(int vpl) {
  switch (vpl) {
    case 1: return reinterpret_cast<const void*>(&route_choose_kernel<T, 1>);
    case 2: return reinterpret_cast<const void*>(&route_choose_kernel<T, 2>);
    case 4: return reinterpret_cast<const void*>(&route_choose_kernel<T, 4>);
    case 8: return reinterpret_cast<const void*>(&route_choose_kernel<T, 8>);
    case 16: return reinterpret_cast<const void*>(&route_choose_kernel<T, 16>);
    default: return reinterpret_cast<const void*>(&route_choose_kernel<T, 32>);
  }
}
int values_per_lane(int E) { return E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : E <= 256 ? 8 : E <= 512 ? 16 : 32; }

// Calls F<T>() for the element type.
#define AGG_FOR_TYPE(dtype, ...)                    \
  [&]() -> cudaError_t {                            \
    if ((dtype) == kTypeF32) {                      \
      using T = float;                              \
      __VA_ARGS__                                   \
    }                                               \
    if ((dtype) == kTypeF16) {                      \
      using T = __half;                             \
      __VA_ARGS__                                   \
    }                                               \
    using T = __nv_bfloat16;                        \
    __VA_ARGS__                                     \
  }()

}  // namespace

// One cluster serves up to 512 tokens and 1536 choices (one block places them all);
// beyond that blocks of at least 32 tokens, sixteen warps' pairs, one block per SM, and
// from 152 * kBlockTokens tokens on as many as hold them.
// (One cluster and two kernels: 64 experts, k 4: 256 tokens 5.9 us and 6.4, 384 7.0 and
// 6.6; 256 experts, k 8: 192 tokens 8.1 and 8.5, 256 tokens 9.4 and 8.6; 128 experts, k 1:
// 384 tokens 5.3 and 6.9.  Blocks of 16 tokens took 7.8 us against 7.2 for 2048 tokens of
// 64 experts, of 64 tokens 7.7.)
int route_blocks(int64_t T, int k) {
  if (T <= 512 && T * k <= 1536) return 1;
  const int64_t b = (T + 31) / 32, least = (T + kBlockTokens - 1) / kBlockTokens;
  return static_cast<int>(b < 152 ? b : least < 152 ? 152 : least);
}
// A cluster's blocks: one for as few tokens as it takes, else eight.
// (64 experts, k 4: 16 tokens 3.7 us by one block, 4.0 by eight, 32 tokens 4.1 and 4.0;
// 256 experts, k 8: 4.8 and 4.8, 5.8 and 5.0.)
int cluster_blocks(int64_t T) { return T <= 16 ? 1 : 8; }

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  const int vpl = values_per_lane(a.E), blocks = route_blocks(a.T, a.k);
  const size_t smem = place_smem(a.E);
  void* args[] = {const_cast<RouteArgs*>(&a)};
  return AGG_FOR_TYPE(a.dtype, {
    if (blocks == 1) {
      const void* fn = route_one_fn<T>(vpl);
      if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
        if (e != cudaSuccess) return e;
      }
      const int cluster = cluster_blocks(a.T);
      return launch_args(fn, dim3(cluster), kRouteThreads, smem, stream, args, cluster);
    }
    cudaError_t e = launch_args(route_choose_fn<T>(vpl), dim3(blocks), kRouteThreads, 0, stream, args);
    if (e != cudaSuccess) return e;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(route_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(smem))) != cudaSuccess)
      return e;
    return launch_args(reinterpret_cast<const void*>(&route_place_kernel), dim3(blocks), kRouteThreads,
                       smem, stream, args);
  });
}

cudaError_t launch_route_backward(const RouteArgs& a, const float* dweights, void* dlogits,
                                  cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const int64_t want = (a.T + 7) / 8;
  const int grid = static_cast<int>(want < 152 * 8 ? want : 152 * 8);
  return AGG_FOR_TYPE(a.dtype, {
    return launch(route_backward_kernel<T>, dim3(grid), 256, stream, a, dweights, static_cast<T*>(dlogits));
  });
}

cudaError_t launch_gather(int64_t T_, int k, int64_t H, int dtype, const void* x, int64_t ldx,
                          const int32_t* order, void* out, cudaStream_t stream) {
  if (T_ == 0) return cudaSuccess;
  return AGG_FOR_TYPE(dtype, {
    constexpr int V = Elem<T>::kVec;
    const bool vec = H % V == 0 && aligned(x, ldx, sizeof(T)) && aligned(out, H, sizeof(T));
    const RowShape s = row_shape(T_ * k, H, vec ? kGatherVec * V : kGatherPieces);
    const dim3 grid(s.x, s.y);
    auto go = [&](auto kernel) {
      return launch(kernel, grid, kRowThreads, stream, T_, k, H, s.log, static_cast<const T*>(x), ldx, order,
                    static_cast<T*>(out));
    };
    if (s.log == kRowLog)
      return vec ? go(gather_kernel<T, V, kGatherVec, false>) : go(gather_kernel<T, 1, kGatherPieces, false>);
    return vec ? go(gather_kernel<T, V, kGatherVec, true>) : go(gather_kernel<T, 1, kGatherPieces, true>);
  });
}

cudaError_t launch_combine(int64_t T_, int k, int64_t H, int dtype, const void* y, int64_t ldy,
                           const int32_t* slots, const float* weights, void* out,
                           cudaStream_t stream) {
  if (T_ == 0) return cudaSuccess;
  return AGG_FOR_TYPE(dtype, {
    constexpr int V = Elem<T>::kVec;
    const bool vec = H % V == 0 && aligned(y, ldy, sizeof(T)) && aligned(out, H, sizeof(T));
    const RowShape s = row_shape(T_, H, vec ? V : kPieces);
    const dim3 grid(s.x, s.y);
    auto go = [&](auto kernel) {
      return launch(kernel, grid, kRowThreads, stream, T_, k, H, s.log, static_cast<const T*>(y), ldy, slots,
                    weights, static_cast<T*>(out));
    };
    if (s.log == kRowLog) return vec ? go(combine_kernel<T, V, 1, false>) : go(combine_kernel<T, 1, kPieces, false>);
    return vec ? go(combine_kernel<T, V, 1, true>) : go(combine_kernel<T, 1, kPieces, true>);
  });
}

cudaError_t launch_combine_backward(int64_t T_, int k, int64_t H, int dtype, const void* dout,
                                    int64_t ldd, const void* y, int64_t ldy, const int32_t* slots,
                                    const float* weights, const int32_t* offsets_end, void* dy,
                                    float* dweights, cudaStream_t stream) {
  if (T_ == 0) return cudaSuccess;
  return AGG_FOR_TYPE(dtype, {
    constexpr int V = Elem<T>::kVec;
    const bool vec = H % V == 0 && aligned(y, ldy, sizeof(T)) && aligned(dout, ldd, sizeof(T)) &&
                     aligned(dy, H, sizeof(T));
    const RowShape s = row_shape(T_, H, vec ? V : kPieces);
    auto go = [&](auto kernel) {
      return launch(kernel, dim3(s.x), kRowThreads, stream, T_, k, H, s.log, static_cast<const T*>(dout), ldd,
                    static_cast<const T*>(y), ldy, slots, weights, offsets_end, static_cast<T*>(dy), dweights);
    };
    if (s.log == kRowLog)
      return vec ? go(combine_backward_kernel<T, V, 1, false>) : go(combine_backward_kernel<T, 1, kPieces, false>);
    return vec ? go(combine_backward_kernel<T, V, 1, true>) : go(combine_backward_kernel<T, 1, kPieces, true>);
  });
}

}  // namespace agg
