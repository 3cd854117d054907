// experts_kernel.cu -- matrix products grouped by expert, for ragged groups, as
// one persistent kernel of CTA pairs for sm_103a.
//
// All four products have the form out[row][wide] = sum over red of W * R, where the
// wide operand W is the MMA's M and the row operand R its N:
//
//   forward          W = w[e] (K x N, wide contiguous: MN-major),  R = x rows (K-major)
//   input gradient   W = w[e] (red contiguous: K-major),           R = dy rows (K-major)
//   weight gradient  W = dy^T (MN-major), R = x^T (MN-major), red = the expert's rows
//   e4m3             W = wq[e] (N x K: K-major), R = xq rows (K-major)
//
// Rows on the N side: a pair's N takes any multiple of 32 up to 256 where its M is
// 256, so a group of 300 rows costs two tiles of 160 and one of 7 rows a tile of 32,
// not 512 and 256 rows.  A lane of the accumulator is then one column of the
// output: a warp's store of one row writes 32 neighbouring elements.
//
// A pair of CTAs (cta_group::2) holds a tile of 256 x w: each CTA stages its 128 of
// the wide dimension and half of the rows, 128 bytes of the sum's dimension a
// k-block, and the even CTA issues the MMAs.
//
//   warp 0      TMA: streams k-blocks of both operands into a ring of stages
//   warp 1      MMA (even CTA, one thread); owns the TMEM allocation
//   warps 2-9   epilogue: TMEM lane quadrant warp % 4, half of the tile's columns
//
// Work: tiles in expert order, and inside an expert in groups of 8 row tiles by all
// wide tiles, so that the tiles in flight share operands in L2.  Unit u of pair p is
// p, p + pairs, ...; every role computes the same list from the offsets, which the
// CTA reads into shared memory first.  Where there are too few tiles for the pairs,
// the sums are cut into S parts (choose_split): each warp stores its part's sums,
// and the warp that arrives last adds the S parts in their order, so that nobody
// waits and the result does not depend on the order of arrival.
//
// e4m3: scales differ per 128 along the sum, so each k-block's sum leaves TMEM and
// is multiplied and added into 32-bit registers (128 columns a thread); two
// accumulators alternate, and the MMA runs on meanwhile.
//
// Rows beyond a group's end belong to the next group: they are multiplied along and
// not stored (rows on the N side do not mix).  In the weight gradient they would
// enter the sums, and an infinity or NaN among them would even survive a product
// with zero, so there the last k-block's surplus rows are overwritten with zeros
// in shared memory before the MMA reads them.
//
// Every wait is bounded; on a timeout the kernel records a status word, drains what
// it has in flight, frees TMEM and returns.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts_kernel.cuh"
#include "fused_kernel.cuh"
#include "moe_rows.cuh"
#include "sm103.cuh"

namespace agg {

namespace {
constexpr int kWBytes = 128 * 128;  // a CTA's wide operand per k-block: 128 x 128 bytes

__host__ __device__ constexpr int rows_per_cta(int BN) { return BN / 2; }
__host__ __device__ constexpr int r_bytes(int BN) { return rows_per_cta(BN) * 128; }
// Stages that fit: 6 of 32 KB, or 10 of 20 KB for short row tiles, where the bytes
// in flight are the weights' alone.
__host__ __device__ constexpr int stages_of(int BN) { return BN == kXRows ? 6 : 10; }
constexpr int kScaleBytes = 8 * 2 * 128 * 4;  // e4m3: each epilogue warp's row scales, two k-blocks
constexpr int kTableBytes = (2 * (kMaxExperts + 1) * 4 + 15) & ~15;
__host__ __device__ constexpr int smem_bytes(int BN, bool fp8) {
  return stages_of(BN) * (kWBytes + r_bytes(BN)) + (fp8 ? kScaleBytes : 0) + kTableBytes + 512 +
         1024 /*alignment*/;
}
static_assert(smem_bytes(kXRows, true) <= 227 * 1024 && smem_bytes(kXFewRows, true) <= 227 * 1024,
              "shared memory of an SM");

__device__ __forceinline__ void set_status(uint32_t* status, uint32_t kind, uint32_t detail) {
  if (atomicCAS(status, 0u, kind) == 0u) atomicExch(status + 1, detail);
}

// tcgen05.mma of e4m3 operands (K = 32), pair form.
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Arrive on a barrier of either CTA of the pair without a cluster-scope release:
// for arrivals that publish no memory writes (an accumulator that has been read:
// tcgen05 fences order that).  The release waits for the warp's earlier stores and
// loads, about a microsecond under load: too long once per k-block.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// ------------------------------------------------------------------ work
// A unit of work, the same for every role of both CTAs.
struct Unit {
  int32_t e;         // expert
  int32_t row0;      // first input row of the tile (weight gradient: of the group)
  int32_t cnt;       // rows of the output in the tile
  int32_t w;         // columns of the MMA: cnt rounded up to a multiple of 32
  int32_t n0;        // first of the wide dimension
  int32_t kt0;       // weight gradient: first output row of the tile
  int32_t kb0, kb1;  // k-blocks
  int32_t red_rows;  // weight gradient: rows of the group
  int32_t tile, part;
};

template <int OP>
__host__ __device__ constexpr int block_k() { return OP == kOpFp8 ? 128 : 64; }

template <int OP, int BN>
struct Schedule {
  const ExpertsParams& p;
  const int32_t* off;   // [E + 1] row offsets
  const int32_t* pre;   // [E + 1] row tiles before each expert
  int32_t wt;           // wide tiles
  int32_t kt;           // weight gradient: output row tiles per expert
  int32_t KB;           // k-blocks of a whole sum
  int32_t split;        // parts of each tile's sum
  int32_t units, pair, pairs;

  __device__ __forceinline__ Schedule(const ExpertsParams& p_, const int32_t* off_,
                                      const int32_t* pre_)
      : p(p_), off(off_), pre(pre_) {
    wt = (p.wide + kXWide - 1) / kXWide;
    pair = blockIdx.x / 2;
    pairs = gridDim.x / 2;
    if constexpr (OP == kOpWeight) {
      kt = (p.out_rows + BN - 1) / BN;
      KB = 0;
      split = 1;
      units = p.E * wt * kt;
    } else {
      kt = 0;
      KB = (p.red + block_k<OP>() - 1) / block_k<OP>();
      const int32_t tiles = pre[p.E] * wt;
      split = choose_split(tiles);
      units = tiles * split;
    }
  }

  // Parts that make the longest pair's share shortest: a round of the pairs costs
  // its k-blocks and about three more for a tile's start and end.
  __device__ __forceinline__ int32_t choose_split(int32_t tiles) const {
    if (tiles == 0 || tiles >= 2 * pairs || p.max_units == 0) return 1;
    int32_t best = 1, cost = 0x7fffffff;
    for (int32_t s = 1; s <= 16 && (s == 1 || (KB >= 4 * s && tiles * s <= p.max_units)); ++s) {
      const int32_t c = ((tiles * s + pairs - 1) / pairs) * ((KB + s - 1) / s + 3);
      if (c < cost) {
        cost = c;
        best = s;
      }
    }
    return best;
  }

  __device__ __forceinline__ bool get(int32_t i, Unit& u) const {
    const int64_t id = static_cast<int64_t>(i) * pairs + pair;
    if (id >= units) return false;
    const int32_t unit = static_cast<int32_t>(id);
    if constexpr (OP == kOpWeight) {
      const int32_t per = wt * kt;
      u.e = unit / per;
      int32_t r = unit - u.e * per;
      const int32_t g = r / (kXGroup * wt);
      r -= g * (kXGroup * wt);
      const int32_t gw = kt - g * kXGroup < kXGroup ? kt - g * kXGroup : kXGroup;
      const int32_t x = r / gw;
      u.n0 = x * kXWide;
      u.kt0 = (g * kXGroup + r - x * gw) * BN;
      u.cnt = p.out_rows - u.kt0 < BN ? p.out_rows - u.kt0 : BN;
      // (the halves of the two CTAs start at multiples of 64 columns)
      u.w = (u.cnt + 127) & ~127;
      u.row0 = off[u.e];
      u.red_rows = off[u.e + 1] - u.row0;
      u.kb0 = 0;
      u.kb1 = (u.red_rows + 63) / 64;
      u.tile = unit;
      u.part = 0;
    } else {
      u.tile = unit / split;
      u.part = unit - u.tile * split;
      // the expert whose row tiles hold this one
      int32_t lo = 0, hi = p.E;
      while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (pre[mid] * wt <= u.tile) lo = mid; else hi = mid;
      }
      u.e = lo;
      const int32_t nt = pre[lo + 1] - pre[lo], cnt = off[lo + 1] - off[lo];
      int32_t r = u.tile - pre[lo] * wt;
      const int32_t g = r / (kXGroup * wt);
      r -= g * (kXGroup * wt);
      const int32_t gw = nt - g * kXGroup < kXGroup ? nt - g * kXGroup : kXGroup;
      const int32_t x = r / gw;
      u.n0 = x * kXWide;
      // the group's rows in nt tiles of equal width, a multiple of 32
      u.w = ((cnt + nt - 1) / nt + 31) & ~31;
      const int32_t first = (g * kXGroup + r - x * gw) * u.w;
      u.row0 = off[lo] + first;
      u.cnt = cnt - first < u.w ? cnt - first : u.w;
      u.kt0 = 0;
      u.red_rows = 0;
      u.kb0 = static_cast<int32_t>(static_cast<int64_t>(KB) * u.part / split);
      u.kb1 = static_cast<int32_t>(static_cast<int64_t>(KB) * (u.part + 1) / split);
    }
    return true;
  }
};

// Offsets to shared memory, checked, and the row tiles before each expert.
// Returns false (to every thread) if the offsets are no layout of the rows.
template <int BN>
__device__ bool load_table(const ExpertsParams& p, int32_t* off, int32_t* pre, int32_t* flag) {
  if (threadIdx.x == 0) *flag = 0;
  for (int e = threadIdx.x; e <= p.E; e += kXThreads)
    off[e] = p.offsets ? p.offsets[e] : (e == 0 ? 0 : p.rows);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kXThreads)
    if (off[e] < 0 || off[e + 1] < off[e] || off[e + 1] > p.rows) *flag = 1;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int32_t carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int32_t n = e < p.E ? off[e + 1] - off[e] : 0;
      int32_t s = n > 0 ? (n - 1) / BN + 1 : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      if (e < p.E) pre[e + 1] = carry + s;
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
  return *flag == 0;
}

struct Ring {
  uint8_t* w;
  uint8_t* r;
  uint64_t* full;   // the pair's bytes are counted on the even CTA's
  uint64_t* empty;
  uint64_t* tfull;  // accumulators, on both CTAs
  uint64_t* tempty; // on the even CTA: 16 epilogue warps
  uint64_t* tail;   // weight gradient: this CTA's last k-block of a group
  volatile int* abort;
};

// ------------------------------------------------------------------ TMA warp
// Two loads of 64 columns, or one of both where the operand is described in blocks.
__device__ __forceinline__ void load_mn(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                        int32_t blk, int32_t col, int32_t row, int32_t e,
                                        int groups) {
  if (blk) {
    tma_load_4d_pair(dst, map, bar, 0, row, col / 64, e);
  } else {
    for (int i = 0; i < groups; ++i)
      tma_load_3d_pair(dst + i * (64 * 128), map, bar, col + i * 64, row, e);
  }
}

template <int OP, int BN>
__device__ void tma_role(const ExpertsParams& p, const Schedule<OP, BN>& sch, const Ring& ring,
                         uint32_t rank, int lane) {
  constexpr int kStagesX = stages_of(BN);
  const uint32_t full0 = mapa_shared(smem_u32(ring.full), 0);
  const uint32_t tail_bar = mapa_shared(smem_u32(ring.tail), rank);
  int stage = 0;
  uint32_t phase = 0, tails = 0, issued = 0, issued_phase = 0;
  bool ok = true;
  Unit u;
  for (int32_t i = 0; ok && sch.get(i, u); ++i) {
    const int32_t half = u.w / 2;
    const int box = OP == kOpWeight ? 0 : (half + BN / 8 - 1) / (BN / 8) - 1;
    const uint32_t r_tx =
        OP == kOpWeight ? static_cast<uint32_t>(2 * 64 * 128) : static_cast<uint32_t>((box + 1) * (BN / 8) * 128);
    const int32_t n = u.n0 + static_cast<int32_t>(rank) * 128;
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
      ok = mbar_wait(&ring.empty[stage], phase ^ 1u, p.timeout_ns, ring.abort, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool tail = OP == kOpWeight && u.red_rows - kb * 64 < 64;
      uint32_t bar = full0 + stage * 8;
      uint8_t* wd = ring.w + stage * kWBytes;
      uint8_t* rd = ring.r + stage * r_bytes(BN);
      if (lane == 0) {
        if (tail) {
          bar = tail_bar;
          mbar_arrive_expect_tx(ring.tail, kWBytes + r_tx);
        } else if (rank == 0) {
          mbar_arrive_expect_tx(&ring.full[stage], 2 * (kWBytes + r_tx));
        } else if (OP == kOpWeight) {
          mbar_arrive_pair(bar);
        }
        if constexpr (OP == kOpForward) {
          load_mn(wd, &p.tm_w, bar, p.w_blk, n, kb * 64, u.e, 2);
        } else if constexpr (OP == kOpWeight) {
          load_mn(wd, &p.tm_w, bar, p.w_blk, n, u.row0 + kb * 64, 0, 2);
        } else {
          tma_load_3d_pair(wd, &p.tm_w, bar, kb * block_k<OP>(), n, u.e);
        }
        if constexpr (OP == kOpWeight)
          load_mn(rd, &p.tm_r[0], bar, p.r_blk, u.kt0 + static_cast<int32_t>(rank) * half,
                  u.row0 + kb * 64, 0, 2);
        else
          tma_load_2d_pair(rd, &p.tm_r[box], bar, kb * block_k<OP>(),
                           u.row0 + static_cast<int32_t>(rank) * half);
        if (!tail) {
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        }
      }
      if (OP == kOpWeight && tail) {
        // this CTA's rows have landed: zeros over the rows of the next group, up
        // to the end of the last 16 that the MMA reads
        ok = mbar_wait(ring.tail, tails & 1u, p.timeout_ns, ring.abort, p.status);
        ++tails;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int valid = u.red_rows - kb * 64, end = (valid + 15) & ~15;
        const int n16 = (end - valid) * 8;  // 16-byte pieces per block of 64 columns
        for (int j = lane; j < 4 * n16; j += 32) {
          const int blk = j / n16, o = valid * 128 + (j - blk * n16) * 16;
          uint8_t* base = blk < 2 ? wd + blk * (64 * 128) : rd + (blk - 2) * (64 * 128);
          *reinterpret_cast<uint4*>(base + o) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full0 + stage * 8);
        __syncwarp();
      }
      if (++stage == kStagesX) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (!ok && lane == 0) {
    set_status(p.status, kStatusPipelineTimeout, 0x100u | rank);
    *ring.abort = 1;
    if (rank == 0) {
      volatile int never = 0;
      for (int s = 0; s < kStagesX; ++s)
        if (issued & (1u << s)) mbar_wait(&ring.full[s], (issued_phase >> s) & 1u, 20000000ull, &never);
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ MMA (one thread)
template <int OP, int BN>
__device__ void mma_role(const ExpertsParams& p, const Schedule<OP, BN>& sch, const Ring& ring,
                         uint32_t tmem) {
  constexpr int kStagesX = stages_of(BN);
  constexpr bool kWMn = OP == kOpForward || OP == kOpWeight;
  constexpr bool kRMn = OP == kOpWeight;
  const uint32_t w0 = smem_u32(ring.w), r0 = smem_u32(ring.r);
  int stage = 0;
  uint32_t phase = 0, acc = 0;
  bool ok = true;
  Unit u;
  for (int32_t i = 0; ok && sch.get(i, u); ++i) {
    const uint32_t idesc = idesc_f16_f32(kXWide, u.w, kWMn, kRMn) |
                           (OP != kOpFp8 && p.bf16 ? kIdescAbBf16 : 0u);
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
      const uint32_t d = tmem + (acc & 1u) * 256u;
      const bool first = OP == kOpFp8 || kb == u.kb0;
      if (first) {
        if (!(ok = mbar_wait(&ring.tempty[acc & 1u], ((acc >> 1) & 1u) ^ 1u, p.timeout_ns,
                             ring.abort, p.status)))
          break;
        tc_fence_after();
      }
      // (the weight gradient's last k-block is zeroed by both CTAs' threads)
      if (OP == kOpWeight)
        ok = mbar_wait_cluster(&ring.full[stage], phase, p.timeout_ns, ring.abort, p.status);
      else
        ok = mbar_wait(&ring.full[stage], phase, p.timeout_ns, ring.abort, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ws = w0 + stage * kWBytes, rs = r0 + stage * r_bytes(BN);
      int steps = 4;
      if (OP == kOpWeight) {
        const int valid = u.red_rows - kb * 64;
        if (valid < 64) steps = (valid + 15) / 16;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (OP == kOpWeight && k >= steps) break;
        // 128-byte swizzle.  K-major: groups of 8 rows 1024 B apart, 32 B further
        // per step.  MN-major: blocks of 64 columns 8 KB apart, groups of 8 rows
        // 1024 B apart, 16 rows (2 KB) per step.
        const uint64_t wd = kWMn ? smem_desc_sw128(ws + k * 2048, 64 * 128, 1024)
                                 : smem_desc_sw128(ws + k * 32, 16, 1024);
        const uint64_t rd = kRMn ? smem_desc_sw128(rs + k * 2048, 64 * 128, 1024)
                                 : smem_desc_sw128(rs + k * 32, 16, 1024);
        const uint32_t add = (!first || k > 0) ? 1u : 0u;
        if constexpr (OP == kOpFp8)
          mma_f8_pair(d, wd, rd, idesc, add);
        else
          mma_f16_pair(d, wd, rd, idesc, add);
      }
      mma_commit_pair_both(&ring.empty[stage]);
      if (++stage == kStagesX) {
        stage = 0;
        phase ^= 1u;
      }
      if (OP == kOpFp8 || kb == u.kb1 - 1) {
        mma_commit_pair_both(&ring.tfull[acc & 1u]);
        ++acc;
      }
    }
  }
  if (!ok) {
    set_status(p.status, kStatusPipelineTimeout, 0x200u);
    *ring.abort = 1;
  }
}

// ------------------------------------------------------------------ epilogue
// 16 rows of one output column per lane.
struct Out {
  void* base;
  int64_t ldo;
  int type;
  bool col_ok;
  int64_t row0;
  int32_t cnt;
  int64_t col;
  __device__ __forceinline__ void store(int32_t c0, const float (&v)[16]) const {
    if (!col_ok) return;
    const int32_t n = cnt - c0 < 16 ? cnt - c0 : 16;
    if (type == kTypeF32) {
      float* o = static_cast<float*>(base) + (row0 + c0) * ldo + col;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) o[i * ldo] = v[i];
    } else if (type == kTypeF16) {
      __half* o = static_cast<__half*>(base) + (row0 + c0) * ldo + col;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) o[i * ldo] = __float2half_rn(v[i]);
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(base) + (row0 + c0) * ldo + col;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) o[i * ldo] = __float2bfloat16_rn(v[i]);
    }
  }
};

template <int OP, int BN>
__device__ void epilogue_role(const ExpertsParams& p, const Schedule<OP, BN>& sch,
                              const Ring& ring, uint32_t rank, int ew, int lane, uint32_t tmem,
                              float* scale_buf) {
  constexpr int kCols = BN / 2;  // columns of a warp, at most
  const int quad = (threadIdx.x >> 5) & 3, half = ew >> 2;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const uint32_t tempty0 = mapa_shared(smem_u32(ring.tempty), 0);
  uint32_t acc = 0;
  Unit u;
  for (int32_t i = 0; sch.get(i, u); ++i) {
    const int c_n = u.w / 32, c_first = half * c_n;  // this warp's 16-column chunks
    const int64_t col = static_cast<int64_t>(u.n0) + rank * 128 + quad * 32 + lane;
    const Out out{p.out, p.ldo, p.out_type, col < p.wide,
                  OP == kOpWeight ? static_cast<int64_t>(u.e) * p.out_rows + u.kt0 : u.row0, u.cnt, col};
    const bool split = sch.split > 1;
    // this warp's part of a split sum: [columns][32 lanes]
    const int64_t slab = static_cast<int64_t>(kCols) * 32;
    float* part = nullptr;
    if (split)
      part = p.partials + ((static_cast<int64_t>(u.tile) * sch.split + u.part) * 16 + rank * 8 + ew) * slab + lane;

    if (u.kb0 == u.kb1) {  // an expert without rows: its weights' gradient is zero
      const float zero[16] = {};
      for (int c = 0; c < c_n; ++c) out.store((c_first + c) * 16, zero);
      continue;
    }
    if constexpr (OP == kOpFp8) {
      float sums[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) sums[c] = 0.0f;
      const int32_t KB = sch.KB, NB = (p.wide + 127) / 128, nb = u.n0 / 128 + static_cast<int>(rank);
      const float* ws = p.ws + (static_cast<int64_t>(u.e) * NB + (nb < NB ? nb : NB - 1)) * KB;
      const float* xs = p.xs + u.row0 + c_first * 16;
      const int32_t left = u.cnt - c_first * 16;  // rows from this warp's first column on
      constexpr int kPer = (kCols + 31) / 32;
      float nx[kPer], nw;
      auto fetch = [&](int32_t kb) {
        nw = __ldg(ws + kb);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          nx[j] = j * 32 + lane < left && j * 32 + lane < c_n * 16
                      ? __ldg(xs + static_cast<int64_t>(kb) * p.rows + j * 32 + lane) : 0.0f;
      };
      fetch(u.kb0);
      for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
        float* buf = scale_buf + (kb & 1) * 128;
#pragma unroll
        for (int j = 0; j < kPer; ++j) buf[j * 32 + lane] = nx[j] * nw;
        if (kb + 1 < u.kb1) fetch(kb + 1);
        __syncwarp();
        if (!mbar_wait(&ring.tfull[acc & 1u], (acc >> 1) & 1u, p.timeout_ns, ring.abort, p.status)) {
          set_status(p.status, kStatusPipelineTimeout, 0x300u | rank);
          *ring.abort = 1;
          return;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c) {
          if (c < c_n) {
            uint32_t v[16];
            tmem_ld16(lane_base + (acc & 1u) * 256u + (c_first + c) * 16, v);
            tmem_ld_wait();
            if (c == c_n - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_pair(tempty0 + (acc & 1u) * 8);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 s = *reinterpret_cast<const float4*>(buf + c * 16 + q * 4);
              sums[c * 16 + q * 4 + 0] = fmaf(__uint_as_float(v[q * 4 + 0]), s.x, sums[c * 16 + q * 4 + 0]);
              sums[c * 16 + q * 4 + 1] = fmaf(__uint_as_float(v[q * 4 + 1]), s.y, sums[c * 16 + q * 4 + 1]);
              sums[c * 16 + q * 4 + 2] = fmaf(__uint_as_float(v[q * 4 + 2]), s.z, sums[c * 16 + q * 4 + 2]);
              sums[c * 16 + q * 4 + 3] = fmaf(__uint_as_float(v[q * 4 + 3]), s.w, sums[c * 16 + q * 4 + 3]);
            }
          }
        }
        ++acc;
      }
#pragma unroll
      for (int c = 0; c < kCols / 16; ++c) {
        if (c < c_n) {
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = sums[c * 16 + j];
          if (split) {
#pragma unroll
            for (int j = 0; j < 16; ++j) __stcg(part + (c * 16 + j) * 32, v[j]);
          } else {
            out.store((c_first + c) * 16, v);
          }
        }
      }
    } else {
      if (!mbar_wait(&ring.tfull[acc & 1u], (acc >> 1) & 1u, p.timeout_ns, ring.abort, p.status)) {
        set_status(p.status, kStatusPipelineTimeout, 0x300u | rank);
        *ring.abort = 1;
        return;
      }
      tc_fence_after();
      for (int c = 0; c < c_n; ++c) {
        uint32_t r[16];
        tmem_ld16(lane_base + (acc & 1u) * 256u + (c_first + c) * 16, r);
        tmem_ld_wait();
        if (c == c_n - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(tempty0 + (acc & 1u) * 8);
        }
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
        if (split) {
#pragma unroll
          for (int j = 0; j < 16; ++j) __stcg(part + (c * 16 + j) * 32, v[j]);
        } else {
          out.store((c_first + c) * 16, v);
        }
      }
      ++acc;
    }
    if (split) {
      // the warp that comes last adds the parts, in their order
      __threadfence();
      __syncwarp();
      uint32_t* count = p.arrivals + static_cast<int64_t>(u.tile) * 16 + rank * 8 + ew;
      uint32_t before = 0;
      if (lane == 0) before = atomicAdd(count, 1u);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before == static_cast<uint32_t>(sch.split - 1)) {
        __threadfence();
        if (lane == 0) *count = 0;  // for the next run
        const float* first = p.partials + (static_cast<int64_t>(u.tile) * sch.split * 16 + rank * 8 + ew) * slab + lane;
        for (int c = 0; c < c_n; ++c) {
          float v[16] = {};
          for (int s = 0; s < sch.split; ++s)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              v[j] += __ldcg(first + s * 16 * slab + (c * 16 + j) * 32);
          out.store((c_first + c) * 16, v);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int OP, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kXThreads, 1)
    experts_kernel(const __grid_constant__ ExpertsParams p) {
  constexpr int kStagesX = stages_of(BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ring ring;
  ring.w = smem;
  ring.r = smem + kStagesX * kWBytes;
  float* scales = reinterpret_cast<float*>(ring.r + kStagesX * r_bytes(BN));
  int32_t* off = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(scales) +
                                            (OP == kOpFp8 ? kScaleBytes : 0));
  int32_t* pre = off + kMaxExperts + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(off) + kTableBytes);
  ring.full = bars;
  ring.empty = bars + kStagesX;
  ring.tfull = bars + 2 * kStagesX;
  ring.tempty = ring.tfull + 2;
  ring.tail = ring.tempty + 2;
  uint64_t* drain = ring.tail + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  ring.abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* flag = reinterpret_cast<int32_t*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStagesX; ++s) {
      mbar_init(&ring.full[s], OP == kOpWeight ? 2 : 1);
      mbar_init(&ring.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ring.tfull[b], 1);
      mbar_init(&ring.tempty[b], 16);
    }
    mbar_init(ring.tail, 1);
    mbar_init(drain, 1);
    *tmem_slot = 0;
    *ring.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  const bool valid = load_table<BN>(p, off, pre, flag);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (valid) {
    const Schedule<OP, BN> sch(p, off, pre);
    if (warp == 0) {
      tma_role<OP, BN>(p, sch, ring, rank, lane);
    } else if (warp == 1) {
      if (rank == 0 && lane == 0) mma_role<OP, BN>(p, sch, ring, tmem);
    } else {
      epilogue_role<OP, BN>(p, sch, ring, rank, warp - 2, lane, tmem, scales + (warp - 2) * 256);
    }
  } else if (threadIdx.x == 0) {
    set_status(p.status, kStatusOffsets, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (rank == 0 && warp == 1 && lane == 0) {
    mma_commit_pair_local(drain);
    volatile int never = 0;
    mbar_wait(drain, 0, p.timeout_ns, &never);
  }
  if (*ring.abort || *reinterpret_cast<volatile uint32_t*>(p.status) != 0u) {
    // after a timeout loads that no barrier of ours counts may still be landing
    if (threadIdx.x == 0) __nanosleep(100000);
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int OP>
const void* fn_of(bool few) {
  if constexpr (OP == kOpWeight)
    return reinterpret_cast<const void*>(&experts_kernel<OP, kXRows>);
  else
    return few ? reinterpret_cast<const void*>(&experts_kernel<OP, kXFewRows>)
               : reinterpret_cast<const void*>(&experts_kernel<OP, kXRows>);
}
const void* kernel_of(int op, bool few) {
  switch (op) {
    case kOpForward: return fn_of<kOpForward>(few);
    case kOpInput: return fn_of<kOpInput>(few);
    case kOpWeight: return fn_of<kOpWeight>(few);
    default: return fn_of<kOpFp8>(few);
  }
}
}  // namespace

cudaError_t experts_prepare(int* pairs) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int least = sms / 2;
  for (int op = 0; op < 4 && e == cudaSuccess; ++op)
    for (int few = 0; few < 2 && e == cudaSuccess; ++few) {
      const void* fn = kernel_of(op, few != 0);
      const int smem = smem_bytes(few && op != kOpWeight ? kXFewRows : kXRows, op == kOpFp8);
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) break;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
      cfg.blockDim = dim3(kXThreads);
      cfg.dynamicSmemBytes = static_cast<size_t>(smem);
      int clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg);
      if (clusters < least) least = clusters;
    }
  *pairs = least;
  return e;
}

cudaError_t launch_experts(const ExpertsParams& p, int op, bool few, int grid,
                           cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kXThreads);
  cfg.dynamicSmemBytes =
      static_cast<size_t>(smem_bytes(few && op != kOpWeight ? kXFewRows : kXRows, op == kOpFp8));
  cfg.stream = stream;
  void* args[] = {const_cast<ExpertsParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, kernel_of(op, few), args);
}

}  // namespace agg
