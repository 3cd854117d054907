// experts_kernel.cu -- matrix products grouped by expert, for ragged groups, as
// one persistent kernel of CTA pairs for sm_103a.
//
// All four products have the form out[row][wide] = sum over red of W * R, where the
// wide operand W is the MMA's M and the row operand R its N:
//
//   forward          W = w[e] (K x N, wide contiguous: MN-major),  R = x rows (K-major)
//   input gradient   W = w[e] (red contiguous: K-major),           R = dy rows (K-major)
//   weight gradient  W = dy^T (MN-major), R = x^T (MN-major), red = the expert's rows
//   e4m3             W = wq[e] (N x K: K-major), R = xq rows (K-major); for long
//                    groups the other way round, rows on the M side
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
//   warps 2-17  epilogue: TMEM lane quadrant warp % 4, a quarter of the tile's columns
//   warp 18     weight gradient: zeros over the rows behind a group's end;
//               e4m3: the scales of each k-block into shared memory
//
// Work: tiles in expert order, and inside an expert in groups of 8 row tiles by all
// wide tiles, so that the tiles in flight share operands in L2.  Unit u of pair p is
// p, p + pairs, ...; every role computes the same list from the offsets, which the
// CTA reads into shared memory first.  Where there are too few tiles for the pairs,
// the sums are cut into S parts (choose_split): each warp stores its part's sums,
// and the warp that arrives last adds the S parts in their order, so that nobody
// waits and the result does not depend on the order of arrival.
//
// Sums leave TMEM in segments and are added in 32-bit registers (64 columns a
// thread); two accumulators alternate, and the MMA runs on meanwhile.  A segment is
//   e4m3           one k-block: its sum is multiplied by both operands' scales,
//   fp32 outputs   8 k-blocks: the tensor core's additions lose about a last bit
//                  each, so the error of one long accumulation grows with its length
//                  (1.1e-6 of the result over 1024 terms, 4.5e-7 in segments),
//   16-bit outputs 128 k-blocks (the rounding of the output hides their error).
//
// Rows beyond a group's end belong to the next group: they are multiplied along and
// not stored (rows on the N side do not mix).  In the weight gradient they would
// enter the sums, and an infinity or NaN among them would even survive a product
// with zero, so there the last k-block's surplus rows are overwritten with zeros
// in shared memory before the MMA reads them.
//
// Measured, bf16, one expert: forward of 8192 x 4096 x 4096 146 us (1.88 PFLOP/s, the
// tensor pipe active for 90 % of the cycles; a k-block's operands take the L2-to-SM path
// as long as its MMAs take the tensor cores); weight gradient to fp32 175 us; 64 rows on
// 32 experts of 4096 x 4096 131 us (the hit weights at 6.9 TB/s).  e4m3: the same product
// 126 us (2.2 PFLOP/s; bound by the epilogue's work on each k-block), 64 rows of 16384 x
// 7168 28 us (4.2 TB/s of weights: 28 tiles in two parts are 56 units for 76 pairs).  A
// call of one tile, repeated, takes 4.4 us, with inputs that change 5.2.
//
// Every wait is bounded; on a timeout the kernel records a status word, drains what
// it has in flight, frees TMEM and returns.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts_kernel.cuh"
#include "fused_kernel.cuh"
#include "moe_rows.cuh"
#include "moe_types.cuh"
#include "sm103.cuh"

namespace agg {

namespace {
constexpr int kWBytes = 128 * 128;  // a CTA's wide operand per k-block: 128 x 128 bytes
// k-blocks per stage of the ring.  The MMA thread's work around a stage (a wait, a
// fence, a commit) took about 0.2 us, as long as the MMAs of one k-block; two k-blocks
// a stage halve it.
constexpr int kSub = kXSub;
constexpr int kGroupBytes = kSub * 64 * 128;  // MN-major: 64 columns of a stage

__host__ __device__ constexpr int rows_per_cta(int BN) { return BN / 2; }
__host__ __device__ constexpr int r_bytes(int BN) { return rows_per_cta(BN) * 128; }
// Stages that fit: 3 of 64 KB, or 5 of 40 KB for short row tiles, where the bytes in
// flight are nearly the weights' alone.
__host__ __device__ constexpr int stages_of(int BN) { return (BN == kXRows ? 6 : 10) / kSub; }
constexpr int kScaleBatch = 4;  // e4m3: k-blocks whose scales are handed over at once; two such batches
__host__ __device__ constexpr int scale_bytes(int op, int BN) {
  return op == kOpFp8 ? 2 * kScaleBatch * BN * 4 : op == kOpFp8Long ? 2 * kScaleBatch * 2 * 128 * 4 : 0;
}
// An epilogue warp's buffer for rows of output on their way: 8 of 128 bytes, or 4.
__host__ __device__ constexpr int out_buffer(int op) { return op == kOpFp8Long ? 0 : op == kOpFp8 ? 512 : 1024; }
__host__ __device__ constexpr int out_bytes(int op) { return kXEpiWarps * out_buffer(op); }
constexpr int kTableBytes = (2 * (kMaxExperts + 1) * 4 + 15) & ~15;
constexpr int kUnitBytes = kXEpiWarps * 48;  // the epilogue warps' units
__host__ __device__ constexpr int smem_bytes(int op, int BN) {
  return stages_of(BN) * kSub * (kWBytes + r_bytes(BN)) + scale_bytes(op, BN) +
         out_bytes(op) + kTableBytes + kUnitBytes + 512 /*barriers*/ + 1024 /*alignment*/;
}
static_assert(smem_bytes(kOpForward, kXRows) <= 227 * 1024 && smem_bytes(kOpForward, kXFewRows) <= 227 * 1024 &&
                  smem_bytes(kOpWeight, kXRows) <= 227 * 1024 && smem_bytes(kOpFp8, kXFewRows) <= 227 * 1024 &&
                  smem_bytes(kOpFp8Long, kXRows) <= 227 * 1024,
              "shared memory of an SM");

// After a wait has run out: how long what is in flight is waited for.
constexpr uint64_t kDrainNs = 20000000;

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

// cluster_sync in two steps, and an arrival that publishes no memory writes.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on a barrier of either CTA of the pair without a cluster-scope release:
// for arrivals that publish no memory writes (an accumulator that has been read:
// tcgen05 fences order that).  The release waits for the warp's earlier stores and
// loads, about a microsecond under load: too long once per k-block.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// A value that is the same in all lanes, so that the compiler knows it: what it
// computes from such values stays in uniform registers, where the MMA and TMA
// instructions take their operands.
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// True in one lane of a converged warp, the same one every time.  (Not lane == 0: of a
// branch on this the compiler knows that one thread runs it, and issues MMAs and loads
// from uniform registers; on a lane number it moved every operand there first.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A wait of a whole warp.  The vote keeps its control flow uniform: the warp goes on, or
// gives up, together (TMEM loads are a warp's), and what it computes around the wait (the
// MMA's descriptors) stays in uniform registers.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                          volatile int* abort, const volatile uint32_t* gstatus) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, timeout_ns, abort, gstatus));
}

// 32 TMEM lanes x 8 columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Accumulators: two of 256 TMEM columns.  For e4m3 with short row tiles one holds four
// k-blocks of 64 columns side by side, so that they are handed over together: a
// hand-over costs the epilogue about 300 cycles, as much as a k-block's sums.
constexpr int kAccCols = 256;
constexpr int kFewBlocks = kAccCols / kXFewRows;
static_assert(kScaleBatch == kFewBlocks, "scales are handed over with the accumulators");

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
  int32_t whole;     // and those that k-blocks may hold as they are: more where zeros follow
                     // (the inputs' last row) or the 16 rows of an MMA step end with the group
  int32_t tile, part;
};
static_assert(sizeof(Unit) <= kUnitBytes / kXEpiWarps, "an epilogue warp's unit");

__host__ __device__ constexpr bool is_fp8(int op) { return op == kOpFp8 || op == kOpFp8Long; }
template <int OP>
__host__ __device__ constexpr int block_k() { return is_fp8(OP) ? 128 : 64; }

// Division by a number that stays: n < 2^31; floor(2^32 / d) gives the quotient or one
// less.  (A hardware division takes about a hundred cycles; a role that decodes its
// next unit with five of them holds the ring up at every tile.)
struct Divisor {
  uint32_t d, m;
  __device__ __forceinline__ explicit Divisor(uint32_t d_) : d(d_), m(0xffffffffu / d_) {}
  __device__ __forceinline__ Divisor(uint32_t d_, uint32_t m_) : d(d_), m(m_) {}
  __device__ __forceinline__ uint32_t div(uint32_t n, uint32_t& rest) const {
    uint32_t q = __umulhi(n, m);
    rest = n - q * d;
    if (rest >= d) {
      ++q;
      rest -= d;
    }
    return q;
  }
};

// The work of a launch, in shared memory.
struct Table {
  const int32_t* off;   // [E + 1] row offsets
  const int32_t* pre;   // [E + 1] row tiles before each expert
  const int32_t* head;  // parts of each tile's sum, floor((2^32 - 1) / parts), units; and from
                        // kInverse on floor((2^32 - 1) / n) for n up to 8
  static constexpr int kInverse = 3;
};

// Parts of a sum that make the longest pair's share shortest: a round of the pairs costs
// its k-blocks and about six more for a tile's start and end; with parts price.once more, for
// their way through memory, and at the end each part as long as the one CTA that adds a
// tile's parts takes to read it, price.part.  (Rows of 64, one expert, bf16: 4096 x
// 512 13.7 us whole, 10.3 in four parts, 12.5 in sixteen; 1024 x 2048 7.2 and, in four,
// 9.0.  Tiles of 256: 200 rows of 1024 x 2048 10.7 and 15.7; 234 of 2896 x 752 16.7 and,
// in three, 15.5.  e4m3: 1 row of 3472 x 952 10.5 and, in four, 9.1; 64 of 16384 x 7168
// 28.2 in two parts and one round, 34.4 in five parts and two rounds.)  Each lane of a
// warp tries one number.
__device__ __forceinline__ int32_t choose_split(int32_t tiles, int32_t KB, int32_t max_units, SplitPrice price) {
  const int32_t pairs = static_cast<int32_t>(gridDim.x / 2);
  if (tiles == 0 || tiles >= 2 * pairs || max_units == 0) return 1;
  const int32_t s = static_cast<int32_t>(threadIdx.x & 31) + 1;
  const bool can = s == 1 || (s <= kMaxSplit && KB >= kMinPart * s && tiles * s <= max_units);
  const int32_t rounds = (tiles * s + pairs - 1) / pairs;
  const uint32_t cost = can ? static_cast<uint32_t>(rounds * ((KB + s - 1) / s + 6 + (s > 1 ? price.once : 0)) + (s > 1 ? s * price.part : 0))
                            : 0x03ffffffu;
  // (the smallest number among the cheapest)
  const uint32_t best = __reduce_min_sync(0xffffffffu, min(cost, 0x03ffffffu) * 32 + (s - 1));
  return static_cast<int32_t>(best & 31u) + 1;
}

// The units of a pair in order: unit i is number pair + i * pairs of the list.  A role
// asks for them one after the other.  (Cheap to make: the epilogue makes it anew for
// each tile, so that nothing of it takes registers while sums are added.)
template <int OP, int BN>
struct Schedule {
  const ExpertsParams& p;
  const int32_t* off;
  const int32_t* pre;
  int32_t wt;           // tiles of the wide dimension
  int32_t kt;           // weight gradient: output row tiles per expert
  int32_t KB;           // k-blocks of a whole sum
  int32_t split;        // parts of each tile's sum
  int32_t units, pair, pairs;
  const int32_t* inverse;
  Divisor by_split, by_group, by_expert;  // parts; tiles of 8 row tiles; weight gradient: of an expert
  // the expert of the last unit, its first tile, row tiles and their height
  int32_t e, tile0, nt, height;

  static __device__ __forceinline__ int32_t wide_tiles(const ExpertsParams& p) {
    return (p.wide + kXWide - 1) / kXWide;
  }
  static __device__ __forceinline__ int32_t row_tiles(const ExpertsParams& p) {
    return OP == kOpWeight ? p.row_tiles : 0;
  }
  static __device__ __forceinline__ int32_t k_blocks(const ExpertsParams& p) {
    return OP == kOpWeight ? 0 : (p.red + block_k<OP>() - 1) / block_k<OP>();
  }
  // By one warp, once the table's `tiles` row tiles are known: its head.
  // (In the weight gradient the tiles are the weights', and the sum that counts is the
  // longest group's, of `longest` rows.)
  static __device__ __forceinline__ void fill_head(const ExpertsParams& p, int32_t tiles, int32_t longest,
                                                   int32_t* head) {
    if (OP == kOpWeight) tiles = p.E * row_tiles(p);
    tiles *= wide_tiles(p);
    const int32_t split = choose_split(tiles, OP == kOpWeight ? longest / 64 : k_blocks(p), p.max_units,
                                       split_price(OP, OP == kOpWeight ? p.step < kXRows : BN != kXRows));
    if ((threadIdx.x & 31) == 0) {
      head[0] = split;
      head[1] = static_cast<int32_t>(split == 1 ? 0xffffffffu : 0xffffffffu / static_cast<uint32_t>(split));
      head[2] = tiles * split;
    }
  }

  __device__ __forceinline__ Schedule(const ExpertsParams& p_, const Table& t)
      : p(p_), off(t.off), pre(t.pre), wt(wide_tiles(p_)), kt(row_tiles(p_)), KB(k_blocks(p_)),
        split(t.head[0]), units(t.head[2]), pair(static_cast<int32_t>(blockIdx.x / 2)),
        pairs(static_cast<int32_t>(gridDim.x / 2)), inverse(t.head + Table::kInverse),
        by_split(static_cast<uint32_t>(split), static_cast<uint32_t>(t.head[1])),
        by_group(static_cast<uint32_t>(kXGroup * wt), p_.inv_group),
        by_expert(OP == kOpWeight ? static_cast<uint32_t>(wt * kt) : 1u, p_.inv_expert), e(-1), tile0(0),
        nt(0), height(0) {}

  // Tile `r` of an expert with n row tiles: groups of 8 row tiles, in a group all wide
  // tiles, the row tiles innermost.
  __device__ __forceinline__ void place(uint32_t r, int32_t n, int32_t& x, int32_t& row_tile) const {
    uint32_t rest;
    const int32_t g = static_cast<int32_t>(by_group.div(r, rest));
    const uint32_t gw = static_cast<uint32_t>(n - g * kXGroup < kXGroup ? n - g * kXGroup : kXGroup);
    uint32_t q = __umulhi(rest, inverse[gw]);
    rest -= q * gw;
    if (rest >= gw) {
      ++q;
      rest -= gw;
    }
    x = static_cast<int32_t>(q);
    row_tile = g * kXGroup + static_cast<int32_t>(rest);
  }

  __device__ __forceinline__ void enter(int32_t tile) {
    int32_t lo = e < 0 ? 0 : e, hi = p.E;
    while (hi - lo > 1) {  // the expert whose row tiles hold this one
      const int32_t mid = (lo + hi) >> 1;
      if (pre[mid] * wt <= tile) lo = mid; else hi = mid;
    }
    e = lo;
    tile0 = pre[lo] * wt;
    nt = pre[lo + 1] - pre[lo];
    // its rows in nt tiles of equal height, a multiple of 32 (rows on the M side: 256)
    const int32_t cnt = off[lo + 1] - off[lo];
    // (unsigned: the sum passes 2^31 for a group of more than 2.139e9 rows)
    const uint32_t most = nt == 1 ? cnt : (static_cast<uint32_t>(cnt) + nt - 1u) / static_cast<uint32_t>(nt);
    height = OP == kOpFp8Long ? BN : static_cast<int32_t>((most + 31u) & ~31u);
  }

  __device__ __forceinline__ bool get(int32_t i, Unit& u) {
    const int64_t id = static_cast<int64_t>(i) * pairs + pair;
    if (id >= units) return false;
    const uint32_t unit = static_cast<uint32_t>(id);
    int32_t x, row_tile;
    uint32_t part = 0;
    u.tile = static_cast<int32_t>(unit);
    if (split > 1) u.tile = static_cast<int32_t>(by_split.div(unit, part));
    u.part = static_cast<int32_t>(part);
    int32_t blocks = KB;  // k-blocks of the whole sum
    if constexpr (OP == kOpWeight) {
      uint32_t r;
      u.e = static_cast<int32_t>(by_expert.div(static_cast<uint32_t>(u.tile), r));
      place(r, kt, x, row_tile);
      u.n0 = x * kXWide;
      u.kt0 = row_tile * p.step;
      u.cnt = p.out_rows - u.kt0 < p.step ? p.out_rows - u.kt0 : p.step;
      // (the halves of the two CTAs start at multiples of 64 columns)
      u.w = (u.cnt + 127) & ~127;
      u.row0 = off[u.e];
      u.red_rows = off[u.e + 1] - u.row0;
      u.whole = off[u.e + 1] == p.rows || (u.red_rows & 15) == 0 ? 0x7fffffff : u.red_rows;
      blocks = (u.red_rows + 63) / 64;
    } else {
      if (e < 0 || u.tile >= tile0 + nt * wt) enter(u.tile);
      u.e = e;
      place(static_cast<uint32_t>(u.tile - tile0), nt, x, row_tile);
      u.n0 = x * kXWide;
      const int32_t cols = p.wide - u.n0;
      u.w = OP != kOpFp8Long ? height : cols < kXWide ? (cols + 31) & ~31 : kXWide;
      const int32_t first = row_tile * height, left = off[e + 1] - off[e] - first;
      u.row0 = off[e] + first;
      u.cnt = left < height ? left : height;
      u.kt0 = 0;
      u.red_rows = u.whole = 0;
    }
    u.kb0 = 0;
    u.kb1 = blocks;
    if (split > 1) {
      uint32_t rest;
      u.kb0 = static_cast<int32_t>(by_split.div(static_cast<uint32_t>(blocks * u.part), rest));
      u.kb1 = static_cast<int32_t>(by_split.div(static_cast<uint32_t>(blocks * (u.part + 1)), rest));
    }
    return true;
  }
};

// Offsets to shared memory, checked, and the row tiles before each expert.
// Returns false (to every thread) if the offsets are no layout of the rows.
template <int OP, int BN>
__device__ bool load_table(const ExpertsParams& p, int32_t* off, int32_t* pre, int32_t* head, int32_t* flag) {
  if (threadIdx.x == 0) *flag = 0;
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
    off[e] = p.offsets ? p.offsets[e] : (e == 0 ? 0 : p.rows);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x)
    if (off[e] < 0 || off[e + 1] < off[e] || off[e + 1] > p.rows) *flag = 1;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int32_t carry = 0, longest = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int32_t n = e < p.E ? off[e + 1] - off[e] : 0;
      int32_t s = n > 0 ? (n - 1) / BN + 1 : 0;
      longest = n > longest ? n : longest;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      if (e < p.E) pre[e + 1] = carry + s;
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) pre[0] = 0;
    if (OP == kOpWeight) longest = __reduce_max_sync(0xffffffffu, longest);
    Schedule<OP, BN>::fill_head(p, carry, longest, head);
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
  uint64_t* tempty; // on the even CTA: the epilogue warps of both
  uint64_t* tail;   // weight gradient, by stage: this CTA's part of a group's last k-block
  uint64_t* zfull;  // and, on the even CTA: both CTAs' parts zeroed behind the group's end
  uint64_t* sfull;  // e4m3: scales of a k-block, by slot
  uint64_t* sempty; // e4m3: this CTA's epilogue warps are through with them
  float* scales;    // two batches: [k-block][BN], long groups [k-block][column block][128]
  uint8_t* stage_out;  // a buffer of out_buffer(OP) bytes for each epilogue warp
  Unit* units;         // an epilogue warp's unit, beside the sums that fill its registers
  volatile int* abort;
};

// ------------------------------------------------------------------ TMA warp
// The loads of a stage's two k-blocks of one operand: one TMA instruction where the
// operand's extent allows a view in blocks of 128 bytes, two otherwise.  (The TMA
// unit takes its instructions one by one; two an operand and stage measured the same.)
// MN-major: 128 columns from col (a map of 64, `half`: 64) by 128 rows of the sum's
// dimension from row.
__device__ __forceinline__ void load_mn(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                        int32_t blk, int32_t col, int32_t row, int32_t e, bool half) {
  if (blk) {
    tma_load_4d_pair(dst, map, bar, 0, row, col / 64, e);
  } else {
    tma_load_3d_pair(dst, map, bar, col, row, e);
    if (!half) tma_load_3d_pair(dst + kGroupBytes, map, bar, col + 64, row, e);
  }
}
// K-major: rows of e from row, k-blocks kb and kb + 1 (bk elements each).
__device__ __forceinline__ void load_k(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                       int32_t blk, int32_t kb, int32_t bk, int32_t row, int32_t e,
                                       int32_t second) {
  if (blk) {
    tma_load_4d_pair(dst, map, bar, 0, row, kb, e);
  } else {
    for (int s = 0; s < kSub; ++s)
      tma_load_3d_pair(dst + s * second, map, bar, (kb + s) * bk, row, e);
  }
}

// Box height of the row operand's loads (rows of a CTA, rounded up to its four sizes).
template <int BN>
__device__ __forceinline__ int32_t box_of(int32_t half) {
  return (half + BN / 8 - 1) / (BN / 8);
}

template <int OP, int BN>
__device__ void tma_role(const ExpertsParams& p, const Table& table, const Ring& ring,
                         uint32_t rank, int lane) {
  Schedule<OP, BN> sch(p, table);
  constexpr int kStagesX = stages_of(BN);
  const uint32_t full0 = mapa_shared(smem_u32(ring.full), 0);
  [[maybe_unused]] const uint32_t tail0 = mapa_shared(smem_u32(ring.tail), rank);
  int stage = 0;
  uint32_t phase = 0, issued = 0, filled = 0;  // bit s: stage s used; its loads' parity
  bool ok = true;
  Unit u;
  for (int32_t i = 0; ok && sch.get(i, u); ++i) {
    const int32_t half = u.w / 2;
    const int32_t boxes = OP == kOpFp8Long ? kXRowBoxes : box_of<BN>(half);
    const int32_t height = OP == kOpWeight ? half : boxes * (BN / 8);
    const uint32_t tx = static_cast<uint32_t>(kSub * (kWBytes + height * 128));
    const int32_t n = u.n0 + static_cast<int32_t>(rank) * 128;
    for (int32_t kb0 = u.kb0; kb0 < u.kb1; kb0 += kSub) {
      const int n_sub = u.kb1 - kb0 < kSub ? u.kb1 - kb0 : kSub;
      ok = mbar_wait(&ring.empty[stage], phase ^ 1u, p.timeout_ns, ring.abort, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (elect_one()) {
        const bool tail = OP == kOpWeight && u.whole - (kb0 + n_sub) * 64 < 0;
        uint32_t bar = full0 + stage * 8;
        if (tail) {
          bar = tail0 + stage * 8;  // counted here: zero_role passes it on
          mbar_arrive_expect_tx(&ring.tail[stage], tx);
        } else {
          if (rank == 0) mbar_arrive_expect_tx(&ring.full[stage], 2 * tx);
          issued |= 1u << stage;
          filled ^= 1u << stage;
        }
        uint8_t* wd = ring.w + stage * (kSub * kWBytes);
        uint8_t* rd = ring.r + stage * (kSub * r_bytes(BN));
        const int32_t mine = static_cast<int32_t>(rank) * half;
        if constexpr (OP == kOpFp8Long) {
          load_k(wd, &p.tm_r[kXRowBoxes - 1], bar, p.r_blk, kb0, 128,
                 u.row0 + static_cast<int32_t>(rank) * 128, 0, kWBytes);
          load_k(rd, &p.tm_w, bar, p.w_blk, kb0, 128, u.n0 + mine, u.e, r_bytes(BN));
        } else if constexpr (OP == kOpWeight) {
          load_mn(wd, &p.tm_w, bar, p.w_blk, n, u.row0 + kb0 * 64, 0, false);
          load_mn(rd, &p.tm_r[half == 64], bar, p.r_blk, u.kt0 + mine, u.row0 + kb0 * 64, 0, half == 64);
        } else {
          if constexpr (OP == kOpForward)
            load_mn(wd, &p.tm_w, bar, p.w_blk, n, kb0 * 64, u.e, false);
          else
            load_k(wd, &p.tm_w, bar, p.w_blk, kb0, block_k<OP>(), n, u.e, kWBytes);
          load_k(rd, &p.tm_r[boxes - 1], bar, p.r_blk, kb0, block_k<OP>(), u.row0 + mine, 0,
                 height * 128);
        }
      }
      __syncwarp();
      if (++stage == kStagesX) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (!ok && elect_one()) {  // (the lane that counted its loads)
    set_status(p.status, kStatusPipelineTimeout, 0x100u | rank);
    *ring.abort = 1;
    if (rank == 0) {
      volatile int never = 0;
      for (int s = 0; s < kStagesX; ++s)
        if (issued & (1u << s)) mbar_wait(&ring.full[s], ((filled >> s) & 1u) ^ 1u, kDrainNs, &never);
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ zeros (weight gradient)
// The last k-block of a group that ends inside it and inside 16 rows (the last group's is
// filled with zeros by the load, no rows are behind it: 1000 rows of 1024 x 1024 took
// 10.9 us through here, 9.9 past it): once this CTA's part has landed,
// zeros over the rows of the next group, up to the end of the last 16 that the MMA
// reads; then the k-block is passed on.  A warp of its own: the TMA warp, waiting for
// its own loads here, would leave the ring to run dry once per tile.
template <int BN>
__device__ void zero_role(const ExpertsParams& p, const Table& table,
                          const Ring& ring, uint32_t rank, int lane) {
  Schedule<kOpWeight, BN> sch(p, table);
  constexpr int kStagesX = stages_of(BN);
  const uint32_t zfull0 = mapa_shared(smem_u32(ring.zfull), 0);
  uint32_t stages = 0, used = 0;  // stages so far; bit s: parity of stage s's tails
  Unit u;
  for (int32_t i = 0; sch.get(i, u); ++i) {
    stages += static_cast<uint32_t>((u.kb1 - u.kb0 + kSub - 1) / kSub);
    if (u.whole - u.kb1 * 64 >= 0) continue;  // whole k-blocks, or a part before the last
    const int valid = u.red_rows & 63;
    const uint32_t stage = (stages - 1) % kStagesX;
    const int first = ((u.kb1 - u.kb0 - 1) % kSub) * 64 + valid;  // of the stage's 128 rows
    bool ok = mbar_wait(&ring.tail[stage], (used >> stage) & 1u, p.timeout_ns, ring.abort, p.status);
    used ^= 1u << stage;
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if (lane == 0) {
        set_status(p.status, kStatusPipelineTimeout, 0x400u | rank);
        *ring.abort = 1;
      }
      break;
    }
    const int n16 = (((valid + 15) & ~15) - valid) * 8;  // 16-byte pieces per block of 64 columns
    for (int j = lane; j < 4 * n16; j += 32) {
      const int blk = j / n16, o = first * 128 + (j - blk * n16) * 16;
      uint8_t* base = blk < 2 ? ring.w + stage * (kSub * kWBytes) + blk * kGroupBytes
                              : ring.r + stage * (kSub * r_bytes(BN)) + (blk - 2) * kGroupBytes;
      *reinterpret_cast<uint4*>(base + o) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(zfull0 + stage * 8);
    __syncwarp();
  }
}

// ------------------------------------------------------------------ scales (e4m3)
// A row's scale times a weight block's, in one float: a multiply-add then does a k-block's
// share of a sum.  Below 2^-126 the product is off by up to 2^-150, and a k-block's share
// (a sum of codes is below 2^24.7) by 2^-125.  Beyond the largest float it is that one,
// so that sums of zero stay zero; a scale that is infinite itself stays so.
constexpr float kMaxFloat = 3.402823466e38f;
__device__ __forceinline__ float scale_product(float x, float w) {
  const float p = x * w;
  return fabsf(p) > kMaxFloat && fabsf(x) <= kMaxFloat && fabsf(w) <= kMaxFloat ? copysignf(kMaxFloat, p) : p;
}
// put(product) stores a batch's products; they are looked at one by one only where the
// largest scales' product is out of range (all of them: 8192 x 4096 x 4096 1.2 % slower).
template <typename Put>
__device__ __forceinline__ void scale_products(float largest_x, float largest_w, const Put& put) {
  if (largest_x * largest_w > kMaxFloat)
    put([](float x, float w) { return scale_product(x, w); });
  else
    put([](float x, float w) { return x * w; });
}

// For each k-block the scales of the tile's rows times this CTA's weights' scale (its
// 128 of the wide dimension are one block), a batch of k-blocks per hand-over.
template <int BN>
__device__ void scale_role(const ExpertsParams& p, const Table& table,
                           const Ring& ring, uint32_t rank, int lane) {
  Schedule<kOpFp8, BN> sch(p, table);
  constexpr int kPer = BN / 32;
  uint32_t batch = 0;
  bool ok = true;
  Unit u;
  for (int32_t i = 0; ok && sch.get(i, u); ++i) {
    const int32_t NB = (p.wide + 127) / 128, nb = u.n0 / 128 + static_cast<int>(rank);
    const float* ws = p.ws + (static_cast<int64_t>(u.e) * NB + (nb < NB ? nb : NB - 1)) * sch.KB;
    const float* xs = p.xs + u.row0 + lane;
    for (int32_t kb0 = u.kb0; kb0 < u.kb1; kb0 += kScaleBatch, ++batch) {
      const int32_t n = u.kb1 - kb0 < kScaleBatch ? u.kb1 - kb0 : kScaleBatch;
      float x[kScaleBatch][kPer], w[kScaleBatch], largest_x = 0.0f, largest_w = 0.0f;
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j) {
        w[j] = j < n ? ws[kb0 + j] : 0.0f;
#pragma unroll
        for (int r = 0; r < kPer; ++r)
          x[j][r] = j < n && r * 32 + lane < u.cnt
                        ? xs[static_cast<int64_t>(kb0 + j) * p.rows + r * 32] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j) {
        largest_w = fmaxf(largest_w, fabsf(w[j]));
#pragma unroll
        for (int r = 0; r < kPer; ++r) largest_x = fmaxf(largest_x, fabsf(x[j][r]));
      }
      const uint32_t slot = batch & 1u;
      ok = mbar_wait(&ring.sempty[slot], ((batch >> 1) & 1u) ^ 1u, p.timeout_ns, ring.abort, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      scale_products(largest_x, largest_w, [&](auto product) {
#pragma unroll
        for (int j = 0; j < kScaleBatch; ++j)
#pragma unroll
          for (int r = 0; r < kPer; ++r)
            ring.scales[(slot * kScaleBatch + j) * BN + r * 32 + lane] = product(x[j][r], w[j]);
      });
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.sfull[slot]);
    }
  }
  if (!ok && lane == 0) {
    set_status(p.status, kStatusPipelineTimeout, 0x500u | rank);
    *ring.abort = 1;
  }
}

// Long groups: this CTA's 128 rows' scales times those of the tile's two column blocks,
// [k-block][column block][row], a batch of k-blocks per hand-over.
template <int BN>
__device__ void scale_long_role(const ExpertsParams& p, const Table& table,
                                const Ring& ring, uint32_t rank, int lane) {
  Schedule<kOpFp8Long, BN> sch(p, table);
  uint32_t batch = 0;
  bool ok = true;
  Unit u;
  for (int32_t i = 0; ok && sch.get(i, u); ++i) {
    const int32_t NB = (p.wide + 127) / 128, nb = u.n0 / 128;
    const float* w0 = p.ws + (static_cast<int64_t>(u.e) * NB + nb) * sch.KB;
    const float* w1 = nb + 1 < NB ? w0 + sch.KB : w0;
    const int32_t first = static_cast<int32_t>(rank) * 128 + lane;
    const float* xs = p.xs + u.row0 + first;
    for (int32_t kb0 = u.kb0; kb0 < u.kb1; kb0 += kScaleBatch, ++batch) {
      const int32_t n = u.kb1 - kb0 < kScaleBatch ? u.kb1 - kb0 : kScaleBatch;
      float x[kScaleBatch][4], a[kScaleBatch], b[kScaleBatch], largest_x = 0.0f, largest_w = 0.0f;
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j) {
        a[j] = j < n ? w0[kb0 + j] : 0.0f;
        b[j] = j < n ? w1[kb0 + j] : 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          x[j][r] = j < n && first + r * 32 < u.cnt
                        ? xs[static_cast<int64_t>(kb0 + j) * p.rows + r * 32] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j) {
        largest_w = fmaxf(largest_w, fmaxf(fabsf(a[j]), fabsf(b[j])));
#pragma unroll
        for (int r = 0; r < 4; ++r) largest_x = fmaxf(largest_x, fabsf(x[j][r]));
      }
      const uint32_t slot = batch & 1u;
      ok = mbar_wait(&ring.sempty[slot], ((batch >> 1) & 1u) ^ 1u, p.timeout_ns, ring.abort, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      float* out = ring.scales + slot * (kScaleBatch * 256) + lane;
      scale_products(largest_x, largest_w, [&](auto product) {
#pragma unroll
        for (int j = 0; j < kScaleBatch; ++j)
          if (j < n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              out[j * 256 + r * 32] = product(x[j][r], a[j]);
              out[j * 256 + 128 + r * 32] = product(x[j][r], b[j]);
            }
      });
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.sfull[slot]);
    }
  }
  if (!ok && lane == 0) {
    set_status(p.status, kStatusPipelineTimeout, 0x500u | rank);
    *ring.abort = 1;
  }
}

// ------------------------------------------------------------------ MMA (one warp)
// The warp waits and computes together; lane 0 issues.
template <int OP, int BN>
__device__ void mma_role(const ExpertsParams& p, const Table& table, const Ring& ring,
                         int lane, uint32_t tmem) {
  Schedule<OP, BN> sch(p, table);
  constexpr int kStagesX = stages_of(BN);
  constexpr bool kWMn = OP == kOpForward || OP == kOpWeight;
  constexpr bool kRMn = OP == kOpWeight;
  // 128-byte swizzle.  K-major: groups of 8 rows 1024 B apart, 32 B further per step.
  // MN-major: blocks of 64 columns kGroupBytes apart, groups of 8 rows 1024 B apart, 16 rows
  // (2 KB) per step.  (The address is the descriptor's lowest field, in units of 16.)
  const uint64_t w0 = kWMn ? smem_desc_sw128(smem_u32(ring.w), kGroupBytes, 1024)
                           : smem_desc_sw128(smem_u32(ring.w), 16, 1024);
  const uint64_t r0 = kRMn ? smem_desc_sw128(smem_u32(ring.r), kGroupBytes, 1024)
                           : smem_desc_sw128(smem_u32(ring.r), 16, 1024);
  constexpr uint32_t kWStep = (kWMn ? 2048 : 32) / 16, kRStep = (kRMn ? 2048 : 32) / 16;
  constexpr uint32_t kWSecond = (kWMn ? 64 * 128 : kWBytes) / 16;  // the second k-block
  int stage = 0;
  uint32_t acc = 0, full_phase = 0, zeroed = 0;  // bit s: parity of stage s's barriers
  bool ok = true;
  auto accumulator = [&] {  // wait until it has been read
    const bool r = warp_wait(&ring.tempty[acc & 1u], ((acc >> 1) & 1u) ^ 1u, p.timeout_ns, ring.abort,
                             p.status);
    tc_fence_after();
    return r;
  };
  Unit u;
  for (int32_t i = 0; ok && sch.get(i, u); ++i) {
    const int32_t kb_end = uniform(u.kb1), kb_begin = uniform(u.kb0), width = uniform(u.w);
    [[maybe_unused]] const int32_t red_rows = uniform(u.red_rows), whole = uniform(u.whole);
    const uint32_t idesc = idesc_f16_f32(kXWide, width, kWMn, kRMn) |
                           (!is_fp8(OP) && p.bf16 ? kIdescAbBf16 : 0u);
    const uint32_t r_second = kRMn ? 64 * 128 / 16
                              : OP == kOpFp8Long ? r_bytes(BN) / 16
                                                 : static_cast<uint32_t>(box_of<BN>(width / 2) * (BN / 8) * 128 / 16);
    const int32_t segment = OP == kOpFp8Long ? 1 : OP == kOpFp8 ? kFewBlocks : p.segment;
    int32_t left = 0;  // k-blocks left of the segment
    for (int32_t kb0 = kb_begin; kb0 < kb_end; kb0 += kSub) {
      const int n_sub = kb_end - kb0 < kSub ? kb_end - kb0 : kSub;
      bool first = false;
      if (OP != kOpFp8Long && left <= 0) {
        if (!(ok = accumulator())) break;
        left = segment;
        first = true;
      }
      int last_steps = 4;  // of the stage's last k-block
      if (OP == kOpWeight && red_rows - (kb0 + n_sub) * 64 < 0)
        last_steps = (red_rows - (kb0 + n_sub - 1) * 64 + 15) / 16;
      if (OP == kOpWeight && whole - (kb0 + n_sub) * 64 < 0) {
        // a group's last k-block comes through both CTAs' zeroing warps
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&ring.zfull[stage], (zeroed >> stage) & 1u,
                                                       p.timeout_ns, ring.abort, p.status));
        zeroed ^= 1u << stage;
      } else {
        ok = warp_wait(&ring.full[stage], (full_phase >> stage) & 1u, p.timeout_ns, ring.abort,
                       p.status);
        full_phase ^= 1u << stage;
      }
      if (!ok) break;
      tc_fence_after();
      const uint64_t ws = w0 + static_cast<uint32_t>(stage * (kSub * kWBytes / 16));
      const uint64_t rs = r0 + static_cast<uint32_t>(stage * (kSub * r_bytes(BN) / 16));
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        if (s >= n_sub) break;
        if (OP == kOpFp8Long && !(ok = accumulator())) break;
        const uint32_t d = tmem + (acc & 1u) * kAccCols +
                           (OP == kOpFp8 ? (kFewBlocks - left + s) * kXFewRows : 0);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (OP == kOpWeight && s == n_sub - 1 && k >= last_steps) break;
            const uint64_t wd = ws + (s * kWSecond + k * kWStep);
            const uint64_t rd = rs + (s * r_second + k * kRStep);
            if constexpr (is_fp8(OP))
              mma_f8_pair(d, wd, rd, idesc, k > 0 ? 1u : 0u);
            else
              mma_f16_pair(d, wd, rd, idesc, (!first || s > 0 || k > 0) ? 1u : 0u);
          }
          if (OP == kOpFp8Long) mma_commit_pair_both(&ring.tfull[acc & 1u]);
        }
        if (OP == kOpFp8Long) ++acc;
      }
      if (!ok) break;
      if (elect_one()) mma_commit_pair_both(&ring.empty[stage]);
      if (++stage == kStagesX) stage = 0;
      if (OP != kOpFp8Long) {
        left -= n_sub;
        if (left <= 0 || kb0 + kSub >= kb_end) {
          left = 0;
          if (elect_one()) mma_commit_pair_both(&ring.tfull[acc & 1u]);
          ++acc;
        }
      }
      __syncwarp();
    }
  }
  if (!ok && lane == 0) {
    set_status(p.status, kStatusPipelineTimeout, 0x200u);
    *ring.abort = 1;
  }
}

// ------------------------------------------------------------------ epilogue
// 8 rows of one output column per lane, 32 columns a warp.  They are turned in shared
// memory (a buffer per warp) so that a store instruction writes 16 bytes a lane, 64 or
// 128 contiguous bytes of each row: stores of one element a lane, at the LSU's rate of
// one instruction per about 7 cycles, took 7000 cycles for a 256 x 256 tile.
template <int kBytes>  // of the buffer
struct Out {
  void* base;
  int64_t ldo, row0, col;  // col: the warp's first
  int type;
  int32_t cnt, cols;       // rows of the tile; columns of the output from col on
  uint8_t* stage;
  __device__ __forceinline__ void store(int32_t c0, const float (&v)[8], int lane) const {
    __syncwarp();  // the buffer has been read
    if (type == kTypeF32) {
      constexpr int kRows = kBytes / 128;  // rows at a time
      float* s = reinterpret_cast<float*>(stage) + lane;
#pragma unroll
      for (int r0 = 0; r0 < 8; r0 += kRows) {
        if (r0 > 0) __syncwarp();
#pragma unroll
        for (int i = 0; i < kRows; ++i) s[i * 32] = v[r0 + i];
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kRows; h += 4) {
          const int r = h + (lane >> 3), row = r0 + r, part = (lane & 7) * 4;
          const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 128 + part * 4);
          if (c0 + row < cnt && part < cols)
            *reinterpret_cast<uint4*>(static_cast<float*>(base) + (row0 + c0 + row) * ldo + col + part) = x;
        }
      }
    } else {
      uint16_t* s = reinterpret_cast<uint16_t*>(stage) + lane;
      if (type == kTypeF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i * 32] = __half_as_ushort(__float2half_rn(v[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i * 32] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
      }
      __syncwarp();
      const int row = lane >> 2, part = (lane & 3) * 8;
      const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 64 + part * 2);
      if (c0 + row < cnt && part < cols)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + (row0 + c0 + row) * ldo + col + part) = x;
    }
  }
};

// 16 columns of an output row in one store of 32 bytes (16-bit outputs whose rows are
// 32-byte aligned): whole sectors, half the instructions.
__device__ __forceinline__ void store_row16(void* base, int type, int64_t at, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = type == kTypeF16 ? Elem<__half>::pair(v[2 * i], v[2 * i + 1])
                            : Elem<__nv_bfloat16>::pair(v[2 * i], v[2 * i + 1]);
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                   static_cast<uint16_t*>(base) + at),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// After this warp has stored its part of a split sum: true for the warp that comes
// last and adds the parts.
template <int kWarps>
__device__ __forceinline__ bool last_part(const ExpertsParams& p, const Unit& u, int32_t split,
                                          uint32_t rank, int ew, int lane) {
  __threadfence();
  __syncwarp();
  uint32_t* count = p.arrivals + (static_cast<int64_t>(u.tile) * 2 + rank) * kWarps + ew;
  uint32_t before = 0;
  if (lane == 0) before = atomicAdd(count, 1u);
  before = __shfl_sync(0xffffffffu, before, 0);
  if (before != static_cast<uint32_t>(split - 1)) return false;
  __threadfence();
  if (lane == 0) *count = 0;  // for the next run
  return true;
}

// 8 columns of one output row per lane (N % 8 == 0: all inside or none).
__device__ __forceinline__ void store_row8(void* base, int type, int64_t at, const float (&v)[8]) {
  if (type == kTypeF32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else if (type == kTypeF16) {
    *reinterpret_cast<uint4*>(static_cast<__half*>(base) + at) = Elem<__half>::pack(v);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) = Elem<__nv_bfloat16>::pack(v);
  }
}

// Zeros to n rows of up to 32 columns (`cols` are left of the output) from element `at` on.
__device__ __forceinline__ void store_zeros(const ExpertsParams& p, int64_t at, int32_t n, int32_t cols, int lane) {
  const int size = p.out_type == kTypeF32 ? 4 : 2, per = 2 * size;  // lanes of a row, 16 bytes each
  const int part = (lane & (per - 1)) * (16 / size);
  uint8_t* to = static_cast<uint8_t*>(p.out) + (at + part) * size;
  if (part < cols)
    for (int r = lane / per; r < n; r += 32 / per)
      *reinterpret_cast<uint4*>(to + r * p.ldo * size) = make_uint4(0, 0, 0, 0);
}

// The sum of a split tile's parts for 8 columns, in the order of the parts, the loads of
// four parts in flight.
__device__ __forceinline__ void add_parts(const float* first, int64_t next, int32_t parts, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  for (int32_t s0 = 0; s0 < parts; s0 += 4) {
    float x[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[u][j] = s0 + u < parts ? __ldcg(first + (s0 + u) * next + j * 32) : 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s0 + u < parts)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += x[u][j];
  }
}

// e4m3, long groups: a lane is a row here, so a k-block's scale is one number per
// thread (the row's times that of the warp's 64 columns, which lie in one block).  With
// the scales on the columns, reading them took as much of the shared memory's time as
// the MMA's operands.  scale_long_role prepares them, four k-blocks at a time: loads
// from global memory in this loop stalled it for half of its time.
template <int BN>
__device__ void epilogue_long(const ExpertsParams& p, const Table& table,
                              const Ring& ring, uint32_t rank, int ew, int lane, uint32_t tmem) {
  constexpr int kCols = 64;
  const int quad = (threadIdx.x >> 5) & 3, c_first = (ew >> 2) * kCols;
  uint32_t acc = 0, batch = 0;
  for (int32_t i = 0;; ++i) {
    float sums[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) sums[c] = 0.0f;
    {
      Unit u;
      if (!Schedule<kOpFp8Long, BN>(p, table).get(i, u)) break;
      const int cols = u.w - c_first;  // a multiple of 32
      const int n16 = cols <= 0 ? 0 : cols >= kCols ? kCols / 16 : cols / 16;
      const uint32_t from0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c_first;
      const uint32_t tempty0 = mapa_shared(smem_u32(ring.tempty), 0);
      const float* scale0 = ring.scales + (c_first >> 7) * 128 + quad * 32 + lane;
      bool ok = true;
      for (int32_t left = u.kb1 - u.kb0; ok && left > 0; left -= kScaleBatch, ++batch) {
        const uint32_t slot = batch & 1u;
        ok = warp_wait(&ring.sfull[slot], (batch >> 1) & 1u, p.timeout_ns, ring.abort, p.status);
        // the batch's scales to registers: a load in the loop would be waited for
        float s[kScaleBatch];
#pragma unroll
        for (int j = 0; j < kScaleBatch; ++j) s[j] = scale0[(slot * kScaleBatch + j) * 256];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.sempty[slot]);
#pragma unroll
        for (int j = 0; j < kScaleBatch; ++j) {
          if (!ok || j >= left) break;
          ok = warp_wait(&ring.tfull[acc & 1u], (acc >> 1) & 1u, p.timeout_ns, ring.abort, p.status);
          tc_fence_after();
          const uint32_t from = from0 + (acc & 1u) * kAccCols;
          if (n16 == kCols / 16) {
#pragma unroll
            for (int c = 0; c < kCols / 16; ++c) {
              uint32_t v[16];
              tmem_ld16(from + c * 16, v);
              tmem_ld_wait();
              if (c == kCols / 16 - 1) {  // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(tempty0 + (acc & 1u) * 8);
              }
#pragma unroll
              for (int q = 0; q < 16; ++q)
                sums[c * 16 + q] = fmaf(__uint_as_float(v[q]), s[j], sums[c * 16 + q]);
            }
          } else {  // the last columns
#pragma unroll
            for (int c = 0; c < kCols / 16 - 1; ++c)
              if (c < n16) {
                uint32_t v[16];
                tmem_ld16(from + c * 16, v);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 16; ++q)
                  sums[c * 16 + q] = fmaf(__uint_as_float(v[q]), s[j], sums[c * 16 + q]);
              }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(tempty0 + (acc & 1u) * 8);
          }
          ++acc;
        }
      }
      if (!ok) {
        set_status(p.status, kStatusPipelineTimeout, 0x300u | rank);
        *ring.abort = 1;
        return;
      }
    }
    Unit u;  // (found anew: kept in shared memory as by epilogue_role, 8192 x 4096 x 4096 took
             // 130 us against 126, from other registers in the loop above)
    Schedule<kOpFp8Long, BN> sch(p, table);
    sch.get(i, u);
    const int32_t split = sch.split;
    const int32_t row = static_cast<int32_t>(rank) * 128 + quad * 32 + lane;
    const int64_t col = static_cast<int64_t>(u.n0) + c_first;
    const int64_t at = (static_cast<int64_t>(u.row0) + row) * p.ldo + col;
    const int32_t left = p.wide - static_cast<int32_t>(col);  // columns of the output from here
    const int n = left <= 0 ? 0 : left >= kCols ? kCols / 8 : left / 8;
    auto eight = [&](int c, float (&v)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = sums[c * 8 + j];
    };
    if (split == 1 && n == kCols / 8 && p.rows32) {
      if (row < u.cnt)
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = sums[c + j];
          store_row16(p.out, p.out_type, at + c, v);
        }
      continue;
    }
    if (split == 1) {
#pragma unroll
      for (int c = 0; c < kCols / 8; ++c)
        if (c < n && row < u.cnt) {
          float v[8];
          eight(c, v);
          store_row8(p.out, p.out_type, at + c * 8, v);
        }
      continue;
    }
    constexpr int kWarps = kXEpiWarps;
    constexpr int64_t kSlab = kCols * 32, kNext = 2 * kWarps * kSlab;
    float* first = p.partials +
                   ((static_cast<int64_t>(u.tile) * split * 2 + rank) * kWarps + ew) * kSlab + lane;
    float* part = first + u.part * kNext;
#pragma unroll
    for (int c = 0; c < kCols / 8; ++c)
      if (c < n) {
        float v[8];
        eight(c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) __stcg(part + (c * 8 + j) * 32, v[j]);
      }
    if (last_part<kWarps>(p, u, split, rank, ew, lane))
      for (int c = 0; c < n; ++c) {
        float v[8];
        add_parts(first + c * 8 * 32, kNext, split, v);
        if (row < u.cnt) store_row8(p.out, p.out_type, at + c * 8, v);
      }
  }
}

template <int OP, int BN>
__device__ void epilogue_role(const ExpertsParams& p, const Table& table,
                              const Ring& ring, uint32_t rank, int ew, int lane, uint32_t tmem) {
  constexpr int kCols = BN / 4;  // columns of a warp, at most
  const int quad = (threadIdx.x >> 5) & 3, quarter = ew >> 2;
  uint32_t acc = 0;
  for (int32_t i = 0;; ++i) {
    float sums[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) sums[c] = 0.0f;
    {
      Unit u;
      if (!Schedule<OP, BN>(p, table).get(i, u)) break;
      if (lane == 0) ring.units[ew] = u;
      const int n8 = u.w / 32, c_first = quarter * n8 * 8;  // this warp's columns, in eights
      if (OP == kOpWeight && u.red_rows == 0 && table.head[0] == 1) {
        // an expert without rows (2 rows, 61 experts of 864 x 352: 21 us, by the sums 26)
        const int32_t col = u.n0 + static_cast<int32_t>(rank) * 128 + quad * 32;
        store_zeros(p, (static_cast<int64_t>(u.e) * p.out_rows + u.kt0 + c_first) * p.ldo + col,
                    n8 * 8 < u.cnt - c_first ? n8 * 8 : u.cnt - c_first, p.wide - col, lane);
        continue;
      }
      const uint32_t from0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c_first;
      const uint32_t tempty0 = mapa_shared(smem_u32(ring.tempty), 0);
      const int32_t seg = OP == kOpFp8 ? kFewBlocks : p.segment;
      for (int32_t left = u.kb1 - u.kb0; left > 0; left -= seg, ++acc) {
        const uint32_t slot = acc & 1u, phase = (acc >> 1) & 1u;
        bool ok = true;
        if constexpr (OP == kOpFp8)
          ok = warp_wait(&ring.sfull[slot], phase, p.timeout_ns, ring.abort, p.status);
        if (!ok || !warp_wait(&ring.tfull[slot], phase, p.timeout_ns, ring.abort, p.status)) {
          set_status(p.status, kStatusPipelineTimeout, 0x300u | rank);
          *ring.abort = 1;
          return;
        }
        tc_fence_after();
        const uint32_t from = from0 + slot * kAccCols;
        if constexpr (OP == kOpFp8) {
          // four k-blocks side by side: this warp's columns of each, times their scales
          const float* scale = ring.scales + slot * (kFewBlocks * BN) + c_first;
          // (two at a time: a wait for the loads costs as much as the sums of a k-block)
#pragma unroll
          for (int j0 = 0; j0 < kFewBlocks; j0 += 2) {
            if (j0 < left) {
              uint32_t v[2][kCols];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (n8 == kCols / 8)
                  tmem_ld16(from + (j0 + j) * BN, v[j]);
                else
                  tmem_ld8(from + (j0 + j) * BN, *reinterpret_cast<uint32_t(*)[8]>(v[j]));
              }
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < kCols; q += 4)
                  if (q < n8 * 8 && j0 + j < left) {
                    const float4 f = *reinterpret_cast<const float4*>(scale + (j0 + j) * BN + q);
                    sums[q] = fmaf(__uint_as_float(v[j][q]), f.x, sums[q]);
                    sums[q + 1] = fmaf(__uint_as_float(v[j][q + 1]), f.y, sums[q + 1]);
                    sums[q + 2] = fmaf(__uint_as_float(v[j][q + 2]), f.z, sums[q + 2]);
                    sums[q + 3] = fmaf(__uint_as_float(v[j][q + 3]), f.w, sums[q + 3]);
                  }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_pair(tempty0 + slot * 8);
            mbar_arrive(&ring.sempty[slot]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c) {
            if (c < n8) {
              uint32_t v[8];
              tmem_ld8(from + c * 8, v);
              tmem_ld_wait();
              if (c == n8 - 1) {  // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(tempty0 + slot * 8);
              }
#pragma unroll
              for (int q = 0; q < 8; ++q) sums[c * 8 + q] += __uint_as_float(v[q]);
            }
          }
        }
      }
    }
    // (the unit again: its fields would take the registers of the loop above.  Finding it
    // anew cost about 0.3 us a tile: weight gradient of 4096 rows, 16 experts of 4096 x 4096,
    // 206 us, so 194; e4m3 of 4085 rows, 47 experts of 784 x 2664, 47.8 and 43.5.)
    __syncwarp();
    const Unit u = ring.units[ew];
    const int32_t split = table.head[0];
    const int n8 = u.w / 32, c_first = quarter * n8 * 8;
    const int32_t col = u.n0 + static_cast<int32_t>(rank) * 128 + quad * 32;
    const Out<out_buffer(OP)> out{p.out, p.ldo,
                  OP == kOpWeight ? static_cast<int64_t>(u.e) * p.out_rows + u.kt0 : u.row0, col,
                  p.out_type, u.cnt, p.wide - col, ring.stage_out + ew * out_buffer(OP)};
    auto eight = [&](int c, float (&v)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = sums[c * 8 + j];
    };
    if (split == 1) {
#pragma unroll
      for (int c = 0; c < kCols / 8; ++c)
        if (c < n8) {
          float v[8];
          eight(c, v);
          out.store(c_first + c * 8, v, lane);
        }
      continue;
    }
    // this warp's part, [columns][32 lanes]; the warp that comes last adds the parts,
    // in their order
    constexpr int64_t kSlab = static_cast<int64_t>(kCols) * 32;
    constexpr int64_t kNext = 2 * kXEpiWarps * kSlab;
    float* first = p.partials +
                   ((static_cast<int64_t>(u.tile) * split * 2 + rank) * kXEpiWarps + ew) * kSlab + lane;
    float* part = first + u.part * kNext;
#pragma unroll
    for (int c = 0; c < kCols / 8; ++c)
      if (c < n8) {
        float v[8];
        eight(c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) __stcg(part + (c * 8 + j) * 32, v[j]);
      }
    if (last_part<kXEpiWarps>(p, u, split, rank, ew, lane))
      for (int c = 0; c < n8; ++c) {
        float v[8];
        add_parts(first + c * 8 * 32, kNext, split, v);
        out.store(c_first + c * 8, v, lane);
      }
  }
}

// ------------------------------------------------------------------ kernel
template <int OP, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(OP), 1)
    experts_kernel(const __grid_constant__ ExpertsParams p) {
  constexpr int kStagesX = stages_of(BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ring ring;
  ring.w = smem;
  ring.r = smem + kStagesX * kSub * kWBytes;
  ring.scales = reinterpret_cast<float*>(ring.r + kStagesX * kSub * r_bytes(BN));
  ring.stage_out = reinterpret_cast<uint8_t*>(ring.scales) + scale_bytes(OP, BN);
  int32_t* off = reinterpret_cast<int32_t*>(ring.stage_out + out_bytes(OP));
  int32_t* pre = off + kMaxExperts + 1;
  ring.units = reinterpret_cast<Unit*>(reinterpret_cast<uint8_t*>(off) + kTableBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ring.units) + kUnitBytes);
  ring.full = bars;
  ring.empty = bars + kStagesX;
  ring.tfull = bars + 2 * kStagesX;
  ring.tempty = ring.tfull + 2;
  ring.tail = ring.tempty + 2;
  ring.zfull = ring.tail + kStagesX;
  ring.sfull = ring.zfull + kStagesX;
  ring.sempty = ring.sfull + 2;
  uint64_t* drain = ring.sempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  ring.abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* flag = reinterpret_cast<int32_t*>(tmem_slot + 2);
  int32_t* head = flag + 1;  // [Table::kInverse + kXGroup + 1]
  const Table table{off, pre, head};

  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStagesX; ++s) {
      mbar_init(&ring.full[s], 1);
      mbar_init(&ring.empty[s], 1);
      mbar_init(&ring.tail[s], 1);
      mbar_init(&ring.zfull[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ring.tfull[b], 1);
      mbar_init(&ring.tempty[b], 2 * kXEpiWarps);
      mbar_init(&ring.sfull[b], 1);
      mbar_init(&ring.sempty[b], kXEpiWarps);
    }
    mbar_init(drain, 1);
    *tmem_slot = 0;
    *ring.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if (warp == 3 && lane <= kXGroup)
    head[Table::kInverse + lane] = static_cast<int32_t>(lane ? 0xffffffffu / static_cast<uint32_t>(lane) : 0u);
  if (warp == 2 && lane <= kXRowBoxes)  // the descriptors' first use would wait for them
    tma_prefetch_desc(lane == kXRowBoxes ? &p.tm_w : &p.tm_r[OP == kOpWeight ? lane & 1 : lane]);
  tc_fence_before();
  cluster_arrive();  // barriers initialised, TMEM allocated; the table is read meanwhile
  pdl_wait();        // from here on global memory is read
  const bool valid = load_table<OP, BN>(p, off, pre, head, flag);
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  if (valid) {
    if (warp == 0) {
      tma_role<OP, BN>(p, table, ring, rank, lane);
    } else if (warp == 1) {
      if (rank == 0) mma_role<OP, BN>(p, table, ring, lane, tmem);
    } else if (warp < 2 + kXEpiWarps) {
      if constexpr (OP == kOpFp8Long)
        epilogue_long<BN>(p, table, ring, rank, warp - 2, lane, tmem);
      else
        epilogue_role<OP, BN>(p, table, ring, rank, warp - 2, lane, tmem);
    } else if constexpr (OP == kOpWeight) {
      zero_role<BN>(p, table, ring, rank, lane);
    } else if constexpr (OP == kOpFp8) {
      scale_role<BN>(p, table, ring, rank, lane);
    } else if constexpr (OP == kOpFp8Long) {
      scale_long_role<BN>(p, table, ring, rank, lane);
    }
  } else if (threadIdx.x == 0) {
    set_status(p.status + 2, kStatusOffsets, 0);
  }
  tc_fence_before();
  // This CTA's epilogue has waited for every accumulator of the pair, so every MMA and load
  // of the pair is through, unless a wait of this CTA ran out (a wait of the peer's alone
  // leaves nothing of the pair's in flight then):
  if (__syncthreads_or(*ring.abort)) {
    if (rank == 0 && warp == 1 && elect_one()) {  // the thread that issued the MMAs
      mma_commit_pair_local(drain);
      volatile int never = 0;
      mbar_wait(drain, 0, kDrainNs, &never);
    }
    // loads that no barrier of ours counts may still be landing
    if (threadIdx.x == 0) __nanosleep(100000);
    __syncthreads();
  }
  // (relaxed: the pair only leaves together, what it wrote is published by its end)
  tc_fence_before();
  cluster_arrive_relaxed();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The kernel of a product: its variant, threads and shared memory.
struct Variant {
  const void* fn;
  int threads, smem;
};
template <int OP, int BN>
Variant variant_of() {
  return {reinterpret_cast<const void*>(&experts_kernel<OP, BN>), threads_of(OP),
          smem_bytes(OP, BN)};
}
Variant variant(int op, bool few) {
  switch (op) {
    case kOpForward: return few ? variant_of<kOpForward, kXFewRows>() : variant_of<kOpForward, kXRows>();
    case kOpInput: return few ? variant_of<kOpInput, kXFewRows>() : variant_of<kOpInput, kXRows>();
    case kOpWeight: return variant_of<kOpWeight, kXRows>();
    default: return few ? variant_of<kOpFp8, kXFewRows>() : variant_of<kOpFp8Long, kXRows>();
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
      const Variant v = variant(op, few != 0);
      e = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
      if (e != cudaSuccess) break;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
      cfg.blockDim = dim3(static_cast<unsigned>(v.threads));
      cfg.dynamicSmemBytes = static_cast<size_t>(v.smem);
      int clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, v.fn, &cfg);
      if (clusters < least) least = clusters;
    }
  *pairs = least;
  return e;
}

cudaError_t launch_experts(const ExpertsParams& p, int op, bool few, int grid,
                           cudaStream_t stream) {
  const Variant v = variant(op, few);
  void* args[] = {const_cast<ExpertsParams*>(&p)};
  return launch_args(v.fn, dim3(static_cast<unsigned>(grid)), v.threads, static_cast<size_t>(v.smem), stream, args);
}

}  // namespace agg
