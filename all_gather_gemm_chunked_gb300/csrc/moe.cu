// moe.cu -- host side of include/ag_moe.h: argument checks, the plan of the
// products by expert (workspace, status) and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <mutex>
#include <new>

#include "ag_moe.h"
#include "experts_kernel.cuh"
#include "fused_kernel.cuh"
#include "host.h"
#include "moe_rows.cuh"

using agg::aligned16;
using agg::cuda_fail;
using agg::DeviceGuard;
using agg::encode_tiled;
using agg::fail;
using agg::log_msg;

static_assert(AG_MOE_F32 == agg::kTypeF32 && AG_MOE_E4M3 == agg::kTypeE4m3 &&
                  AG_GEMM_F16 == agg::kTypeF16 && AG_GEMM_BF16 == agg::kTypeBf16 &&
                  AG_MOE_MAX_EXPERTS == agg::kMaxExperts && AG_MOE_MAX_TOP_K == agg::kMaxTopK &&
                  AG_MOE_SCALE_BLOCK == agg::kScaleBlock,
              "public and internal values");

namespace {

constexpr int64_t kMaxTokens = 1LL << 28;   // (the router then takes 4097 blocks)
constexpr int64_t kMaxRowLen = 1LL << 24;   // columns of a moved row (grid limit)

bool float_type(int dtype) {
  return dtype == AG_GEMM_F16 || dtype == AG_GEMM_BF16 || dtype == AG_MOE_F32;
}
int esize(int dtype) { return dtype == AG_MOE_F32 ? 4 : dtype == AG_MOE_E4M3 ? 1 : 2; }

// ------------------------------------------------------------------ router, rows
int check_route(int64_t T, int E, int k, int dtype) {
  if (!float_type(dtype)) return fail(AG_GEMM_ERR_INVALID, "logits must be fp16, bf16 or fp32 (got type %d)", dtype);
  if (E < 1 || E > agg::kMaxExperts)
    return fail(AG_GEMM_ERR_INVALID, "experts must be in [1, %d] (got %d)", agg::kMaxExperts, E);
  if (k < 1 || k > agg::kMaxTopK || k > E)
    return fail(AG_GEMM_ERR_INVALID, "top_k must be in [1, min(experts, %d)] (got %d)", agg::kMaxTopK, k);
  if (T < 0) return fail(AG_GEMM_ERR_INVALID, "tokens must not be negative (got %lld)", (long long)T);
  if (T > kMaxTokens || T * k >= (1LL << 31))
    return fail(AG_GEMM_ERR_UNSUPPORTED, "too many tokens: at most %lld, and tokens * top_k below 2^31",
                (long long)kMaxTokens);
  return AG_GEMM_OK;
}

int check_rows(int64_t T, int k, int64_t H, int dtype) {
  if (!float_type(dtype)) return fail(AG_GEMM_ERR_INVALID, "rows must be fp16, bf16 or fp32 (got type %d)", dtype);
  if (k < 1 || k > agg::kMaxTopK)
    return fail(AG_GEMM_ERR_INVALID, "top_k must be in [1, %d] (got %d)", agg::kMaxTopK, k);
  if (T < 0 || H < 1) return fail(AG_GEMM_ERR_INVALID, "need T >= 0 and H >= 1 (got %lld, %lld)", (long long)T, (long long)H);
  if (T * k >= (1LL << 31) || T > kMaxTokens || H > kMaxRowLen)
    return fail(AG_GEMM_ERR_UNSUPPORTED, "too many rows (T * top_k below 2^31) or columns (at most %lld)",
                (long long)kMaxRowLen);
  return AG_GEMM_OK;
}

agg::RouteArgs route_args(int64_t T, int E, int k, int dtype, const void* logits, int64_t ld,
                          int normalize) {
  agg::RouteArgs a;
  std::memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.T = T;
  a.ld = ld;
  a.E = E;
  a.k = k;
  a.dtype = dtype;
  a.normalize = normalize;
  return a;
}

int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? AG_GEMM_OK : cuda_fail(e, what);
}

}  // namespace

// ------------------------------------------------------------------ plan
struct ag_moe_plan {
  int E = 0;
  int64_t K = 0, N = 0;
  int dtype = 0;
  int device = 0;
  int pairs = 0;
  uint32_t* status = nullptr;    // [4], then the arrival counters
  uint32_t* arrivals = nullptr;
  int64_t arrival_count = 0;
  float* partials = nullptr;     // null until the first run that may split its sums
  uint64_t timeout_ns = 2000000000ull;
  cudaEvent_t done = nullptr;
  // The last run that may split its sums, and so use the workspace: `done` is recorded
  // behind it, and the next such run on another stream waits for it.  Others share
  // nothing with it but the status word; an event behind each would cost a call a
  // quarter of its host time (4.5 us against 3.4).
  agg::StreamId last_stream;
  bool has_run = false;
  bool loose = false;  // a run without an event since the last status or reset
  bool cleared = false;  // a reset since the last status: runs on other streams wait for `done` too
  // The same inside a graph capture: branches of one capture are put in order.
  cudaEvent_t captured = nullptr;
  agg::StreamId captured_stream;
  unsigned long long capture_id = 0;
};

namespace {

// Workspace of split sums: 40 MB hold 608 units of short tiles or 152 of long
// ones.  Sums are split only where there are fewer than two tiles a pair.  A plan gets it
// with its first run that may split: many plans of a model never do.
constexpr int64_t kPartialBytes = 608 * agg::split_unit_bytes(true);
static_assert(kPartialBytes == 152 * agg::split_unit_bytes(false), "both tile heights");
int max_units(bool few) { return static_cast<int>(kPartialBytes / agg::split_unit_bytes(few)); }

cudaError_t allocate_partials(ag_moe_plan* p) {
  // (allowed while a stream is being captured: the allocation is no part of the graph)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return e;
  e = cudaMalloc(&p->partials, static_cast<size_t>(kPartialBytes));
  if (e != cudaSuccess) p->partials = nullptr;
  const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
  return e != cudaSuccess ? e : back;
}

// Whether a sum of so many k-blocks can be split: whether that pays in the best case, all
// parts running at once.  (More tiles than pairs make it pay less: the parts' rounds
// then save no more of the k-blocks, and cost more.)
bool may_split(int64_t KB, agg::SplitPrice price) {
  for (int64_t s = 2; s <= agg::kMaxSplit && s * agg::kMinPart <= KB; ++s)
    if ((KB + s - 1) / s + price.once + s * price.part < KB) return true;
  return false;
}

// Rows of a product: with a tile's height beyond them, row numbers stay below 2^31.
constexpr int64_t kMaxRows = (1LL << 31) - 256;
static_assert(agg::kXRows <= 256 && agg::kXSub * 64 <= 256, "rows beyond the last that a tile or a stage reaches");

// k-blocks of a segment where the output is fp32, and where it has 16 bits: each of a
// k-block's four additions in the tensor core loses up to 2^-23 of the sum, always towards
// zero, so 8 k-blocks cost up to 4e-6 and 128 up to 6e-5, an eighth of fp16's half last
// bit.  (Sums of 2^22 positive fp16 products in one segment were off by 1.6e-3, in
// segments of 128 k-blocks by 2.2e-4, the rounding of the output.)
constexpr int kSegment = 8, kSegment16 = 128;

struct Prepared {
  cudaError_t e;
  int pairs;
};
Prepared prepare_once(int device) {
  constexpr int kDevices = 64;
  static std::mutex mu;
  static Prepared of[kDevices];
  static bool done[kDevices];
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= kDevices) return {cudaErrorInvalidDevice, 0};
  if (!done[device]) {
    of[device].e = agg::experts_prepare(&of[device].pairs);
    done[device] = of[device].e == cudaSuccess;
  }
  return of[device];
}

void free_plan(ag_moe_plan* p) {
  if (p->done) cudaEventDestroy(p->done);
  if (p->captured) cudaEventDestroy(p->captured);
  if (p->status) cudaFree(p->status);
  if (p->partials) cudaFree(p->partials);
  delete p;
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == AG_MOE_E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// An operand whose sum runs along the memory rows' length: two k-blocks of 128 bytes by
// `height` rows of one of E matrices (extent len x rows).  With whole blocks the length
// is described in blocks and one box brings both.
bool whole_blocks(int dtype, int64_t len) { return len * esize(dtype) % 128 == 0; }
int encode_k_major(CUtensorMap* map, int dtype, const void* base, int64_t len, int64_t rows,
                   int64_t ld, int64_t E, int64_t ld_e, int height) {
  const int es = esize(dtype);
  const cuuint64_t in = 128 / es;
  if (whole_blocks(dtype, len)) {
    const cuuint64_t dims[4] = {in, (cuuint64_t)rows, (cuuint64_t)len / in, (cuuint64_t)E};
    const cuuint64_t strides[3] = {(cuuint64_t)ld * es, 128, (cuuint64_t)ld_e * es};
    const cuuint32_t box[4] = {(cuuint32_t)in, (cuuint32_t)height, agg::kXSub, 1};
    return encode_tiled(map, map_type(dtype), base, 4, dims, strides, box);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)len, (cuuint64_t)rows, (cuuint64_t)E};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * es, (cuuint64_t)ld_e * es};
  const cuuint32_t box[3] = {(cuuint32_t)in, (cuuint32_t)height, 1};
  return encode_tiled(map, map_type(dtype), base, 3, dims, strides, box);
}

// An operand whose sum runs across the memory rows (2-byte elements): 128 rows (two
// k-blocks) by 64 columns; with cols % 64 == 0 in blocks of 64 columns, two of them a
// box, so that a CTA's 128 columns are one load.
int encode_mn_major(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t ld,
                    int64_t E, int64_t ld_e, int blocks = 2) {
  if (whole_blocks(AG_GEMM_F16, cols)) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)cols / 64, (cuuint64_t)E};
    const cuuint64_t strides[3] = {(cuuint64_t)ld * 2, 128, (cuuint64_t)ld_e * 2};
    const cuuint32_t box[4] = {64, 64 * agg::kXSub, (cuuint32_t)blocks, 1};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, 4, dims, strides, box);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)E};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld_e * 2};
  const cuuint32_t box[3] = {64, 64 * agg::kXSub, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, 3, dims, strides, box);
}

int check_matrix(const char* name, const void* p, int64_t ld, int64_t cols, int dtype) {
  if (!p) return fail(AG_GEMM_ERR_INVALID, "%s is NULL", name);
  if (!aligned16(p)) return fail(AG_GEMM_ERR_INVALID, "%s must be 16-byte aligned", name);
  if (ld < cols || ld * esize(dtype) % 16 != 0)
    return fail(AG_GEMM_ERR_INVALID, "%s: row pitch %lld must be at least %lld and a multiple of 16 bytes",
                name, (long long)ld, (long long)cols);
  if (ld >= (1LL << 36)) return fail(AG_GEMM_ERR_UNSUPPORTED, "%s: row pitch too large", name);
  return AG_GEMM_OK;
}

int check_run(ag_moe_plan* p, bool fp8, int64_t rows, const int32_t* offsets, int out_dtype) {
  if (!p) return fail(AG_GEMM_ERR_INVALID, "plan is NULL");
  if ((p->dtype == AG_MOE_E4M3) != fp8)
    return fail(AG_GEMM_ERR_INVALID, fp8 ? "ag_fp8_forward needs an AG_MOE_E4M3 plan"
                                         : "this product needs an fp16 or bf16 plan (AG_MOE_E4M3: ag_fp8_forward)");
  if (rows < 0 || rows > kMaxRows)
    return fail(AG_GEMM_ERR_INVALID, "rows must be in [0, %lld] (got %lld)", (long long)kMaxRows, (long long)rows);
  if (!offsets && p->E != 1)
    return fail(AG_GEMM_ERR_INVALID, "offsets may be NULL only for one expert (the plan has %d)", p->E);
  const bool ok = out_dtype == AG_MOE_F32 ||
                  (fp8 ? out_dtype == AG_GEMM_F16 || out_dtype == AG_GEMM_BF16 : out_dtype == p->dtype);
  if (!ok) return fail(AG_GEMM_ERR_INVALID, "out_dtype %d does not fit the plan's type %d", out_dtype, p->dtype);
  return AG_GEMM_OK;
}

// Row tiles that the groups of so many rows can make.
int64_t most_row_tiles(const ag_moe_plan* p, int64_t rows, bool few) {
  return rows / (few ? agg::kXFewRows : agg::kXRows) + (rows < p->E ? rows : p->E);
}

// Short row tiles where the groups are short on average: 64 rows a tile leave ten
// stages for the weights in flight, 256 read the weights once where a group is longer.
// (32 experts of 4096 x 4096, bf16: 64 rows each 166 us short, 167 long, 80 rows 177 and
// 169; e4m3: 80 rows 118 and 130, 96 rows 130 and 131, 128 rows 155 and 135.)
// And where all of them run at once: a k-block of 256 rows takes 0.23 us, of 64 0.14.
// (One expert, 200 rows of 1024 x 2048, 32 short tiles: 7.5 us against 10.7; e4m3 7.3
// against 10.1.  In two rounds of short tiles 1200 rows of 1024 x 2048 took 10.7 against
// 12.1 us, 600 of 2048 x 3000 18.4 against 15.0; e4m3 1088 of 4096 x 2048 22.2 against 21.2.)
bool few_rows(const ag_moe_plan* p, int64_t rows, int64_t wide) {
  return rows <= static_cast<int64_t>(p->dtype == AG_MOE_E4M3 ? 96 : 64) * p->E ||
         most_row_tiles(p, rows, true) * ((wide + agg::kXWide - 1) / agg::kXWide) <= p->pairs;
}

int run(ag_moe_plan* p, agg::ExpertsParams& x, int op, bool few, int64_t row_tiles,
        void* stream_v) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  x.E = p->E;
  x.bf16 = p->dtype == AG_GEMM_BF16;
  x.segment = x.out_type == AG_MOE_F32 ? kSegment : kSegment16;
  x.arrivals = p->arrivals;
  x.status = p->status;
  // (8192 x 4096 x 4096, e4m3: 125 us with 32-byte stores, 134 with rows 16 bytes off)
  x.rows32 = x.out_type != AG_MOE_F32 && (reinterpret_cast<uintptr_t>(x.out) & 31u) == 0 && x.ldo % 16 == 0;
  x.timeout_ns = p->timeout_ns;
  const int64_t wide_tiles = (x.wide + agg::kXWide - 1) / agg::kXWide;
  if ((row_tiles + agg::kXGroup) * wide_tiles >= (1LL << 30))
    return fail(AG_GEMM_ERR_UNSUPPORTED, "more than 2^30 tiles");
  x.inv_group = 0xffffffffu / static_cast<uint32_t>(agg::kXGroup * wide_tiles);
  x.inv_expert = op == agg::kOpWeight ? 0xffffffffu / static_cast<uint32_t>(wide_tiles * x.row_tiles) : 0;
  const bool fp8 = op == agg::kOpFp8;
  const int64_t kb = op == agg::kOpWeight ? x.rows / 64 : (x.red + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64);
  // (where the tiles' number does not depend on offsets, two rounds of them never split)
  const bool plenty = (op == agg::kOpWeight || !x.offsets) && (row_tiles - 1) * wide_tiles >= 2 * p->pairs;
  const bool split = !plenty && may_split(kb, agg::split_price(fp8 && !few ? agg::kOpFp8Long : op,
                                                    op == agg::kOpWeight ? x.step < agg::kXRows : few));
  x.max_units = split ? max_units(few) : 0;
  cudaError_t e = split && !p->partials ? allocate_partials(p) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "workspace of split sums");
  x.partials = p->partials;
  // A captured run is ordered by its graph: an event of the streams outside cannot be
  // waited on there, nor one of the graph outside.
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  unsigned long long capture_id = 0;
  if ((e = cudaStreamGetCaptureInfo(stream, &capture, &capture_id)) != cudaSuccess)
    return cuda_fail(e, "cudaStreamGetCaptureInfo");
  const bool captured = capture != cudaStreamCaptureStatusNone;
  const bool ordered = split || (p->cleared && !captured);
  const agg::StreamId id = ordered ? agg::StreamId(stream, captured) : agg::StreamId();
  const bool wait = ordered && (captured ? p->capture_id == capture_id && p->captured_stream != id
                                         : p->has_run && p->last_stream != id);
  if (wait && (e = cudaStreamWaitEvent(stream, captured ? p->captured : p->done, 0)) != cudaSuccess)
    return cuda_fail(e, "cudaStreamWaitEvent");
  // no more pairs than there can be units
  const int64_t parts = !split ? 1 : kb / agg::kMinPart < agg::kMaxSplit ? kb / agg::kMinPart : agg::kMaxSplit;
  const int64_t units = row_tiles * wide_tiles * parts;
  const int pairs = static_cast<int>(units < p->pairs ? units : p->pairs);
  if ((e = agg::launch_experts(x, op, few, 2 * pairs, stream)) != cudaSuccess)
    return cuda_fail(e, "experts kernel launch");
  if (!split) {
    p->loose = true;
  } else if ((e = cudaEventRecord(captured ? p->captured : p->done, stream)) != cudaSuccess) {
    return cuda_fail(e, "cudaEventRecord");
  } else if (captured) {
    p->captured_stream = id;
    p->capture_id = capture_id;
  } else {
    p->last_stream = id;
    p->has_run = true;
  }
  log_msg(3, "plan %p: experts product %d enqueued, %d rows", static_cast<void*>(p), op, x.rows);
  return AG_GEMM_OK;
}

// The row operand, once for each height of box that its tiles can have.
int encode_rows(agg::ExpertsParams& x, int dtype, const void* base, int64_t len, int64_t rows,
                int64_t ld, bool few) {
  const int step = (few ? agg::kXFewRows : agg::kXRows) / 8;
  const int64_t half = (rows + 31) / 32 * 16;  // of a CTA, in a tile of all rows
  const int most = (dtype == AG_MOE_E4M3 && !few) || half >= 4 * step ? agg::kXRowBoxes
                                                                   : static_cast<int>((half + step - 1) / step);
  x.r_blk = whole_blocks(dtype, len);
  for (int i = 0; i < agg::kXRowBoxes; ++i) {
    if (i >= most) {
      x.tm_r[i] = x.tm_r[i - 1];
      continue;
    }
    if (int rc = encode_k_major(&x.tm_r[i], dtype, base, len, rows, ld, 1, rows * ld, (i + 1) * step)) return rc;
  }
  return AG_GEMM_OK;
}

// Forward and input gradient: out rows x wide over red.
int run_rows(ag_moe_plan* p, int op, int64_t rows, const void* in, int64_t ld_in,
             const int32_t* offsets, const void* w, int64_t ldw, int64_t ldw_e, void* out,
             int64_t ld_out, int out_dtype, void* stream) {
  const bool fwd = op == agg::kOpForward;
  if (int rc = check_run(p, false, rows, offsets, out_dtype)) return rc;
  const int64_t red = fwd ? p->K : p->N, wide = fwd ? p->N : p->K;
  if (rows == 0) return AG_GEMM_OK;
  if (int rc = check_matrix(fwd ? "x" : "dy", in, ld_in, red, p->dtype)) return rc;
  if (int rc = check_matrix("w", w, ldw, p->N, p->dtype)) return rc;
  if (int rc = check_matrix(fwd ? "y" : "dx", out, ld_out, wide, out_dtype)) return rc;
  if (p->E > 1 && (ldw_e < p->K * ldw || ldw_e % 8 != 0 || ldw_e >= (1LL << 38)))
    return fail(AG_GEMM_ERR_INVALID, "w: the experts' distance %lld must be at least K rows and a multiple of 16 bytes",
                (long long)ldw_e);
  if (p->E == 1) ldw_e = p->K * ldw;
  DeviceGuard dg(p->device);
  const bool few = few_rows(p, rows, wide);
  agg::ExpertsParams x{};
  int rc = fwd ? encode_mn_major(&x.tm_w, w, p->N, p->K, ldw, p->E, ldw_e)
               : encode_k_major(&x.tm_w, p->dtype, w, p->N, p->K, ldw, p->E, ldw_e, 128);
  if (rc || (rc = encode_rows(x, p->dtype, in, red, rows, ld_in, few))) return rc;
  x.w_blk = whole_blocks(p->dtype, p->N);
  x.offsets = offsets;
  x.rows = static_cast<int32_t>(rows);
  x.wide = static_cast<int32_t>(wide);
  x.red = static_cast<int32_t>(red);
  x.out_type = out_dtype;
  x.out = out;
  x.ldo = ld_out;
  return run(p, x, op, few, most_row_tiles(p, rows, few), stream);
}

}  // namespace

extern "C" {

int64_t ag_moe_route_workspace(int64_t T, int E, int top_k) {
  if (int rc = check_route(T, E, top_k, AG_MOE_F32)) return rc;
  const int blocks = agg::route_blocks(T, top_k);
  return blocks == 1 ? 0 : static_cast<int64_t>(blocks) * E * 4;
}

int ag_moe_route(int64_t T, int E, int top_k, int dtype, const void* logits, int64_t ld,
                 int normalize, float* weights, int32_t* experts, int32_t* offsets,
                 int32_t* order, int32_t* slots, void* workspace, void* stream) {
  if (int rc = check_route(T, E, top_k, dtype)) return rc;
  if (!offsets || (T > 0 && (!logits || !weights || !experts || !order || !slots)))
    return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (ld < E) return fail(AG_GEMM_ERR_INVALID, "row pitch %lld is less than %d experts", (long long)ld, E);
  if (agg::route_blocks(T, top_k) > 1 && !workspace)
    return fail(AG_GEMM_ERR_INVALID, "workspace is NULL (see ag_moe_route_workspace)");
  agg::RouteArgs a = route_args(T, E, top_k, dtype, logits, ld, normalize);
  a.weights = weights;
  a.experts = experts;
  a.offsets = offsets;
  a.order = order;
  a.slots = slots;
  a.counts = static_cast<int32_t*>(workspace);
  return launched(agg::launch_route(a, static_cast<cudaStream_t>(stream)), "router launch");
}

int ag_moe_route_backward(int64_t T, int E, int top_k, int dtype, const void* logits, int64_t ld,
                          int normalize, const float* weights, const int32_t* experts,
                          const float* dweights, void* dlogits, void* stream) {
  if (int rc = check_route(T, E, top_k, dtype)) return rc;
  if (T == 0) return AG_GEMM_OK;
  if (!logits || !weights || !experts || !dweights || !dlogits)
    return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (ld < E) return fail(AG_GEMM_ERR_INVALID, "row pitch %lld is less than %d experts", (long long)ld, E);
  agg::RouteArgs a = route_args(T, E, top_k, dtype, logits, ld, normalize);
  a.weights = const_cast<float*>(weights);
  a.experts = const_cast<int32_t*>(experts);
  return launched(agg::launch_route_backward(a, dweights, dlogits, static_cast<cudaStream_t>(stream)),
                  "router gradient launch");
}

int ag_moe_gather(int64_t T, int top_k, int64_t H, int dtype, const void* x, int64_t ldx,
                  const int32_t* order, void* out, void* stream) {
  if (int rc = check_rows(T, top_k, H, dtype)) return rc;
  if (T == 0) return AG_GEMM_OK;
  if (!x || !order || !out) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (ldx < H) return fail(AG_GEMM_ERR_INVALID, "row pitch %lld is less than %lld columns", (long long)ldx, (long long)H);
  return launched(agg::launch_gather(T, top_k, H, dtype, x, ldx, order, out,
                                     static_cast<cudaStream_t>(stream)), "gather launch");
}

int ag_moe_combine(int64_t T, int top_k, int64_t H, int dtype, const void* y, int64_t ldy,
                   const int32_t* slots, const float* weights, void* out, void* stream) {
  if (int rc = check_rows(T, top_k, H, dtype)) return rc;
  if (T == 0) return AG_GEMM_OK;
  if (!y || !slots || !out) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (ldy < H) return fail(AG_GEMM_ERR_INVALID, "row pitch %lld is less than %lld columns", (long long)ldy, (long long)H);
  return launched(agg::launch_combine(T, top_k, H, dtype, y, ldy, slots, weights, out,
                                      static_cast<cudaStream_t>(stream)), "combine launch");
}

int ag_moe_combine_backward(int64_t T, int top_k, int64_t H, int dtype, const void* dout,
                            int64_t ldd, const void* y, int64_t ldy, const int32_t* slots,
                            const float* weights, const int32_t* offsets_end, void* dy,
                            float* dweights, void* stream) {
  if (int rc = check_rows(T, top_k, H, dtype)) return rc;
  if (T == 0) return AG_GEMM_OK;
  if (!dout || !y || !slots || !weights || !dy || !dweights)
    return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (ldd < H || ldy < H)
    return fail(AG_GEMM_ERR_INVALID, "row pitches %lld, %lld are less than %lld columns", (long long)ldd,
                (long long)ldy, (long long)H);
  return launched(agg::launch_combine_backward(T, top_k, H, dtype, dout, ldd, y, ldy, slots, weights,
                                               offsets_end, dy, dweights,
                                               static_cast<cudaStream_t>(stream)),
                  "combine gradient launch");
}

int ag_fp8_quantize_rows(int64_t rows, int64_t K, int dtype, const void* x, int64_t ldx,
                         int64_t src_rows, const int32_t* order, int top_k, void* q,
                         float* scales, void* stream) {
  if (!float_type(dtype)) return fail(AG_GEMM_ERR_INVALID, "x must be fp16, bf16 or fp32 (got type %d)", dtype);
  if (rows < 0 || rows >= (1LL << 31) || src_rows < 0 || (!order && src_rows < rows))
    return fail(AG_GEMM_ERR_INVALID, "rows must be in [0, 2^31) and, without order, at most src_rows (got %lld of %lld)",
                (long long)rows, (long long)src_rows);
  if (K < 16 || K % 16 != 0 || K > kMaxRowLen)
    return fail(AG_GEMM_ERR_INVALID, "K must be a multiple of 16, at most %lld (got %lld)", (long long)kMaxRowLen,
                (long long)K);
  if (order && (top_k < 1 || top_k > agg::kMaxTopK))
    return fail(AG_GEMM_ERR_INVALID, "top_k must be in [1, %d] (got %d)", agg::kMaxTopK, top_k);
  if (rows == 0) return AG_GEMM_OK;
  if (int rc = check_matrix("x", x, ldx, K, dtype)) return rc;
  if (!q || !scales) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (!aligned16(q)) return fail(AG_GEMM_ERR_INVALID, "q must be 16-byte aligned");
  return launched(agg::launch_quantize_rows(rows, K, dtype, x, ldx, src_rows, order, top_k, q, scales,
                                            static_cast<cudaStream_t>(stream)),
                  "row quantisation launch");
}

int ag_fp8_quantize_weights(int E, int64_t K, int64_t N, int dtype, const void* w, void* q,
                            float* scales, void* stream) {
  if (!float_type(dtype)) return fail(AG_GEMM_ERR_INVALID, "w must be fp16, bf16 or fp32 (got type %d)", dtype);
  if (E < 1 || E > agg::kMaxExperts)
    return fail(AG_GEMM_ERR_INVALID, "experts must be in [1, %d] (got %d)", agg::kMaxExperts, E);
  if (K < 16 || K % 16 != 0 || N < 8 || N % 8 != 0 || K > kMaxRowLen || N > kMaxRowLen)
    return fail(AG_GEMM_ERR_INVALID, "need K %% 16 == 0 and N %% 8 == 0, at most %lld (got %lld, %lld)",
                (long long)kMaxRowLen, (long long)K, (long long)N);
  if (E * ((K + 127) / 128) * ((N + 127) / 128) >= (1LL << 31))
    return fail(AG_GEMM_ERR_UNSUPPORTED, "more than 2^31 scale blocks");
  if (!w || !q || !scales) return fail(AG_GEMM_ERR_INVALID, "a pointer is NULL");
  if (!aligned16(w) || !aligned16(q)) return fail(AG_GEMM_ERR_INVALID, "w and q must be 16-byte aligned");
  return launched(agg::launch_quantize_weights(E, K, N, dtype, w, q, scales, static_cast<cudaStream_t>(stream)),
                  "weight quantisation launch");
}

ag_moe_plan* ag_moe_plan_create(int E, int64_t K, int64_t N, int dtype) {
  if (dtype != AG_GEMM_F16 && dtype != AG_GEMM_BF16 && dtype != AG_MOE_E4M3) {
    fail(AG_GEMM_ERR_INVALID, "dtype must be AG_GEMM_F16, AG_GEMM_BF16 or AG_MOE_E4M3 (got %d)", dtype);
    return nullptr;
  }
  if (E < 1 || E > agg::kMaxExperts) {
    fail(AG_GEMM_ERR_INVALID, "experts must be in [1, %d] (got %d)", agg::kMaxExperts, E);
    return nullptr;
  }
  const int kmod = dtype == AG_MOE_E4M3 ? 16 : 8;
  if (K < kmod || K % kmod != 0 || N < 8 || N % 8 != 0 || K > kMaxRowLen || N > kMaxRowLen) {
    fail(AG_GEMM_ERR_INVALID, "need K %% %d == 0 and N %% 8 == 0, both in (0, %lld] (got %lld, %lld)", kmod,
         (long long)kMaxRowLen, (long long)K, (long long)N);
    return nullptr;
  }
  if (E * ((K + 255) / 256) * ((N + 255) / 256) >= (1LL << 30)) {
    fail(AG_GEMM_ERR_UNSUPPORTED, "more than 2^30 weight tiles");
    return nullptr;
  }
  int device = 0, major = 0, minor = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&device)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device)) != cudaSuccess) {
    cuda_fail(e, "device query");
    return nullptr;
  }
  if (major != 10 || minor != 3) {
    fail(AG_GEMM_ERR_UNSUPPORTED, "needs an sm_103 (GB300) device, found sm_%d%d", major, minor);
    return nullptr;
  }
  const Prepared pre = prepare_once(device);
  if (pre.e != cudaSuccess || pre.pairs < 1) {
    if (pre.e == cudaSuccess) fail(AG_GEMM_ERR_UNSUPPORTED, "experts kernel clusters do not fit");
    else cuda_fail(pre.e, "experts kernel occupancy");
    return nullptr;
  }
  ag_moe_plan* p = new (std::nothrow) ag_moe_plan();
  if (!p) {
    fail(AG_GEMM_ERR_OOM, "host allocation failed");
    return nullptr;
  }
  p->E = E;
  p->K = K;
  p->N = N;
  p->dtype = dtype;
  p->device = device;
  p->pairs = pre.pairs;
  p->arrival_count = static_cast<int64_t>(max_units(true)) * 2 * agg::kXEpiWarps;
  const size_t words = static_cast<size_t>(4 + p->arrival_count) * sizeof(uint32_t);
  agg::Clearer clearer;
  if ((e = cudaMalloc(&p->status, words)) != cudaSuccess ||
      (e = clearer.clear(p->status, words)) != cudaSuccess ||
      (e = cudaEventCreateWithFlags(&p->done, cudaEventDisableTiming)) != cudaSuccess ||
      (e = cudaEventCreateWithFlags(&p->captured, cudaEventDisableTiming)) != cudaSuccess ||
      (e = clearer.finish()) != cudaSuccess) {
    cuda_fail(e, "plan allocation");
    free_plan(p);
    return nullptr;
  }
  p->arrivals = p->status + 4;
  log_msg(2, "plan %p: %d experts, K=%lld N=%lld dtype=%d, %d pairs", static_cast<void*>(p), E,
          (long long)K, (long long)N, dtype, p->pairs);
  return p;
}

void ag_moe_plan_destroy(ag_moe_plan* plan) {
  if (!plan) return;
  log_msg(2, "plan %p destroyed", static_cast<void*>(plan));
  DeviceGuard dg(plan->device);
  free_plan(plan);
}

int ag_moe_plan_device(const ag_moe_plan* plan) {
  if (!plan) return fail(AG_GEMM_ERR_INVALID, "plan is NULL");
  return plan->device;
}

int ag_moe_plan_tile_rows(const ag_moe_plan* plan, int64_t rows, int input_gradient) {
  if (!plan) return fail(AG_GEMM_ERR_INVALID, "plan is NULL");
  if (rows < 0 || rows > kMaxRows)
    return fail(AG_GEMM_ERR_INVALID, "rows must be in [0, %lld] (got %lld)", (long long)kMaxRows, (long long)rows);
  if (input_gradient && plan->dtype == AG_MOE_E4M3)
    return fail(AG_GEMM_ERR_INVALID, "an AG_MOE_E4M3 plan has no input gradient");
  return few_rows(plan, rows, input_gradient ? plan->K : plan->N) ? agg::kXFewRows : agg::kXRows;
}

int64_t ag_moe_plan_status_word(ag_moe_plan* plan) {
  if (!plan) return fail(AG_GEMM_ERR_INVALID, "plan is NULL");
  DeviceGuard dg(plan->device);
  cudaError_t e;
  if (plan->loose && (e = cudaDeviceSynchronize()) != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  if (!plan->loose && plan->has_run && (e = cudaEventSynchronize(plan->done)) != cudaSuccess)
    return cuda_fail(e, "cudaEventSynchronize");
  plan->loose = plan->cleared = false;
  uint32_t w[4] = {0, 0, 0, 0};
  if ((e = cudaMemcpy(w, plan->status, sizeof(w), cudaMemcpyDeviceToHost)) != cudaSuccess)
    return cuda_fail(e, "status read");
  const int i = w[0] != agg::kStatusOk ? 0 : 2;
  return static_cast<int64_t>(w[i]) | (static_cast<int64_t>(w[i + 1]) << 32);
}

int ag_moe_plan_status(ag_moe_plan* plan) {
  const int64_t w = ag_moe_plan_status_word(plan);
  if (w < 0) return static_cast<int>(w);
  const uint32_t kind = static_cast<uint32_t>(w & 0xFF);
  if (kind == agg::kStatusOk) return AG_GEMM_OK;
  if (kind == agg::kStatusOffsets)
    return fail(AG_GEMM_ERR_INVALID, "offsets decrease or leave [0, rows]: the run wrote nothing");
  return fail(AG_GEMM_ERR_TIMEOUT, "device wait timed out (status 0x%llx)", (unsigned long long)w);
}

int ag_moe_plan_reset(ag_moe_plan* plan, void* stream_v) {
  if (!plan) return fail(AG_GEMM_ERR_INVALID, "plan is NULL");
  DeviceGuard dg(plan->device);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  const agg::StreamId id(stream, agg::is_captured(stream));
  cudaError_t e;
  if (plan->loose && (e = cudaDeviceSynchronize()) != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  if (!plan->loose && plan->has_run && plan->last_stream != id &&
      (e = cudaStreamWaitEvent(stream, plan->done, 0)) != cudaSuccess)
    return cuda_fail(e, "cudaStreamWaitEvent");
  plan->loose = false;
  if ((e = cudaMemsetAsync(plan->status, 0, static_cast<size_t>(4 + plan->arrival_count) * sizeof(uint32_t),
                           stream)) != cudaSuccess ||
      (e = cudaEventRecord(plan->done, stream)) != cudaSuccess)
    return cuda_fail(e, "plan reset");
  plan->last_stream = id;
  plan->has_run = true;
  plan->cleared = true;
  return AG_GEMM_OK;
}

int ag_moe_plan_set_timeout_ns(ag_moe_plan* plan, int64_t ns) {
  if (!plan) return fail(AG_GEMM_ERR_INVALID, "plan is NULL");
  if (ns <= 0) return fail(AG_GEMM_ERR_INVALID, "timeout must be positive");
  plan->timeout_ns = static_cast<uint64_t>(ns);
  return AG_GEMM_OK;
}

int ag_moe_forward(ag_moe_plan* plan, int64_t rows, const void* x, int64_t ldx,
                   const int32_t* offsets, const void* w, int64_t ldw, int64_t ldw_expert,
                   void* y, int64_t ldy, int out_dtype, void* stream) {
  return run_rows(plan, agg::kOpForward, rows, x, ldx, offsets, w, ldw, ldw_expert, y, ldy, out_dtype, stream);
}

int ag_moe_backward_input(ag_moe_plan* plan, int64_t rows, const void* dy, int64_t lddy,
                          const int32_t* offsets, const void* w, int64_t ldw, int64_t ldw_expert,
                          void* dx, int64_t lddx, int out_dtype, void* stream) {
  return run_rows(plan, agg::kOpInput, rows, dy, lddy, offsets, w, ldw, ldw_expert, dx, lddx, out_dtype, stream);
}

int ag_moe_backward_weight(ag_moe_plan* plan, int64_t rows, const void* x, int64_t ldx,
                           const void* dy, int64_t lddy, const int32_t* offsets, void* dw,
                           int out_dtype, void* stream) {
  if (int rc = check_run(plan, false, rows, offsets, out_dtype)) return rc;
  if (!dw) return fail(AG_GEMM_ERR_INVALID, "dw is NULL");
  if (!aligned16(dw)) return fail(AG_GEMM_ERR_INVALID, "dw must be 16-byte aligned");
  DeviceGuard dg(plan->device);
  if (rows == 0) {
    const size_t bytes = static_cast<size_t>(plan->E) * plan->K * plan->N * esize(out_dtype);
    return launched(cudaMemsetAsync(dw, 0, bytes, static_cast<cudaStream_t>(stream)), "zero gradient");
  }
  if (int rc = check_matrix("x", x, ldx, plan->K, plan->dtype)) return rc;
  if (int rc = check_matrix("dy", dy, lddy, plan->N, plan->dtype)) return rc;
  agg::ExpertsParams p{};
  int rc;
  if ((rc = encode_mn_major(&p.tm_w, dy, plan->N, rows, lddy, 1, rows * lddy)) ||
      (rc = encode_mn_major(&p.tm_r[0], x, plan->K, rows, ldx, 1, rows * ldx)) ||
      (rc = encode_mn_major(&p.tm_r[1], x, plan->K, rows, ldx, 1, rows * ldx, 1)))
    return rc;
  p.w_blk = whole_blocks(plan->dtype, plan->N);
  p.r_blk = whole_blocks(plan->dtype, plan->K);
  p.offsets = offsets;
  p.rows = static_cast<int32_t>(rows);
  p.wide = static_cast<int32_t>(plan->N);
  p.out_rows = static_cast<int32_t>(plan->K);
  // Half tiles where all of them run at once: half the rows to store and half of x to
  // load per k-block.  (3754 rows of 608 x 376: 16.2 us against 22.4; 64 of 4096 x 512:
  // 7.4 against 8.2.  Twice as many tiles as pairs would cost a second round.)
  const int64_t halves = plan->E * ((plan->K + 127) / 128) * ((plan->N + agg::kXWide - 1) / agg::kXWide);
  p.step = halves <= plan->pairs ? agg::kXRows / 2 : agg::kXRows;
  p.row_tiles = (p.out_rows + p.step - 1) / p.step;
  p.out_type = out_dtype;
  p.out = dw;
  p.ldo = plan->N;
  return run(plan, p, agg::kOpWeight, false, static_cast<int64_t>(plan->E) * p.row_tiles, stream);
}

int ag_fp8_forward(ag_moe_plan* plan, int64_t rows, const void* xq, const float* xs,
                   const int32_t* offsets, const void* wq, const float* ws, void* y, int64_t ldy,
                   int out_dtype, void* stream) {
  if (int rc = check_run(plan, true, rows, offsets, out_dtype)) return rc;
  if (rows == 0) return AG_GEMM_OK;
  if (int rc = check_matrix("xq", xq, plan->K, plan->K, AG_MOE_E4M3)) return rc;
  if (int rc = check_matrix("wq", wq, plan->K, plan->K, AG_MOE_E4M3)) return rc;
  if (int rc = check_matrix("y", y, ldy, plan->N, out_dtype)) return rc;
  if (!xs || !ws) return fail(AG_GEMM_ERR_INVALID, "scales are NULL");
  DeviceGuard dg(plan->device);
  const bool few = few_rows(plan, rows, plan->N);
  agg::ExpertsParams p{};
  int rc;
  if ((rc = encode_k_major(&p.tm_w, AG_MOE_E4M3, wq, plan->K, plan->N, plan->K, plan->E, plan->K * plan->N, 128)) ||
      (rc = encode_rows(p, AG_MOE_E4M3, xq, plan->K, rows, plan->K, few)))
    return rc;
  p.w_blk = whole_blocks(AG_MOE_E4M3, plan->K);
  p.offsets = offsets;
  p.rows = static_cast<int32_t>(rows);
  p.wide = static_cast<int32_t>(plan->N);
  p.red = static_cast<int32_t>(plan->K);
  p.out_type = out_dtype;
  p.out = y;
  p.ldo = ldy;
  p.xs = xs;
  p.ws = ws;
  return run(plan, p, agg::kOpFp8, few, most_row_tiles(plan, rows, few), stream);
}

}  // extern "C"
