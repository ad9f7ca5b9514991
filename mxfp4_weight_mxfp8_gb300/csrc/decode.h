// Launchers of the decode step's kernels around the expert layer, used by
// decode_api.cu, and the argument structures that they take.
#pragma once

#include "common.cuh"

namespace moe {

struct AppendArgs {
  moe_kv_cache_t c;
  const uint16_t* x[2];      // keys, values: BF16 rows
  int64_t token_stride[2], head_stride[2];
  const int64_t* slots;
  int tokens;
};

struct AttendArgs {
  moe_kv_cache_t c;
  moe_kv_batch_t b;
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  int q_heads, group;        // group: query heads of one cache head
  int window;
  float scale;
  uint16_t* out;
  float* lse;
  uint8_t* workspace;
  // Requests that share prefixes (kv_attend.cuh): the groups' rows of the block table, the pages that each request skips,
  // and the rows' outputs and (base 2) log-sum-exps over the prefixes.
  const int32_t* rows;
  const int32_t* skipped;
  float* partial;
  float* partial_lse;
  // Of the requests' own part: its arrival counters (3 * kAttendMaxCtas, zero) and room for its pieces.
  uint32_t* counters;
  float* pieces;
  // Where the prefixes' pieces are found: the groups' first units of the work, their sum and what an item counts as; their
  // first query tokens, prefixes and first blocks of 8 rows.
  long long* group_unit;
  const int32_t* group_token;
  const int32_t* group_prefix;
  const int32_t* group_block;
  const int32_t* shared;  // blocks of rows in all; 0: nothing is shared
  int early;  // kPrefix: whether it may work while the launch before it runs
};

// Items of more units of work may be cut between CTAs in the 128-row form (the others' all may).
constexpr int kAttendRowsLong = 16;
constexpr int kAttendRowsCtas = 240;
// Pieces of an item are joined in runs of about the square root of their number; so many are merged as they are. (Those of
// the 128-row form always are.)
constexpr int kAttendMerged = 32;
__host__ __device__ inline int attend_join_width(int pieces) {
  int width = 8;
  while (width * width < pieces) ++width;
  return width;
}
// Dimensions c4 .. c4 + 3 of row i in a piece of the prefixes' 128-row form, whose threads hold rows: quad by quad (other
// pieces are row by row).
__host__ __device__ constexpr int attend_quad_at(int i, int c4) { return c4 * 128 + i * 4; }

constexpr int kAttendMaxCtas = 512;

// Tiles of 128 that so many cache tokens take (any number up to 2^31 - 1).
__host__ __device__ inline int attend_tiles(int tokens) { return static_cast<int>((static_cast<uint32_t>(tokens) + 127u) / 128u); }

enum AttendMode : int { kWhole = 0, kPrefix = 1, kSuffix = 2 };

struct AttendMaps {
  CUtensorMap k, v;          // [pages * kv_heads][page_tokens][head_dim]; a box is a page's span of a head
};

cudaError_t launch_norm(const moe_norm_t& a, cudaStream_t stream);
cudaError_t launch_rope(const moe_rope_t& a, cudaStream_t stream);
cudaError_t launch_route(const moe_route_t& a, cudaStream_t stream);
cudaError_t launch_kv_plan(const moe_kv_plan_t& a, cudaStream_t stream);
cudaError_t launch_kv_fork(const moe_kv_fork_t& a, cudaStream_t stream);
cudaError_t launch_kv_copy(const moe_kv_cache_t& c, const int32_t* moves, const int32_t* count, int capacity, cudaStream_t stream);
cudaError_t launch_kv_reclaim(const moe_kv_reclaim_t& a, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_kv_attend(const AttendArgs& a, cudaStream_t stream);
cudaError_t launch_kv_attend_shared(const AttendArgs& a, const moe_kv_prefixes_t& p, void* scratch, cudaStream_t stream);
// The forms of 8 * tile query rows and of 128, in each mode.
cudaError_t launch_kv_attend_decode(const AttendArgs& a, const AttendMaps& maps, int tile, int shift, int sms, cudaStream_t stream);
cudaError_t launch_kv_attend_decode_prefix(const AttendArgs& a, const AttendMaps& maps, int tile, int shift, int sms, cudaStream_t stream);
cudaError_t launch_kv_attend_decode_suffix(const AttendArgs& a, const AttendMaps& maps, int tile, int shift, int sms, cudaStream_t stream);
// Their CTAs on so many SMs: each may leave two pieces of an item, of (head_dim + 2) floats a row.
int kv_attend_decode_ctas(int head_dim, int tile, int sms);
int kv_attend_rows_ctas(int sms);
// Joins the pieces that the prefixes' launch (its rows of a row tile, CTAs) left with the requests' own parts.
cudaError_t launch_kv_attend_merge(const AttendArgs& a, int rows, int ctas, cudaStream_t stream);
cudaError_t launch_kv_attend_rows(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream);
cudaError_t launch_kv_attend_rows_prefix(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream);
cudaError_t launch_kv_attend_rows_suffix(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream);

// What moe_norm refuses (null: nothing); `plan`: its codes go to a layer's plan.
const char* norm_fault(const moe_norm_t* n, bool plan);

const char* rope_fault(const moe_rope_t* r);

// Launches a kernel; `chained`: by programmatic dependent launch, for kernels that wait for what they need themselves.
template <class... Params, class... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, bool chained, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Sets this thread's error detail (moe_last_error_detail) and returns `status`.
int fail(int status, const char* format, ...);

}  // namespace moe
