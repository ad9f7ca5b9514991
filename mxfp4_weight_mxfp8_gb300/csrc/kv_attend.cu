// Attention over the paged 8-bit cache (moe_kv_attend, moe_kv_attend_shared in
// include/moe.h): which form a call takes, and the plan of shared prefixes.
//
// Requests in groups that share a prefix take four launches: a small plan, each
// request's own tokens, the prefix of every group for all of the group's rows at
// once (its keys and values read once, not once for each request), and the merging
// of what the two left.
#include <cudaTypedefs.h>

#include <atomic>

#include "decode.h"
#include "ptx.cuh"

namespace moe {
namespace {

using ptx::grid_launch_dependents;

cudaError_t encode_map(CUtensorMap* map, const uint8_t* data, const moe_kv_cache_t& c) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> entry{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 encode = entry.load(std::memory_order_acquire);
  if (encode == nullptr) {
    cudaDriverEntryPointQueryResult found{};
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", reinterpret_cast<void**>(&encode),
                                                           12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (encode == nullptr || found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    entry.store(encode, std::memory_order_release);
  }
  const cuuint64_t D = c.head_dim, P = c.page_tokens;
  const cuuint64_t dims[3] = {D, P, static_cast<cuuint64_t>(c.pages) * c.kv_heads};
  const cuuint64_t strides[2] = {D, D * P};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(D < 128 ? D : 128), static_cast<cuuint32_t>(P), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(data), dims, strides, box, elem,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Call {
  AttendMaps maps;
  int shift = 4, sms = 0;
  cudaError_t open(const moe_kv_cache_t& c) {
    while ((1 << shift) < c.page_tokens) ++shift;
    cudaError_t e = encode_map(&maps.k, c.k, c);
    if (e == cudaSuccess) e = encode_map(&maps.v, c.v, c);
    int device = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    return e;
  }
};

// The row tile that a call takes, in eights of rows; 0: the form of 128 rows.
int row_tile(const AttendArgs& a) {
  // Row tiles of 8, 16, 24 or 32, by the rows that a request has on average over the call, requests without rows and
  // padding included (the host knows no more): a wider tile costs its softmax and TMEM columns whether rows use them or
  // not, a narrower one reads the cache again (64 requests of up to 4096 tokens, heads of 128: 8 rows take 62 us in tiles
  // of 8, 73 in 16; 16 rows 74 in 16, 83 in 24; 24 rows 84 in 24, 96 in 32).
  // Many more rows are the 128-row form's (up to head_dim 128: there the two groups' scores and outputs fill the TMEM). The
  // same requests with 40 rows each take 151 us here and 161 there, with heads of 64 138 and 131; with 48 rows 178 and 162,
  // 166 and 131; two requests of 30 thousand tokens with 40 rows 62 and 91.
  const long long rows = static_cast<long long>(a.b.tokens) * a.group;
  if (a.c.head_dim <= 128 && rows > 44ll * a.b.requests) return 0;
  if (rows <= 8ll * a.b.requests) return 1;
  if (rows <= 16ll * a.b.requests || a.c.head_dim == 256) return 2;
  return rows <= 24ll * a.b.requests ? 3 : 4;
}

cudaError_t launch_whole(const AttendArgs& a, const Call& c, int tile, cudaStream_t stream) {
  return tile ? launch_kv_attend_decode(a, c.maps, tile, c.shift, c.sms, stream) : launch_kv_attend_rows(a, c.maps, c.shift, c.sms, stream);
}

// ------------------------------------------------------------- shared prefixes
// Prefixes are shared from this much saved work on, in tiles of 8 rows: what two launches, their starts and the merging cost.
// One prefix of 8192 tokens, 64 query heads on 8 of 128: 8 requests, 3020 tiles, take 37.9 us with it and 36.9 without, 4
// requests 36.8 and 27.0, 16 requests 39.1 and 57.6; 64 requests on 1024 tokens, 3558 tiles, 54.2 and 43.7, on 2048 50.6 and
// 63.4 (and 4 to 7 us go to looking where nothing is shared in the end). Heads of 64 turn at the same number. A tile of 256
// takes twice as long: 8 requests on 8192 tokens, 1638 tiles, 54.3 and 63.1, 64 on 2048, 3276 tiles, 109 and 125.
constexpr int least_tiles(int head_dim) { return head_dim == 256 ? 1600 : 3700; }
// And of those only groups for whom it saves a share of their prefix's work: what rows fill already many row tiles of their
// own reads a prefix as often either way (16 requests with up to 300 rows of 256 each: 506 us with it, 460 without).
constexpr int kLeastShare = 4;
// What a tile costs in row tiles of 8, 16, 24, 32 rows and (0) in the form of 128, in tenths of the first (from 64 ragged
// requests with 8 to 32 rows, 62 to 96 us, and 1.95 us a tile and SM in the form of 128).
constexpr int kTileCost[] = {21, 10, 12, 14, 15};

// The plan's share of what the host knows.
struct SharedWork {
  int shift;
  int group, kv_heads;        // query heads of one cache head; those
  int own;                    // cost of a tile of the prefix to a request
  int rows, cost;             // of the prefixes' launch: rows of a row tile, a tile's cost
};

// Scratch: the groups' first query tokens, prefixes (tokens) and rows of the block table, the pages that each request skips;
// the arrival counters of the requests' part, the groups' first blocks of 8 rows and units of work; then each row's log-sum-exp and output over its prefix.
struct Scratch {
  int32_t *start, *prefix, *row, *skipped;
  uint32_t* counters;
  int32_t* block;
  long long* unit;
  float *lse, *out;
  Scratch(void* p, const AttendArgs& a) {
    start = static_cast<int32_t*>(p);
    prefix = start + 2 * MOE_KV_MAX_REQUESTS;
    row = prefix + MOE_KV_MAX_REQUESTS;
    skipped = row + MOE_KV_MAX_REQUESTS;
    counters = reinterpret_cast<uint32_t*>(skipped + MOE_KV_MAX_REQUESTS);
    block = reinterpret_cast<int32_t*>(counters + 3 * kAttendMaxCtas);
    unit = reinterpret_cast<long long*>(block + 2 * MOE_KV_MAX_REQUESTS);
    out = reinterpret_cast<float*>(static_cast<uint8_t*>(p) + MOE_KV_SHARED_HEADER);
    lse = out + static_cast<int64_t>(a.b.tokens) * a.q_heads * a.c.head_dim;
  }
};
static_assert(7 * MOE_KV_MAX_REQUESTS * 4 + 3 * kAttendMaxCtas * 4 + (MOE_KV_MAX_REQUESTS + 2) * 8 <= MOE_KV_SHARED_HEADER, "the plan's room");
static_assert((7 * MOE_KV_MAX_REQUESTS + 3 * kAttendMaxCtas) % 2 == 0, "alignment of the units");

// What of a group's prefix its requests can share: whole pages that every query of theirs sees and the tables have. Of
// requests without queries nothing is asked; a prefix that only one request reads is left to that. Groups that do not cover
// the requests in order share nothing, nor do requests whose query rows do not follow each other (a group's rows would not be
// theirs), nor does a call in which that would save less than p.least_tiles tiles.
// A thread to a request, and to a group; everything that is read is on its way at once.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) kv_shared_kernel(const moe_kv_batch_t b, const moe_kv_prefixes_t p, const SharedWork w, Scratch s) {
  __shared__ int s_least[kThreads], s_row[kThreads], s_count[kThreads], s_start[kThreads + 1], s_first[kThreads + 1], s_warp[kThreads / 32];
  __shared__ unsigned long long s_saved;
  const int tid = threadIdx.x;
  grid_launch_dependents();  // (the next launch waits for this one's end before it reads what is written here)
  const auto token = [&](int at) { return min(max(at, 0), b.tokens); };
  int from = 0, to = 0, behind = 0, start = 0, prefix = 0;  // a request's query rows, its tokens; a group's
  if (tid < b.requests) {
    from = b.query_start[tid];
    to = b.query_start[tid + 1];
    behind = max(b.seq_lens[tid], 0);
  }
  if (tid < p.groups) {
    start = p.group_start[tid];
    prefix = p.prefix_lens[tid];
  }
  if (tid == 0) s_start[p.groups] = p.group_start[p.groups];
  for (int i = tid; i < 3 * kAttendMaxCtas; i += kThreads) s.counters[i] = 0;
  if (tid == 0) s_saved = 0;
  s_least[tid] = s_row[tid] = 0x7FFFFFFF;
  s_count[tid] = 0;
  if (tid < p.groups) s_start[tid] = start;
  if (tid < b.requests) s_first[tid] = token(from);
  if (tid == b.requests - 1) s_first[b.requests] = token(to);
  __syncthreads();
  bool fine = from <= to;
  if (tid < p.groups) fine = fine && start <= s_start[tid + 1];
  fine = __syncthreads_and(fine) && s_start[0] == 0 && s_start[p.groups] == b.requests;
  int group = 0;
  if (tid < b.requests && fine) {
    int hi = p.groups;  // s_start[group] <= tid < s_start[hi]
    while (hi - group > 1) {
      const int mid = (group + hi) >> 1;
      if (s_start[mid] <= tid) group = mid;
      else hi = mid;
    }
    const int n = token(to) - token(from);
    if (n > 0) {
      atomicMin(s_least + group, behind - n);
      atomicMin(s_row + group, tid);
      atomicAdd(s_count + group, 1);
    }
  }
  __syncthreads();
  int tokens = 0, blocks = 0;
  if (tid < p.groups && fine && s_count[tid] > 1) {
    const long long room = static_cast<long long>(b.table_width) << w.shift;
    tokens = static_cast<int>(min(static_cast<long long>(min(prefix, s_least[tid])), room));
    tokens = max(tokens, 0) >> w.shift << w.shift;
    if (tokens) {
      const long long rows = static_cast<long long>(s_first[s_start[tid + 1]] - s_first[start]) * w.group;  // of the group
      const long long own = static_cast<long long>(s_count[tid]) * w.own, less = own - (rows + w.rows - 1) / w.rows * w.cost;
      const long long saved = less * w.kv_heads * attend_tiles(tokens) / 10;
      if (p.least_tiles > 1 && kLeastShare * less < own) {
        tokens = 0;
      } else {
        atomicAdd(&s_saved, static_cast<unsigned long long>(max(saved, 1ll)));
        blocks = static_cast<int>((rows + 7) / 8);
      }
    }
  }
  __syncthreads();
  if (s_saved < static_cast<unsigned long long>(p.least_tiles)) tokens = blocks = 0;
  // The blocks of 8 rows of the groups before this one, of those that share.
  int sum = blocks;
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += u;
  }
  if (lane == 31) s_warp[warp] = sum;
  const int row = s_row[tid];
  s_least[tid] = tokens >> w.shift;
  __syncthreads();
  if (tid < b.requests) s.skipped[tid] = s_least[group];  // (0 everywhere where nothing is fine)
  for (int k = 0; k < warp; ++k) sum += s_warp[k];
  if (tid < p.groups) {
    s.start[tid] = s_first[fine ? start : 0];  // (the merging launch takes it as it is)
    s.prefix[tid] = tokens;
    s.row[tid] = tokens ? row : 0;
    s.block[tid] = sum - blocks;
  }
  if (tid == p.groups - 1) {
    s.block[p.groups] = sum;
    s.start[p.groups] = s_first[fine ? b.requests : 0];
  }
}

}  // namespace

cudaError_t launch_kv_attend(const AttendArgs& a, cudaStream_t stream) {
  Call c;
  const cudaError_t e = c.open(a.c);
  if (e != cudaSuccess) return e;
  return launch_whole(a, c, row_tile(a), stream);
}

cudaError_t launch_kv_attend_shared(const AttendArgs& whole, const moe_kv_prefixes_t& p, void* scratch, cudaStream_t stream) {
  Call c;
  cudaError_t e = c.open(whole.c);
  if (e != cudaSuccess) return e;
  const Scratch s(scratch, whole);
  AttendArgs a = whole, b = whole;  // the requests' own part, their prefixes'
  a.counters = s.counters;
  a.skipped = s.skipped;
  a.shared = b.shared = s.block + p.groups;
  a.partial = b.partial = s.out;
  a.partial_lse = b.partial_lse = s.lse;
  b.rows = s.row;
  b.group_unit = s.unit;
  b.group_token = s.start;
  b.group_prefix = s.prefix;
  b.group_block = s.block;
  b.b.query_start = s.start;
  b.b.seq_lens = s.prefix;
  b.b.requests = p.groups;
  const int own_tile = row_tile(whole), tile = row_tile(b), own_rows = own_tile ? 8 * own_tile : 128;
  const long long rows = static_cast<long long>(whole.b.tokens) * whole.group, average = (rows + whole.b.requests - 1) / whole.b.requests;
  const SharedWork work = {c.shift, a.group, a.c.kv_heads, static_cast<int>((average + own_rows - 1) / own_rows) * kTileCost[own_tile],
                           tile ? 8 * tile : 128, kTileCost[tile]};
  moe_kv_prefixes_t prefixes = p;
  if (p.least_tiles == 0) prefixes.least_tiles = least_tiles(whole.c.head_dim);
  // What the call can save at most, were its whole table one prefix: less than that, and no plan is asked (4 requests on a
  // prefix of 481 tokens: 10.6 us, some 5 more with it).
  const long long table_tiles = ((static_cast<long long>(whole.b.table_width) << c.shift) + 127) / 128;
  if (static_cast<double>(whole.b.requests) * work.own * work.kv_heads * static_cast<double>(table_tiles) / 10 < prefixes.least_tiles)
    return launch_whole(whole, c, own_tile, stream);
  // (A small batch's few warps are through their barriers sooner.)
  if (whole.b.requests <= 128) kv_shared_kernel<128><<<1, 128, 0, stream>>>(whole.b, prefixes, work, s);
  else kv_shared_kernel<1024><<<1, 1024, 0, stream>>>(whole.b, prefixes, work, s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // The prefixes' part works while the other's last CTAs run, if there is room for the pieces of both (not for twice the form
  // of 128 rows, whose work is long).
  const auto piece_bytes = [&](int t) {
    return 8ull * (t ? 8 * t * kv_attend_decode_ctas(a.c.head_dim, t, c.sms) : 128 * kv_attend_rows_ctas(c.sms)) * (a.c.head_dim + 2);
  };
  const size_t theirs = (piece_bytes(tile) + 255) / 256 * 256, room = MOE_KV_WORKSPACE_BYTES - MOE_KV_WORKSPACE_HEADER;
  b.early = theirs + piece_bytes(own_tile) <= room;
  a.pieces = reinterpret_cast<float*>(a.workspace + MOE_KV_WORKSPACE_HEADER + (b.early ? theirs : 0));
  e = own_tile ? launch_kv_attend_decode_suffix(a, c.maps, own_tile, c.shift, c.sms, stream)
               : launch_kv_attend_rows_suffix(a, c.maps, c.shift, c.sms, stream);
  if (e != cudaSuccess) return e;
  e = tile ? launch_kv_attend_decode_prefix(b, c.maps, tile, c.shift, c.sms, stream)
           : launch_kv_attend_rows_prefix(b, c.maps, c.shift, c.sms, stream);
  if (e != cudaSuccess) return e;
  return launch_kv_attend_merge(b, tile ? 8 * tile : 128, tile ? kv_attend_decode_ctas(a.c.head_dim, tile, c.sms) : kv_attend_rows_ctas(c.sms), stream);
}

}  // namespace moe
