// Pages that several requests hold: rows that go on from others, the free list,
// pages moved (moe_kv_fork, moe_kv_reclaim, moe_kv_copy in include/moe.h).
//
// Fork: who takes a page is a prefix sum over the requests, which every CTA
// takes for itself; the rows are copied a warp to a row. Reclaim: the pages that
// some row holds are bits of a map; a page's place among the free ones is a
// count of the bits before it (one CTA with the map in its shared memory, without
// launches in between, is 2 us quicker up to some 2000 entries, and three times
// slower at 16 thousand: not kept). Copy: bytes.
//
// Latency bounds the tables: a fork of 1000 requests with its copies takes 7.7 us, a
// free list from 1000 requests 6.4 us, against 2.5 for any launch. The bytes bound a
// pool's compaction: 64 requests, 198 MB moved, 41 us in all, 34 of them the copy's.
#include "decode.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
static_assert(MOE_KV_MAX_REQUESTS <= 1024, "a CTA has a thread for every request");

__device__ __forceinline__ int pages_for(int tokens, int shift) {  // (any length up to 2^31 - 1)
  return static_cast<int>((static_cast<uint32_t>(tokens) + (1u << shift) - 1) >> shift);
}

// ------------------------------------------------------------------------ fork
template <int kForkThreads>
__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(const moe_kv_fork_t a, int shift) {
  constexpr int kWarps = kForkThreads / 32;
  __shared__ int s_first[MOE_KV_MAX_REQUESTS];  // [row] the first request that goes on from it
  __shared__ int s_parent[kForkThreads], s_len[kForkThreads], s_last[kForkThreads];  // [request]; s_last: its last page, where taken
  __shared__ int s_warp[kWarps], s_longest[kWarps], s_moved[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << shift;
  for (int i = tid; i < a.rows; i += kForkThreads) s_first[i] = 0x7FFFFFFF;
  __syncthreads();
  int p = -1, len = 0, flags = 0;
  if (tid < a.requests) {
    p = a.parents[tid];
    if (p < -1 || p >= a.rows) {
      flags |= 1;
      p = -1;
    }
    if (p >= 0) {
      atomicMin(s_first + p, tid);
      len = a.seq_lens[p];
      if (len < 0) {
        flags |= 1;
        len = 0;
      }
    }
  }
  const long long head = *a.free_head;
  const int needed = pages_for(len, shift);
  if (needed > a.table_width) flags |= 4;
  int entry = -1;
  if (len & (P - 1) && needed <= a.table_width) entry = a.block_table[p * a.table_stride + needed - 1];
  __syncthreads();
  const bool wants = entry >= 0 && s_first[p] != tid;
  const uint32_t votes = __ballot_sync(kAll, wants);
  if (lane == 0) s_warp[warp] = __popc(votes);
  __syncthreads();
  int total = lane < kWarps ? s_warp[lane] : 0, before = lane < warp ? total : 0;
  total = __reduce_add_sync(kAll, total);
  before = __reduce_add_sync(kAll, before) + __popc(votes & ((1u << lane) - 1));
  int page = -1;
  if (wants) {
    const long long at = head + before;
    if (at >= 0 && at < a.free_count) page = a.free_pages[at];
  }
  if (tid < a.requests) {
    s_parent[tid] = p;
    s_len[tid] = len;
    s_last[tid] = wants ? page : -2;
  }
  const bool moved = wants && page >= 0;
  if (blockIdx.x == 0) {
    if (tid < a.requests) {
      a.out_lens[tid] = len;
      a.moves[3 * tid] = moved ? entry : -1;
      a.moves[3 * tid + 1] = moved ? page : -1;
      a.moves[3 * tid + 2] = moved ? len & (P - 1) : 0;
    }
    if (total && (head < 0 || head + total > a.free_count)) flags |= 8;
    flags = __reduce_or_sync(kAll, flags);
    const int longest = __reduce_max_sync(kAll, len), count = __popc(__ballot_sync(kAll, moved));
    if (lane == 0) {
      s_longest[warp] = longest;
      s_moved[warp] = count | flags << 16;
    }
    __syncthreads();
    if (warp == 0) {
      const int w = lane < kWarps ? s_moved[lane] : 0;
      const int all = __reduce_add_sync(kAll, w & 0xFFFF), bits = __reduce_or_sync(kAll, w >> 16);
      const int most = __reduce_max_sync(kAll, lane < kWarps ? s_longest[lane] : 0);
      if (lane == 0) {
        a.counts[0] = all;
        a.counts[1] = static_cast<int>(min(head + total, 0x7FFFFFFFll));
        a.counts[2] = most;
        a.counts[3] = bits;
      }
    }
  }
  __syncthreads();

  // The rows, a warp to 128 entries of one.
  const int parts = (a.table_width + 127) / 128;
  const long long units = static_cast<long long>(a.requests) * parts;
  for (long long u = static_cast<long long>(blockIdx.x) * kWarps + warp; u < units; u += static_cast<long long>(gridDim.x) * kWarps) {
    const int r = static_cast<int>(u / parts), j0 = static_cast<int>(u - static_cast<long long>(r) * parts) * 128 + lane;
    const int from = s_parent[r], n = pages_for(s_len[r], shift), last = s_last[r];
    const int32_t* src = a.block_table + from * a.table_stride;
    int32_t* dst = a.out_table + r * a.out_stride;
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + 32 * i;
      v[i] = j < a.table_width && j < n ? src[j] : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + 32 * i;
      if (j < a.table_width) dst[j] = j == n - 1 && last != -2 ? last : v[i];
    }
  }
}

// --------------------------------------------------------------------- reclaim
// Workspace: counts of the marking (error bits), then the map, a bit to a page, then (compaction) the place of each page that
// leaves among those.
struct Map {
  uint32_t* errors;
  uint32_t* bits;
  int32_t* leaver;
  int words;
  __host__ __device__ explicit Map(const moe_kv_reclaim_t& a)
      : errors(static_cast<uint32_t*>(a.workspace)), bits(errors + 128), words((a.pages + 31) / 32) {
    leaver = reinterpret_cast<int32_t*>(bits + (words + 3) / 4 * 4);
  }
};

constexpr int kReclaimThreads = 256;

// The launches of a call are chained: each starts while the one before it runs, and waits for its end where it needs it (what
// that one wrote it reads from the second level).
__global__ void __launch_bounds__(kReclaimThreads) kv_clear_kernel(const moe_kv_reclaim_t a) {
  const Map m(a);
  ptx::grid_launch_dependents();
  for (int i = blockIdx.x * kReclaimThreads + threadIdx.x; i < (m.words + 3) / 4; i += gridDim.x * kReclaimThreads)
    reinterpret_cast<uint4*>(m.bits)[i] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x == 0 && threadIdx.x == 0) *m.errors = 0;
}

// The entries that a row's length covers.
__device__ __forceinline__ int held_entries(const moe_kv_reclaim_t& a, int r, int shift, uint32_t& errors) {
  const int len = a.seq_lens[r];
  if (len < 0) errors |= 1;
  const int n = pages_for(max(len, 0), shift);
  if (n > a.table_width) errors |= 4;
  return min(n, a.table_width);
}

__global__ void __launch_bounds__(kReclaimThreads) kv_mark_kernel(const moe_kv_reclaim_t a, int shift) {
  const Map m(a);
  uint32_t errors = 0;
  const int r = blockIdx.y, n = held_entries(a, r, shift, errors);
  const int32_t* row = a.block_table + r * a.table_stride;
  const int stride = gridDim.x * kReclaimThreads;
  int j = blockIdx.x * kReclaimThreads + threadIdx.x, page = j < n ? row[j] : -1;
  ptx::grid_dependency_wait();  // the map is clear
  ptx::grid_launch_dependents();
  while (j < n) {
    if (page < 0 || page >= a.pages) errors |= 2;
    else atomicOr(m.bits + (page >> 5), 1u << (page & 31));
    j += stride;
    if (j < n) page = row[j];
  }
  errors = __reduce_or_sync(kAll, errors);
  if (errors && (threadIdx.x & 31) == 0) atomicOr(m.errors, errors);
}

// The sum of x over the CTA, everywhere.
__device__ __forceinline__ long long block_sum(int x, int* s_part) {
  x = __reduce_add_sync(kAll, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = x;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kReclaimThreads / 32; ++w) sum += s_part[w];
  return sum;
}

// Where the k-th move is listed: below the room that moves have, whatever another call with the same workspace makes of the
// map meanwhile (its counts are wrong then, but nothing is written or read outside).
__device__ __forceinline__ int32_t* move_at(const moe_kv_reclaim_t& a, int k) {
  return a.moves + 3ll * min(static_cast<uint32_t>(k), static_cast<uint32_t>(max(a.pages / 2, 1) - 1));
}

// Each CTA lists the pages of a run of words: free ones, or what leaves and where it goes.
template <bool kCompact>
__global__ void __launch_bounds__(kReclaimThreads) kv_list_kernel(const moe_kv_reclaim_t a, int shift, int words_per) {
  __shared__ int s_part[kReclaimThreads / 32], s_scan[kReclaimThreads / 32], s_first[kReclaimThreads];
  __shared__ uint32_t s_word[kReclaimThreads];
  const Map m(a);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int begin = blockIdx.x * words_per, end = min(begin + words_per, m.words);  // (begin is a multiple of 4)
  ptx::grid_dependency_wait();  // the marks are made
  ptx::grid_launch_dependents();
  int held = 0, before = 0;
  const uint4* quads = reinterpret_cast<const uint4*>(m.bits);
#pragma unroll 4
  for (int i = tid; i < (m.words + 3) / 4; i += kReclaimThreads) {
    const uint4 w = __ldcg(quads + i);  // (what is past the last word is clear)
    const int c = __popc(w.x) + __popc(w.y) + __popc(w.z) + __popc(w.w);
    held += c;
    before += 4 * i < begin ? c : 0;
  }
  const int n = static_cast<int>(block_sum(held, s_part));
  int at = static_cast<int>(block_sum(before, s_part));  // pages held before the CTA's first word
  int kept = 0;                                          // held pages before page n, which stay
  if (kCompact) {
    for (int i = tid; i <= n >> 5 && i < m.words; i += kReclaimThreads)
      kept += __popc(i < n >> 5 ? __ldcg(m.bits + i) : __ldcg(m.bits + i) & ((1u << (n & 31)) - 1));
    kept = static_cast<int>(block_sum(kept, s_part));
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.counts[0] = a.counts[1] = n;
    a.counts[2] = kCompact ? n - kept : 0;
    a.counts[3] = static_cast<int>(__ldcg(m.errors));
  }
  // Words, a lane to a page.
  for (int base = begin; base < end; base += kReclaimThreads) {
    const uint32_t word = base + tid < end ? __ldcg(m.bits + base + tid) : 0;
    const int own = __popc(word);
    int in = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kAll, in, d);
      if (lane >= d) in += u;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = in;
    __syncthreads();
    int first = at, total = 0;
#pragma unroll
    for (int w = 0; w < kReclaimThreads / 32; ++w) {
      first += w < warp ? s_scan[w] : 0;
      total += s_scan[w];
    }
    first += in - own;  // held before this thread's word
    at += total;
    s_word[tid] = word;
    s_first[tid] = first;
    __syncthreads();
    for (int k = warp; k < kReclaimThreads && base + k < end; k += kReclaimThreads / 32) {
      const uint32_t bits = s_word[k];
      const int page = (base + k) * 32 + lane, rank = s_first[k] + __popc(bits & ((1u << lane) - 1));  // held before it
      const bool mine = bits >> lane & 1;
      if (page >= a.pages) continue;
      if (!kCompact) {
        if (!mine) a.free_pages[min(static_cast<uint32_t>(n + (page - rank)), static_cast<uint32_t>(a.pages - 1))] = page;
      } else {
        if (page >= n) {
          a.free_pages[page] = page;
          if (mine) {
            m.leaver[page] = rank - kept;
            move_at(a, rank - kept)[0] = page;
          }
        } else if (!mine) {
          int32_t* move = move_at(a, page - rank);
          move[1] = page;
          move[2] = 1 << shift;
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kReclaimThreads) kv_rename_kernel(const moe_kv_reclaim_t a, int shift) {
  const Map m(a);
  uint32_t errors = 0;
  const int r = blockIdx.y, used = held_entries(a, r, shift, errors);
  ptx::grid_dependency_wait();  // the moves are listed
  const int n = __ldcg(a.counts);
  const int32_t* row = a.block_table + r * a.table_stride;
  int32_t* out = a.out_table + r * a.out_stride;
  for (int j = blockIdx.x * kReclaimThreads + threadIdx.x; j < a.table_width; j += gridDim.x * kReclaimThreads) {
    int page = j < used ? row[j] : -1;
    if (page >= a.pages) page = -1;
    if (page >= n) page = __ldcg(move_at(a, __ldcg(m.leaver + page)) + 1);
    out[j] = max(page, -1);
  }
}

// ------------------------------------------------------------------------ copy
constexpr int kCopyThreads = 128;

// A unit is a move's keys or values of some heads, of a few thousand bytes; a CTA takes units in turn, eight words of a thread
// on their way together.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const moe_kv_cache_t c, const int32_t* moves, const int32_t* count, int capacity, int heads_per) {
  ptx::grid_dependency_wait();
  const int n = count ? min(max(__ldcg(count), 0), capacity) : capacity;
  const int head_words = c.page_tokens * c.head_dim / 16, parts = (c.kv_heads + heads_per - 1) / heads_per;
  const long long page_words = static_cast<long long>(c.kv_heads) * head_words;
  for (long long u = blockIdx.x; u < 2ll * n * parts; u += gridDim.x) {
    const long long which = u / parts;
    const int h0 = static_cast<int>(u - which * parts) * heads_per, heads = min(heads_per, c.kv_heads - h0);
    const int32_t* move = moves + 3 * (which >> 1);
    const int from = __ldcg(move), to = __ldcg(move + 1), tokens = min(__ldcg(move + 2), c.page_tokens);
    if (from < 0 || to < 0 || from >= c.pages || to >= c.pages || from == to || tokens <= 0) continue;
    uint8_t* scales = which & 1 ? c.v_scale : c.k_scale;
    uint4* data = reinterpret_cast<uint4*>(which & 1 ? c.v : c.k) + h0 * head_words;
    const uint4* src = data + from * page_words;
    uint4* dst = data + to * page_words;
    const int words = tokens * c.head_dim / 16, all = words * heads;
    for (int base = threadIdx.x; base < all; base += 8 * kCopyThreads) {
      uint4 v[8];
      int at[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = base + e * kCopyThreads, h = i / words;
        at[e] = h * head_words + i - h * words;
        if (i < all) v[e] = src[at[e]];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (base + e * kCopyThreads < all) dst[at[e]] = v[e];
    }
    if (threadIdx.x < heads)
      scales[static_cast<long long>(to) * c.kv_heads + h0 + threadIdx.x] = scales[static_cast<long long>(from) * c.kv_heads + h0 + threadIdx.x];
  }
}

int shift_of(int page_tokens) {
  int shift = 4;
  while ((1 << shift) < page_tokens) ++shift;
  return shift;
}

}  // namespace

cudaError_t launch_kv_fork(const moe_kv_fork_t& a, cudaStream_t stream) {
  const int threads = a.requests <= 256 ? 256 : 1024;
  const long long warps = static_cast<long long>(a.requests) * ((a.table_width + 127) / 128);
  const long long ctas = (warps + threads / 32 - 1) / (threads / 32);
  const int grid = static_cast<int>(ctas < 152 ? ctas : 152);
  if (threads == 256) kv_fork_kernel<256><<<grid, 256, 0, stream>>>(a, shift_of(a.page_tokens));
  else kv_fork_kernel<1024><<<grid, 1024, 0, stream>>>(a, shift_of(a.page_tokens));
  return cudaGetLastError();
}

cudaError_t launch_kv_copy(const moe_kv_cache_t& c, const int32_t* moves, const int32_t* count, int capacity, cudaStream_t stream) {
  // Heads of about 16 KB to a unit, of a page of 64 tokens two heads of 128 (a fork with 56 moves of up to 64 tokens of 8 heads
  // takes 6.2 us so, 6.6 with a page's keys to a unit, 7.1 with a head; one of 1000 requests with few moves 7.9, 7.9 and 12.1;
  // a compaction 41, 42 and 50). The most CTAs, from 12 to 64 an SM, make no difference.
  int heads_per = 16384 / (c.page_tokens * c.head_dim);
  heads_per = heads_per < 1 ? 1 : heads_per > c.kv_heads ? c.kv_heads : heads_per;
  const long long units = 2ll * capacity * ((c.kv_heads + heads_per - 1) / heads_per);
  return launch_chained(kv_copy_kernel, static_cast<int>(units < 152 * 16 ? units : 152 * 16), kCopyThreads, 0, true, stream, c, moves, count, capacity, heads_per);
}

cudaError_t launch_kv_reclaim(const moe_kv_reclaim_t& a, cudaStream_t stream) {
  const int shift = shift_of(a.page_tokens), words = (a.pages + 31) / 32;
  const auto least = [](int x, int y) { return x < y ? x : y; };
  kv_clear_kernel<<<least((words + 4 * kReclaimThreads - 1) / (4 * kReclaimThreads), 152), kReclaimThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  const dim3 rows(least((a.table_width + kReclaimThreads - 1) / kReclaimThreads, 8), a.requests);
  if (e == cudaSuccess) e = launch_chained(kv_mark_kernel, rows, kReclaimThreads, 0, true, stream, a, shift);
  const int ctas = least((words + 7) / 8, 152), words_per = ((words + ctas - 1) / ctas + 3) / 4 * 4, grid = (words + words_per - 1) / words_per;
  const bool compact = a.out_table != nullptr;
  if (e == cudaSuccess) e = launch_chained(compact ? kv_list_kernel<true> : kv_list_kernel<false>, grid, kReclaimThreads, 0, true, stream, a, shift, words_per);
  if (e == cudaSuccess && compact) e = launch_chained(kv_rename_kernel, rows, kReclaimThreads, 0, true, stream, a, shift);
  return e;
}

}  // namespace moe
