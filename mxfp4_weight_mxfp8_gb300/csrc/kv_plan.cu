// Block tables and slots of a step's new tokens (moe_kv_plan in include/moe.h).
//
// Two prefix sums over the requests (new tokens, new pages) and then one
// independent item per new token: its request by binary search, its page from
// the table or, past the pages held, from the free list at the request's place
// in it. A page is entered in the table by the token that starts it (a page
// taken by this call always starts with a new token), so nothing waits for
// anything but the sums, which every CTA takes for itself.
//
// Latency bounds it: 64 requests with a token each take 2.7 us, about a launch;
// 1000 requests with 300 thousand new tokens take 5.9 us, where the 3.4 MB
// alone would take 0.5 and the sums (four dependent loads and two scans) 3.
#include "decode.h"

namespace moe {
namespace {

// A thread to a request: kPlanThreads at least as many as the requests.
static_assert(MOE_KV_MAX_REQUESTS <= 1024, "a CTA has a thread for every request");

// A request's cached and new tokens; both 0 where they are no lengths.
__device__ __forceinline__ bool lengths(const moe_kv_plan_t& a, int r, int& c, int& q) {
  c = a.context_lens[r];
  q = a.query_lens[r];
  const bool ok = c >= 0 && q >= 0 && static_cast<long long>(c) + q <= 0x7FFFFFFF - a.page_tokens;
  if (!ok) c = q = 0;
  return ok;
}

// seq_lens over context_lens: every CTA of the plan has read those by now.
__global__ void __launch_bounds__(1024) kv_lengths_kernel(const moe_kv_plan_t a) {
  int c, q;
  if (threadIdx.x >= a.requests) return;
  lengths(a, threadIdx.x, c, q);
  a.seq_lens[threadIdx.x] = c + q;
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const moe_kv_plan_t a, int shift, bool store_lengths) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ long long s_start[kPlanThreads + 1];  // new tokens before request r
  __shared__ long long s_pages[kPlanThreads];      // new pages before request r
  __shared__ int s_context[kPlanThreads];
  __shared__ long long s_warp[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = a.page_tokens;

  long long tsum = 0, psum = 0;  // of request tid
  int flags = 0, longest = 0;
  const long long head = *a.free_head;
  if (tid < a.requests) {
    int c, q;
    if (!lengths(a, tid, c, q)) flags |= 1;
    s_context[tid] = c;
    longest = c + q;
    const int held = (c + P - 1) >> shift, needed = (c + q + P - 1) >> shift;
    if (needed > a.table_width) flags |= 4;
    if (store_lengths && blockIdx.x == 0) a.seq_lens[tid] = c + q;
    tsum = q;
    psum = needed - held;
  }
  long long tin = tsum, pin = psum;  // inclusive sums over the warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, tin, d), v = __shfl_up_sync(0xFFFFFFFFu, pin, d);
    if (lane >= d) {
      tin += u;
      pin += v;
    }
  }
  if (lane == 31) {
    s_warp[0][warp] = tin;
    s_warp[1][warp] = pin;
  }
  __syncthreads();
  // Every warp sums the warps' totals for itself: lane w, warp w's.
  long long tw = lane < kWarps ? s_warp[0][lane] : 0, pw = lane < kWarps ? s_warp[1][lane] : 0;
  long long tbase = lane < warp ? tw : 0, pbase = lane < warp ? pw : 0;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    tw += __shfl_xor_sync(0xFFFFFFFFu, tw, d);
    pw += __shfl_xor_sync(0xFFFFFFFFu, pw, d);
    tbase += __shfl_xor_sync(0xFFFFFFFFu, tbase, d);
    pbase += __shfl_xor_sync(0xFFFFFFFFu, pbase, d);
  }
  const long long total = tw, pages = pw;
  if (tid < a.requests) {
    s_start[tid] = tbase + tin - tsum;
    s_pages[tid] = pbase + pin - psum;
    if (blockIdx.x == 0) a.query_start[tid] = static_cast<int>(min(s_start[tid], 0x7FFFFFFFll));
  }
  if (tid == 0) s_start[a.requests] = total;
  if (blockIdx.x == 0) {
    if (total > a.tokens) flags |= 2;
    if (head < 0 || head + pages > a.free_count) flags |= pages ? 8 : 0;
    flags = (__syncthreads_or(flags & 1) ? 1 : 0) | (__syncthreads_or(flags & 2) ? 2 : 0) |
            (__syncthreads_or(flags & 4) ? 4 : 0) | (__syncthreads_or(flags & 8) ? 8 : 0);
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    __shared__ int s_longest[kWarps];
    if (lane == 0) s_longest[warp] = longest;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) longest = max(longest, s_longest[w]);
      a.query_start[a.requests] = static_cast<int>(min(total, 0x7FFFFFFFll));
      a.counts[0] = static_cast<int>(min(total, 0x7FFFFFFFll));
      a.counts[1] = static_cast<int>(min(head + pages, 0x7FFFFFFFll));
      a.counts[2] = longest;
      a.counts[3] = flags;
    }
  }
  __syncthreads();

  for (long long t = blockIdx.x * kPlanThreads + tid; t < a.tokens;
       t += static_cast<long long>(gridDim.x) * kPlanThreads) {
    if (t >= total) {
      a.positions[t] = 0;
      a.slots[t] = -1;
      continue;
    }
    int lo = 0, hi = a.requests;  // s_start[lo] <= t < s_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int c = s_context[lo], pos = c + static_cast<int>(t - s_start[lo]);
    const int j = pos >> shift, held = (c + P - 1) >> shift;
    int32_t* row = a.block_table + lo * a.table_stride;
    int page = -1;
    if (j < held) {
      if (j < a.table_width) page = row[j];
    } else {
      const long long at = head + s_pages[lo] + (j - held);
      if (j < a.table_width) {
        if (at >= 0 && at < a.free_count) page = a.free_pages[at];
        if ((pos & (P - 1)) == 0) row[j] = page;
      }
    }
    a.positions[t] = pos;
    a.slots[t] = page >= 0 ? (static_cast<int64_t>(page) << shift) + (pos & (P - 1)) : -1;
  }
}

}  // namespace

cudaError_t launch_kv_plan(const moe_kv_plan_t& a, cudaStream_t stream) {
  int shift = 4;
  while ((1 << shift) < a.page_tokens) ++shift;
  // A thread to a request: 256 threads while that is enough (64 requests: 2.7 us, against 3.6 with 1024). Every CTA
  // takes the sums again, so one to an SM (1000 requests, 300 thousand tokens: 5.9 us; 6.5 with 100 CTAs, 7.0 with 304).
  const int threads = a.requests <= 256 ? 256 : 1024;
  int grid = (a.tokens + threads - 1) / threads;
  grid = grid < 1 ? 1 : (grid > 152 ? 152 : grid);
  // Lengths stepped in place are written by a launch of their own, unless one CTA does all (each thread its own request's).
  const bool later = a.seq_lens == a.context_lens && grid > 1;
  if (threads == 256) kv_plan_kernel<256><<<grid, 256, 0, stream>>>(a, shift, !later);
  else kv_plan_kernel<1024><<<grid, 1024, 0, stream>>>(a, shift, !later);
  if (later) kv_lengths_kernel<<<1, 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
