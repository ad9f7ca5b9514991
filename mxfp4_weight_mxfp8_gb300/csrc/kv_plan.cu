// Block tables and slots of a step's new tokens (moe_kv_plan in include/moe.h).
//
// Two prefix sums over the requests (new tokens, new pages) and then one
// independent item per new token: its request by binary search, its page from
// the table or, past the pages held, from the free list at the request's place
// in it. A page is entered in the table by the token that starts it (a page
// taken by this call always starts with a new token), so nothing waits for
// anything but the sums, which every CTA takes for itself.
#include "kernels.h"

namespace moe {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanPerThread = MOE_KV_MAX_REQUESTS / kPlanThreads;

struct PlanSums {
  long long tokens, pages;
};

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const moe_kv_plan_t a, int shift) {
  __shared__ long long s_start[MOE_KV_MAX_REQUESTS + 1];  // new tokens before request r
  __shared__ long long s_pages[MOE_KV_MAX_REQUESTS];      // new pages before request r
  __shared__ int s_context[MOE_KV_MAX_REQUESTS];
  __shared__ long long s_warp[2][kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = a.page_tokens;

  long long tok[kPlanPerThread], pag[kPlanPerThread], tsum = 0, psum = 0;
  int flags = 0, longest = 0;
#pragma unroll
  for (int i = 0; i < kPlanPerThread; ++i) {
    const int r = tid * kPlanPerThread + i;
    int c = 0, q = 0;
    if (r < a.requests) {
      c = a.context_lens[r];
      q = a.query_lens[r];
      if (c < 0 || q < 0 || static_cast<long long>(c) + q > 0x7FFFFFFF - P) {
        flags |= 1;
        c = q = 0;
      }
      s_context[r] = c;
      longest = max(longest, c + q);
      if (((c + q + P - 1) >> shift) > a.table_width) flags |= 4;
      if (blockIdx.x == 0) a.seq_lens[r] = c + q;
    }
    tok[i] = tsum;
    pag[i] = psum;
    tsum += q;
    psum += ((c + q + P - 1) >> shift) - ((c + P - 1) >> shift);
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
  long long tbase = tin - tsum, pbase = pin - psum, total = 0, pages = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      tbase += s_warp[0][w];
      pbase += s_warp[1][w];
    }
    total += s_warp[0][w];
    pages += s_warp[1][w];
  }
#pragma unroll
  for (int i = 0; i < kPlanPerThread; ++i) {
    const int r = tid * kPlanPerThread + i;
    if (r < a.requests) {
      s_start[r] = tbase + tok[i];
      s_pages[r] = pbase + pag[i];
      if (blockIdx.x == 0)
        a.query_start[r] = static_cast<int>(min(tbase + tok[i], 0x7FFFFFFFll));
    }
  }
  if (tid == 0) s_start[a.requests] = total;
  const long long head = *a.free_head;
  if (blockIdx.x == 0) {
    if (total > a.tokens) flags |= 2;
    if (head < 0 || head + pages > a.free_count) flags |= pages ? 8 : 0;
    flags = __syncthreads_or(flags & 1) | __syncthreads_or(flags & 2) * 2 |
            __syncthreads_or(flags & 4) * 4 | __syncthreads_or(flags & 8) * 8;
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    __shared__ int s_longest[kPlanThreads / 32];
    if (lane == 0) s_longest[warp] = longest;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kPlanThreads / 32; ++w) longest = max(longest, s_longest[w]);
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
  int grid = (a.tokens + kPlanThreads * 4 - 1) / (kPlanThreads * 4);
  grid = grid < 1 ? 1 : (grid > 152 ? 152 : grid);
  kv_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(a, shift);
  return cudaGetLastError();
}

}  // namespace moe
