// Causal attention of new tokens over the paged 8-bit cache (moe_kv_attend in
// include/moe.h).
//
// One CTA per (token, query head): its warps take the visible keys in turn,
// each with a running maximum, sum and output row, joined in shared memory.
#include <cuda_fp16.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kAttendWarps = 4;
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float2 decode2(uint32_t codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
}

template <int D>
__global__ void __launch_bounds__(32 * kAttendWarps) kv_attend_kernel(const AttendArgs a, int shift) {
  constexpr int kPer = D / 32;  // values of a row in a lane: consecutive
  __shared__ float s_m[kAttendWarps], s_l[kAttendWarps], s_o[kAttendWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, h = blockIdx.y;
  if (t >= a.b.query_start[a.b.requests]) return;
  int lo = 0, hi = a.b.requests;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.b.query_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t room = static_cast<int64_t>(a.b.table_width) << shift;
  const int seq = a.b.seq_lens[lo];
  const int pos = seq - (a.b.query_start[lo + 1] - t);
  const int from = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int kvh = h / a.group;
  float q[kPer], o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.q_token_stride + h * a.q_head_stride + lane * kPer + i]) << 16);
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = from + warp; j <= pos && j < room; j += kAttendWarps) {
    const int page = a.b.block_table[lo * a.b.table_stride + (j >> shift)];
    if (page < 0 || page >= a.c.pages) continue;
    const int64_t ph = static_cast<int64_t>(page) * a.c.kv_heads + kvh;
    const int64_t at = ((ph << shift) + (j & (a.c.page_tokens - 1))) * D + lane * kPer;
    float dot = 0.0f, v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const float2 f = decode2(*reinterpret_cast<const uint16_t*>(a.c.k + at + i));
      dot += q[i] * f.x + q[i + 1] * f.y;
      const float2 g = decode2(*reinterpret_cast<const uint16_t*>(a.c.v + at + i));
      v[i] = g.x;
      v[i + 1] = g.y;
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) dot += __shfl_xor_sync(kAll, dot, d);
    const float s = dot * pow2f(a.c.k_scale[ph] - 127) * a.scale;
    const float sv = pow2f(a.c.v_scale[ph] - 127);
    const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + p * (v[i] * sv);
    m = mn;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_o[warp][lane * kPer + i] = o[i];
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, s_m[w]);
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
  for (int w = 0; w < kAttendWarps; ++w) {
    const float f = s_m[w] == -INFINITY ? 0.0f : expf(s_m[w] - top);
    sum += s_l[w] * f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] += s_o[w][lane * kPer + i] * f;
  }
  const int64_t row = static_cast<int64_t>(t) * a.q_heads + h;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    a.out[row * D + lane * kPer + i] = __bfloat16_as_ushort(__float2bfloat16(sum == 0.0f ? 0.0f : o[i] / sum));
  if (a.lse != nullptr && lane == 0) a.lse[row] = top + logf(sum);
}

}  // namespace

cudaError_t launch_kv_attend(const AttendArgs& a, cudaStream_t stream) {
  int shift = 4;
  while ((1 << shift) < a.c.page_tokens) ++shift;
  const dim3 grid(a.b.tokens, a.q_heads);
  if (a.c.head_dim == 64)
    kv_attend_kernel<64><<<grid, 32 * kAttendWarps, 0, stream>>>(a, shift);
  else if (a.c.head_dim == 128)
    kv_attend_kernel<128><<<grid, 32 * kAttendWarps, 0, stream>>>(a, shift);
  else
    kv_attend_kernel<256><<<grid, 32 * kAttendWarps, 0, stream>>>(a, shift);
  return cudaGetLastError();
}

}  // namespace moe
