// The pieces of attention over shared prefixes, joined with the requests' own parts
// (kv_attend.cuh: kPrefix, kSuffix).
//
// A CTA takes 8 rows of an item: they have the same pieces. The factors of all
// pieces' rows first, in shared memory, then a thread its four dimensions of one row
// over the pieces, eight loads in flight, a warp 8 rows by 4 quads: whole sectors in
// either layout of a piece. Everything lies in L2. The launch takes some 4 us of 512
// rows' 80 (64 requests on a prefix of 8192 tokens, 64 query heads on 8 of 128, 10 MB
// of pieces); four CTAs of 32 dimensions each in the place of one of 128 make it 2 to 4
// us more, even where there are few rows.
#include "decode.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D>
__global__ void __launch_bounds__(2 * D) kv_attend_merge_kernel(const AttendArgs a, int tile_rows, int grid) {
  constexpr int kWarps = D / 16;
  __shared__ float s_factor[kAttendRowsCtas][8], s_sum[kAttendRowsCtas][8], s_other[8], s_lse[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = a.b.requests, heads = a.c.kv_heads;
  // The plan is there since before the launch before this one started; that one's units and pieces when it has ended.
  const int work = __ldcg(a.shared) * heads;
  if (blockIdx.x == 0 && work == 0) ptx::grid_dependency_wait();
  for (int at = blockIdx.x; at < work; at += gridDim.x) {
    const int block = at / heads, head = at - block * heads;
    int g = 0;
    for (int hi = groups; hi - g > 1;) {  // group_block[g] <= block < group_block[hi]
      const int mid = (g + hi) >> 1;
      if (__ldcg(a.group_block + mid) <= block) g = mid;
      else hi = mid;
    }
    const int first = __ldcg(a.group_block + g), token0 = __ldcg(a.group_token + g), prefix = __ldcg(a.group_prefix + g);
    const int token1 = min(__ldcg(a.group_token + g + 1), a.b.tokens);
    const int row0 = (block - first) * 8, tile = row0 / tile_rows, i0 = row0 - tile * tile_rows;
    // This thread's row, its quad, and its place among the outputs' rows.
    const int i = lane & 7, c4 = (warp * 4 + (lane >> 3)) * 4, row = row0 + i, token = token0 + row / a.group;
    const bool used = token < token1;
    const int64_t dst = static_cast<int64_t>(used ? token : token0) * a.q_heads + head * a.group + row % a.group;
    ptx::grid_dependency_wait();
    // What is needed first is on its way together.
    const int32_t status = __ldcg(reinterpret_cast<const int32_t*>(a.workspace));
    const long long total = __ldcg(a.group_unit + groups), units_before = __ldcg(a.group_unit + g);
    const int weight = static_cast<int>(__ldcg(a.group_unit + groups + 1));
    const float4 own = __ldcg(reinterpret_cast<const float4*>(a.partial + dst * D + c4));
    const float lse_of_row = __ldcg(a.partial_lse + dst);
    if (status != MOE_OK) return;  // (after an error nothing is to be used)
    const int units = attend_tiles(prefix) + weight;
    const long long ctas = min(static_cast<long long>(grid), total), item = units_before + (static_cast<long long>(tile) * heads + head) * units;
    const int c0 = static_cast<int>(((item + 1) * ctas - 1) / total), c1 = static_cast<int>(((item + units) * ctas - 1) / total);
    if (c0 == c1 || (tile_rows == 128 && weight > 0 && units <= kAttendRowsLong)) continue;  // one CTA's, which has joined it
    const int pieces = c1 - c0 + 1, width = tile_rows != 128 && pieces > kAttendMerged ? attend_join_width(pieces) : 1, count = (pieces + width - 1) / width;
    const int64_t floats = static_cast<int64_t>(tile_rows) * (D + 2);
    const float* base = reinterpret_cast<const float*>(a.workspace + MOE_KV_WORKSPACE_HEADER) + c0 * 2 * floats;
    const auto piece = [&](int e) { return base + (e == 0 ? 1 : static_cast<int64_t>(e) * 2 * width) * floats; };

    for (int k = tid; k < count * 8; k += 2 * D) {
      const float* p = piece(k >> 3) + static_cast<int64_t>(tile_rows) * D + i0 + (k & 7);
      s_factor[k >> 3][k & 7] = __ldcg(p);
      s_sum[k >> 3][k & 7] = __ldcg(p + tile_rows);
    }
    __syncthreads();
    for (int r = warp; r < 8; r += kWarps) {  // a row to a warp, pieces to a lane
      const float lse = __shfl_sync(kAll, lse_of_row, r);
      float top = lse;
      for (int e = lane; e < count; e += 32) top = fmaxf(top, s_factor[e][r]);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
      const float ref = top > -INFINITY ? top : 0.0f, other = exp2_fast(lse - ref);
      float sum = 0.0f;
      for (int e = lane; e < count; e += 32) {
        s_factor[e][r] = exp2_fast(s_factor[e][r] - ref);
        sum = fmaf(s_sum[e][r], s_factor[e][r], sum);
      }
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
      sum += other;
      const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      for (int e = lane; e < count; e += 32) s_factor[e][r] *= inv;
      if (lane == 0) {
        s_other[r] = other * inv;
        s_lse[r] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
    }
    __syncthreads();
    const float f0 = s_other[i];
    float4 o = make_float4(own.x * f0, own.y * f0, own.z * f0, own.w * f0);
    const int quad = tile_rows == 128 ? attend_quad_at(i0 + i, c4) : (i0 + i) * D + c4;
    for (int e0 = 0; e0 < count; e0 += 8) {
      float4 v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e0 + e < count) v[e] = __ldcg(reinterpret_cast<const float4*>(piece(e0 + e) + quad));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e0 + e >= count) continue;
        const float f = s_factor[e0 + e][i];
        o = make_float4(fmaf(v[e].x, f, o.x), fmaf(v[e].y, f, o.y), fmaf(v[e].z, f, o.z), fmaf(v[e].w, f, o.w));
      }
    }
    __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
    if (used) *reinterpret_cast<uint2*>(a.out + dst * D + c4) = *reinterpret_cast<uint2*>(w);
    if (used && a.lse != nullptr && tid < 8) a.lse[dst] = s_lse[i];
    __syncthreads();  // the factors' room is free again
  }
}

template <int D>
cudaError_t launch_dim(const AttendArgs& a, int rows, int ctas, cudaStream_t stream) {
  // Every block of 8 rows that there may be: each group's rows are rounded up.
  const long long blocks = (static_cast<long long>(a.b.tokens) * a.group + 7) / 8 + a.b.requests;
  const long long work = blocks * a.c.kv_heads, most = 152 * 8;  // (a call that shares nothing pays for the CTAs)
  return launch_chained(kv_attend_merge_kernel<D>, static_cast<int>(work < most ? work : most), 2 * D, 0, true, stream, a, rows, ctas);
}

}  // namespace

cudaError_t launch_kv_attend_merge(const AttendArgs& a, int rows, int ctas, cudaStream_t stream) {
  if (a.c.head_dim == 64) return launch_dim<64>(a, rows, ctas, stream);
  if (a.c.head_dim == 128) return launch_dim<128>(a, rows, ctas, stream);
  return launch_dim<256>(a, rows, ctas, stream);
}

}  // namespace moe
