// Routing: router logits -> the top-k expert ids and weights of each token
// (moe_route in include/moe.h).
//
// One warp per token, the token's logits in registers: element e = lane +
// 32 * i. Scores, keys and sums are FP32. The softmax's sum halves the 1024
// places (i against i + 16, ... in registers, then lanes 16, 8, ... apart), a
// fixed order. Keys become ordered 32-bit integers and the k winners are
// taken one by one: a warp maximum, then the lowest index that has it.
#include <cuda_fp16.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;
constexpr uint32_t kAll = 0xFFFFFFFFu;
// Ordered forms: a larger key is a larger integer. Absent elements (past the
// last expert, or taken already) are 0, below the masked ones.
constexpr uint32_t kMaskedKey = 0x007FFFFFu;  // -inf

__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 and +0 are equal keys
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) {
  return __ldg(p);
}
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}
template <>
__device__ __forceinline__ float load_logit<__half>(const __half* p) {
  return __half2float(*p);
}

// Sum of the warp's 32 * N values by halving the 1024 places they fill.
template <int N>
__device__ __forceinline__ float tree_sum(float (&v)[N]) {
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
#pragma unroll
    for (int i = 0; i < half; ++i)
      if (i + half < N) v[i] += v[i + half];
  }
  float s = v[0];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kAll, s, d);
  return s;
}

template <typename T, int N>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const moe_route_t a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const T* row = static_cast<const T*>(a.logits) + t * a.row_stride;
  const int E = a.experts;

  float x[N], score[N];
  uint32_t masked = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < E ? load_logit<T>(row + e) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (!(x[i] > -INFINITY)) masked |= 1u << i;  // -inf or NaN
  if (a.scoring == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) score[i] = __fdiv_rn(1.0f, 1.0f + expf(-x[i]));
  } else {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = fminf(x[i], 3.402823466e38f);
      if (!(masked >> i & 1)) top = fmaxf(top, x[i]);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    float part[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      score[i] = (masked >> i & 1) ? 0.0f : expf(x[i] - top);
      part[i] = score[i];
    }
    const float sum = tree_sum<N>(part);
#pragma unroll
    for (int i = 0; i < N; ++i) score[i] = __fdiv_rn(score[i], sum);
  }

  const bool by_sum = a.groups > 1 && a.group_score == 2;
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    float f = x[i];
    if (a.bias != nullptr)
      f = e < E ? score[i] + __ldg(a.bias + e) : -INFINITY;
    else if (by_sum)
      f = score[i];
    key[i] = (masked >> i & 1) || f != f ? kMaskedKey : ordered(f);
    if (e >= E) key[i] = 0;
  }

  if (a.groups > 1) {
    const int size = E / a.groups;
    float rank = -INFINITY;  // lane g: group g's
    for (int g = 0; g < a.groups; ++g) {
      float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        if (e >= g * size && e < (g + 1) * size) {
          const float f = unordered(key[i]);
          b2 = fmaxf(b2, fminf(b1, f));
          b1 = fmaxf(b1, f);
        }
      }
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) {
        const float o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
      if (lane == g) rank = a.group_score == 2 ? b1 + b2 : b1;
    }
    uint32_t mine = rank != rank ? kMaskedKey : ordered(rank);
    int before = 0;  // groups ahead of this lane's
    for (int g = 0; g < a.groups; ++g) {
      const uint32_t other = __shfl_sync(kAll, mine, g);
      before += other > mine || (other == mine && g < lane);
    }
    const uint32_t kept = __ballot_sync(kAll, lane < a.groups && before < a.group_topk);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(kept >> (e / size) & 1)) key[i] = kMaskedKey;
    }
  }

  int id = 0;
  float w = 0.0f;
  for (int k = 0; k < a.topk; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kAll, best);
    int mine = 0x7FFFFFFF;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (key[i] == top) mine = lane + 32 * i;
    const int e = __reduce_min_sync(kAll, mine);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e == lane + 32 * i) {
        key[i] = 0;
        s = score[i];
      }
    s = __shfl_sync(kAll, s, e & 31);
    if (lane == k) {
      id = e;
      w = top == kMaskedKey ? 0.0f : s;
    }
  }
  if (a.renormalize) {
    float sum = w;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  if (lane < a.topk) {
    a.ids[static_cast<int64_t>(t) * a.topk + lane] = id;
    a.weights[static_cast<int64_t>(t) * a.topk + lane] = w * a.scale;
  }
}

template <typename T>
cudaError_t launch_type(const moe_route_t& a, cudaStream_t stream) {
  const int grid = (a.tokens + kRouteWarps - 1) / kRouteWarps, block = 32 * kRouteWarps;
  if (a.experts <= 128)
    route_kernel<T, 4><<<grid, block, 0, stream>>>(a);
  else if (a.experts <= 256)
    route_kernel<T, 8><<<grid, block, 0, stream>>>(a);
  else if (a.experts <= 384)
    route_kernel<T, 12><<<grid, block, 0, stream>>>(a);
  else if (a.experts <= 512)
    route_kernel<T, 16><<<grid, block, 0, stream>>>(a);
  else
    route_kernel<T, 32><<<grid, block, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const moe_route_t& a, cudaStream_t stream) {
  if (a.dtype == MOE_F32) return launch_type<float>(a, stream);
  if (a.dtype == MOE_BF16) return launch_type<__nv_bfloat16>(a, stream);
  return launch_type<__half>(a, stream);
}

}  // namespace moe
