// Routing: router logits -> the top-k expert ids and weights of each token
// (moe_route in include/moe.h).
//
// One warp per token, the token's logits in registers: element e = lane +
// 32 * i. Scores, keys and sums are FP32. The softmax's sum halves the 1024
// places (i against i + 16, ... in registers, then lanes 16, 8, ... apart), a
// fixed order. Keys become ordered 32-bit integers. The topk-th largest of the
// 32 lanes' maxima is a bound that at least topk keys reach and few others do;
// the keys that reach it are sorted one to a lane.
#include <cuda_fp16.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;
constexpr int kRouteCtas = 152 * 6;
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

// Order of two candidates: the larger key, then the lower index.
__device__ __forceinline__ bool ahead(uint32_t k0, int e0, uint32_t k1, int e1) {
  return k0 > k1 || (k0 == k1 && e0 < e1);
}

// The k-th largest of the 32 lanes' values (1 <= k <= 32), by a bitonic sort.
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, int k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d >= 1; d /= 2) {
      const uint32_t o = __shfl_xor_sync(kAll, v, d);
      const bool descending = !(lane & size) || size == 32, lower = !(lane & d);
      v = descending == lower ? max(v, o) : min(v, o);
    }
  return __shfl_sync(kAll, v, k - 1);
}

template <typename T, int N>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const moe_route_t a) {
  __shared__ __align__(16) uint32_t s_keys[kRouteWarps][32 * N];  // a warp's keys, then its candidates' scores
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.experts;
  uint32_t* keys = s_keys[warp];
  const bool by_sum = a.groups > 1 && a.group_score == 2;
  float bias[N];
  if (a.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) bias[i] = lane + 32 * i < E ? __ldg(a.bias + lane + 32 * i) : 0.0f;
  }

  for (int t = blockIdx.x * kRouteWarps + warp; t < a.tokens; t += gridDim.x * kRouteWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.row_stride;
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

    uint32_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f = x[i];
      if (a.bias != nullptr) f = score[i] + bias[i];
      else if (by_sum) f = score[i];
      key[i] = (masked >> i & 1) || f != f ? kMaskedKey : ordered(f);
      if (lane + 32 * i >= E) key[i] = 0;
    }

    if (a.groups > 1) {
      // A group to a run of lanes: its two largest keys, from shared memory.
      const int size = E / a.groups;
      const int each = a.groups <= 1 ? 32 : a.groups <= 2 ? 16 : a.groups <= 4 ? 8 : a.groups <= 8 ? 4 : a.groups <= 16 ? 2 : 1;
      const int group = lane / each;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) keys[lane + 32 * i] = key[i];
      __syncwarp();
      uint32_t b1 = 0, b2 = 0;
      if (group < a.groups) {
        for (int j = lane % each; j < size; j += each) {
          const uint32_t v = keys[group * size + j];
          b2 = max(b2, min(b1, v));
          b1 = max(b1, v);
        }
      }
      for (int d = each / 2; d >= 1; d >>= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
        b2 = max(max(b2, o2), min(b1, o1));
        b1 = max(b1, o1);
      }
      const float rank = a.group_score == 2 ? unordered(b1) + unordered(b2) : unordered(b1);
      const uint32_t mine = rank != rank ? kMaskedKey : ordered(rank);
      int before = 0;  // groups ahead of this lane's
      for (int g = 0; g < a.groups; ++g) {
        const uint32_t other = __shfl_sync(kAll, mine, g * each);
        before += other > mine || (other == mine && g < group);
      }
      const uint32_t kept = __ballot_sync(kAll, group < a.groups && before < a.group_topk);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !(kept >> (e / size * each) & 1)) key[i] = kMaskedKey;
      }
    }

    // Candidates: the keys from the topk-th largest of the lanes' maxima on. At least topk keys are that large, and
    // with spread keys only a few more.
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) best = max(best, key[i]);
    const uint32_t cut = kth_largest(best, a.topk, lane);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) mine += key[i] >= cut;
    int at = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kAll, at, d);
      if (lane >= d) at += o;
    }
    const int count = __shfl_sync(kAll, at, 31);
    at -= mine;
    int id = 0;
    float w = 0.0f;
    if (count <= 32) {
      // One to a lane, sorted.
      float* scores = reinterpret_cast<float*>(keys) + 64;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (key[i] >= cut) {
          keys[at] = key[i];
          keys[32 + at] = lane + 32 * i;
          scores[at] = score[i];
          ++at;
        }
      __syncwarp();
      uint32_t k = lane < count ? keys[lane] : 0;
      int e = lane < count ? static_cast<int>(keys[32 + lane]) : 0x7FFFFFFF;
      int from = lane;  // where its score lies
#pragma unroll
      for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int d = size / 2; d >= 1; d /= 2) {
          const uint32_t ok = __shfl_xor_sync(kAll, k, d);
          const uint32_t oe = __shfl_xor_sync(kAll, static_cast<uint32_t>(e) | static_cast<uint32_t>(from) << 16, d);
          const int other = static_cast<int>(oe & 0xFFFFu);
          const bool descending = !(lane & size) || size == 32, lower = !(lane & d);
          const bool first = ahead(k, e & 0xFFFF, ok, other);
          if ((descending == lower) != first) {
            k = ok;
            e = other;
            from = static_cast<int>(oe >> 16);
          }
        }
      if (lane < a.topk) {
        id = e & 0xFFFF;
        w = k == kMaskedKey ? 0.0f : scores[from];
      }
    } else {
      // Too many equal keys or too large a topk: one by one, a warp maximum, then the lowest index that has it.
      for (int k = 0; k < a.topk; ++k) {
        best = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) best = max(best, key[i]);
        const uint32_t top = __reduce_max_sync(kAll, best);
        int own = 0x7FFFFFFF;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
          if (key[i] == top) own = lane + 32 * i;
        const int e = __reduce_min_sync(kAll, own);
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
}

template <typename T>
cudaError_t launch_type(const moe_route_t& a, cudaStream_t stream) {
  // Warps that stay over their tokens, so the bias is read once; more than the SMs hold at a time, to even out the end.
  const int ctas = (a.tokens + kRouteWarps - 1) / kRouteWarps, grid = ctas < kRouteCtas ? ctas : kRouteCtas;
  const int block = 32 * kRouteWarps;
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
