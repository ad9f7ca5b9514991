// Routing: router logits -> the top-k expert ids and weights of each token
// (moe_route in include/moe.h).
//
// One warp per token, the token's logits in registers: element e = lane +
// 32 * i. Scores, keys and sums are FP32. The softmax's sum halves the 1024
// places (i against i + 16, ... in registers, then lanes 16, 8, ... apart), a
// fixed order. Keys become ordered 32-bit integers. The topk-th largest of the
// 32 lanes' maxima is a bound that at least topk keys reach and few others do;
// the keys that reach it are sorted one to a lane.
//
// Ids are the formula's bit for bit, so every key is computed as written: expf,
// a correctly rounded reciprocal or quotient, one addition of the bias. That,
// not memory, bounds large calls: 16381 tokens of 384 experts with a bias and
// group limits take 25.6 us (1.07 TB/s; the 27 MB alone would take 4.0), with
// the schedulers issuing in 70 % of the cycles (about 1340 warp instructions a
// token, a third of them the 384 sigmoids). One token takes 3.7 us and 64 take
// 3.4, of which a launch is about 2.5.
#include <cuda_fp16.h>

#include "decode.h"

namespace moe {
namespace {

constexpr int kRouteWarps = 4;
constexpr int kRouteSms = 152;
constexpr uint32_t kAll = 0xFFFFFFFFu;
// Ordered forms: a larger key is a larger integer. Absent elements (past the
// last expert, or taken already) are 0, below the masked ones.
constexpr uint32_t kMaskedKey = 0x007FFFFFu;  // -inf

__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 and +0 are equal keys
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
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

// 1 / (1 + exp(-x)); the reciprocal is the division's value, correctly rounded.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

template <typename T, int N>
__global__ void __launch_bounds__(32 * kRouteWarps, N <= 12 ? 6 : N <= 16 ? 4 : 3) route_kernel(const moe_route_t a) {
  // A warp's keys by expert (groups), then its candidates (key, expert) as they come and in order.
  constexpr int kOrdered = 72, kKeys = 32 * N > kOrdered + 64 ? 32 * N : kOrdered + 64;
  __shared__ __align__(16) uint32_t s_keys[kRouteWarps][kKeys];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.experts;
  uint32_t* keys = s_keys[warp];
  const bool sigmoids = a.scoring == MOE_SCORE_SIGMOID;
  const bool by_sum = a.groups > 1 && a.group_score == 2;
  const bool scored = a.bias != nullptr || by_sum;  // the keys need every score; else the logits order them
  float bias[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    bias[i] = a.bias != nullptr && lane + 32 * i < E ? __ldg(a.bias + lane + 32 * i) : 0.0f;
    if (bias[i] != bias[i]) bias[i] = -INFINITY;  // a NaN key counts as masked
  }
  // A group to a run of lanes.
  const int size = E / a.groups;
  const int each = a.groups <= 2 ? 16 : a.groups <= 4 ? 8 : a.groups <= 8 ? 4 : a.groups <= 16 ? 2 : 1;
  const int group = lane / each;

  for (int t = blockIdx.x * kRouteWarps + warp; t < a.tokens; t += gridDim.x * kRouteWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.row_stride;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      x[i] = e < E ? load_logit<T>(row + e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fminf(fmaxf(x[i], -INFINITY), 3.402823466e38f);  // NaN: masked; +inf: the largest number
    // A logit's score is exp(x - top) / sum, or its sigmoid.
    float top = 0.0f, sum = 1.0f;
    uint32_t key[N];
    if (!sigmoids) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) top = fmaxf(top, x[i]);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
      if (top == -INFINITY) top = 0.0f;
      float score[N];
#pragma unroll
      for (int i = 0; i < N; ++i) score[i] = expf(x[i] - top);
      float part[N];
#pragma unroll
      for (int i = 0; i < N; ++i) part[i] = score[i];
      sum = tree_sum<N>(part);
      if (scored) {
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = ordered(x[i] > -INFINITY ? __fdiv_rn(score[i], sum) + bias[i] : -INFINITY);
      }
    } else if (scored) {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = ordered(x[i] > -INFINITY ? sigmoid(x[i]) + bias[i] : -INFINITY);
    }
    if (!scored) {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = ordered(x[i]);
    }
    if (E < 32 * N) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane + 32 * i >= E) key[i] = 0;
    }

    if (a.groups > 1) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) keys[lane + 32 * i] = key[i];
      __syncwarp();
      uint32_t b1 = 0, b2 = 0;  // the group's two largest
      if (group < a.groups) {
#pragma unroll 4
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
      if (group < a.groups && before >= a.group_topk) {
#pragma unroll 4
        for (int j = lane % each; j < size; j += each) keys[group * size + j] = kMaskedKey;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = keys[lane + 32 * i];
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
    uint32_t won = kMaskedKey;
    __syncwarp();
    if (count <= 32) {
      // One to a lane; its place is the number of those ahead of it: the larger key, then the lower index.
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (key[i] >= cut) {
          *reinterpret_cast<uint2*>(keys + 2 * at) = make_uint2(key[i], lane + 32 * i);
          ++at;
        }
      __syncwarp();
      const uint2 own = *reinterpret_cast<const uint2*>(keys + 2 * lane);
      if (lane < 4) *reinterpret_cast<uint2*>(keys + 2 * (count + lane)) = make_uint2(0, 0);  // the last four read together
      __syncwarp();
      int place = 0;
      for (int j = 0; j < count; j += 4) {
        const uint4 o0 = *reinterpret_cast<const uint4*>(keys + 2 * j), o1 = *reinterpret_cast<const uint4*>(keys + 2 * j + 4);
        place += o0.x > own.x || (o0.x == own.x && o0.y < own.y);
        place += o0.z > own.x || (o0.z == own.x && o0.w < own.y);
        place += o1.x > own.x || (o1.x == own.x && o1.y < own.y);
        place += o1.z > own.x || (o1.z == own.x && o1.w < own.y);
      }
      __syncwarp();
      if (lane < count) *reinterpret_cast<uint2*>(keys + kOrdered + 2 * place) = own;
      __syncwarp();
      const uint2 mine2 = *reinterpret_cast<const uint2*>(keys + kOrdered + 2 * lane);
      if (lane < a.topk) {
        won = mine2.x;
        id = static_cast<int>(mine2.y);
      }
    } else {
      // Too many equal keys or too large a topk: one by one, a warp maximum, then the lowest index that has it.
      for (int k = 0; k < a.topk; ++k) {
        best = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) best = max(best, key[i]);
        const uint32_t largest = __reduce_max_sync(kAll, best);
        int own = 0x7FFFFFFF;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
          if (key[i] == largest) own = lane + 32 * i;
        const int e = __reduce_min_sync(kAll, own);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (e == lane + 32 * i) key[i] = 0;
        if (lane == k) {
          id = e;
          won = largest;
        }
      }
    }
    // The winners' scores again, from their logits.
    float w = 0.0f;
    if (lane < a.topk && won != kMaskedKey) {
      float v = load_logit<T>(row + id);
      if (sigmoids) w = sigmoid(v);
      else w = __fdiv_rn(expf(fminf(v, 3.402823466e38f) - top), sum);
    }
    if (a.renormalize) {
      float all = w;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) all += __shfl_xor_sync(kAll, all, d);
      w = all > 0.0f ? __fdiv_rn(w, all) : 0.0f;
    }
    if (lane < a.topk) {
      a.ids[static_cast<int64_t>(t) * a.topk + lane] = id;
      a.weights[static_cast<int64_t>(t) * a.topk + lane] = w * a.scale;
    }
  }
}

template <typename T, int N>
cudaError_t launch_size(const moe_route_t& a, cudaStream_t stream) {
  // Warps that stay over their tokens, so the bias is read once; no more than are resident together (16381 tokens:
  // 25.6 us, against 27.4 with a warp for every token).
  const int ctas = (a.tokens + kRouteWarps - 1) / kRouteWarps, resident = kRouteSms * (N <= 12 ? 6 : N <= 16 ? 4 : 3);
  route_kernel<T, N><<<ctas < resident ? ctas : resident, 32 * kRouteWarps, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const moe_route_t& a, cudaStream_t stream) {
  if (a.experts <= 128) return launch_size<T, 4>(a, stream);
  if (a.experts <= 256) return launch_size<T, 8>(a, stream);
  if (a.experts <= 384) return launch_size<T, 12>(a, stream);
  if (a.experts <= 512) return launch_size<T, 16>(a, stream);
  return launch_size<T, 32>(a, stream);
}

}  // namespace

cudaError_t launch_route(const moe_route_t& a, cudaStream_t stream) {
  if (a.dtype == MOE_F32) return launch_type<float>(a, stream);
  if (a.dtype == MOE_BF16) return launch_type<__nv_bfloat16>(a, stream);
  return launch_type<__half>(a, stream);
}

}  // namespace moe
