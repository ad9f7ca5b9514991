// Quantizing new keys and values into the paged cache (moe_kv_append in
// include/moe.h).
//
// The tokens of one page follow one another in `slots`; the first of them (its
// row is 0, or the slot before is not its predecessor) stands for the page, and
// a warp for each head's keys and values takes the whole run: one pass for
// max|x|, the page's scale (grown if need be, with the earlier codes rounded
// again), one pass that encodes.
// Scales are powers of two, so growing one loses only what the smaller codes'
// last places hold.
#include "kernels.h"

namespace moe {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kAppendCtas = 152 * 8;  // as many as are resident together, about
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float finite_abs(uint32_t bf16_bits) {
  const uint32_t b = bf16_bits & 0x7FFFu;
  return b < 0x7F80u ? __uint_as_float(b << 16) : 0.0f;
}

// Codes of the two BF16 values of a word, scaled by 2^-E; infinities saturate.
__device__ __forceinline__ uint32_t encode2(uint32_t word, float inv) {
  const float2 v = make_float2(__uint_as_float(word << 16) * inv, __uint_as_float(word & 0xFFFF0000u) * inv);
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t rescale2(uint32_t codes, float shift) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  float2 f = __half22float2(__half2(h));
  f.x *= shift;
  f.y *= shift;
  const uint32_t moved = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  uint32_t nan = 0;  // a NaN keeps its code, sign included
  if ((codes & 0x7Fu) == 0x7Fu) nan |= 0xFFu;
  if ((codes & 0x7F00u) == 0x7F00u) nan |= 0xFF00u;
  return (moved & ~nan) | (codes & nan);
}

// Largest finite magnitude of a lane's share of `run` rows, kUnroll loads in flight.
template <int D>
__device__ __forceinline__ float rows_amax(const uint16_t* x, int64_t stride, int run, int lane) {
  constexpr int kChunks = D / 8, kUnroll = 8;  // a chunk: 8 values, 16 bytes
  float amax = 0.0f;
  for (int base = lane; base < run * kChunks; base += 32 * kUnroll) {
    uint4 w[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int i = base + 32 * j;
      w[j] = i < run * kChunks ? *reinterpret_cast<const uint4*>(x + (i / kChunks) * stride + (i % kChunks) * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t words[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) amax = fmaxf(amax, fmaxf(finite_abs(words[q]), finite_abs(words[q] >> 16)));
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, d));
  return amax;
}

// A warp for each (keys or values, head); a CTA's warps go over the pages that start in its window of tokens.
template <int D>
__global__ void __launch_bounds__(32 * kAppendWarps) kv_append_kernel(const AppendArgs a, int shift, int window) {
  constexpr int kChunks = D / 8, kUnroll = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = a.c.page_tokens, item = blockIdx.y * kAppendWarps + warp;
  if (item >= 2 * a.c.kv_heads) return;
  const int which = item & 1, head = item >> 1, w0 = blockIdx.x * window;
  const int64_t limit = static_cast<int64_t>(a.c.pages) << shift, stride = a.token_stride[which];
  uint8_t* scales = which ? a.c.v_scale : a.c.k_scale;

  bool leads = false;  // the lane's token of the window is the first of its page
  if (lane < window && w0 + lane < a.tokens) {
    const int64_t slot = a.slots[w0 + lane], before = w0 + lane > 0 ? a.slots[w0 + lane - 1] : -1;
    leads = slot >= 0 && slot < limit && ((slot & (P - 1)) == 0 || before != slot - 1);
  }
  for (uint32_t leaders = __ballot_sync(kAll, leads); leaders; leaders &= leaders - 1) {
    const int t = w0 + __ffs(leaders) - 1;
    const int64_t slot = a.slots[t], page = slot >> shift;
    const int first = static_cast<int>(slot & (P - 1));
    uint8_t* scale = scales + page * a.c.kv_heads + head;
    const int old = first != 0 ? static_cast<int>(*scale) - 127 : -128;
    int run = 0;  // rows of this page, this one included
    for (int base = 0; base < P - first; base += 32) {
      const int i = base + lane;
      const bool in = i < P - first && t + i < a.tokens && a.slots[t + i] == slot + i;
      const uint32_t votes = __ballot_sync(kAll, in);
      const int n = votes == kAll ? 32 : __ffs(~votes) - 1;
      run += n;
      if (n < 32) break;
    }
    const uint16_t* x = a.x[which] + t * stride + head * a.head_stride[which];
    uint8_t* codes = (which ? a.c.v : a.c.k) + ((page * a.c.kv_heads + head) << shift) * D;
    int E = mx_exponent(rows_amax<D>(x, stride, run, lane), false);
    if (old >= E) {
      E = old;
    } else if (first != 0) {
      const float down = pow2f(max(old - E, -126));
      for (int i = lane; i < first * (D / 4); i += 32) {
        uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
        const uint32_t c = *p;
        *p = rescale2(c & 0xFFFFu, down) | rescale2(c >> 16, down) << 16;
      }
    }
    if (lane == 0 && E != old) *scale = static_cast<uint8_t>(E + 127);
    // The rows again (from the caches by now), encoded.
    const float inv = pow2f(-E);
    for (int base = lane; base < run * kChunks; base += 32 * kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int i = base + 32 * j;
        if (i < run * kChunks) w[j] = *reinterpret_cast<const uint4*>(x + (i / kChunks) * stride + (i % kChunks) * 8);
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int i = base + 32 * j;
        uint2 o;
        o.x = encode2(w[j].x, inv) | encode2(w[j].y, inv) << 16;
        o.y = encode2(w[j].z, inv) | encode2(w[j].w, inv) << 16;
        if (i < run * kChunks) *reinterpret_cast<uint2*>(codes + (first + i / kChunks) * D + (i % kChunks) * 8) = o;
      }
    }
  }
}

template <int D>
cudaError_t launch_dim(const AppendArgs& a, int shift, cudaStream_t stream) {
  // Windows of one token where that already gives every SM work (a decode step), up to 32 for long prompts, whose pages
  // start only every page_tokens tokens.
  const int columns = (2 * a.c.kv_heads + kAppendWarps - 1) / kAppendWarps;
  int window = 1;
  while (window < 32 && static_cast<int64_t>(a.tokens) * columns > window * kAppendCtas) window *= 2;
  const dim3 grid((a.tokens + window - 1) / window, columns);
  kv_append_kernel<D><<<grid, 32 * kAppendWarps, 0, stream>>>(a, shift, window);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  int shift = 4;
  while ((1 << shift) < a.c.page_tokens) ++shift;
  if (a.c.head_dim == 64) return launch_dim<64>(a, shift, stream);
  if (a.c.head_dim == 128) return launch_dim<128>(a, shift, stream);
  return launch_dim<256>(a, shift, stream);
}

}  // namespace moe
