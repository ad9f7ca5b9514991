// Quantizing new keys and values into the paged cache (moe_kv_append in
// include/moe.h).
//
// The tokens of one page follow one another in `slots`; the first of them (its
// row is 0, or the slot before is not its predecessor) stands for the page and
// its warps take the whole run: one pass for max|x|, the page's scale (grown
// if need be, with the earlier codes rounded again), one pass that encodes.
// Scales are powers of two, so growing one loses only what the smaller codes'
// last places hold.
#include "kernels.h"

namespace moe {
namespace {

constexpr int kAppendWarps = 4;
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

template <int D>
__global__ void __launch_bounds__(32 * kAppendWarps) kv_append_kernel(const AppendArgs a, int shift) {
  constexpr int kChunks = D / 8;  // 8 values: 16 bytes of BF16, 8 of codes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, P = a.c.page_tokens;
  const int64_t slot = a.slots[t], limit = static_cast<int64_t>(a.c.pages) << shift;
  if (slot < 0 || slot >= limit) return;
  const int first = static_cast<int>(slot & (P - 1));
  if (first != 0 && t > 0 && a.slots[t - 1] == slot - 1) return;
  int run = 0;  // rows of this page, this one included
  for (int base = 0; base < P - first; base += 32) {
    const int i = base + lane;
    const bool in = i < P - first && t + i < a.tokens && a.slots[t + i] == slot + i;
    const uint32_t votes = __ballot_sync(kAll, in);
    const int n = votes == kAll ? 32 : __ffs(~votes) - 1;
    run += n;
    if (n < 32) break;
  }
  const int64_t page = slot >> shift;
  for (int item = warp; item < 2 * a.c.kv_heads; item += kAppendWarps) {
    const int which = item & 1, head = item >> 1;
    const uint16_t* x = a.x[which] + t * a.token_stride[which] + head * a.head_stride[which];
    uint8_t* scales = which ? a.c.v_scale : a.c.k_scale;
    uint8_t* codes = (which ? a.c.v : a.c.k) + ((page * a.c.kv_heads + head) << shift) * D;
    float amax = 0.0f;
    for (int i = lane; i < run * kChunks; i += 32) {
      const uint4 w = *reinterpret_cast<const uint4*>(x + (i / kChunks) * a.token_stride[which] + (i % kChunks) * 8);
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(finite_abs(words[j]), finite_abs(words[j] >> 16)));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, d));
    int E = mx_exponent(amax, false);
    uint8_t* scale = scales + page * a.c.kv_heads + head;
    if (first != 0) {
      const int old = static_cast<int>(*scale) - 127;
      if (old >= E) {
        E = old;
      } else {
        const float down = pow2f(max(old - E, -126));
        for (int i = lane; i < first * (D / 4); i += 32) {
          uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
          const uint32_t c = *p;
          *p = rescale2(c & 0xFFFFu, down) | rescale2(c >> 16, down) << 16;
        }
      }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = static_cast<uint8_t>(E + 127);
    const float inv = pow2f(-E);
    for (int i = lane; i < run * kChunks; i += 32) {
      const uint4 w = *reinterpret_cast<const uint4*>(x + (i / kChunks) * a.token_stride[which] + (i % kChunks) * 8);
      uint2 o;
      o.x = encode2(w.x, inv) | encode2(w.y, inv) << 16;
      o.y = encode2(w.z, inv) | encode2(w.w, inv) << 16;
      *reinterpret_cast<uint2*>(codes + (first + i / kChunks) * D + (i % kChunks) * 8) = o;
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  int shift = 4;
  while ((1 << shift) < a.c.page_tokens) ++shift;
  if (a.c.head_dim == 64)
    kv_append_kernel<64><<<a.tokens, 32 * kAppendWarps, 0, stream>>>(a, shift);
  else if (a.c.head_dim == 128)
    kv_append_kernel<128><<<a.tokens, 32 * kAppendWarps, 0, stream>>>(a, shift);
  else
    kv_append_kernel<256><<<a.tokens, 32 * kAppendWarps, 0, stream>>>(a, shift);
  return cudaGetLastError();
}

}  // namespace moe
