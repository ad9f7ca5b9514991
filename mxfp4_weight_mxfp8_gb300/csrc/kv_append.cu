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
//
// 11 prompts of up to 1500 tokens (8 heads of 128, 77 MB) take 18.4 us, 4.2
// TB/s, where the bytes alone would take 11.4: a CTA's page is a chain of slot
// lookups, row loads, a maximum over the item and stores, about 2 us long, and
// the schedulers issue in 56 % of the cycles meanwhile. A decode step of 64
// tokens takes 2.7 us, about a launch. Rows are held in registers between the
// two passes, so they are read once.
#include "decode.h"

namespace moe {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kAppendCtas = 152 * 8;  // as many as are resident together, about
constexpr uint32_t kAll = 0xFFFFFFFFu;

// Largest magnitude bits of a word's two BF16 values, running.
__device__ __forceinline__ uint32_t larger2(uint32_t m, uint32_t word) { return __vmaxu2(m, word & 0x7FFF7FFFu); }

// The same over the finite values only.
__device__ __forceinline__ uint32_t larger2_finite(uint32_t m, uint32_t word) {
  const uint32_t v = word & 0x7FFF7FFFu;
  return __vmaxu2(m, v & ~__vcmpgeu2(v, 0x7F807F80u));
}

// Codes of a word's two BF16 values times 2^-E (exact in BF16); infinities saturate.
__device__ __forceinline__ uint32_t encode2(uint32_t word, __nv_bfloat162 inv) {
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&word), inv);
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&v);
  return __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)), __NV_SATFINITE, __NV_E4M3);
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

// kSplit warps for each (keys or values, head); a CTA's warps go over the pages that start in its window of tokens.
// Up to kHeld chunks a lane stay in registers between the two passes; what a page holds beyond that is read again.
template <int D, int kSplit>
__global__ void __launch_bounds__(32 * kAppendWarps, kSplit == 1 ? 2 : 4) kv_append_kernel(const AppendArgs a, int shift, int window) {
  constexpr int kChunks = D / 8, kHeld = 8, kBatch = 32 * kHeld * kSplit;  // a chunk: 8 values, 16 bytes
  __shared__ uint32_t s_most[2][kAppendWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % kSplit;
  const int P = a.c.page_tokens, item = (blockIdx.y * kAppendWarps + warp) / kSplit;
  if (item >= 2 * a.c.kv_heads) return;
  const int which = item & 1, head = item >> 1, w0 = blockIdx.x * window;
  const int64_t limit = static_cast<int64_t>(a.c.pages) << shift, stride = which ? a.token_stride[1] : a.token_stride[0];
  uint8_t* scales = which ? a.c.v_scale : a.c.k_scale;

  bool leads = false;  // the lane's token of the window is the first of its page
  if (lane < window && w0 + lane < a.tokens) {
    const int64_t slot = a.slots[w0 + lane], before = w0 + lane > 0 ? a.slots[w0 + lane - 1] : -1;
    leads = slot >= 0 && slot < limit && ((slot & (P - 1)) == 0 || before != slot - 1);
  }
  int turn = 0;
  for (uint32_t leaders = __ballot_sync(kAll, leads); leaders; leaders &= leaders - 1, turn ^= 1) {
    const int t = w0 + __ffs(leaders) - 1;
    const int64_t slot = a.slots[t], page = slot >> shift;
    const int first = static_cast<int>(slot & (P - 1));
    uint8_t* scale = scales + page * a.c.kv_heads + head;
    const int old = first != 0 ? static_cast<int>(*scale) - 127 : -128;
    // Rows of this page, this one included; the lookups of up to 128 go out together.
    bool in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 32 * j + lane;
      in[j] = i < P - first && t + i < a.tokens && a.slots[t + i] == slot + i;
    }
    int run = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t votes = __ballot_sync(kAll, in[j]);
      if (run == 32 * j) run += votes == kAll ? 32 : __ffs(~votes) - 1;
    }
    const uint16_t* x = (which ? a.x[1] : a.x[0]) + t * stride + head * (which ? a.head_stride[1] : a.head_stride[0]);
    uint8_t* codes = (which ? a.c.v : a.c.k) + ((page * a.c.kv_heads + head) << shift) * D;
    // A lane's chunks lie 32 apart, so kStep rows apart in the same columns.
    constexpr int kStep = 32 / kChunks;
    const int chunks = run * kChunks, mine = part * 32 * kHeld + lane;
    const uint16_t* src = x + (mine / kChunks) * stride + (mine % kChunks) * 8;
    uint8_t* dst = codes + first * D + mine * 8;
    const int64_t step = kStep * stride;
    uint4 held[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      held[j] = mine + 32 * j < chunks ? *reinterpret_cast<const uint4*>(src + j * step) : make_uint4(0, 0, 0, 0);
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) most = larger2(larger2(larger2(larger2(most, held[j].x), held[j].y), held[j].z), held[j].w);
    for (int base = mine + kBatch; base < chunks; base += kBatch)
#pragma unroll 4
      for (int i = base; i < base + 32 * kHeld && i < chunks; i += 32) {
        const uint4 w = *reinterpret_cast<const uint4*>(x + (i / kChunks) * stride + (i % kChunks) * 8);
        most = larger2(larger2(larger2(larger2(most, w.x), w.y), w.z), w.w);
      }
    if (__any_sync(kAll, max(most & 0xFFFFu, most >> 16) >= 0x7F80u)) {  // infinities or NaN: once more without them
      most = 0;
      for (int i = part * 32 + lane; i < chunks; i += 32 * kSplit) {
        const uint4 w = *reinterpret_cast<const uint4*>(x + (i / kChunks) * stride + (i % kChunks) * 8);
        most = larger2_finite(larger2_finite(larger2_finite(larger2_finite(most, w.x), w.y), w.z), w.w);
      }
    }
    most = __reduce_max_sync(kAll, max(most & 0xFFFFu, most >> 16));
    if (kSplit > 1) {  // over the item's warps (two sets of words: the next page's do not meet this one's)
      if (lane == 0) s_most[turn][warp] = most;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / kSplit), "r"(32 * kSplit) : "memory");
#pragma unroll
      for (int j = 0; j < kSplit; ++j) most = max(most, s_most[turn][warp / kSplit * kSplit + j]);
    }
    const float amax = __uint_as_float(most << 16);
    int E = mx_exponent(amax, false);
    if (old >= E) {
      E = old;
    } else if (first != 0) {
      const float down = pow2f(max(old - E, -126));
      for (int i = part * 32 + lane; i < first * (D / 4); i += 32 * kSplit) {
        uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
        const uint32_t c = *p;
        *p = rescale2(c & 0xFFFFu, down) | rescale2(c >> 16, down) << 16;
      }
    }
    const __nv_bfloat162 inv = __float2bfloat162_rn(pow2f(-E));
    auto encode = [&](const uint4& w) {
      return make_uint2(encode2(w.x, inv) | encode2(w.y, inv) << 16, encode2(w.z, inv) | encode2(w.w, inv) << 16);
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (mine + 32 * j < chunks) *reinterpret_cast<uint2*>(dst + j * 256) = encode(held[j]);
    for (int base = mine + kBatch; base < chunks; base += kBatch)
      for (int i = base; i < base + 32 * kHeld && i < chunks; i += 32)
        *reinterpret_cast<uint2*>(codes + first * D + i * 8) =
            encode(*reinterpret_cast<const uint4*>(x + (i / kChunks) * stride + (i % kChunks) * 8));
    // Every warp of the item has read the old scale before its barrier above.
    if (part == 0 && lane == 0 && E != old) *scale = static_cast<uint8_t>(E + 127);
  }
}

template <int D, int kSplit>
cudaError_t launch_split(const AppendArgs& a, int shift, int window, cudaStream_t stream) {
  const int columns = (2 * a.c.kv_heads * kSplit + kAppendWarps - 1) / kAppendWarps;
  const dim3 grid((a.tokens + window - 1) / window, columns);
  kv_append_kernel<D, kSplit><<<grid, 32 * kAppendWarps, 0, stream>>>(a, shift, window);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const AppendArgs& a, int shift, cudaStream_t stream) {
  // A token to a CTA, a warp to an item, while that is no more CTAs than are resident together (a decode step of 64
  // tokens: 2.7 us, against 4.2 the other way; prompts of 12 thousand tokens: 90 us, against 18.4).
  const int columns = (2 * a.c.kv_heads + kAppendWarps - 1) / kAppendWarps;
  if (static_cast<int64_t>(a.tokens) * columns <= kAppendCtas) return launch_split<D, 1>(a, shift, 1, stream);
  // More tokens: windows of up to 32, a lane to a token (the pages of prompts start every page_tokens tokens; with
  // windows of 8 those prompts take 23.5 us), four warps to an item.
  int window = 2;
  while (window < 32 && static_cast<int64_t>(a.tokens) * columns * 4 > static_cast<int64_t>(window) * kAppendCtas) window *= 2;
  return launch_split<D, 4>(a, shift, window, stream);
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
