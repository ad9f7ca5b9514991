// Rotary positions of queries and keys (moe_rope in include/moe.h).
//
// The angle of a pair is position * turns, a whole number of 2^-64 turns: the
// product modulo 2^64 drops whole turns exactly, and its upper half is the angle
// to 2^-32 of a turn, whatever the position. A lane keeps the sines of its
// eight pairs and takes the same dimensions of one head after the other, so
// they are computed once for several heads; every element is read and written
// once and the bytes bound it.
#include "decode.h"

namespace moe {
namespace {

constexpr int kRopeThreads = 128;

// Tensor `which` of the two.
struct Rows {
  const uint16_t* from;
  uint16_t* to;
  int64_t token, head, to_token, to_head;
};

__device__ __forceinline__ void sin_cos(uint64_t turns, int position, float amplitude, float& sin, float& cos) {
  const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns;
  // Half turns in [-1, 1).
  sincospif(static_cast<float>(static_cast<int32_t>(at >> 32)) * 0x1p-31f, &sin, &cos);
  sin *= amplitude;
  cos *= amplitude;
}

__device__ __forceinline__ uint32_t pack(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The pair (a, b), turned; the roundings written out, so that both kernels give the same bits.
__device__ __forceinline__ float first_of(float a, float b, float sin, float cos) { return __fmaf_rn(a, cos, -__fmul_rn(b, sin)); }
__device__ __forceinline__ float second_of(float a, float b, float sin, float cos) { return __fmaf_rn(b, cos, __fmul_rn(a, sin)); }

// A head's row is `units` units: rotated ones (8 pairs: two 16-byte words), then copied ones (a word each, where the output
// is another tensor). `slots` lanes, a power of two, share the units of a head; the heads of a token go by in turn, `heads`
// of them to a CTA's y.
template <bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const moe_rope_t a, int slots, int heads_per) {
  const int pairs = a.rotary_dim / 2, rotated = pairs / 8, all_heads = a.q_heads + a.k_heads;
  const int copied = (a.head_dim - a.rotary_dim) / 8;
  const int slot = threadIdx.x & (slots - 1), groups = kRopeThreads / slots, first = blockIdx.y * heads_per;
  const int last = min(first + heads_per, all_heads);
  const int t = blockIdx.x;
  const int position = a.positions[t];
  const Rows q{static_cast<const uint16_t*>(a.q) + t * a.q_token_stride, static_cast<uint16_t*>(a.q_out) + t * a.q_out_token_stride,
               0, a.q_head_stride, 0, a.q_out_head_stride};
  const Rows k{static_cast<const uint16_t*>(a.k) + t * a.k_token_stride, static_cast<uint16_t*>(a.k_out) + t * a.k_out_token_stride,
               0, a.k_head_stride, 0, a.k_out_head_stride};
  for (int u = slot; u < rotated; u += slots) {
    float sin[8], cos[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sin_cos(a.turns[u * 8 + j], position, a.amplitude, sin[j], cos[j]);
    const int at0 = kInterleaved ? u * 16 : u * 8, at1 = kInterleaved ? at0 + 8 : at0 + pairs;
#pragma unroll 2
    for (int h = first + threadIdx.x / slots; h < last; h += groups) {
      const bool key = h >= a.q_heads;
      const uint16_t* from = key ? k.from + (h - a.q_heads) * k.head : q.from + h * q.head;
      uint16_t* to = key ? k.to + (h - a.q_heads) * k.to_head : q.to + h * q.to_head;
      const uint4 x = *reinterpret_cast<const uint4*>(from + at0), y = *reinterpret_cast<const uint4*>(from + at1);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
      uint32_t xo[4], yo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kInterleaved) {
          const float a0 = low(xs[j]), b0 = high(xs[j]), a1 = low(ys[j]), b1 = high(ys[j]);
          xo[j] = pack(first_of(a0, b0, sin[j], cos[j]), second_of(a0, b0, sin[j], cos[j]));
          yo[j] = pack(first_of(a1, b1, sin[4 + j], cos[4 + j]), second_of(a1, b1, sin[4 + j], cos[4 + j]));
        } else {
          const float a0 = low(xs[j]), a1 = high(xs[j]), b0 = low(ys[j]), b1 = high(ys[j]);
          xo[j] = pack(first_of(a0, b0, sin[2 * j], cos[2 * j]), first_of(a1, b1, sin[2 * j + 1], cos[2 * j + 1]));
          yo[j] = pack(second_of(a0, b0, sin[2 * j], cos[2 * j]), second_of(a1, b1, sin[2 * j + 1], cos[2 * j + 1]));
        }
      }
      *reinterpret_cast<uint4*>(to + at0) = make_uint4(xo[0], xo[1], xo[2], xo[3]);
      *reinterpret_cast<uint4*>(to + at1) = make_uint4(yo[0], yo[1], yo[2], yo[3]);
    }
  }
  for (int i = threadIdx.x; i < copied * (last - first); i += kRopeThreads) {
    const int h = first + i / copied, at = a.rotary_dim + i % copied * 8;
    const bool key = h >= a.q_heads;
    const uint16_t* from = key ? k.from + (h - a.q_heads) * k.head : q.from + h * q.head;
    uint16_t* to = key ? k.to + (h - a.q_heads) * k.to_head : q.to + h * q.to_head;
    if (from != to) *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(from + at);
  }
}

// The same element by element, for rows and dimensions that do not come in 16-byte words.
__global__ void __launch_bounds__(kRopeThreads) rope_elements_kernel(const moe_rope_t a) {
  const int pairs = a.rotary_dim / 2, all_heads = a.q_heads + a.k_heads, rest = a.head_dim - a.rotary_dim;
  const int t = blockIdx.x, position = a.positions[t];
  const uint16_t* qf = static_cast<const uint16_t*>(a.q) + t * a.q_token_stride;
  const uint16_t* kf = static_cast<const uint16_t*>(a.k) + t * a.k_token_stride;
  uint16_t* qt = static_cast<uint16_t*>(a.q_out) + t * a.q_out_token_stride;
  uint16_t* kt = static_cast<uint16_t*>(a.k_out) + t * a.k_out_token_stride;
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) {
    float sin, cos;
    sin_cos(a.turns[i], position, a.amplitude, sin, cos);
    const int at0 = a.interleaved ? 2 * i : i, at1 = a.interleaved ? 2 * i + 1 : i + pairs;
    for (int h = blockIdx.y; h < all_heads; h += gridDim.y) {
      const bool key = h >= a.q_heads;
      const uint16_t* from = key ? kf + (h - a.q_heads) * a.k_head_stride : qf + h * a.q_head_stride;
      uint16_t* to = key ? kt + (h - a.q_heads) * a.k_out_head_stride : qt + h * a.q_out_head_stride;
      const float x = low(from[at0]), y = low(from[at1]);
      const uint32_t both = pack(first_of(x, y, sin, cos), second_of(x, y, sin, cos));
      to[at0] = static_cast<uint16_t>(both);
      to[at1] = static_cast<uint16_t>(both >> 16);
    }
  }
  for (int h = blockIdx.y; h < all_heads; h += gridDim.y) {
    const bool key = h >= a.q_heads;
    const uint16_t* from = key ? kf + (h - a.q_heads) * a.k_head_stride : qf + h * a.q_head_stride;
    uint16_t* to = key ? kt + (h - a.q_heads) * a.k_out_head_stride : qt + h * a.q_out_head_stride;
    if (from != to)
      for (int i = threadIdx.x; i < rest; i += kRopeThreads) to[a.rotary_dim + i] = from[a.rotary_dim + i];
  }
}

// A tensor's rows as an outer run of equally spaced blocks of bytes.
struct Blocks {
  int64_t at, stride, bytes, count;
};

Blocks blocks_of(const void* p, int64_t token, int64_t head, int tokens, int heads, int dim) {
  const int64_t x = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p));
  if (tokens == 1) token = (heads - 1) * head + dim;  // (any)
  if (heads == 1) head = dim;
  if (token >= head) return {x, 2 * token, 2 * ((heads - 1) * head + dim), tokens};
  return {x, 2 * head, 2 * ((tokens - 1) * token + dim), heads};
}

// Whether two tensors share bytes: blocks equally far apart may lie side by side, others only in separate ranges.
bool meet(const Blocks& a, const Blocks& b) {
  if (a.at >= b.at + (b.count - 1) * b.stride + b.bytes || b.at >= a.at + (a.count - 1) * a.stride + a.bytes) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  const int64_t off = ((b.at - a.at) % a.stride + a.stride) % a.stride;
  return off < a.bytes || a.stride - off < b.bytes;
}

// Whether a tensor's rows share bytes with each other.
bool folded(int64_t token, int64_t head, int tokens, int heads, int dim) {
  if (tokens == 1) return heads > 1 && head < dim;
  if (heads == 1) return token < dim;
  return token >= head ? head < dim || token < (heads - 1) * head + dim : token < dim || head < (tokens - 1) * token + dim;
}

}  // namespace

const char* rope_fault(const moe_rope_t* r) {
  if (r == nullptr) return "null argument";
  if (r->tokens < 0) return "tokens < 0";
  if (r->q_heads < 1 || r->q_heads > 1024 || r->k_heads < 0 || r->k_heads > 1024) return "heads out of range";
  if (r->head_dim < 2 || r->head_dim > MOE_ROPE_MAX_DIM) return "head_dim out of range";
  if (r->rotary_dim < 2 || r->rotary_dim % 2 != 0 || r->rotary_dim > r->head_dim) return "rotary_dim must be even, 2 .. head_dim";
  if (!(r->amplitude - r->amplitude == 0.0f)) return "amplitude not finite";
  if (r->q_token_stride < 0 || r->q_head_stride < 0 || r->k_token_stride < 0 || r->k_head_stride < 0 || r->q_out_token_stride < 0 ||
      r->q_out_head_stride < 0 || r->k_out_token_stride < 0 || r->k_out_head_stride < 0)
    return "strides must not be negative";
  if (r->tokens == 0) return nullptr;
  if (!r->positions || !r->turns || !r->q || !r->q_out || (r->k_heads && (!r->k || !r->k_out))) return "null pointer";
  const auto off = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (off(r->positions, 4) || off(r->turns, 8) || off(r->q, 2) || off(r->k, 2) || off(r->q_out, 2) || off(r->k_out, 2))
    return "misaligned pointer";
  const int T = r->tokens, D = r->head_dim;
  if (folded(r->q_out_token_stride, r->q_out_head_stride, T, r->q_heads, D) ||
      (r->k_heads && folded(r->k_out_token_stride, r->k_out_head_stride, T, r->k_heads, D)))
    return "an output's rows overlap";
  const bool q_same = r->q == r->q_out && r->q_token_stride == r->q_out_token_stride && r->q_head_stride == r->q_out_head_stride;
  const bool k_same = r->k == r->k_out && r->k_token_stride == r->k_out_token_stride && r->k_head_stride == r->k_out_head_stride;
  const Blocks q = blocks_of(r->q, r->q_token_stride, r->q_head_stride, T, r->q_heads, D);
  const Blocks qo = blocks_of(r->q_out, r->q_out_token_stride, r->q_out_head_stride, T, r->q_heads, D);
  const Blocks at = {static_cast<int64_t>(reinterpret_cast<uintptr_t>(r->positions)), 0, 4ll * T, 1};
  const Blocks table = {static_cast<int64_t>(reinterpret_cast<uintptr_t>(r->turns)), 0, 4ll * r->rotary_dim, 1};
  if ((!q_same && meet(q, qo)) || meet(at, qo) || meet(table, qo)) return "an output overlaps an input (only q_out may be q, k_out k)";
  if (r->k_heads) {
    const Blocks k = blocks_of(r->k, r->k_token_stride, r->k_head_stride, T, r->k_heads, D);
    const Blocks ko = blocks_of(r->k_out, r->k_out_token_stride, r->k_out_head_stride, T, r->k_heads, D);
    if ((!k_same && meet(k, ko)) || meet(q, ko) || meet(k, qo) || meet(at, ko) || meet(table, ko))
      return "an output overlaps an input (only q_out may be q, k_out k)";
    if (meet(qo, ko)) return "the outputs overlap";
  }
  return nullptr;
}

cudaError_t launch_rope(const moe_rope_t& a, cudaStream_t stream) {
  const auto words = [](const void* p, int64_t token, int64_t head) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && token % 8 == 0 && head % 8 == 0);
  };
  const int heads = a.q_heads + a.k_heads;
  const bool whole = a.rotary_dim % 16 == 0 && a.head_dim % 8 == 0 && words(a.q, a.q_token_stride, a.q_head_stride) &&
                     words(a.q_out, a.q_out_token_stride, a.q_out_head_stride) &&
                     (a.k_heads == 0 || (words(a.k, a.k_token_stride, a.k_head_stride) && words(a.k_out, a.k_out_token_stride, a.k_out_head_stride)));
  // Heads of one token shared out while there are fewer CTAs than are resident together.
  const auto parts = [&](int per) {
    int n = 1;
    while (n < heads && static_cast<int64_t>(a.tokens) * n < 152 * 8 && heads / n > per) n *= 2;
    return n;
  };
  if (!whole) {
    rope_elements_kernel<<<dim3(a.tokens, parts(1)), kRopeThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  int slots = 1;
  while (slots < a.rotary_dim / 16 && slots < 32) slots *= 2;
  const int groups = kRopeThreads / slots, n = parts(groups), per = (heads + n - 1) / n;
  const dim3 grid(a.tokens, (heads + per - 1) / per);
  if (a.interleaved) rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a, slots, per);
  else rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a, slots, per);
  return cudaGetLastError();
}

}  // namespace moe
