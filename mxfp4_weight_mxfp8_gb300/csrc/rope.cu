// Rotary positions of queries and keys (moe_rope in include/moe.h).
//
// The angle of a pair is position * turns, a whole number of 2^-64 turns: the
// product modulo 2^64 drops whole turns exactly, and its upper half is that angle
// to 2^-32 of a turn, whatever the position; the table's own rounding, 2^-65, is
// 2^-34 of a turn at position 2^31. A CTA takes a token's heads, so the
// sines are computed once for all of them; every element is read and written once
// and the bytes bound it: 12592 tokens of 72 heads of 128, half of each turned,
// 464 MB, take 71 us, 6.5 TB/s, 96 % of a copy's rate (sines for each head anew made
// it 9 more). A decode step's 64 tokens are their launch, 2.6 us, heads shared out so that
// the GPU is full.
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

// A head's row is a number of units of two 16-byte words each: rotated ones (8 pairs), then copied ones, where the output is
// another tensor: 32 at most. `slots` lanes, a power of two, have one each, so a warp takes whole rows; the heads of a token
// go by in turn, `heads_per` of them to a CTA's y.
static_assert(MOE_ROPE_MAX_DIM <= 32 * 16, "a lane for every unit of a head");
template <bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const moe_rope_t a, int slots, int heads_per, int units) {
  __shared__ __align__(16) float s_sin[MOE_ROPE_MAX_DIM / 2], s_cos[MOE_ROPE_MAX_DIM / 2];
  const int pairs = a.rotary_dim / 2, rotated = pairs / 8, all_heads = a.q_heads + a.k_heads;
  const int u = threadIdx.x & (slots - 1), groups = kRopeThreads / slots, first = blockIdx.y * heads_per;
  const int last = min(first + heads_per, all_heads), t = blockIdx.x;
  const Rows q{static_cast<const uint16_t*>(a.q) + t * a.q_token_stride, static_cast<uint16_t*>(a.q_out) + t * a.q_out_token_stride,
               0, a.q_head_stride, 0, a.q_out_head_stride};
  const Rows k{static_cast<const uint16_t*>(a.k) + t * a.k_token_stride, static_cast<uint16_t*>(a.k_out) + t * a.k_out_token_stride,
               0, a.k_head_stride, 0, a.k_out_head_stride};
  const auto from_of = [&](int h) { return h >= a.q_heads ? k.from + (h - a.q_heads) * k.head : q.from + h * q.head; };
  const auto to_of = [&](int h) { return h >= a.q_heads ? k.to + (h - a.q_heads) * k.to_head : q.to + h * q.to_head; };
  const bool turned = u < rotated;
  const int at0 = !turned ? a.rotary_dim + (u - rotated) * 16 : kInterleaved ? u * 16 : u * 8;
  const int at1 = !turned || kInterleaved ? at0 + 8 : at0 + pairs;
  const bool has0 = u < units, has1 = has0 && at1 < a.head_dim;  // (a copied unit may be one word)
  // Two heads' elements are on their way while the sines are computed; then always the next two.
  int h = first + threadIdx.x / slots;
  uint4 x[2], y[2];
  const auto load = [&](int from) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (from + e * groups < last) {
        const uint16_t* p = from_of(from + e * groups);
        if (has0) x[e] = *reinterpret_cast<const uint4*>(p + at0);
        if (has1) y[e] = *reinterpret_cast<const uint4*>(p + at1);
      }
  };
  load(h);
  const int position = a.positions[t];
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) sin_cos(a.turns[i], position, a.amplitude, s_sin[i], s_cos[i]);
  __syncthreads();
  float sin[8], cos[8];
  if (turned) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<float4*>(sin + j) = *reinterpret_cast<const float4*>(s_sin + u * 8 + j);
      *reinterpret_cast<float4*>(cos + j) = *reinterpret_cast<const float4*>(s_cos + u * 8 + j);
    }
  }
  for (; h < last; h += 2 * groups) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (h + e * groups >= last) continue;
      uint4 xo = x[e], yo = y[e];
      if (turned) {
        const uint32_t xs[4] = {x[e].x, x[e].y, x[e].z, x[e].w}, ys[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
        uint32_t p[4], r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kInterleaved) {
            const float a0 = low(xs[j]), b0 = high(xs[j]), a1 = low(ys[j]), b1 = high(ys[j]);
            p[j] = pack(first_of(a0, b0, sin[j], cos[j]), second_of(a0, b0, sin[j], cos[j]));
            r[j] = pack(first_of(a1, b1, sin[4 + j], cos[4 + j]), second_of(a1, b1, sin[4 + j], cos[4 + j]));
          } else {
            const float a0 = low(xs[j]), a1 = high(xs[j]), b0 = low(ys[j]), b1 = high(ys[j]);
            p[j] = pack(first_of(a0, b0, sin[2 * j], cos[2 * j]), first_of(a1, b1, sin[2 * j + 1], cos[2 * j + 1]));
            r[j] = pack(second_of(a0, b0, sin[2 * j], cos[2 * j]), second_of(a1, b1, sin[2 * j + 1], cos[2 * j + 1]));
          }
        }
        xo = make_uint4(p[0], p[1], p[2], p[3]);
        yo = make_uint4(r[0], r[1], r[2], r[3]);
      }
      uint16_t* to = to_of(h + e * groups);
      if (!turned && to == from_of(h + e * groups)) continue;  // in place: as it is
      if (has0) *reinterpret_cast<uint4*>(to + at0) = xo;
      if (has1) *reinterpret_cast<uint4*>(to + at1) = yo;
    }
    load(h + 2 * groups);
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

// A tensor's rows: blocks of bytes, one to a token and head, in bytes from each other. (A table is one block.)
struct Spread {
  int64_t at, token, head, tokens, heads, bytes;
};

Spread table_of(const void* p, int64_t bytes) { return {static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), 0, 0, 1, 1, bytes}; }

Spread rows_of(const void* p, int64_t token, int64_t head, int64_t tokens, int64_t heads, int64_t dim) {
  Spread r{static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), 2 * token, 2 * head, tokens, heads, 2 * dim};
  if (r.heads > 1 && r.head == r.bytes) {  // one block
    r.bytes *= r.heads;
    r.heads = 1;
  }
  if (r.tokens == 1) r.token = 0;
  if (r.heads == 1) r.head = 0;
  return r;
}

// Whether a run of blocks of a_bytes meets one of b_bytes, `off` bytes further, by a difference of `low` .. `high` strides.
bool runs_meet(int64_t off, int64_t stride, int64_t low, int64_t high, int64_t a_bytes, int64_t b_bytes) {
  // The least d from `low` on that brings b's block past the end of what lies before a's.
  int64_t d = low;
  if (stride > 0) {
    const int64_t x = -b_bytes - off;  // off + d * stride > -b_bytes
    const int64_t least = (x >= 0 ? x / stride : -((-x + stride - 1) / stride)) + 1;
    if (least > d) d = least;
  }
  return d <= high && off + d * stride > -b_bytes && off + d * stride < a_bytes;
}

int64_t end_of(const Spread& r) { return r.at + (r.tokens - 1) * r.token + (r.heads - 1) * r.head + r.bytes; }

// Whether two tensors share bytes. Of rows whose tokens are equally far apart (heads side by side in a fused projection,
// in any order) exactly; of others only those in separate ranges are known not to.
bool meet(const Spread& a, const Spread& b) {
  if (a.at >= end_of(b) || b.at >= end_of(a)) return false;
  if (a.tokens > 1 && b.tokens > 1 && a.token != b.token) return true;
  const int64_t stride = a.tokens > 1 ? a.token : b.token, low = 1 - a.tokens, high = b.tokens - 1;
  if (a.head == b.head || a.heads == 1 || b.heads == 1) {
    const int64_t head = a.heads > 1 ? a.head : b.head;
    for (int64_t d = 1 - a.heads; d < b.heads; ++d)
      if (runs_meet(b.at - a.at + d * head, stride, low, high, a.bytes, b.bytes)) return true;
    return false;
  }
  for (int64_t i = 0; i < a.heads; ++i)
    for (int64_t j = 0; j < b.heads; ++j)
      if (runs_meet(b.at + j * b.head - a.at - i * a.head, stride, low, high, a.bytes, b.bytes)) return true;
  return false;
}

// Whether a tensor's rows share bytes with each other.
bool folded(const Spread& r) {
  if (r.tokens > 1 && r.token < r.bytes) return true;
  for (int64_t d = 1; d < r.heads; ++d)
    if (runs_meet(d * r.head, r.token, 1 - r.tokens, r.tokens - 1, r.bytes, r.bytes)) return true;
  return false;
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
  const Spread q = rows_of(r->q, r->q_token_stride, r->q_head_stride, T, r->q_heads, D);
  const Spread qo = rows_of(r->q_out, r->q_out_token_stride, r->q_out_head_stride, T, r->q_heads, D);
  const Spread at = table_of(r->positions, 4ll * T), table = table_of(r->turns, 4ll * r->rotary_dim);
  const bool q_same = r->q == r->q_out && r->q_token_stride == r->q_out_token_stride && r->q_head_stride == r->q_out_head_stride;
  if (folded(qo)) return "an output's rows overlap";
  if ((!q_same && meet(q, qo)) || meet(at, qo) || meet(table, qo)) return "an output overlaps an input (only q_out may be q, k_out k)";
  if (r->k_heads) {
    const Spread k = rows_of(r->k, r->k_token_stride, r->k_head_stride, T, r->k_heads, D);
    const Spread ko = rows_of(r->k_out, r->k_out_token_stride, r->k_out_head_stride, T, r->k_heads, D);
    const bool k_same = r->k == r->k_out && r->k_token_stride == r->k_out_token_stride && r->k_head_stride == r->k_out_head_stride;
    if (folded(ko)) return "an output's rows overlap";
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
  // Nothing is copied in place.
  const bool copies = a.q != a.q_out || (a.k_heads && a.k != a.k_out);
  const int units = a.rotary_dim / 16 + (copies ? (a.head_dim - a.rotary_dim + 15) / 16 : 0);
  int slots = 1;
  while (slots < units) slots *= 2;
  const int groups = kRopeThreads / slots, n = parts(groups), per = (heads + n - 1) / n;
  const dim3 grid(a.tokens, (heads + per - 1) / per);
  if (a.interleaved) rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a, slots, per, units);
  else rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a, slots, per, units);
  return cudaGetLastError();
}

}  // namespace moe
