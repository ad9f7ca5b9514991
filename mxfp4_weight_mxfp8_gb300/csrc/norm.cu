// Residual addition and root-mean-square norm, with outputs in 16 or 32 bits
// and in MXFP8 (moe_norm in include/moe.h).
//
// One pass: a row stays in registers between its sum of squares and its
// outputs, so each input is read once and each output written once, and the
// bytes bound it: 16381 rows of 3584 in BF16 with residual and all outputs, 530 MB,
// take 79 us, 6.7 TB/s, 99 % of a copy's rate. A thread holds chunks of 8 elements;
// a row of up to 1024 is a warp's, without a barrier, a longer one a CTA's, with one
// (one row of 3584: 2.5 us, a launch). Four neighbouring lanes hold a block of 32,
// whose largest magnitude takes two shuffles.
#include <cuda_fp16.h>

#include <cmath>

#include "decode.h"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kChunk = 8;  // elements

// Eight elements as they lie in memory: 16 bytes of a 16-bit type, 32 of FP32.
template <int kWords>
struct Raw {
  uint4 w[kWords > 0 ? kWords : 1];
};

// Elements i .. i + 7 of a row of n; those from n on are zero. kReadOnly: of memory that the kernel does not write (x and the
// residual may be outputs too).
template <int kWords, bool kVector, bool kReadOnly = false>
__device__ __forceinline__ Raw<kWords> load(const void* row, int i, int n) {
  Raw<kWords> r;
  if constexpr (kVector) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + static_cast<int64_t>(i) * 2 * kWords);
#pragma unroll
    for (int j = 0; j < kWords; ++j) r.w[j] = i >= n ? make_uint4(0, 0, 0, 0) : kReadOnly ? __ldg(p + j) : p[j];
  } else if constexpr (kWords == 1) {
    const uint16_t* p = static_cast<const uint16_t*>(row) + i;
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = (i + 2 * j < n ? p[2 * j] : 0u) | (i + 2 * j + 1 < n ? static_cast<uint32_t>(p[2 * j + 1]) << 16 : 0u);
    r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(row) + i;
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < n ? p[j] : 0u;
    r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
    r.w[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
  return r;
}

template <int kWords>
__device__ __forceinline__ void unpack(const Raw<kWords>& r, bool half, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const uint32_t w[4] = {r.w[j].x, r.w[j].y, r.w[j].z, r.w[j].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (kWords == 2) {
        v[4 * j + k] = __uint_as_float(w[k]);
      } else if (half) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      } else {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  }
}

// Elements i .. i + 7 into a row of n, rounded to its type.
template <int kWords, bool kVector>
__device__ __forceinline__ void store(void* row, int i, int n, bool half, const float (&v)[8]) {
  uint32_t w[4 * kWords];
#pragma unroll
  for (int j = 0; j < 4 * kWords; ++j) {
    if constexpr (kWords == 2) {
      w[j] = __float_as_uint(v[j]);
    } else if (half) {
      const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  if constexpr (kVector) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(row) + static_cast<int64_t>(i) * 2 * kWords);
#pragma unroll
    for (int j = 0; j < kWords; ++j) p[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  } else if constexpr (kWords == 1) {
    uint16_t* p = static_cast<uint16_t*>(row) + i;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[j] = static_cast<uint16_t>(w[j / 2] >> (j % 2 * 16));
  } else {
    uint32_t* p = static_cast<uint32_t*>(row) + i;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[j] = w[j];
  }
}

// The weights of elements i .. i + 7.
template <bool kVector>
__device__ __forceinline__ void load_weight(const moe_norm_t& a, int i, float (&v)[8]) {
  if (a.weight_dtype == MOE_F32)
    unpack(load<2, kVector, true>(a.weight, i, a.hidden), false, v);
  else
    unpack(load<1, kVector, true>(a.weight, i, a.hidden), a.weight_dtype == MOE_F16, v);
}

// The sum over a row's threads: a warp's, or the CTA's through `red`.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float x, float* red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  if constexpr (!kWarpRow) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = lane < warps ? red[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  }
  return x;
}

template <bool kWarpRow>
__device__ __forceinline__ float row_max(float x, float* red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  if constexpr (!kWarpRow) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = lane < warps ? red[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  }
  return x;
}

// XW, RW: 16-byte words of a chunk of x, of the residual (0: none). kHeld: chunks that a thread holds.
template <int XW, int RW, int kHeld, bool kVector, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 128 : 1024) norm_kernel(const moe_norm_t a) {
  __shared__ float red[kWarpRow ? 1 : 3][32];
  const int lane = threadIdx.x & 31, step = kWarpRow ? 32 : blockDim.x, at = kWarpRow ? lane : threadIdx.x;
  const int64_t t = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= a.tokens) return;
  const bool half = a.dtype == MOE_F16, res_half = a.residual_dtype == MOE_F16;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.x_stride * (2 * XW);
  const uint8_t* residual = static_cast<const uint8_t*>(a.residual) + (RW ? t * a.residual_stride * (2 * RW) : 0);

  Raw<XW> xr[kHeld];
  Raw<RW> rr[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int i = (j * step + at) * kChunk;
    xr[j] = load<XW, kVector>(x, i, a.hidden);
    if constexpr (RW > 0) rr[j] = load<RW, kVector>(residual, i, a.hidden);
  }
  float h[kHeld][8], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    unpack(xr[j], half, h[j]);
    if constexpr (RW > 0) {
      float r[8];
      unpack(rr[j], res_half, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[j][k] += r[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(h[j][k], h[j][k], sum);
  }
  sum = row_sum<kWarpRow>(sum, red[0]);
  if (a.residual_out != nullptr) {
    const int size = a.residual_dtype == MOE_F32 ? 4 : 2;
    uint8_t* to = static_cast<uint8_t*>(a.residual_out) + t * a.residual_out_stride * size;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = (j * step + at) * kChunk;
      if (i >= a.hidden) continue;
      if (size == 4) store<2, kVector>(to, i, a.hidden, false, h[j]);
      else store<1, kVector>(to, i, a.hidden, res_half, h[j]);
    }
  }
  const float n = static_cast<float>(a.hidden);
  float eps = a.eps;
  if (!(sum < INFINITY)) {
    // Past FP32's range (or not finite): the row times a power of two that brings its largest magnitude to [1, 2).
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(h[j][k]));
    top = row_max<kWarpRow>(top, red[kWarpRow ? 0 : 1]);
    if (top < INFINITY) {  // (a NaN stays one in the sum)
      const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      const float down = pow2f(-e);
      sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[j][k] *= down;
          sum = fmaf(h[j][k], h[j][k], sum);
        }
      sum = row_sum<kWarpRow>(sum, red[kWarpRow ? 0 : 2]);
      eps *= down;
      eps *= down;
    }
  }
  const float r = rsqrtf(sum / n + eps);
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int c = j * step + at, i = c * kChunk;
    const bool in = i < a.hidden;
    float y[8];
    {
      float w[8];
      load_weight<kVector>(a, i, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = h[j][k] * r * (w[k] + a.weight_offset);
    }
    if (a.out != nullptr && in)
      store<XW, kVector>(static_cast<uint8_t*>(a.out) + t * a.out_stride * (2 * XW), i, a.hidden, half, y);
    if (a.codes != nullptr) {
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(y[k]));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      if (!in) continue;  // (blocks of 32 are in or out as a whole)
      const int E = mx_exponent(top, false);
      const float inv = pow2f(-E);
      uint32_t code[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        code[k] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * k] * inv, y[2 * k + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint2*>(a.codes + t * a.hidden + i) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
      if ((c & 3) == 0) a.scales[t * (a.hidden / kBlock) + c / 4] = static_cast<uint8_t>(E + 127);
    }
  }
}

template <int XW, int RW, bool kVector>
cudaError_t launch_row(const moe_norm_t& a, cudaStream_t stream) {
  const int chunks = (a.hidden + kChunk - 1) / kChunk;
  if (chunks <= 128) {
    // A warp to a row, four rows to a CTA.
    const int grid = a.tokens / 4 + (a.tokens % 4 != 0);
    if (!kVector || chunks > 64) norm_kernel<XW, RW, 4, kVector, true><<<grid, 128, 0, stream>>>(a);
    else if (chunks > 32) norm_kernel<XW, RW, 2, true, true><<<grid, 128, 0, stream>>>(a);
    else norm_kernel<XW, RW, 1, true, true><<<grid, 128, 0, stream>>>(a);
  } else {
    const int threads = (chunks + 63) / 64 * 32;
    norm_kernel<XW, RW, 2, kVector, false><<<a.tokens, threads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <int XW, int RW>
cudaError_t launch_words(const moe_norm_t& a, bool vector, cudaStream_t stream) {
  return vector ? launch_row<XW, RW, true>(a, stream) : launch_row<XW, RW, false>(a, stream);
}

template <int XW>
cudaError_t launch_x(const moe_norm_t& a, bool vector, cudaStream_t stream) {
  if (a.residual == nullptr) return launch_words<XW, 0>(a, vector, stream);
  return a.residual_dtype == MOE_F32 ? launch_words<XW, 2>(a, vector, stream) : launch_words<XW, 1>(a, vector, stream);
}

int size_of(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// Rows that start on 16-byte boundaries (null: nothing to read or write).
bool whole_words(const void* p, int64_t stride, int dtype, int tokens) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (tokens == 1 || stride * size_of(dtype) % 16 == 0));
}

struct Span {
  const void* p;
  int64_t stride, bytes;  // of a row and the next one; of a row
};

// Whether rows of two tensors share bytes. Rows equally far apart may lie side by side (columns of one buffer); of others
// only those in separate ranges are known not to meet.
bool meet(const Span& a, const Span& b, int64_t rows) {
  if (a.p == nullptr || b.p == nullptr) return false;
  const int64_t x = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p)), y = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p));
  if (x >= y + (rows - 1) * b.stride + b.bytes || y >= x + (rows - 1) * a.stride + a.bytes) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  const int64_t off = ((y - x) % a.stride + a.stride) % a.stride;
  return off < a.bytes || a.stride - off < b.bytes;
}

}  // namespace

const char* norm_fault(const moe_norm_t* n, bool plan) {
  if (n == nullptr) return "null argument";
  if (n->tokens < 0) return "tokens < 0";
  if (n->hidden < 1 || n->hidden > MOE_MAX_HIDDEN) return "hidden out of range";
  const auto known = [](int d) { return d == MOE_F32 || d == MOE_BF16 || d == MOE_F16; };
  if (!known(n->dtype) || !known(n->weight_dtype) || ((n->residual || n->residual_out) && !known(n->residual_dtype)))
    return "dtype of x, residual or weight";
  if (!(n->eps >= 1e-30f) || !std::isfinite(n->eps) || !std::isfinite(n->weight_offset)) return "eps must be finite and at least 1e-30, weight_offset finite";
  if ((n->codes == nullptr) != (n->scales == nullptr)) return "codes and scales come together";
  if (plan && n->codes) return "codes and scales are the handle's";
  if ((n->codes || plan) && n->hidden % kBlock != 0) return "MXFP8 needs hidden to be a multiple of 32";
  if (n->x_stride < 0 || (n->residual && n->residual_stride < 0)) return "strides must not be negative";
  if ((n->out && n->out_stride < n->hidden) || (n->residual_out && n->residual_out_stride < n->hidden))
    return "an output's rows overlap (stride < hidden)";
  if (n->tokens == 0) return nullptr;
  if (!n->x || !n->weight || (!n->out && !n->codes && !plan)) return "null pointer (x, weight, and out or codes)";
  const auto off = [](const void* p, uintptr_t k) { return (reinterpret_cast<uintptr_t>(p) & (k - 1)) != 0; };
  if (off(n->x, size_of(n->dtype)) || off(n->out, size_of(n->dtype)) || off(n->weight, size_of(n->weight_dtype)) ||
      off(n->residual, size_of(n->residual_dtype)) || off(n->residual_out, size_of(n->residual_dtype)) || off(n->codes, 8))
    return "misaligned pointer";
  const int64_t w = size_of(n->dtype), r = size_of(n->residual_dtype), h = n->hidden;
  const Span in[] = {{n->x, n->x_stride * w, h * w}, {n->residual, n->residual_stride * r, h * r}, {n->weight, 0, h * size_of(n->weight_dtype)}};
  const Span out[] = {{n->out, n->out_stride * w, h * w}, {n->residual_out, n->residual_out_stride * r, h * r}, {n->codes, h, h}, {n->scales, h / kBlock, h / kBlock}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i)
      if (!(o == i && o < 2 && out[o].p == in[i].p && (out[o].stride == in[i].stride || n->tokens == 1)) && meet(out[o], in[i], n->tokens))
        return "an output overlaps an input (only out may be x, residual_out residual)";
    for (int i = 0; i < o; ++i)
      if (meet(out[o], out[i], n->tokens)) return "two outputs overlap";
  }
  return nullptr;
}

cudaError_t launch_norm(const moe_norm_t& a, cudaStream_t stream) {
  const bool vector = a.hidden % kChunk == 0 && whole_words(a.x, a.x_stride, a.dtype, a.tokens) &&
                      whole_words(a.out, a.out_stride, a.dtype, a.tokens) && whole_words(a.weight, 0, a.weight_dtype, 1) &&
                      whole_words(a.residual, a.residual_stride, a.residual_dtype, a.tokens) &&
                      whole_words(a.residual_out, a.residual_out_stride, a.residual_dtype, a.tokens);
  return a.dtype == MOE_F32 ? launch_x<2>(a, vector, stream) : launch_x<1>(a, vector, stream);
}

}  // namespace moe
