// Launchers of the decode step's kernels around the expert layer, used by
// decode_api.cu, and the argument structures that they take.
#pragma once

#include "common.cuh"

namespace moe {

struct AppendArgs {
  moe_kv_cache_t c;
  const uint16_t* x[2];      // keys, values: BF16 rows
  int64_t token_stride[2], head_stride[2];
  const int64_t* slots;
  int tokens;
};

struct AttendArgs {
  moe_kv_cache_t c;
  moe_kv_batch_t b;
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  int q_heads, group;        // group: query heads of one cache head
  int window;
  float scale;
  uint16_t* out;
  float* lse;
  uint8_t* workspace;
};

struct AttendMaps {
  CUtensorMap k, v;          // [pages * kv_heads][page_tokens][head_dim]; a box is a page's span of a head
};

cudaError_t launch_route(const moe_route_t& a, cudaStream_t stream);
cudaError_t launch_kv_plan(const moe_kv_plan_t& a, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_kv_attend(const AttendArgs& a, cudaStream_t stream);
cudaError_t launch_kv_attend_rows(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream);

// Sets this thread's error detail (moe_last_error_detail) and returns `status`.
int fail(int status, const char* format, ...);

}  // namespace moe
