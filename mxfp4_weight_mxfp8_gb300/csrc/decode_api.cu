// C entries of the decode step around the layer: argument checks, launches.
#include <cmath>

#include "decode.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  return moe::fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int refuse(const char* what) { return moe::fail(MOE_ERR_ARG, "%s", what); }

bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

const char* cache_fault(const moe_kv_cache_t* c) {
  if (c == nullptr || !c->k || !c->v || !c->k_scale || !c->v_scale) return "null cache pointer";
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return "cache not 16-byte aligned";
  if (c->pages < 1 || c->kv_heads < 1 || c->kv_heads > 1024) return "cache pages or heads out of range";
  if (static_cast<int64_t>(c->pages) * c->kv_heads > 0x7FFFFFFF) return "pages * kv_heads past 2^31";
  if (!page_size_ok(c->page_tokens)) return "page_tokens must be 16, 32, 64 or 128";
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return "head_dim must be 64, 128 or 256";
  return nullptr;
}

// Strides of BF16 rows read with 16-byte loads.
bool strides_ok(int64_t token, int64_t head) {
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0;
}

}  // namespace

extern "C" {

int moe_route(const moe_route_t* r, void* stream) {
  if (r == nullptr) return refuse("null argument");
  if (r->tokens < 0) return refuse("tokens < 0");
  if (r->experts < 1 || r->experts > MOE_MAX_EXPERTS) return refuse("experts out of range");
  if (r->topk < 1 || r->topk > MOE_ROUTE_MAX_TOPK || r->topk > r->experts)
    return refuse("topk out of range");
  if (r->dtype != MOE_F32 && r->dtype != MOE_BF16 && r->dtype != MOE_F16)
    return refuse("dtype of the logits");
  if (r->scoring != MOE_SCORE_SOFTMAX && r->scoring != MOE_SCORE_SIGMOID) return refuse("scoring");
  if (r->groups < 1 || r->groups > MOE_ROUTE_MAX_GROUPS || r->experts % r->groups != 0)
    return refuse("groups must divide experts, at most 32");
  if (r->group_topk < 1 || r->group_topk > r->groups) return refuse("group_topk out of range");
  if (r->group_score != 1 && r->group_score != 2) return refuse("group_score must be 1 or 2");
  if (r->groups > 1 && r->group_score == 2 && r->experts / r->groups < 2)
    return refuse("group_score 2 needs two experts to a group");
  if (r->row_stride < r->experts) return refuse("row_stride < experts");
  if (!std::isfinite(r->scale)) return refuse("scale not finite");
  if (r->tokens == 0) return MOE_OK;
  if (!r->logits || !r->ids || !r->weights) return refuse("null pointer");
  if (!aligned(r->logits, r->dtype == MOE_F32 ? 4 : 2) || !aligned(r->bias, 4) ||
      !aligned(r->ids, 4) || !aligned(r->weights, 4))
    return refuse("misaligned pointer");
  return launched(moe::launch_route(*r, static_cast<cudaStream_t>(stream)), "moe_route");
}

int moe_kv_plan(const moe_kv_plan_t* p, void* stream) {
  if (p == nullptr) return refuse("null argument");
  if (p->requests < 1 || p->requests > MOE_KV_MAX_REQUESTS) return refuse("requests out of range");
  if (!page_size_ok(p->page_tokens)) return refuse("page_tokens must be 16, 32, 64 or 128");
  if (p->tokens < 0 || p->free_count < 0 || p->table_width < 1 || p->table_stride < p->table_width)
    return refuse("tokens, free_count or table size out of range");
  if (!p->context_lens || !p->query_lens || !p->free_head || !p->block_table || !p->query_start ||
      !p->seq_lens || !p->counts || (p->tokens && (!p->positions || !p->slots)) ||
      (p->free_count && !p->free_pages))
    return refuse("null pointer");
  if (!aligned(p->context_lens, 4) || !aligned(p->query_lens, 4) || !aligned(p->free_pages, 4) ||
      !aligned(p->free_head, 4) || !aligned(p->block_table, 4) || !aligned(p->query_start, 4) ||
      !aligned(p->seq_lens, 4) || !aligned(p->positions, 4) || !aligned(p->slots, 8) ||
      !aligned(p->counts, 4))
    return refuse("misaligned pointer");
  if (p->free_head >= p->counts && p->free_head < p->counts + 4)
    return refuse("free_head must not lie in this call's counts");
  // Every CTA reads the inputs for itself, some when others have written: only lengths stepped in place are provided for.
  const int64_t per = 4ll * p->requests;
  const struct { const void* at; int64_t bytes; } in[] = {{p->context_lens, per}, {p->query_lens, per}, {p->free_pages, 4ll * p->free_count}, {p->free_head, 4}},
      out[] = {{p->query_start, per + 4}, {p->seq_lens, per}, {p->positions, 4ll * p->tokens}, {p->slots, 8ll * p->tokens}, {p->counts, 16}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (overlap(o.at, o.bytes, i.at, i.bytes) && !(o.at == p->seq_lens && i.at == p->context_lens && p->seq_lens == p->context_lens))
        return refuse("an output overlaps an input (only seq_lens may be context_lens)");
  return launched(moe::launch_kv_plan(*p, static_cast<cudaStream_t>(stream)), "moe_kv_plan");
}

int moe_kv_append(const moe_kv_cache_t* cache, const void* k, int64_t k_token_stride,
                  int64_t k_head_stride, const void* v, int64_t v_token_stride,
                  int64_t v_head_stride, const int64_t* slots, int tokens, void* stream) {
  if (const char* fault = cache_fault(cache)) return refuse(fault);
  if (tokens < 0) return refuse("tokens < 0");
  if (!strides_ok(k_token_stride, k_head_stride) || !strides_ok(v_token_stride, v_head_stride))
    return refuse("strides must be multiples of 8 elements, not negative");
  if (tokens == 0) return MOE_OK;
  if (!k || !v || !slots) return refuse("null pointer");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return refuse("misaligned pointer");
  moe::AppendArgs a{};
  a.c = *cache;
  a.x[0] = static_cast<const uint16_t*>(k);
  a.x[1] = static_cast<const uint16_t*>(v);
  a.token_stride[0] = k_token_stride;
  a.token_stride[1] = v_token_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  a.slots = slots;
  a.tokens = tokens;
  return launched(moe::launch_kv_append(a, static_cast<cudaStream_t>(stream)), "moe_kv_append");
}

int moe_kv_attend(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, const void* q,
                  int64_t q_token_stride, int64_t q_head_stride, int q_heads, float scale,
                  int window, void* out, float* lse, void* workspace, void* stream) {
  if (const char* fault = cache_fault(cache)) return refuse(fault);
  if (batch == nullptr) return refuse("null argument");
  if (batch->requests < 1 || batch->requests > MOE_KV_MAX_REQUESTS)
    return refuse("requests out of range");
  if (batch->tokens < 0 || batch->table_width < 1 || batch->table_stride < batch->table_width)
    return refuse("tokens or table size out of range");
  if (q_heads < 1 || q_heads > 1024 || q_heads % cache->kv_heads != 0)
    return refuse("q_heads must be a multiple of kv_heads, at most 1024");
  if (!strides_ok(q_token_stride, q_head_stride))
    return refuse("strides must be multiples of 8 elements, not negative");
  if (window < 0) return refuse("window < 0");
  if (!std::isfinite(scale)) return refuse("scale not finite");
  if (batch->tokens == 0) return MOE_OK;
  if (!batch->block_table || !batch->query_start || !batch->seq_lens || !q || !out || !workspace)
    return refuse("null pointer");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4) ||
      !aligned(batch->block_table, 4) || !aligned(batch->query_start, 4) ||
      !aligned(batch->seq_lens, 4))
    return refuse("misaligned pointer");
  moe::AttendArgs a{};
  a.c = *cache;
  a.b = *batch;
  a.q = static_cast<const uint16_t*>(q);
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.q_heads = q_heads;
  a.group = q_heads / cache->kv_heads;
  a.window = window;
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.workspace = static_cast<uint8_t*>(workspace);
  return launched(moe::launch_kv_attend(a, static_cast<cudaStream_t>(stream)), "moe_kv_attend");
}

int moe_kv_sync_status(void* workspace, void* stream) {
  if (workspace == nullptr || !aligned(workspace, 16)) return refuse("null or misaligned workspace");
  int32_t status = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&status, workspace, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && status != MOE_OK) {
    e = cudaMemsetAsync(workspace, 0, MOE_KV_WORKSPACE_HEADER, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e == cudaSuccess ? status : launched(e, "moe_kv_sync_status");
}

int moe_kv_set_timeout(void* workspace, uint64_t nanoseconds, void* stream) {
  if (workspace == nullptr || !aligned(workspace, 16)) return refuse("null or misaligned workspace");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(static_cast<uint8_t*>(workspace) + 8, &nanoseconds, 8, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return launched(e, "moe_kv_set_timeout");
}

int moe_kv_debug_withhold(void* workspace, int cta, void* stream) {
  if (workspace == nullptr || !aligned(workspace, 16)) return refuse("null or misaligned workspace");
  if (cta < -1) return refuse("cta < -1");
  const int32_t word = cta + 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(static_cast<uint8_t*>(workspace) + 4, &word, 4, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return launched(e, "moe_kv_debug_withhold");
}

}  // extern "C"
