// C entries of the decode step around the layer: argument checks, launches.
#include <cmath>

#include "decode.h"
#include "twice.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

// A range of an argument's bytes.
struct Bytes {
  const void* at;
  int64_t bytes;
};

bool overlap(const Bytes& a, const Bytes& b) { return overlap(a.at, a.bytes, b.at, b.bytes); }

// Bytes of a table of int32 rows, from its first row's first to its last row's last.
int64_t table_bytes(int rows, int64_t stride, int width) { return 4 * ((rows - 1) * stride + width); }

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

// The arguments of an attend call (null: nothing to refuse).
const char* attend_args(moe::AttendArgs* a, const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, const void* q, int64_t q_token_stride,
                        int64_t q_head_stride, int q_heads, float scale, int window, void* out, float* lse, void* workspace) {
  if (const char* fault = cache_fault(cache)) return fault;
  if (batch == nullptr) return "null argument";
  if (batch->requests < 1 || batch->requests > MOE_KV_MAX_REQUESTS) return "requests out of range";
  if (batch->tokens < 0 || batch->table_width < 1 || batch->table_stride < batch->table_width) return "tokens or table size out of range";
  if (q_heads < 1 || q_heads > 1024 || q_heads % cache->kv_heads != 0) return "q_heads must be a multiple of kv_heads, at most 1024";
  if (!strides_ok(q_token_stride, q_head_stride)) return "strides must be multiples of 8 elements, not negative";
  if (window < 0) return "window < 0";
  if (!std::isfinite(scale)) return "scale not finite";
  if (batch->tokens == 0) return nullptr;
  if (!batch->block_table || !batch->query_start || !batch->seq_lens || !q || !out || !workspace) return "null pointer";
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4) || !aligned(batch->block_table, 4) ||
      !aligned(batch->query_start, 4) || !aligned(batch->seq_lens, 4))
    return "misaligned pointer";
  a->c = *cache;
  a->b = *batch;
  a->q = static_cast<const uint16_t*>(q);
  a->q_token_stride = q_token_stride;
  a->q_head_stride = q_head_stride;
  a->q_heads = q_heads;
  a->group = q_heads / cache->kv_heads;
  a->window = window;
  a->scale = scale;
  a->out = static_cast<uint16_t*>(out);
  a->lse = lse;
  a->workspace = static_cast<uint8_t*>(workspace);
  return nullptr;
}

// x modulo 1 in units of 2^-64, rounded, modulo 2^64.
uint64_t fraction_of(moe::Twice x) {
  if (!std::isfinite(x.hi)) return 0;
  const auto whole = [&] {  // of x, which keeps the rest, 0 .. 1
    double n = std::floor(x.hi);
    x = moe::quick_sum(x.hi - n, x.lo);
    if (x.hi < 0.0) {
      n -= 1.0;
      x = x + 1.0;
    }
    return n;
  };
  whole();
  x = moe::times_two_to(x, 32);
  const uint64_t upper = static_cast<uint64_t>(whole());
  x = moe::times_two_to(x, 32);
  const uint64_t lower = static_cast<uint64_t>(whole());
  return (upper << 32) + lower + (x.hi >= 0.5 ? 1 : 0);
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

int moe_norm(const moe_norm_t* n, void* stream) {
  if (const char* fault = moe::norm_fault(n, false)) return refuse(fault);
  if (n->tokens == 0) return MOE_OK;
  return launched(moe::launch_norm(*n, static_cast<cudaStream_t>(stream)), "moe_norm");
}

int moe_rope(const moe_rope_t* r, void* stream) {
  if (const char* fault = moe::rope_fault(r)) return refuse(fault);
  if (r->tokens == 0) return MOE_OK;
  return launched(moe::launch_rope(*r, static_cast<cudaStream_t>(stream)), "moe_rope");
}

int moe_rope_turns(int rotary_dim, double base, int scaling, double factor, double trained, double low, double high,
                   uint64_t* turns) {
  if (turns == nullptr) return refuse("null pointer");
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > MOE_ROPE_MAX_DIM) return refuse("rotary_dim out of range");
  if (!(base > 1.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor)) return refuse("base or factor out of range");
  if (scaling != MOE_ROPE_LINEAR && scaling != MOE_ROPE_BANDS && scaling != MOE_ROPE_RAMP) return refuse("scaling");
  if (scaling != MOE_ROPE_LINEAR && (!(trained > 0.0) || !std::isfinite(trained) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return refuse("trained, low or high out of range");
  // The pair that turns n times over the trained length: trained * base^(-2i / rotary_dim) = tau n.
  const auto index = [&](double n) { return rotary_dim * std::log(trained / (moe::kTau.hi * n)) / (2.0 * std::log(base)); };
  double from = 0.0, to = 1.0;
  if (scaling == MOE_ROPE_RAMP) {
    from = std::fmax(std::floor(index(high)), 0.0);
    to = std::fmin(std::ceil(index(low)), rotary_dim - 1.0);
    if (to <= from) to = from + 0.001;  // a step
  }
  // From here on with twice a double's bits: a table of 64 is read at positions up to 2^31.
  const moe::Twice rate = moe::log_of(base) / moe::Twice(rotary_dim);
  for (int i = 0; i < rotary_dim / 2; ++i) {
    moe::Twice f = i ? moe::exp_of(rate * (-2.0 * i)) : 1.0, keep = 0.0;
    if (scaling == MOE_ROPE_BANDS) keep = (f / moe::kTau * trained - low) / (moe::Twice(high) - low);
    if (scaling == MOE_ROPE_RAMP) keep = moe::Twice(1.0) - moe::Twice(i - from) / (moe::Twice(to) - from);
    keep = keep.hi > 1.0 ? 1.0 : keep.hi > 0.0 ? keep : 0.0;
    f = f * keep + f / factor * (moe::Twice(1.0) - keep);
    turns[i] = fraction_of(f / moe::kTau);
  }
  return MOE_OK;
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

int moe_kv_fork(const moe_kv_fork_t* f, void* stream) {
  if (f == nullptr) return refuse("null argument");
  if (f->requests < 1 || f->requests > MOE_KV_MAX_REQUESTS || f->rows < 1 || f->rows > MOE_KV_MAX_REQUESTS)
    return refuse("requests or rows out of range");
  if (!page_size_ok(f->page_tokens)) return refuse("page_tokens must be 16, 32, 64 or 128");
  if (f->free_count < 0 || f->table_width < 1 || f->table_width > 1 << 30 || f->table_stride < f->table_width || f->out_stride < f->table_width)
    return refuse("free_count or table size out of range");
  if (!f->parents || !f->block_table || !f->seq_lens || !f->free_head || !f->out_table || !f->out_lens || !f->moves || !f->counts ||
      (f->free_count && !f->free_pages))
    return refuse("null pointer");
  const Bytes in[] = {{f->parents, 4ll * f->requests}, {f->block_table, table_bytes(f->rows, f->table_stride, f->table_width)},
                      {f->seq_lens, 4ll * f->rows}, {f->free_pages, 4ll * f->free_count}, {f->free_head, 4}};
  const Bytes out[] = {{f->out_table, table_bytes(f->requests, f->out_stride, f->table_width)}, {f->out_lens, 4ll * f->requests},
                       {f->moves, 12ll * f->requests}, {f->counts, 16}};
  for (const Bytes& o : out) {
    if (!aligned(o.at, 4)) return refuse("misaligned pointer");
    for (const Bytes& i : in)
      if (overlap(o, i)) return refuse("an output overlaps an input");
    for (const Bytes& p : out)
      if (&p != &o && overlap(o, p)) return refuse("two outputs overlap");
  }
  for (const Bytes& i : in)
    if (!aligned(i.at, 4)) return refuse("misaligned pointer");
  return launched(moe::launch_kv_fork(*f, static_cast<cudaStream_t>(stream)), "moe_kv_fork");
}

int moe_kv_copy(const moe_kv_cache_t* cache, const int32_t* moves, const int32_t* count, int capacity, void* stream) {
  if (const char* fault = cache_fault(cache)) return refuse(fault);
  if (capacity < 0) return refuse("capacity < 0");
  if (capacity == 0) return MOE_OK;
  if (!moves) return refuse("null pointer");
  if (!aligned(moves, 4) || !aligned(count, 4)) return refuse("misaligned pointer");
  return launched(moe::launch_kv_copy(*cache, moves, count, capacity, static_cast<cudaStream_t>(stream)), "moe_kv_copy");
}

int moe_kv_reclaim(const moe_kv_reclaim_t* r, void* stream) {
  if (r == nullptr) return refuse("null argument");
  if (r->requests < 1 || r->requests > MOE_KV_MAX_REQUESTS) return refuse("requests out of range");
  if (!page_size_ok(r->page_tokens)) return refuse("page_tokens must be 16, 32, 64 or 128");
  if (r->pages < 1 || r->pages > 1 << 30) return refuse("pages out of range");
  if (r->table_width < 1 || r->table_width > 1 << 30 || r->table_stride < r->table_width) return refuse("table size out of range");
  if ((r->out_table == nullptr) != (r->moves == nullptr)) return refuse("out_table and moves come together");
  if (r->out_table && r->out_stride < r->table_width) return refuse("table size out of range");
  if (!r->block_table || !r->seq_lens || !r->free_pages || !r->counts || !r->workspace) return refuse("null pointer");
  if (!aligned(r->workspace, 16)) return refuse("misaligned pointer");
  const int64_t table = table_bytes(r->requests, r->table_stride, r->table_width);
  const Bytes in[] = {{r->block_table, table}, {r->seq_lens, 4ll * r->requests}};
  const Bytes out[] = {{r->free_pages, 4ll * r->pages}, {r->counts, 16},
                       {r->workspace, static_cast<int64_t>(MOE_KV_RECLAIM_BYTES(r->pages))},
                       {r->moves, r->moves ? 12ll * (r->pages > 1 ? r->pages / 2 : 1) : 0},
                       {r->out_table, r->out_table ? table_bytes(r->requests, r->out_stride, r->table_width) : 0}};
  const bool in_place = r->out_table == r->block_table && r->out_stride == r->table_stride;
  for (const Bytes& o : out) {
    if (!aligned(o.at, 4)) return refuse("misaligned pointer");
    for (const Bytes& i : in)
      if (overlap(o, i) && !(in_place && o.at == r->out_table && i.at == r->block_table))
        return refuse("an output overlaps an input (only out_table may be block_table)");
    for (const Bytes& p : out)
      if (&p != &o && overlap(o, p)) return refuse("two outputs overlap");
  }
  for (const Bytes& i : in)
    if (!aligned(i.at, 4)) return refuse("misaligned pointer");
  return launched(moe::launch_kv_reclaim(*r, static_cast<cudaStream_t>(stream)), "moe_kv_reclaim");
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
  moe::AttendArgs a{};
  if (const char* fault = attend_args(&a, cache, batch, q, q_token_stride, q_head_stride, q_heads, scale, window, out, lse, workspace))
    return refuse(fault);
  if (batch->tokens == 0) return MOE_OK;
  return launched(moe::launch_kv_attend(a, static_cast<cudaStream_t>(stream)), "moe_kv_attend");
}

size_t moe_kv_shared_bytes(int tokens, int q_heads, int head_dim) {
  if (tokens < 0 || q_heads < 1 || q_heads > 1024 || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return 0;
  return MOE_KV_SHARED_HEADER + 4ull * tokens * q_heads * (head_dim + 1);
}

int moe_kv_attend_shared(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, const moe_kv_prefixes_t* prefixes, const void* q,
                         int64_t q_token_stride, int64_t q_head_stride, int q_heads, float scale, void* out, float* lse,
                         void* workspace, void* scratch, void* stream) {
  moe::AttendArgs a{};
  if (const char* fault = attend_args(&a, cache, batch, q, q_token_stride, q_head_stride, q_heads, scale, 0, out, lse, workspace))
    return refuse(fault);
  if (prefixes == nullptr) return refuse("null argument");
  if (prefixes->groups < 1 || prefixes->groups > batch->requests) return refuse("groups out of range");
  if (prefixes->least_tiles < 0) return refuse("least_tiles < 0");
  if (batch->tokens == 0) return MOE_OK;
  if (!prefixes->group_start || !prefixes->prefix_lens || !scratch) return refuse("null pointer");
  if (!aligned(prefixes->group_start, 4) || !aligned(prefixes->prefix_lens, 4) || !aligned(scratch, 16)) return refuse("misaligned pointer");
  return launched(moe::launch_kv_attend_shared(a, *prefixes, scratch, static_cast<cudaStream_t>(stream)), "moe_kv_attend_shared");
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
