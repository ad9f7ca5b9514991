// Attention over the paged 8-bit cache for many query rows: prompt chunks
// (moe_kv_attend in include/moe.h; kv_attend.cu has the decode form).
//
// Here the 128 query rows of an item are the tensor core's 128-row operand and
// a tile's 128 tokens the columns: S[row][token] = Q x K^T and O[row][dim] +=
// P x V, so a row's weights need no other row. Scores are taken of the cache's
// codes as they are, queries split into e4m3 hi + e5m2 lo, two products into one
// accumulator: together they hold the 8 significant bits of a BF16 query exactly
// down to 2^-13 of its row's largest magnitude, and what is smaller within 2^-21
// of that. Weights must keep their precision however small they are (kv_attend.cu
// says why), so they are two BF16 numbers, hi + lo, 16 bits at every magnitude,
// and two products again. They go back into TMEM, in the place of the scores that
// they come from, and are read from there: shared memory has no room for them.
// For that the values are widened to BF16, code times page scale, which is exact.
// A row's weights are held against a reference; one that outgrows it by 2^8
// raises it, and the weights and outputs so far follow.
//
// Two groups take a CTA's tiles in turn, one in its softmax while the other's
// products run; in a group two warpgroups share the rows, each with half of the
// columns (two threads to a row). At an item's end each thread takes a quarter of
// its row's output from both groups' TMEM.
//
// Softmax and widening bound it: two chunks of up to 700 tokens on 3300 to 6000
// earlier ones (64 query heads on 8 of 128, 162 GFLOP) take 313 us, 517 TFLOP/s.
// A group's next scores cannot start before its weights have been used: it
// waits for both products (some 2 thousand cycles, and widens its next values
// meanwhile), the other group's tile half hidden behind it. Values widened only
// then, into one buffer for each group, made it 350 us.
// Short items are bound by their starts and ends (queries, first scores and
// maxima, the output): prompts of 1130 and 870 tokens without earlier ones take
// 139 us, 240 TFLOP/s; with the groups joined in shared memory, not by reading
// each other's TMEM, 162.
#include "kv_attend.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;
constexpr int kGroups = 2;                        // each two warpgroups: threads 0-255, 256-511
constexpr int kGroupThreads = 2 * kCompute;
constexpr int kAllCompute = kGroups * kGroupThreads;
constexpr int kProducerWarp = kAllCompute / 32;   // one for the keys, one for the values
constexpr int kIssueWarp = kProducerWarp + 2;     // one for each group
constexpr int kThreads = kAllCompute + 128;

template <int D>
struct RowsShape {
  static constexpr int kRows = moe::kRows;
  static constexpr int kHalves = 1;
  static constexpr int kSpan = D;                 // 128 or 64: one box, one swizzle span a row
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kPartialFloats = kRows * (D + 2);
  static constexpr int kGroupTmem = 256;          // scores 128 columns, output D
  // Keys and values in rings of their own: a tile's keys are done with long before its values. A value stage holds the wide
  // form, and the codes as they come: behind it, or (from 128 dimensions on) in its second half, where a token's wide row
  // of the second 64 dimensions lies over its own codes.
  static constexpr int kKeyStages = D == 128 ? 2 : 4, kStages = 4;
  static constexpr int kWideBytes = kTile * D * 2, kKeyStride = kTileBytes, kValueStride = kWideBytes + (D == 128 ? 0 : kTileBytes);
  static constexpr int kRing = 0, kWide = kKeyStages * kTileBytes;
  static constexpr int kValuesAt = kWide + (D == 128 ? kTileBytes : kWideBytes);
  static constexpr int kQ = kWide + kStages * kValueStride;          // hi, lo; an item's output on its way out
  static constexpr int kRowF = kQ + 2 * kRows * D;                   // [row] factor
  static constexpr int kTops = kRowF + kRows * 4;                    // [group][half][row] maxima, then sums
  static constexpr int kRefs = kTops + kGroups * 2 * kRows * 4;      // [group][row] references
  static constexpr int kRowDst = kRefs + kGroups * kRows * 4;        // [row] its place among the outputs' rows
  static constexpr int kNan = kRowDst + kRows * 8;                  // [row][D / 32]: outputs that saw a NaN apart
  static constexpr int kMeta = kNan + kRows * D / 8;                 // [stage][kMaxPages + 1]
  static constexpr int kBars = (kMeta + kStages * (kMaxPages + 1) * 4 + 15) / 16 * 16;
  static constexpr int kPrefix = kBars + (2 * kKeyStages + 2 * kStages + 4 * kGroups + 1) * 8;  // k_full, k_empty, v_full, v_empty, s_full, o_full, p_ready, drained, q_ready
  static constexpr int smem(int requests) { return kPrefix + (requests + 1) * 8 + 1024; }
  // Each stage is always the same group's: a group waits for its own tiles only, and by a phase's parity would take a stage's
  // tile before last for its last, had the other group's in between not come yet.
  static_assert(kKeyStages % kGroups == 0 && kStages % kGroups == 0, "stages by groups");
  static_assert(kWide % 1024 == 0 && kValueStride % 1024 == 0 && kQ % 1024 == 0, "operand images on swizzle boundaries");
};
// What starting and joining an item costs, in tiles (prompts without earlier tokens: 139 us with 4 and 5, 146 with 6, 153
// with 8; one of 900 tokens with a window of 100: 104 with 4, 100 with 5; the chunks: 313 with any).
constexpr int kItemTiles = 5;
constexpr int kLongUnits = 16;       // longer items may be cut anywhere (one head to a group, 900 tokens: 46 -> 34.6 us)
constexpr int kMaxRowsCtas = 240;  // two pieces each fit the workspace
static_assert(kPartialOffset + 2ll * kMaxRowsCtas * kRows * (128 + 2) * 4 <= MOE_KV_WORKSPACE_BYTES, "workspace");

// Sixteen consecutive TMEM columns of this thread's lane, without the wait.
__device__ __forceinline__ void tmem_load_16_async(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}

// The wait for tcgen05.ld, tied to the registers that it completes.
__device__ __forceinline__ void tmem_wait_16(float (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
               :
               : "memory");
}

// Runs f(column, values, others) over kColumns columns from `taddr`, 16 at a time; the others are on their way meanwhile.
template <int kColumns, class F>
__device__ __forceinline__ void for_columns(uint32_t taddr, F&& f) {
  float u[16], v[16];
  tmem_load_16_async(taddr, u);
#pragma unroll 1
  for (int c = 0; c < kColumns; c += 32) {
    tmem_wait_16(u);
    tmem_load_16_async(taddr + c + 16, v);
    f(c, u, v);
    tmem_wait_16(v);
    if (c + 32 < kColumns) tmem_load_16_async(taddr + c + 32, u);
    f(c + 16, v, u);
  }
}

__device__ __forceinline__ void all_sync() { asm volatile("bar.sync 3, 512;" ::: "memory"); }

// Barrier of the two warps that share rows, or of more; true everywhere if any thread brings true.
template <int kCount>
__device__ __forceinline__ bool sync_any(int id, bool mine) {
  uint32_t any;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %2, 0;\n"
      "barrier.cta.red.or.pred q, %1, %3, p;\n"
      "selp.u32 %0, 1, 0, q; }"
      : "=r"(any)
      : "r"(id), "r"(static_cast<uint32_t>(mine)), "n"(kCount)
      : "memory");
  return any != 0;
}

// Sixteen columns back into TMEM.
__device__ __forceinline__ void tmem_store_16(uint32_t taddr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"f"(r[0]),
      "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]),
      "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "r"(taddr)
      : "memory");
}

// The largest of 16 (NaN loses).
__device__ __forceinline__ float highest(const float (&v)[16]) {
  float big[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) big[j] = fmaxf(fmaxf(v[4 * j], v[4 * j + 1]), fmaxf(v[4 * j + 2], v[4 * j + 3]));
  return fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
}

// This row's weights of `groups` 16 tokens (8 columns of hi pairs, 8 of lo pairs) times a power of two.
__device__ __forceinline__ void scale_weights(uint32_t taddr, int groups, float factor) {
  tmem_wait_stores();
#pragma unroll 1
  for (int g = 0; g < groups; ++g) {
    float w[16];
    tmem_load_16_async(taddr + 16 * g, w);
    tmem_wait_16(w);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t pair = __float_as_uint(w[j]);
      const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(pair << 16) * factor, __uint_as_float(pair & 0xFFFF0000u) * factor);
      w[j] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&v));
    }
    tmem_store_16(taddr + 16 * g, w);
  }
}

// This thread's kColumns columns of an output times a factor.
template <int kColumns>
__device__ __forceinline__ void scale_output(uint32_t taddr, float factor) {
#pragma unroll 1
  for (int c = 0; c < kColumns; c += 16) {
    float o[16];
    tmem_load_16_async(taddr + c, o);
    tmem_wait_16(o);
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] *= factor;
    tmem_store_16(taddr + c, o);
  }
  tmem_wait_stores();
}

// Where a CTA's run of units ends and the next one's starts: inside an item only if the item is long, else at its nearer
// end (a piece costs an item's start and the join, some kItemTiles tiles).
__device__ long long snap(const AttendArgs& a, const long long* prefix, int weight, int shift, long long x, long long total) {
  if (weight == 0 || x <= 0 || x >= total) return x;
  Segment<kRows> s;
  s.find(a, prefix, weight, shift, x, x + 1);
  if (s.units > kLongUnits) return x;
  return 2 * (x - s.item) >= s.units ? s.item + s.units : s.item;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attend_rows_kernel(const AttendArgs a, const __grid_constant__ AttendMaps maps, int shift) {
  using X = RowsShape<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* meta = reinterpret_cast<uint32_t*>(sm + X::kMeta);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + X::kBars);
  uint64_t* k_empty = k_full + X::kKeyStages;
  uint64_t* v_full = k_empty + X::kKeyStages;
  uint64_t* v_empty = v_full + X::kStages;
  uint64_t* s_full = v_empty + X::kStages;   // [group]: scores of its tile in TMEM
  uint64_t* o_full = s_full + kGroups;     // [group]: its tile's output in TMEM
  uint64_t* p_ready = o_full + kGroups;    // [group]: its tile's weights in TMEM, its values widened
  uint64_t* drained = p_ready + kGroups;   // [group]: every product issued has completed
  uint64_t* q_ready = drained + kGroups;
  long long* prefix = reinterpret_cast<long long*>(sm + X::kPrefix);
  __shared__ long long s_sum[kThreads / 32][2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ int s_nans;         // the item has outputs noted in `nans`
  __shared__ Segment<kRows> s_segment;  // the compute warps', kept by one of their threads
  __shared__ long long s_unit;
  __shared__ int32_t s_status;   // the workspace's when the CTA started
  __shared__ long long s_run[2];  // the CTA's units
  int32_t* status = reinterpret_cast<int32_t*>(a.workspace);
  float* partials = reinterpret_cast<float*>(a.workspace + kPartialOffset);

  const int32_t found = tid == 0 ? *static_cast<const volatile int32_t*>(status) : 0;  // (on its way while the work is summed)
  if (tid == 0) {
    for (int i = 0; i < X::kKeyStages; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < X::kStages; ++i) {
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(o_full + i, 1);
      mbar_init(p_ready + i, kGroupThreads);
      mbar_init(drained + i, 1);
    }
    mbar_init(q_ready, kAllCompute);
    fence_mbar_init();
  }
  const int weight = sum_work<kThreads, kRows, kItemTiles>(a, shift, prefix, s_sum);
  const long long total = prefix[a.b.requests];
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  if (blockIdx.x >= ctas) return;
  if (tid == 0 || tid == 32) {
    const int i = tid == 0 ? 0 : 1;
    s_run[i] = snap(a, prefix, weight, shift, total * (blockIdx.x + i) / ctas, total);
  }
  if (tid == 0) s_status = found;
  __syncthreads();
  const long long start = s_run[0], stop = s_run[1];
  if (start >= stop || s_status != MOE_OK) return;  // (an error that nobody has read yet: the arrival counters are anyhow)
  if (warp == kIssueWarp) {
    tmem_alloc(&s_tmem, kGroups * X::kGroupTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;  // group g: scores at 256 g, then weights in their place; output at 256 g + 128

  if (warp == kProducerWarp) {
    produce<X, D, 1>(a, maps, prefix, weight, shift, start, stop, sm, meta, k_full, k_empty, status);
  } else if (warp == kProducerWarp + 1) {
    produce<X, D, 2>(a, maps, prefix, weight, shift, start, stop, sm, meta, v_full, v_empty, status);
  } else if (warp == kIssueWarp || warp == kIssueWarp + 1) {
    constexpr uint32_t kMode = X::kSpan == 128 ? 2 : 4, kGroup = 8 * X::kSpan;
    const uint32_t q_at = smem_addr(sm + X::kQ), wide = smem_addr(sm + X::kWide), ring = smem_addr(sm + X::kRing);
    const int w = warp - kIssueWarp;  // the warpgroup whose products this warp issues
    int k = 0, segments = 0, turn = 0;  // k: the CTA's first tile of the segment; turn: the group's own count
    bool alive = true;
    auto scores = [&](int i) {
      const int stage = i % X::kKeyStages;
      alive = __all_sync(kAll, wait(k_full + stage, (i / X::kKeyStages) & 1, status));
      if (!alive) return;
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t keys = ring + stage * X::kKeyStride;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int st = 0; st < D / 32; ++st)
            mma_f8(tmem + w * X::kGroupTmem, smem_desc(q_at + part * kRows * D + st * 32, 16, kGroup, kMode),
                   smem_desc(keys + st * 32, 16, kGroup, kMode), idesc_f8(kTile, false, false, part == 1), part + st > 0);
        tc_commit(k_empty + stage);
        tc_commit(s_full + w);
      }
      __syncwarp();
    };
    Segment<kRows> s;
    s.find(a, prefix, weight, shift, start, stop);
    for (long long x = start; alive;) {
      const int last = k + s.end - s.begin;
      if (s.begin < s.end) alive = __all_sync(kAll, wait(q_ready, segments++ & 1, status));
      int i = k + ((k & 1) != w);
      if (alive && i < last) scores(i);
      for (bool first = true; i < last && alive; i += 2, ++turn, first = false) {
        alive = __all_sync(kAll, wait(p_ready + w, turn & 1, status));
        if (!alive) break;
        tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t own = tmem + w * X::kGroupTmem, vals = wide + i % X::kStages * X::kValueStride;
#pragma unroll
          for (int st = 0; st < kTile / 16; ++st)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              mma_bf16_tmem(own + 128, own + st * 16 + part * 8, smem_desc(vals + st * 2048, kTile * 128, 1024, 2),
                            idesc_bf16(D, false, true), !first || st + part > 0);
          tc_commit(v_empty + i % X::kStages);
          tc_commit(o_full + w);
        }
        __syncwarp();
        // The next scores take the place of these weights, once those have been used.
        if (i + 2 < last) {
          alive = __all_sync(kAll, wait(o_full + w, turn & 1, status));
          if (alive) scores(i + 2);
        }
      }
      k = last;
      x += s.length;
      if (x >= stop) break;
      s.next(a, prefix, shift, x, stop);
    }
    if (lane == 0) {
      tc_commit(drained + w);
      wait(drained + w, 0, status);
    }
    __syncwarp();
  } else if (warp < kProducerWarp) {
    const int group = tid / kGroupThreads, half = (tid / kCompute) & 1, row = tid & (kCompute - 1);
    const int pair = 4 + group * 4 + (warp & 3);  // the barrier of the two warps that share this row
    constexpr int kHalfTile = kTile / 2, kHalfD = D / 2;
    float* row_f = reinterpret_cast<float*>(sm + X::kRowF);
    float* tops = reinterpret_cast<float*>(sm + X::kTops);
    float* refs = reinterpret_cast<float*>(sm + X::kRefs);
    long long* row_dst = reinterpret_cast<long long*>(sm + X::kRowDst);
    uint32_t* nans = reinterpret_cast<uint32_t*>(sm + X::kNan);
    uint8_t* staged = sm + X::kQ;  // an item's output
    const uint32_t lanes = tmem + group * X::kGroupTmem + (static_cast<uint32_t>(warp & 3) << 21);
    const int widen_row = (warp & 7) * 16 + lane / 2;  // the token of a tile that this thread widens, with its neighbour
    const uint32_t s_at = lanes + half * kHalfTile, o_at = lanes + 128 + half * kHalfD;
    int k = 0, turn = 0;   // the CTA's tile; the group's own count
    bool failed = false;   // a wait ran out: no more waits; agreed on at the barriers
    if (tid == 0) {
      s_unit = start;
      s_segment.find(a, prefix, weight, shift, start, stop);
    }
    all_sync();
    const Segment<kRows>& s = s_segment;
    const uint32_t inverse = inverse_of(a.group);
    for (;;) {
      const Sight sight(a, s, inverse);
      const int rows = sight.rows;
      const int last = k + s.end - s.begin;
      if (s.begin < s.end) {
        // Queries: hi image, lo image, each row scaled by a power of two so that its largest magnitude lies in [128, 256).
        constexpr int kChunks = D / 8;
#pragma unroll
        for (int i = tid; i < kRows * kChunks; i += kAllCompute) {
          const int r = i / kChunks, c = i % kChunks, tok = per_group(s.within + r, inverse);
          uint4 w = make_uint4(0, 0, 0, 0);
          if (r < rows)
            w = *reinterpret_cast<const uint4*>(a.q + (s.q.first + s.token + tok) * a.q_token_stride +
                                                (s.head * a.group + s.within + r - tok * a.group) * a.q_head_stride + c * 8);
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7FFFu, (v[j] >> 16) & 0x7FFFu));
#pragma unroll
          for (int d = 1; d < kChunks; d <<= 1) top = max(top, __shfl_xor_sync(kAll, top, d));
          const int e = max(static_cast<int>(top >> 7) - 127 - 7, -120);
          // A negative scale goes into the queries' signs, so the factors below are not negative.
          const float down = (top == 0 ? 1.0f : pow2f(-e)) * (a.scale < 0.0f ? -1.0f : 1.0f);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            split2_wide(__uint_as_float(v[j] << 16) * down, __uint_as_float(v[j] & 0xFFFF0000u) * down, hi[j], lo[j]);
          uint8_t* dst = sm + X::kQ + c * 8 % 16 + chunk_at<X::kSpan>(r, c / 2);
          *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(dst + kRows * D) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          if (c == 0)
            row_f[r] = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : top == 0 ? 0.0f : fabsf(a.scale) * kLog2e * pow2f(e);
        }
        for (int i = tid; i < kRows * D / 32; i += kAllCompute) nans[i] = 0;
        if (tid == 0) s_nans = 0;
        fence_proxy_async_shared();
        mbar_arrive(q_ready);
        all_sync();
      }
      const int in_tile = per_group(s.within + row, inverse), tok = s.token + in_tile;
      if (tid < kRows)
        row_dst[row] = static_cast<long long>(s.q.first + tok) * a.q_heads + s.head * a.group + s.within + row - in_tile * a.group;
      const int hi = row < rows ? sight.last(row) : -1, lo = row < rows ? sight.first(hi) : 0;
      const float factor = s.begin < s.end ? row_f[row] : 0.0f;
      float l = 0.0f, m = row < rows ? -INFINITY : 0.0f;  // m: the reference of the row's weights
      bool written = false;                               // the group's output in TMEM is this item's
      int at = k + ((k & 1) != group);
      for (; at < last; at += 2, ++turn) {
        const int stage = at % X::kStages;
        if (!failed) failed = !wait(v_full + stage, (at / X::kStages) & 1, status);
        __syncwarp();
        const uint32_t* mt = meta + stage * (kMaxPages + 1);
        const int base = (s.q.tile0 + s.begin + at - k) * kTile, base_half = base + half * kHalfTile;
        const bool edge = sight.edge(base) || mt[kMaxPages] == 0;
        {
          // The values' wide form, while the group's products run: two lanes to a token, half of its dimensions each (the
          // second in an order of its own, so that they meet no bank twice). Both read all before either writes.
          uint8_t* image = sm + X::kWide + stage * X::kValueStride;
          const uint8_t* codes = sm + X::kValuesAt + stage * X::kValueStride;
          constexpr int kChunks = D / 32;
          const int part = lane & 1;
          const Widener<D / 32> widener(sight, mt[widen_row >> shift], edge, base + widen_row, nans, &s_nans);
          uint4 w[kChunks];
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
            w[i] = *reinterpret_cast<const uint4*>(codes + chunk_at<X::kSpan>(widen_row, part * kChunks + (i ^ (D == 128 ? part * 2 : 0))));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kChunks; ++i) widener(w[i], part * kChunks + (i ^ (D == 128 ? part * 2 : 0)), widen_row, image);
          fence_proxy_async_shared();
        }
        // The row's visible tokens among this thread's 16 from column c on, as bits.
        auto visible = [&](int c, uint32_t entry) {
          const int from = min(max(lo - base_half - c, 0), 16), to = entry >> 16 ? min(max(hi - base_half - c, -1), 15) : -1;
          return 0xFFFFu >> (15 - to) & 0xFFFFu << from;
        };
        // Some row's first token may come with any of the group's tiles. (Both warps of the pair hold the same rows.)
        const bool find = !written || __any_sync(kAll, m == -INFINITY && hi >= base && lo < base + kTile);
        if (!failed) failed = !wait(s_full + group, turn & 1, status);
        __syncwarp();
        tc_fence_after_sync();
        if (find) {
          // The reference is raised to the row's largest score, over both halves; what is there already follows.
          float top = -INFINITY;
          for_columns<kHalfTile>(s_at, [&](int c, float (&v)[16], float (&)[16]) {
            const uint32_t entry = mt[(half * kHalfTile + c) >> shift];
            if (edge) {
              const uint32_t seen = visible(c, entry);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (!(seen & 1u << j)) v[j] = -INFINITY;
            }
            const float most = highest(v);
            if (most > -INFINITY) top = fmaxf(top, most * (factor * scale_of(entry & 0xFFu)));
          });
          tops[(group * 2 + half) * kRows + row] = top;
          sync_any<64>(pair, false);
          top = fmaxf(m, fmaxf(top, tops[(group * 2 + (half ^ 1)) * kRows + row]));
          const float keep = m > -INFINITY ? exp2_fast(m - top) : 0.0f;
          l *= keep;
          if (written) scale_output<kHalfD>(o_at, keep);
          m = top;
        }
        const float ref = m > -INFINITY ? m : 0.0f;
        float part = 0.0f, raised = 0.0f;
        for_columns<kHalfTile>(s_at, [&](int c, float (&v)[16], float (&others)[16]) {
          const uint32_t entry = mt[(half * kHalfTile + c) >> shift];
          const float f = factor * scale_of(entry & 0xFFu), off = -(ref + raised);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = fmaf(v[j], f, off);
          if (edge) {
            const uint32_t seen = visible(c, entry);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (!(seen & 1u << j)) v[j] = -INFINITY;
          }
          const float high = highest(v);
          if (__any_sync(kAll, high > kHighest)) {
            // A weight outgrows the reference, which is raised; the tile's weights so far, which lie over their scores, follow.
            tmem_wait_16(others);
            const float up = high > kHighest ? high : 0.0f, keep = exp2_fast(-up);
            scale_weights(s_at, c / 16, keep);
            part *= keep;
            raised += up;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] -= up;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = exp2_fast(v[j]);
          float sum[4], out[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[j] = (v[4 * j] + v[4 * j + 1]) + (v[4 * j + 2] + v[4 * j + 3]);
          part += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t hi_pair, lo_pair;
            split2_bf16(v[2 * j], v[2 * j + 1], hi_pair, lo_pair);
            out[j] = __uint_as_float(hi_pair);
            out[8 + j] = __uint_as_float(lo_pair);
          }
          tmem_store_16(s_at + c, out);
        });
        if (sync_any<64>(pair, raised > 0.0f)) {
          // Both halves of a row go to the larger of their references.
          tops[(group * 2 + half) * kRows + row] = raised;
          sync_any<64>(pair, false);
          const float to = fmaxf(raised, tops[(group * 2 + (half ^ 1)) * kRows + row]);
          const float own = exp2_fast(raised - to), keep = exp2_fast(-to);
          scale_weights(s_at, kHalfTile / 16, own);
          part *= own;
          l *= keep;
          if (written) scale_output<kHalfD>(o_at, keep);
          m += to;
        }
        l += part;
        written = true;
        tmem_wait_stores();
        tc_fence_before_sync();
        mbar_arrive(p_ready + group);
      }
      // The groups' outputs are joined: a thread takes a quarter of its row's columns, from both groups' TMEM (a group may have
      // had no tile).
      if (written && !failed) failed = !wait(o_full + group, (turn - 1) & 1, status);
      const bool any0 = k + (k & 1) < last, any1 = k + !(k & 1) < last;
      k = last;
      tops[(group * 2 + half) * kRows + row] = l;
      if (half == 0) refs[group * kRows + row] = m;
      tc_fence_before_sync();
      failed = sync_any<kAllCompute>(3, failed);
      if (failed) break;
      tc_fence_after_sync();
      constexpr int kOwn = kHalfD / 2;
      const int column = half * kHalfD + group * kOwn;
      const uint32_t out0 = tmem + (static_cast<uint32_t>(warp & 3) << 21) + 128 + column, out1 = out0 + X::kGroupTmem;
      float own[kOwn];
      {
        const float l0 = tops[row] + tops[kRows + row], l1 = tops[2 * kRows + row] + tops[3 * kRows + row];
        const float m0 = refs[row], m1 = refs[kRows + row], mn = fmaxf(m0, m1), safe = mn > -INFINITY ? mn : 0.0f;
        const float f0 = exp2_fast(m0 - safe), f1 = exp2_fast(m1 - safe);
        l = l0 * f0 + l1 * f1;
        m = mn;
#pragma unroll
        for (int c = 0; c < kOwn; c += 16) {
          float u[16], v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) u[j] = v[j] = 0.0f;
          if (any0) tmem_load_16_async(out0 + c, u);
          if (any1) tmem_load_16_async(out1 + c, v);
          tmem_wait_16(u);
          tmem_wait_16(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) own[c + j] = u[j] * f0 + v[j] * f1;
        }
        tc_fence_before_sync();
        if (s.begin < s.end && s_nans) {
          const uint32_t bad = nans[row * (D / 32) + column / 32] >> (column % 32);  // (its lowest kOwn bits)
#pragma unroll
          for (int i = 0; i < kOwn; ++i)
            if (bad & 1u << i) own[i] = __uint_as_float(0x7FC00000u);
        }
      }
      if (s.whole) {
        // Out in whole rows, by way of the queries' room (a thread's own row, 16 bytes at a time, would take an eighth of a
        // wavefront's width a store).
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        if (a.lse != nullptr && tid < rows) a.lse[row_dst[tid]] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        auto cell = [&](int r, int c) { return reinterpret_cast<uint4*>(staged + r * (2 * D) + ((c ^ (r & 7)) << 4)); };
#pragma unroll
        for (int c = 0; c < kOwn; c += 8) {
          __nv_bfloat162 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = __floats2bfloat162_rn(own[c + 2 * j] * inv, own[c + 2 * j + 1] * inv);
          *cell(row, (column + c) / 8) = *reinterpret_cast<uint4*>(w);
        }
        all_sync();
#pragma unroll
        for (int i = tid; i < kRows * D / 8; i += kAllCompute) {
          const int r = i / (D / 8), c = i % (D / 8);
          if (r < rows) *reinterpret_cast<uint4*>(a.out + row_dst[r] * D + c * 8) = *cell(r, c);
        }
      } else {
        float* piece = partials + static_cast<int64_t>(blockIdx.x * 2 + (s.first ? 1 : 0)) * X::kPartialFloats;
        if (tid < kRows) {
          piece[kRows * D + tid] = m;
          piece[kRows * D + kRows + tid] = l;
        }
#pragma unroll
        for (int c = 0; c < kOwn; c += 4)
          *reinterpret_cast<float4*>(piece + row * D + column + c) = make_float4(own[c], own[c + 1], own[c + 2], own[c + 3]);
      }
      if (!s.whole) join_item<kRows, D, kAllCompute, 3>(a, s, row_dst, rows, ctas, total, tid, &s_last);
      all_sync();  // the output's room, the rows' factors and the join word are free again, the segment is done with
      if (tid == 0) {
        s_unit += s_segment.length;
        if (s_unit < stop) s_segment.next(a, prefix, shift, s_unit, stop);
      }
      all_sync();
      if (s_unit >= stop) break;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kGroups * X::kGroupTmem);
  }
}

template <int D>
cudaError_t launch_dim(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kv_attend_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             RowsShape<D>::smem(MOE_KV_MAX_REQUESTS));
  if (e != cudaSuccess) return e;
  const int grid = sms < kMaxRowsCtas ? sms : kMaxRowsCtas;
  kv_attend_rows_kernel<D><<<grid, kThreads, RowsShape<D>::smem(a.b.requests), stream>>>(a, maps, shift);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attend_rows(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream) {
  return a.c.head_dim == 64 ? launch_dim<64>(a, maps, shift, sms, stream) : launch_dim<128>(a, maps, shift, sms, stream);
}

}  // namespace moe
