// Attention over the paged 8-bit cache for many query rows: prompt chunks
// (moe_kv_attend in include/moe.h; kv_attend.cu has the decode form).
//
// Here the 128 query rows of an item are the tensor core's 128-row operand and
// a tile's 128 tokens the columns: S[row][token] = Q x K^T and O[row][dim] +=
// P x V (V read transposed, as it lies in the page), so a row's weights need
// no other row. Queries and weights are split into e4m3 hi + e5m2 lo, two
// products into one accumulator: hi + lo hold the 8 significant bits of a BF16
// query exactly down to 2^-16 of its row's largest magnitude, and a weight of
// 2^-10 of its row's reference or more within 2^-8 of itself (BF16's own
// rounding; below that within 2^-18 of the reference). Weights carry their
// token's value scale, and the reference is a maximum of such products seen so
// far: while none outgrows it, the output stays in TMEM, accumulated in FP32 by
// the tensor core itself, and the scores are read once. Only when one does (and
// on an item's first tile) the maxima are taken first and the output is rescaled.
//
// Two groups take a CTA's tiles in turn, one in its softmax while the other's
// products run; in a group two warpgroups share the rows, each with half of the
// columns (two threads to a row). The groups' results are joined in shared memory.
//
// The softmax bounds it: two chunks of up to 700 tokens on 3300 to 6000 earlier
// ones (64 query heads on 8 of 128, 162 GFLOP) take 279 us, 579 TFLOP/s, where
// both products with their lo parts keep the tensor pipe busy for a quarter of
// that. A tile costs a group some 4 thousand cycles of conversions,
// exponentials and sums and 1.7 thousand of waiting for its own products, the
// other group's tile half hidden behind it; the schedulers issue in half of the
// cycles. Steps of 64 tokens with their scores in turn in two halves hide those
// products and measured 335 us (twice the waits and barriers, and the query
// image read twice as often); a tile's values before the next scores, 303.
// Short items are bound by their starts and ends, some 20 thousand cycles
// (queries 4, first scores and maxima 4, the groups' join and the output 6):
// prompts of 1130 and 870 tokens without earlier ones take 149 us, 224 TFLOP/s.
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
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr int kPartialFloats = kRows * (D + 2);
  static constexpr int kGroupTmem = 256;          // scores 128 columns, output D
  // Keys and values in rings of their own: a tile's keys are done with long before its values.
  static constexpr int kKeyStride = kTileBytes, kValuesAt = kStages * kTileBytes, kValueStride = kTileBytes;
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + 2 * kStages * kTileBytes;        // hi, lo
  static constexpr int kP = kQ + 2 * kRows * D;                      // [group] hi, lo
  static constexpr int kRowF = kP + kGroups * 2 * kRows * kTile;     // [row] factor
  static constexpr int kTops = kRowF + kRows * 4;                    // [group][half][row] maxima, then sums
  static constexpr int kRefs = kTops + kGroups * 2 * kRows * 4;      // [group][row] references, then [group] the value scales'
  static constexpr int kRowDst = kRefs + kGroups * kRows * 4 + 16;   // [row] its place among the outputs' rows
  static constexpr int kNan = kRowDst + kRows * 8;                  // [row][D / 32]: outputs that saw a NaN apart
  static constexpr int kMeta = kNan + kRows * D / 8;                 // [stage][kMaxPages + 1]
  static constexpr int kBars = (kMeta + kStages * (kMaxPages + 1) * 4 + 15) / 16 * 16;
  static constexpr int kPrefix = kBars + (4 * kStages + 4 * kGroups + 1) * 8;  // k_full, k_empty, v_full, v_empty, s_full, o_full, p_ready, drained, q_ready
  static constexpr int smem(int requests) { return kPrefix + (requests + 1) * 8 + 1024; }
  static_assert(kGroups * 2 * kRows * kTile >= kRows * D * 4, "the groups' join fits the weights' room");
};
// What starting and joining an item costs, in tiles (the chunks: 286 us with 4, 281 with 6, 282 with 8; the prompts: 147,
// 151, 151; with a window of 1000 on 4000 tokens: 219, 219, 237).
constexpr int kItemTiles = 6;
constexpr int kLongUnits = 16;       // longer items may be cut anywhere (one head to a group, 900 tokens: 46 -> 34.6 us)
constexpr int kUp = 4;               // weights are held times 2^4, so one may grow to 2^4.75 times its reference's before
constexpr float kHighest = 430.0f;   // it leaves e4m3
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

// Runs f(column, values) over kColumns columns from `taddr`, 16 at a time, the next ones on their way meanwhile.
template <int kColumns, class F>
__device__ __forceinline__ void for_columns(uint32_t taddr, F&& f) {
  float u[16], v[16];
  tmem_load_16_async(taddr, u);
#pragma unroll 1
  for (int c = 0; c < kColumns; c += 32) {
    tmem_wait_16(u);
    tmem_load_16_async(taddr + c + 16, v);
    f(c, u);
    tmem_wait_16(v);
    if (c + 32 < kColumns) tmem_load_16_async(taddr + c + 32, u);
    f(c + 16, v);
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
  uint64_t* k_empty = k_full + X::kStages;
  uint64_t* v_full = k_empty + X::kStages;
  uint64_t* v_empty = v_full + X::kStages;
  uint64_t* s_full = v_empty + X::kStages;   // [group]: scores of its tile in TMEM
  uint64_t* o_full = s_full + kGroups;     // [group]: its tile's output in TMEM
  uint64_t* p_ready = o_full + kGroups;    // [group]: its tile's weights in shared memory
  uint64_t* drained = p_ready + kGroups;   // [group]: every product issued has completed
  uint64_t* q_ready = drained + kGroups;
  long long* prefix = reinterpret_cast<long long*>(sm + X::kPrefix);
  __shared__ long long s_sum[kThreads / 32][2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ int s_nans;         // the item has outputs noted in `nans`
  __shared__ Segment<kRows> s_segment;  // the compute warps', kept by one of their threads
  __shared__ long long s_unit;
  __shared__ long long s_run[2];  // the CTA's units
  int32_t* status = reinterpret_cast<int32_t*>(a.workspace);
  float* partials = reinterpret_cast<float*>(a.workspace + kPartialOffset);

  if (tid == 0) {
    for (int i = 0; i < X::kStages; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
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
  __syncthreads();
  const long long start = s_run[0], stop = s_run[1];
  if (start >= stop) return;
  if (warp == kIssueWarp) {
    tmem_alloc(&s_tmem, kGroups * X::kGroupTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;  // group g: scores at 256 g, output at 256 g + 128

  if (warp == kProducerWarp) {
    produce<X, D, 1>(a, maps, prefix, weight, shift, start, stop, sm, meta, k_full, k_empty, status);
  } else if (warp == kProducerWarp + 1) {
    produce<X, D, 2>(a, maps, prefix, weight, shift, start, stop, sm, meta, v_full, v_empty, status);
  } else if (warp == kIssueWarp || warp == kIssueWarp + 1) {
    constexpr uint32_t kMode = X::kSpan == 128 ? 2 : 4, kGroup = 8 * X::kSpan;
    const uint32_t q_at = smem_addr(sm + X::kQ), p_at = smem_addr(sm + X::kP), ring = smem_addr(sm + X::kRing);
    const int w = warp - kIssueWarp;  // the warpgroup whose products this warp issues
    int k = 0, segments = 0, turn = 0;  // k: the CTA's first tile of the segment; turn: the group's own count
    bool alive = true;
    auto scores = [&](int i) {
      alive = __all_sync(kAll, wait(k_full + i % X::kStages, (i / X::kStages) & 1, status));
      if (!alive) return;
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t keys = ring + (i % X::kStages) * X::kKeyStride;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int st = 0; st < D / 32; ++st)
            mma_f8(tmem + w * X::kGroupTmem, smem_desc(q_at + part * kRows * D + st * 32, 16, kGroup, kMode),
                   smem_desc(keys + st * 32, 16, kGroup, kMode), idesc_f8(kTile, false, false, part == 1), part + st > 0);
        tc_commit(k_empty + i % X::kStages);
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
        // The group's scores have been read: its next tile's go first.
        if (i + 2 < last) scores(i + 2);
        alive = alive && __all_sync(kAll, wait(v_full + i % X::kStages, (i / X::kStages) & 1, status));
        if (!alive) break;
        tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t vals = ring + X::kValuesAt + (i % X::kStages) * X::kValueStride, p = p_at + w * 2 * kRows * kTile;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int st = 0; st < kTile / 32; ++st)
              mma_f8(tmem + w * X::kGroupTmem + 128, smem_desc(p + part * kRows * kTile + st * 32, 16, 1024, 2),
                     smem_desc(vals + st * 32 * X::kSpan, 0, kGroup, kMode), idesc_f8(D, false, true, part == 1),
                     !first || part + st > 0);
          tc_commit(v_empty + i % X::kStages);
          tc_commit(o_full + w);
        }
        __syncwarp();
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
    const int in_group = tid & (kGroupThreads - 1);
    const int pair = 4 + group * 4 + (warp & 3);  // the barrier of the two warps that share this row
    constexpr int kHalfTile = kTile / 2, kHalfD = D / 2;
    float* row_f = reinterpret_cast<float*>(sm + X::kRowF);
    float* tops = reinterpret_cast<float*>(sm + X::kTops);
    float* refs = reinterpret_cast<float*>(sm + X::kRefs);
    int* ref_scale = reinterpret_cast<int*>(refs + kGroups * kRows);
    long long* row_dst = reinterpret_cast<long long*>(sm + X::kRowDst);
    uint32_t* nans = reinterpret_cast<uint32_t*>(sm + X::kNan);
    float* join = reinterpret_cast<float*>(sm + X::kP);
    uint8_t* weights = sm + X::kP + group * 2 * kRows * kTile;
    const uint32_t lanes = tmem + group * X::kGroupTmem + (static_cast<uint32_t>(warp & 3) << 21);
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
      const int before = s.q.seq - s.q.n;
      const int rows = static_cast<int>(min(static_cast<long long>(kRows), static_cast<long long>(s.q.n - s.token) * a.group - s.within));
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
      const int hi = row < rows ? before + tok : -1, lo = row < rows && a.window > 0 ? max(0, hi - a.window + 1) : 0;
      // Tokens that any of the rows sees, and that all see.
      const int all_hi = before + s.token, any_hi = all_hi + per_group(s.within + rows - 1, inverse);
      const int any_lo = a.window > 0 ? max(0, all_hi - a.window + 1) : 0, all_lo = a.window > 0 ? max(0, any_hi - a.window + 1) : 0;
      const bool mixed = any_lo != all_lo || any_hi != all_hi;
      const float factor = s.begin < s.end ? row_f[row] : 0.0f;
      float l = 0.0f, m = row < rows ? -INFINITY : 0.0f;  // m: the reference of the row's weights
      int m_scale = 0;                                    // the reference of the value scales
      bool written = false;                               // the group's output in TMEM is this item's
      int at = k + ((k & 1) != group);
      for (; at < last; at += 2, ++turn) {
        const int stage = at % X::kStages;
        if (!failed) failed = !wait(v_full + stage, (at / X::kStages) & 1, status);  // (for the entries; well before the scores)
        __syncwarp();
        const uint32_t* mt = meta + stage * (kMaxPages + 1);
        const int base = (s.q.tile0 + s.begin + at - k) * kTile, base_half = base + half * kHalfTile;
        const int most = static_cast<int>(mt[kMaxPages] & 0xFFu);
        const bool edge = base < all_lo || base + kTile - 1 > all_hi || !(mt[kMaxPages] >> 8);
        // The row's visible tokens among this thread's 16 from column c on, as bits.
        auto visible = [&](int c, uint32_t entry) {
          const int from = min(max(lo - base_half - c, 0), 16), to = entry >> 16 ? min(max(hi - base_half - c, -1), 15) : -1;
          return 0xFFFFu >> (15 - to) & 0xFFFFu << from;
        };
        // Some row's first token may come with any of the group's tiles. (Both warps of the pair hold the same rows.)
        bool find = !written || most > m_scale || __any_sync(kAll, m == -INFINITY && hi >= base && lo < base + kTile);
        if (!failed) failed = !wait(s_full + group, turn & 1, status);
        __syncwarp();
        tc_fence_after_sync();
        for (int tries = 0;; ++tries) {
          if (find) {
            // The references are raised: the largest value scale, and the row's largest score with its token's value scale
            // (less the largest), over both halves; what is there already follows.
            const int scale = max(m_scale, most), rise = min(scale - m_scale, kFar);
            float top = -INFINITY;
            for_columns<kHalfTile>(s_at, [&](int c, float (&v)[16]) {
              const uint32_t entry = mt[(half * kHalfTile + c) >> shift];
              if (edge) {
                const uint32_t seen = visible(c, entry);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (!(seen & 1u << j)) v[j] = -INFINITY;
              }
              float big[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) big[j] = fmaxf(fmaxf(v[4 * j], v[4 * j + 1]), fmaxf(v[4 * j + 2], v[4 * j + 3]));
              const float most_here = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
              const float drop = static_cast<float>(max(static_cast<int>((entry >> 8) & 0xFFu) - scale, -kFar));
              if (most_here > -INFINITY) top = fmaxf(top, fmaf(most_here, factor * scale_of(entry & 0xFFu), drop));
            });
            float* mine = tops + (group * 2 + half) * kRows + row;
            *mine = top;
            sync_any<64>(pair, false);
            top = fmaxf(m - static_cast<float>(rise), fmaxf(top, tops[(group * 2 + (half ^ 1)) * kRows + row]));
            const float keep = m > -INFINITY ? exp2_fast(m - top) : 0.0f;
            l *= keep;
            if (written) {
              if (!failed) failed = !wait(o_full + group, (turn - 1) & 1, status);
              __syncwarp();
              tc_fence_after_sync();
              const float f = m > -INFINITY ? exp2_fast(m - top + static_cast<float>(m_scale - scale)) : 0.0f;
#pragma unroll 1
              for (int c = 0; c < kHalfD; c += 16) {
                float o[16];
                tmem_load_16_async(o_at + c, o);
                tmem_wait_16(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_store_16(o_at + c, o);
              }
              tmem_wait_stores();
            }
            m = top;
            m_scale = scale;
          }
          // The last tile's weights have been used: these take their place.
          if (written && !failed) failed = !wait(o_full + group, (turn - 1) & 1, status);
          const float ref = m > -INFINITY ? m : 0.0f;
          float part = 0.0f, high = 0.0f;
          for_columns<kHalfTile>(s_at, [&](int c, float (&v)[16]) {
            const uint32_t entry = mt[(half * kHalfTile + c) >> shift];
            const float f = factor * scale_of(entry & 0xFFu);
            // Times 2^kUp and the page's value scale over its reference, both in the exponent.
            const int up = kUp + max(static_cast<int>((entry >> 8) & 0xFFu) - m_scale, -kFar);
            const float off = static_cast<float>(up) - ref;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = exp2_fast(fmaf(v[j], f, off));
            if (edge) {
              const uint32_t seen = visible(c, entry);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (!(seen & 1u << j)) v[j] = 0.0f;
            }
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t his[4], los[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              sum[j / 2] = (v[2 * j] + v[2 * j + 1]) + (v[2 * j + 2] + v[2 * j + 3]);
              high = fmaxf(high, fmaxf(fmaxf(v[2 * j], v[2 * j + 1]), fmaxf(v[2 * j + 2], v[2 * j + 3])));
              uint32_t h0, l0, h1, l1;
              split2_wide_half(v[2 * j], v[2 * j + 1], h0, l0);
              split2_wide_half(v[2 * j + 2], v[2 * j + 3], h1, l1);
              his[j / 2] = h0 | h1 << 16;
              los[j / 2] = l0 | l1 << 16;
            }
            part = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), __uint_as_float(static_cast<uint32_t>(127 - up) << 23), part);
            uint8_t* dst = weights + chunk_at<128>(row, (half * kHalfTile + c) / 16);
            *reinterpret_cast<uint4*>(dst) = make_uint4(his[0], his[1], his[2], his[3]);
            *reinterpret_cast<uint4*>(dst + kRows * kTile) = make_uint4(los[0], los[1], los[2], los[3]);
          });
          find = sync_any<64>(pair, high > kHighest);
          if (!find || tries == 1) {
            l += part;
            break;
          }
        }
        written = true;
        if (edge) {
          // Values that no row sees are dropped, whatever they hold. A NaN that only some rows see is
          // taken out too, and noted for those. (Thread `row` here takes the tile's token of that number.)
          uint8_t* value = sm + X::kRing + X::kValuesAt + stage * X::kValueStride + row * X::kSpan;
          const int token = base + row;
          const bool seen = token >= any_lo && token <= any_hi && (mt[row >> shift] >> 16);
          if (!seen || (mixed && any_nan<D / 32, 2>(reinterpret_cast<const uint4*>(value) + half))) {
#pragma unroll 1
            for (int c = half; c < D / 16; c += 2) {
              uint4* cell = reinterpret_cast<uint4*>(value + c * 16);
              if (!seen) {
                *cell = make_uint4(0, 0, 0, 0);
                continue;
              }
              const uint4 w = *cell;
              uint32_t words[4] = {w.x, w.y, w.z, w.w};
              if (!(nan_code(w.x) | nan_code(w.y) | nan_code(w.z) | nan_code(w.w))) continue;
              // Stored chunk c of the token's row holds the dimensions of chunk c ^ (the row's swizzle).
              const int chunk = X::kSpan == 128 ? (c ^ row) & 7 : c ^ ((row >> 1) & 3);
#pragma unroll 1
              for (int b = 0; b < 16; ++b) {
                if (((words[b >> 2] >> (8 * (b & 3))) & 0x7Fu) != 0x7Fu) continue;
                words[b >> 2] &= ~(0xFFu << (8 * (b & 3)));
                const int dim = chunk * 16 + b;
                s_nans = 1;
                for (int i = 0; i < rows; ++i) {
                  const int last_seen = all_hi + per_group(s.within + i, inverse);
                  if (token <= last_seen && (a.window == 0 || token > last_seen - a.window))
                    atomicOr(nans + i * (D / 32) + dim / 32, 1u << (dim % 32));
                }
              }
              *cell = make_uint4(words[0], words[1], words[2], words[3]);
            }
          }
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        mbar_arrive(p_ready + group);
      }
      // The group's output, this thread's half of the row.
      float acc[kHalfD];
      if (written) {
        if (!failed) failed = !wait(o_full + group, (turn - 1) & 1, status);
        __syncwarp();
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < kHalfD; c += 16) {
          float o[16];
          tmem_load_16_async(o_at + c, o);
          tmem_wait_16(o);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c + j] = o[j];
        }
        tc_fence_before_sync();
      } else {
#pragma unroll
        for (int i = 0; i < kHalfD; ++i) acc[i] = 0.0f;
      }
      k = last;

      // The groups' outputs are joined: each takes a half of its threads' columns, and gives the other half away.
      failed = sync_any<kAllCompute>(3, failed);
      if (failed) break;
      constexpr int kOwn = kHalfD / 2;
      const int column = half * kHalfD + group * kOwn;
      tops[(group * 2 + half) * kRows + row] = l;
      if (half == 0) refs[group * kRows + row] = m;
      if (in_group == 0) ref_scale[group] = m_scale;
      auto cell = [&](int c) { return reinterpret_cast<float4*>(join + row * D + half * kHalfD + ((c ^ (row & 7)) << 2)); };
      float own[kOwn];
      if (group == 0) {
#pragma unroll
        for (int c = 0; c < kOwn / 4; ++c)
          *cell(kOwn / 4 + c) = make_float4(acc[kOwn + 4 * c], acc[kOwn + 4 * c + 1], acc[kOwn + 4 * c + 2], acc[kOwn + 4 * c + 3]);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) own[i] = acc[i];
      } else {
#pragma unroll
        for (int c = 0; c < kOwn / 4; ++c) *cell(c) = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) own[i] = acc[kOwn + i];
      }
      all_sync();
      {
        const float l0 = tops[row] + tops[kRows + row], l1 = tops[2 * kRows + row] + tops[3 * kRows + row];
        const float m0 = refs[row], m1 = refs[kRows + row], mn = fmaxf(m0, m1), safe = mn > -INFINITY ? mn : 0.0f;
        const float f0 = exp2_fast(m0 - safe), f1 = exp2_fast(m1 - safe);
        l = l0 * f0 + l1 * f1;
        m = mn;
        const float g0 = f0 * scale_of(ref_scale[0]) * (1.0f / (1 << kUp)), g1 = f1 * scale_of(ref_scale[1]) * (1.0f / (1 << kUp));
        const float mine = group == 0 ? g0 : g1, other = group == 0 ? g1 : g0;
#pragma unroll
        for (int c = 0; c < kOwn / 4; ++c) {
          const float4 v = *cell(group * (kOwn / 4) + c);
          own[4 * c] = own[4 * c] * mine + v.x * other;
          own[4 * c + 1] = own[4 * c + 1] * mine + v.y * other;
          own[4 * c + 2] = own[4 * c + 2] * mine + v.z * other;
          own[4 * c + 3] = own[4 * c + 3] * mine + v.w * other;
        }
        if (s.begin < s.end && s_nans) {
          const uint32_t bad = nans[row * (D / 32) + column / 32] >> (column % 32);  // (its lowest kOwn bits)
#pragma unroll
          for (int i = 0; i < kOwn; ++i)
            if (bad & 1u << i) own[i] = __uint_as_float(0x7FC00000u);
        }
        const float inv = !s.whole ? 1.0f : l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
#pragma unroll
        for (int c = 0; c < kOwn / 4; ++c)
          *cell(group * (kOwn / 4) + c) = make_float4(own[4 * c] * inv, own[4 * c + 1] * inv, own[4 * c + 2] * inv, own[4 * c + 3] * inv);
      }
      all_sync();
      // Out in whole rows (a thread's own row, 16 bytes at a time, would take an eighth of a wavefront's width a store).
      auto joined = [&](int r, int c) {
        return *reinterpret_cast<const float4*>(join + r * D + c / (kHalfD / 4) * kHalfD + ((c % (kHalfD / 4) ^ (r & 7)) << 2));
      };
      if (s.whole) {
        if (a.lse != nullptr && tid < rows) a.lse[row_dst[tid]] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
#pragma unroll
        for (int i = tid; i < kRows * D / 8; i += kAllCompute) {
          const int r = i / (D / 8), c = i % (D / 8);
          const float4 v0 = joined(r, 2 * c), v1 = joined(r, 2 * c + 1);
          __nv_bfloat162 w[4] = {__floats2bfloat162_rn(v0.x, v0.y), __floats2bfloat162_rn(v0.z, v0.w),
                                 __floats2bfloat162_rn(v1.x, v1.y), __floats2bfloat162_rn(v1.z, v1.w)};
          if (r < rows) *reinterpret_cast<uint4*>(a.out + row_dst[r] * D + c * 8) = *reinterpret_cast<uint4*>(w);
        }
      } else {
        float* piece = partials + static_cast<int64_t>(blockIdx.x * 2 + (s.first ? 1 : 0)) * X::kPartialFloats;
        if (tid < kRows) {
          piece[kRows * D + tid] = m;
          piece[kRows * D + kRows + tid] = l;
        }
#pragma unroll
        for (int i = tid; i < kRows * D / 4; i += kAllCompute)
          *reinterpret_cast<float4*>(piece + i * 4) = joined(i / (D / 4), i % (D / 4));
      }
      if (!s.whole) join_item<kRows, D, kAllCompute, 3>(a, s, row_dst, rows, ctas, total, tid, &s_last);
      all_sync();  // the join's room, the rows' factors and the join word are free again, the segment is done with
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
