// Attention over the paged 8-bit cache for many query rows: prompt chunks
// (moe_kv_attend in include/moe.h; kv_attend.cu has the decode form).
//
// Here the 128 query rows of an item are the tensor core's 128-row operand and
// a tile's 128 tokens the columns: S[row][token] = Q x K^T and O[row][dim] =
// P x V (V read transposed, as it lies in the page), so a thread owns a row and
// its maximum and sum need no other thread. Queries and weights are split
// into e4m3 hi + e5m2 lo, two products into one accumulator: hi + lo hold the
// 8 significant bits of a BF16 query exactly down to 2^-16 of its row's largest
// magnitude, and a weight of 2^-10 of its row's reference or more within 2^-8 of
// itself (BF16's own rounding; below that within 2^-18 of the reference). The
// reference is a maximum of the row's scores seen so far, raised only when a
// weight outgrows it. Each tile's output joins the running one in FP32 registers.
//
// Two warpgroups take a CTA's tiles in turn, one in its softmax while the
// other's products run; their results are joined in shared memory.
#include "kv_attend.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;
constexpr int kGroups = 2;                        // compute warpgroups: warps 0-3, 4-7
constexpr int kProducerWarp = 4 * kGroups;
constexpr int kIssueWarp = kProducerWarp + 1;       // one for each warpgroup
constexpr int kThreads = 128 * (kGroups + 1);    // whole warpgroups: one warp of the last one idles
// Registers a thread: 168 at launch; the last warpgroup gives of its own to the others (2 x 224 + 56 = 3 x 168).
constexpr int kComputeRegs = 224, kIssueRegs = 56;

template <int D>
struct RowsShape {
  static constexpr int kRows = moe::kRows;
  static constexpr int kHalves = 1;
  static constexpr int kSpan = D;                 // 128 or 64: one box, one swizzle span a row
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr int kPartialFloats = kRows * (D + 2);
  static constexpr int kGroupTmem = 256;          // scores 128 columns, output D
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kStages * kStageBytes;           // hi, lo
  static constexpr int kP = kQ + 2 * kRows * D;                      // [group] hi, lo
  static constexpr int kRowF = kP + kGroups * 2 * kRows * kTile;     // [row] factor
  static constexpr int kJoinMl = kRowF + kRows * 4;                  // [row] the second group's maximum and sum
  static constexpr int kNan = kJoinMl + kRows * 8;                   // [row][D / 32]: outputs that saw a NaN apart
  static constexpr int kMeta = kNan + kRows * D / 8;                 // [stage][kMaxPages + 1]
  static constexpr int kBars = (kMeta + kStages * (kMaxPages + 1) * 4 + 15) / 16 * 16;
  static constexpr int kPrefix = kBars + (2 * kStages + 4 * kGroups + 1) * 8;  // full, empty, s_full, o_full, p_ready, drained, q_ready
  static constexpr int smem(int requests) { return kPrefix + (requests + 1) * 8 + 1024; }
  static_assert(kPartialOffset + 2ll * 256 * kPartialFloats * 4 <= MOE_KV_WORKSPACE_BYTES || D == 128, "workspace");
  static_assert(kGroups * 2 * kRows * kTile >= kRows * D * 4, "the groups' join fits the weights' room");
};
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

// Codes of two values: e4m3 hi and e5m2 lo, v = hi + lo.
__device__ __forceinline__ void split2_wide(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack2(v0, v1);
  const float2 f = unpack2(hi);
  lo = __nv_cvt_float2_to_fp8x2(make_float2(v0 - f.x, v1 - f.y), __NV_SATFINITE, __NV_E5M2);
}

// The same in half precision, for weights.
__device__ __forceinline__ void split2_wide_half(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  const __half2 v = __floats2half2_rn(v0, v1);
  hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(v), __NV_SATFINITE, __NV_E4M3);
  const __half2 rest = __hsub2(v, __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3)));
  lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E5M2);
}

__device__ __forceinline__ void both_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

// Barrier of both warpgroups; true everywhere if any thread brings true.
__device__ __forceinline__ bool both_any(bool mine) {
  uint32_t any;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 3, 256, p;\n"
      "selp.u32 %0, 1, 0, q; }"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attend_rows_kernel(const AttendArgs a, const __grid_constant__ AttendMaps maps, int shift) {
  using X = RowsShape<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* meta = reinterpret_cast<uint32_t*>(sm + X::kMeta);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + X::kBars);
  uint64_t* empty = full + X::kStages;
  uint64_t* s_full = empty + X::kStages;   // [group]: scores of its tile in TMEM
  uint64_t* o_full = s_full + kGroups;     // [group]: its tile's output in TMEM
  uint64_t* p_ready = o_full + kGroups;    // [group]: its tile's weights in shared memory
  uint64_t* drained = p_ready + kGroups;   // [group]: every product issued has completed
  uint64_t* q_ready = drained + kGroups;
  long long* prefix = reinterpret_cast<long long*>(sm + X::kPrefix);
  __shared__ long long s_sum[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  int32_t* status = reinterpret_cast<int32_t*>(a.workspace);
  float* partials = reinterpret_cast<float*>(a.workspace + kPartialOffset);

  if (tid == 0) {
    for (int i = 0; i < X::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(o_full + i, 1);
      mbar_init(p_ready + i, kCompute);
      mbar_init(drained + i, 1);
    }
    mbar_init(q_ready, kCompute * kGroups);
    fence_mbar_init();
  }
  sum_work<kThreads, kRows>(a, shift, prefix, s_sum);
  const long long total = prefix[a.b.requests];
  const long long ctas = min(static_cast<long long>(gridDim.x), (total + kItemTiles) / (kItemTiles + 1));
  if (blockIdx.x >= ctas) return;
  const long long start = total * blockIdx.x / ctas, stop = total * (blockIdx.x + 1) / ctas;
  if (warp == kIssueWarp) {
    tmem_alloc(&s_tmem, kGroups * X::kGroupTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;  // group g: scores at 256 g, output at 256 g + 128

  if (warp >= kProducerWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  if (warp == kProducerWarp) {
    produce<X, D>(a, maps, prefix, shift, start, stop, sm, meta, full, empty, status);
  } else if (warp == kIssueWarp || warp == kIssueWarp + 1) {
    constexpr uint32_t kMode = X::kSpan == 128 ? 2 : 4, kGroup = 8 * X::kSpan;
    const uint32_t q_at = smem_addr(sm + X::kQ), p_at = smem_addr(sm + X::kP), ring = smem_addr(sm + X::kRing);
    const int w = warp - kIssueWarp;  // the warpgroup whose products this warp issues
    int k = 0, segments = 0, turn = 0;  // k: the CTA's first tile of the segment; turn: the group's own count
    bool alive = true;
    auto scores = [&](int i) {
      alive = __all_sync(kAll, wait(full + i % X::kStages, (i / X::kStages) & 1, status));
      if (!alive) return;
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t keys = ring + (i % X::kStages) * X::kStageBytes;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int st = 0; st < D / 32; ++st)
            mma_f8(tmem + w * X::kGroupTmem, smem_desc(q_at + part * kRows * D + st * 32, 16, kGroup, kMode),
                   smem_desc(keys + st * 32, 16, kGroup, kMode), idesc_f8(kTile, false, false, part == 1), part + st > 0);
        tc_commit(s_full + w);
      }
      __syncwarp();
    };
    Segment s;
    s.find(a, prefix, shift, kRows, start, stop);
    for (long long x = start; alive;) {
      const int last = k + s.end - s.begin;
      if (s.begin < s.end) alive = __all_sync(kAll, wait(q_ready, segments++ & 1, status));
      int i = k + ((k & 1) != w);
      if (alive && i < last) scores(i);
      for (; i < last && alive; i += 2, ++turn) {
        alive = __all_sync(kAll, wait(p_ready + w, turn & 1, status));
        if (!alive) break;
        tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t vals = ring + (i % X::kStages) * X::kStageBytes + X::kTileBytes, p = p_at + w * 2 * kRows * kTile;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int st = 0; st < kTile / 32; ++st)
              mma_f8(tmem + w * X::kGroupTmem + 128, smem_desc(p + part * kRows * kTile + st * 32, 16, 1024, 2),
                     smem_desc(vals + st * 32 * X::kSpan, 0, kGroup, kMode), idesc_f8(D, false, true, part == 1), part + st > 0);
          tc_commit(empty + i % X::kStages);
          tc_commit(o_full + w);
        }
        __syncwarp();
        // The group's scores have been read: its next tile's follow, while the group takes this output.
        if (i + 2 < last) scores(i + 2);
      }
      k = last;
      x += s.length;
      if (x >= stop) break;
      s.next(a, prefix, shift, kRows, x, stop);
    }
    if (lane == 0) {
      tc_commit(drained + w);
      wait(drained + w, 0, status);
    }
    __syncwarp();
  } else if (warp < kProducerWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
    const int group = warp >> 2, row = tid & (kCompute - 1);
    float* row_f = reinterpret_cast<float*>(sm + X::kRowF);
    float2* join_ml = reinterpret_cast<float2*>(sm + X::kJoinMl);
    uint32_t* nans = reinterpret_cast<uint32_t*>(sm + X::kNan);
    float* join = reinterpret_cast<float*>(sm + X::kP);
    uint8_t* weights = sm + X::kP + group * 2 * kRows * kTile;
    const uint32_t lanes = tmem + group * X::kGroupTmem + (static_cast<uint32_t>(warp & 3) << 21);
    int k = 0, turn = 0;   // the CTA's tile; the group's own count
    bool failed = false;   // a wait of this thread's ran out; no more waits, agreed on at the segment's end
    Segment s;
    s.find(a, prefix, shift, kRows, start, stop);
    for (long long x = start;;) {
      const int row0 = s.row_tile * kRows, before = s.q.seq - s.q.n;
      const int rows = static_cast<int>(min(static_cast<long long>(kRows), static_cast<long long>(s.q.n) * a.group - row0));
      float acc[D], l = 0.0f, m = row < rows ? -INFINITY : 0.0f;  // m: the reference of the weights, not always the maximum
#pragma unroll
      for (int i = 0; i < D; ++i) acc[i] = 0.0f;
      const int last = k + s.end - s.begin;
      bool mixed = false;
      if (s.begin < s.end) {
        // Queries: hi image, lo image, each row scaled by a power of two so that its largest magnitude lies in [128, 256).
        constexpr int kChunks = D / 8;
#pragma unroll 2
        for (int i = tid; i < kRows * kChunks; i += kCompute * kGroups) {
          const int r = i / kChunks, c = i % kChunks, at = row0 + r, tok = at / a.group;
          uint4 w = make_uint4(0, 0, 0, 0);
          if (r < rows)
            w = *reinterpret_cast<const uint4*>(a.q + (s.q.first + tok) * a.q_token_stride +
                                                (s.head * a.group + at - tok * a.group) * a.q_head_stride + c * 8);
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
        for (int i = tid; i < kRows * D / 32; i += kCompute * kGroups) nans[i] = 0;
        fence_proxy_async_shared();
        mbar_arrive(q_ready);
        both_sync();
      }
      const int tok = (row0 + row) / a.group;
      const int hi = row < rows ? before + tok : -1, lo = row < rows && a.window > 0 ? max(0, hi - a.window + 1) : 0;
      // Tokens that any of the rows sees, and that all see.
      const int any_hi = before + (row0 + rows - 1) / a.group, all_hi = before + row0 / a.group;
      const int any_lo = a.window > 0 ? max(0, all_hi - a.window + 1) : 0, all_lo = a.window > 0 ? max(0, any_hi - a.window + 1) : 0;
      mixed = any_lo != all_lo || any_hi != all_hi;
      const float factor = s.begin < s.end ? row_f[row] : 0.0f;
      for (int at = k + ((k & 1) != group); at < last; at += 2, ++turn) {
        const int stage = at % X::kStages;
        if (!failed) failed = !wait(s_full + group, turn & 1, status);
        if (!failed) failed = !wait(full + stage, (at / X::kStages) & 1, status);
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t* mt = meta + stage * (kMaxPages + 1);
        const int base = (s.q.tile0 + s.begin + at - k) * kTile;
        const int most = static_cast<int>(mt[kMaxPages] & 0xFFu);
        const bool edge = base < all_lo || base + kTile - 1 > all_hi || !(mt[kMaxPages] >> 8);
        // One pass over the scores while no weight outgrows its reference by more than the codes hold (2^4.75); else, and
        // on the first tile, one for the maxima before it.
        bool find = __any_sync(kAll, m == -INFINITY);
        for (int tries = 0; tries < 2; ++tries) {
          if (find) {
            float top = m;
            for_columns<kTile>(lanes, [&](int c, float (&v)[16]) {
              const uint32_t entry = mt[c >> shift];
              if (edge) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const int token = base + c + j;
                  if (token < lo || token > hi || !(entry >> 16)) v[j] = -INFINITY;
                }
              }
              float big[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) big[j] = fmaxf(fmaxf(v[4 * j], v[4 * j + 1]), fmaxf(v[4 * j + 2], v[4 * j + 3]));
              const float most_here = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
              if (most_here > -INFINITY) top = fmaxf(top, most_here * (factor * scale_of(entry & 0xFFu)));
            });
            const float keep = m > -INFINITY ? exp2_fast(m - top) : 0.0f;
            m = top;
            l *= keep;
#pragma unroll
            for (int i = 0; i < D; ++i) acc[i] *= keep;
          }
          const float ref = m > -INFINITY ? m : 0.0f;
          float part = 0.0f, high = 0.0f;
          for_columns<kTile>(lanes, [&](int c, float (&v)[16]) {
            const uint32_t entry = mt[c >> shift];
            const float f = factor * scale_of(entry & 0xFFu);
            // Times 2^kUp and the page's value scale over the tile's largest, both in the exponent.
            const int up = kUp + max(static_cast<int>((entry >> 8) & 0xFFu) - most, -100);
            const float off = static_cast<float>(up) - ref;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = exp2_fast(fmaf(v[j], f, off));
            if (edge) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int token = base + c + j;
                if (token < lo || token > hi || !(entry >> 16)) v[j] = 0.0f;
              }
            }
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t his[8], los[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              sum[j & 3] += v[2 * j] + v[2 * j + 1];
              high = fmaxf(high, fmaxf(v[2 * j], v[2 * j + 1]));
              split2_wide_half(v[2 * j], v[2 * j + 1], his[j], los[j]);
            }
            part = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), __uint_as_float(static_cast<uint32_t>(127 - up) << 23), part);
            uint8_t* dst = weights + chunk_at<128>(row, c / 16);
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(his[0] | his[1] << 16, his[2] | his[3] << 16, his[4] | his[5] << 16, his[6] | his[7] << 16);
            *reinterpret_cast<uint4*>(dst + kRows * kTile) =
                make_uint4(los[0] | los[1] << 16, los[2] | los[3] << 16, los[4] | los[5] << 16, los[6] | los[7] << 16);
          });
          find = __any_sync(kAll, high > kHighest);
          if (!find || tries == 1) {
            l += part;
            break;
          }
        }
        if (edge) {
          // Values that no row sees are dropped, whatever they hold. A NaN that only some rows see is
          // taken out too, and noted for those. (Thread `row` here takes the tile's token of that number.)
          uint8_t* value = sm + X::kRing + stage * X::kStageBytes + X::kTileBytes + row * X::kSpan;
          const int token = base + row;
          const bool seen = token >= any_lo && token <= any_hi && (mt[row >> shift] >> 16);
          if (!seen || mixed) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
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
                for (int i = 0; i < rows; ++i) {
                  const int last_seen = before + (row0 + i) / a.group;
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
        // The tile's product joins the running output.
        if (!failed) failed = !wait(o_full + group, turn & 1, status);
        __syncwarp();
        tc_fence_after_sync();
        const float into = scale_of(most) * (1.0f / (1 << kUp));
        float u[16], v[16];
        tmem_load_16_async(lanes + 128, u);
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          tmem_wait_16(u);
          tmem_load_16_async(lanes + 128 + c + 16, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(u[j], into, acc[c + j]);
          tmem_wait_16(v);
          if (c + 32 < D) tmem_load_16_async(lanes + 128 + c + 32, u);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c + 16 + j] = fmaf(v[j], into, acc[c + 16 + j]);
        }
      }
      k = last;

      // The second group's rows join the first's.
      failed = both_any(failed);
      if (failed) break;
      if (group == 1) {
        join_ml[row] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 4; ++c)
          *reinterpret_cast<float4*>(join + row * D + ((c ^ (row & 15)) << 2)) =
              make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
      }
      both_sync();
      if (group == 0) {
        const float2 other = join_ml[row];
        const float mn = fmaxf(m, other.x), safe = mn > -INFINITY ? mn : 0.0f;
        const float f0 = exp2_fast(m - safe), f1 = exp2_fast(other.x - safe);
        m = mn;
        l = l * f0 + other.y * f1;
#pragma unroll
        for (int c = 0; c < D / 4; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(join + row * D + ((c ^ (row & 15)) << 2));
          acc[4 * c] = acc[4 * c] * f0 + v.x * f1;
          acc[4 * c + 1] = acc[4 * c + 1] * f0 + v.y * f1;
          acc[4 * c + 2] = acc[4 * c + 2] * f0 + v.z * f1;
          acc[4 * c + 3] = acc[4 * c + 3] * f0 + v.w * f1;
        }
        if (mixed && s.begin < s.end) {
#pragma unroll
          for (int i = 0; i < D; ++i)
            if (nans[row * (D / 32) + i / 32] >> (i % 32) & 1) acc[i] = __uint_as_float(0x7FC00000u);
        }
        if (s.whole) {
          if (row < rows) {
            const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            const int64_t dst = static_cast<int64_t>(s.q.first + tok) * a.q_heads + s.head * a.group + row0 + row - tok * a.group;
#pragma unroll
            for (int c = 0; c < D; c += 8) {
              __nv_bfloat162 w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = __floats2bfloat162_rn(acc[c + 2 * j] * inv, acc[c + 2 * j + 1] * inv);
              *reinterpret_cast<uint4*>(a.out + dst * D + c) = *reinterpret_cast<uint4*>(w);
            }
            if (a.lse != nullptr) a.lse[dst] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
          }
        } else {
          float* mine = partials + static_cast<int64_t>(blockIdx.x * 2 + (s.first ? 1 : 0)) * X::kPartialFloats;
#pragma unroll
          for (int c = 0; c < D; c += 4)
            *reinterpret_cast<float4*>(mine + row * D + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
          mine[kRows * D + row] = m;
          mine[kRows * D + kRows + row] = l;
          join_item<kRows, D>(a, s, rows, ctas, total, tid, &s_last);
        }
      }
      x += s.length;
      if (x >= stop) break;
      s.next(a, prefix, shift, kRows, x, stop);
      both_sync();  // the join's room, the rows' factors and the join word are free again
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
