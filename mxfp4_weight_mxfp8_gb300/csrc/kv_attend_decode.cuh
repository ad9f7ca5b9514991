// Causal attention of new tokens over the paged 8-bit cache (moe_kv_attend in
// include/moe.h).
//
// An item is 8 * RT query rows of a request and cache head (kv_attend.cuh has
// the work split). In both products the cache's tokens or dimensions are the
// tensor core's 128-row operand: S^T[token][row] = K x Q^T and O^T[dim][row] +=
// V^T x P^T (V read transposed, token-major as it lies in the page). The few
// query rows are the narrow operand. Scores are taken of the keys' codes as they
// are, queries split into two e4m3 numbers, hi + lo / 16, which take two columns
// of the one product (the wide operand is read from shared memory once for
// both): together they hold the 8 significant bits of a BF16 query exactly down
// to 2^-13 of its row's largest magnitude, and what is smaller within 2^-21 of
// that. Weights must keep their precision however small they are (under a
// dominant token of no value the others are all of the output), so they are two
// BF16 numbers, hi + lo, 16 bits at every magnitude, in columns of their own
// again. For that the values are widened to BF16, code times page scale, which
// is exact, in place in shared memory.
// A row's weights are held against a reference, the largest score when it was
// last raised, so a tile needs no maxima and the output stays in TMEM, accumulated
// in FP32 by the tensor core. Only when a weight outgrows the reference by 2^8
// (and on an item's first tile) the maxima are taken first and the output is
// rescaled.
//
// Roles: a producer warp looks up pages and streams tiles by TMA through a ring,
// a warp issues the MMAs, four warps widen the values, do the softmax (thread =
// token) and read the output at the end (thread = dimension).
//
// The cache's bytes bound large decode steps: 64 requests of up to 8192 tokens
// (64 query heads on 8 of 128) take 100 us for 532 MB, 5.3 TB/s, 78 % of a
// copy's rate, with the schedulers issuing in 57 % of the cycles: the widening's
// instructions (the loop without them takes 93 us). Two requests of 100 to 131
// thousand tokens take 53 us for 244 MB: the same, with longer joins. One request
// of 777 tokens takes 10.5 us, all latency. With several rows a request and a
// window (40 requests, up to 24 rows, 1024 tokens of 64: 42 us for 35 MB) an
// item's start and end bound it, twice as long as a tile.
#pragma once

#include "kv_attend.cuh"

namespace moe {
namespace {

constexpr int kProducerWarp = 4;  // after the compute warps 0-3
constexpr int kIssueWarp = 5;
constexpr int kWidenWarp = 6;     // the first of four, in shapes that have them
constexpr float kLo = 1.0f / 16.0f;  // lo parts are held 16 times as large

template <int D, int RT>
struct Shape {
  static constexpr int kRows = 8 * RT;
  static constexpr int kCols = 2 * kRows;                 // N: hi and lo of each row
  static constexpr int kHalves = D >= 128 ? D / 128 : 1;  // 128-byte spans of a cache row
  static constexpr int kSpan = D >= 128 ? 128 : 64;       // bytes of a row in one box: the swizzle's width
  static constexpr int kTileBytes = kTile * D;            // keys or values of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kKeyStride = kStageBytes, kValuesAt = kTileBytes, kValueStride = kStageBytes;
  // Four warps of their own widen the values where one CTA fills an SM (prompts of 900 tokens, 16 heads on 8 of 256: 138 us,
  // 169 without). Elsewhere they take the place of a CTA (16 rows of 128: 81 us, 74 without; 8 rows of 64: 64 and 53).
  static constexpr bool kWideners = D == 256;
  static constexpr int kThreads = kWideners ? 320 : 192;
  // As many CTAs as shared memory and registers hold with two tiles or more in each one's ring (24 rows of 64 in 3 CTAs of
  // 96 registers spill: 119 us for 64 requests of up to 4096 tokens, against 79 in 2).
  static constexpr int kCtasPerSm = D == 256 ? 1 : RT == 1 || (D == 64 && RT == 2) ? 3 : 2;
  static constexpr int kStages = D == 64 ? (RT == 1 ? 4 : RT == 2 ? 3 : 5) : D == 128 && RT != 2 ? 2 : 3;
  static constexpr int kKeyStages = kStages;
  // What starting and joining an item costs, in tiles: more of them the wider the row tile and the shorter a tile's loads
  // (64 ragged requests of 128: 8 rows take 102 us with 2, 106 with 1 or 5; 24 rows 84 with 4, 88 with 7; of 64: 8 rows 54
  // with 3 to 5, 61 with 1).
  static constexpr int kItemTiles = RT + (D == 64 ? 3 : 1);
  // The same for short items, the requests' own behind a shared prefix (36 requests with 32 rows of 64 and up to 1500 tokens
  // behind prefixes of up to 5000, 12 alone: 81 us with 3, 84 with 7; the other shapes turn where they do above).
  static constexpr int kOwnItemTiles = D == 64 ? 3 : kItemTiles;
  static constexpr int kPartialFloats = kRows * (D + 2);  // rows, then maxima, then sums
  static constexpr int kTmem = 2 * kCols + kHalves * kCols <= 64 ? 64 : 2 * kCols + kHalves * kCols <= 128 ? 128 : 256;
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kStages * kStageBytes;  // hi rows, lo rows
  static constexpr int kP = kQ + kCols * D;                 // [64 tokens] hi rows, lo rows
  static constexpr int kRed = kP + kCols * kTile * 2;       // [row][warp] maxima, then sums
  static constexpr int kRef = kRed + kRows * 16;          // [warp][row] the weights' references
  static constexpr int kRowF = kRef + kRows * 16;         // [row] factor
  static constexpr int kRowLo = kRowF + kRows * 4;        // [row] first and last visible token
  static constexpr int kRowHi = kRowLo + kRows * 4;
  static constexpr int kRowDst = kRowHi + kRows * 4;      // [row] its place among the outputs' rows
  static constexpr int kNan = kRowDst + kRows * 8;        // [row][D / 32]: outputs that saw a NaN apart
  static constexpr int kMeta = kNan + kRows * D / 8;      // [stage][kMaxPages + 1]
  static constexpr int kBars = (kMeta + kStages * (kMaxPages + 1) * 4 + 15) / 16 * 16;
  static constexpr int kPrefix = kBars + (2 * kStages + 8) * 8;  // full, empty, s_full[2], o_full, p_ready, q_ready, drained, v_ready[2]
  static constexpr int smem(int requests) { return kPrefix + (requests + 1) * 8 + 1024; }
  static_assert(kPartialOffset + 2ll * kMaxCtas * kPartialFloats * 4 <= MOE_KV_WORKSPACE_BYTES, "workspace");
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0, "operand images on swizzle boundaries");
};

// Eight columns back into TMEM.
__device__ __forceinline__ void tmem_store_8(uint32_t taddr, const float (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(r[0]), "f"(r[1]), "f"(r[2]),
               "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "r"(taddr)
               : "memory");
}

// Eight consecutive TMEM columns of this thread's lane as floats, without the wait.
__device__ __forceinline__ void tmem_load_8_async(uint32_t taddr, float (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
      : "r"(taddr)
      : "memory");
}

// The wait for tcgen05.ld, tied to the registers that it completes.
__device__ __forceinline__ void tmem_wait_8(float (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7])
               :
               : "memory");
}

// Barrier of the compute warps; true everywhere if any thread brings true.
__device__ __forceinline__ bool compute_any(bool mine) {
  uint32_t any;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 1, 128, p;\n"
      "selp.u32 %0, 1, 0, q; }"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0;
}

// Sums of each row's values over the warp into red[row][warp]: lanes trade halves of their rows until one (three) is
// left, so 8 rows take 9 exchanges, not 40.
template <int kRows>
__device__ __forceinline__ void row_sums(float (&v)[kRows], float* red, int lane, int warp) {
  int row = 0, d = 16;
  constexpr int kLeft = kRows == 24 ? 3 : 1;
#pragma unroll
  for (int n = kRows / 2; n >= kLeft; n /= 2, d /= 2) {
    const bool upper = lane & d;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float give = upper ? v[j] : v[j + n], mine = upper ? v[j + n] : v[j];
      v[j] = mine + __shfl_xor_sync(kAll, give, d);
    }
    row += upper ? n : 0;
    if (n == kLeft) {
      d /= 2;
      break;
    }
  }
#pragma unroll
  for (; d >= 1; d /= 2)
#pragma unroll
    for (int j = 0; j < kLeft; ++j) v[j] += __shfl_xor_sync(kAll, v[j], d);
  constexpr int kSame = kRows == 8 ? 4 : kRows == 16 ? 2 : kRows == 24 ? 4 : 1;  // lanes that hold the same rows
  if (lane % kSame == 0) {
#pragma unroll
    for (int j = 0; j < kLeft; ++j) red[(row + j) * 4 + warp] = v[j];
  }
}

// A tile's values, widened in place, the first dimensions over the tile's keys, which its scores have used; thread `tid`
// takes the tile's token of that number. (From 128 dimensions on a token's wide rows lie over the keys and its own codes;
// with 64 they lie over others', so all are read before any is written.)
template <int kMode, int D, int RT>
__device__ __forceinline__ void widen_values(const Widener<kMode, D / 32>& widener, uint8_t* image, int tid) {
  using X = Shape<D, RT>;
  // (Rolled: unrolled, its code crowds the softmax's out of the instruction cache: 106 us for 64 ragged requests, not 101.)
  constexpr int kBatch = D == 64 ? 4 : 2;
#pragma unroll 1
  for (int c = 0; c < D / 16; c += kBatch) {
    uint4 codes[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      codes[i] = *reinterpret_cast<const uint4*>(image + X::kTileBytes + (c + i) / (X::kSpan / 16) * (kTile * X::kSpan) +
                                                 chunk_at<X::kSpan>(tid, (c + i) % (X::kSpan / 16)));
    if (D == 64) compute_sync();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) widener(codes[i], c + i, tid, image);
  }
}

template <int kMode, int D, int RT>
__global__ void __launch_bounds__(Shape<D, RT>::kThreads, Shape<D, RT>::kCtasPerSm)
    kv_attend_kernel(const AttendArgs a, const __grid_constant__ AttendMaps maps, int shift) {
  using X = Shape<D, RT>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* meta = reinterpret_cast<uint32_t*>(sm + X::kMeta);  // page: key scale, value scale << 8, present << 16
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + X::kBars);
  uint64_t* empty = full + X::kStages;
  uint64_t* s_full = empty + X::kStages;  // [2]: scores of a tile in TMEM
  uint64_t* o_full = s_full + 2;          // a tile's output in TMEM
  uint64_t* p_ready = o_full + 1;         // a tile's weights in shared memory
  uint64_t* q_ready = p_ready + 1;        // a segment's queries in shared memory
  uint64_t* drained = q_ready + 1;        // every MMA issued has completed
  uint64_t* v_ready = drained + 1;        // [2]: a tile's values widened by warps of their own
  long long* prefix = reinterpret_cast<long long*>(sm + X::kPrefix);
  __shared__ long long s_sum[X::kThreads / 32][2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ int s_nans;         // the item has outputs noted in `nans`
  __shared__ Segment<kMode, X::kRows> s_first;    // the CTA's first
  __shared__ Segment<kMode, X::kRows> s_segment;  // the compute warps', kept by one of their threads
  __shared__ long long s_unit;
  __shared__ int32_t s_status;   // the workspace's when the CTA started
  int32_t* status = reinterpret_cast<int32_t*>(a.workspace);
  float* partials = pieces_of<kMode>(a);

  if constexpr (kMode == kPrefix) {
    if (!a.early) grid_dependency_wait();
    if (__ldcg(a.shared) == 0) {  // nothing is shared (this launch ends after kSuffix's all the same)
      if (blockIdx.x == 0) grid_dependency_wait();
      return;
    }
  }
  const int32_t found = tid == 0 ? *static_cast<const volatile int32_t*>(status) : 0;  // (on its way while the work is summed)
  if (tid == 0) {
    for (int i = 0; i < X::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_full + 1, 1);
    mbar_init(o_full, 1);
    mbar_init(p_ready, kCompute);
    mbar_init(q_ready, kCompute);
    mbar_init(drained, 1);
    mbar_init(v_ready, kCompute);
    mbar_init(v_ready + 1, kCompute);
    fence_mbar_init();
  }
  if constexpr (kMode == kSuffix) grid_dependency_wait();  // the plan
  const int item_tiles = kMode == kSuffix && *a.shared > 0 ? X::kOwnItemTiles : X::kItemTiles;
  Own<kMode> own;
  const int weight = sum_work<kMode, X::kThreads, X::kRows>(a, item_tiles, shift, prefix, s_sum, own);
  const long long total = prefix[a.b.requests];
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  // (Whatever it does, kPrefix's launch ends after kSuffix's.)
  if (kMode == kPrefix && blockIdx.x == 0 && ctas == 0) grid_dependency_wait();
  if (blockIdx.x >= ctas) return;
  const long long start = total * blockIdx.x / ctas, stop = total * (blockIdx.x + 1) / ctas;
  if (warp == kIssueWarp) {
    tmem_alloc(&s_tmem, X::kTmem);
    tmem_relinquish();  // the SM's other CTA allocates its own
  }
  if (a.b.requests > X::kThreads ? tid == 0 : own.holds(start)) {
    if (a.b.requests > X::kThreads) s_first.find(a, prefix, weight, shift, start, stop);
    else s_first.place(a, tid, own.q, own.from, weight, start, stop);
  }
  if (tid == 0) s_status = found;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // The next launch may start, now that this CTA has its TMEM: that one holds TMEM too while it waits for this one's end.
  if constexpr (kMode != kWhole) grid_launch_dependents();
  const uint32_t tmem = s_tmem, tmem_o = tmem + 2 * X::kCols;

  if (s_status != MOE_OK) {
    // An error that nobody has read yet: its call has left the arrival counters anyhow.
  } else if (warp == kProducerWarp) {
    produce<kMode, X, D, 3>(a, maps, prefix, shift, s_first, start, stop, sm, meta, full, empty, status);
  } else if (warp == kIssueWarp) {
    // Operand descriptors: keys and queries in the 128-byte (64-byte) swizzle, 8-row groups 1024 (512) bytes apart; values
    // M-major, 64 dimensions wide (D = 64: both 64-row halves of the operand read the same 64).
    constexpr uint32_t kValueHalf = kTile * 128, kNext = D == 64 ? 0 : kValueHalf;
    constexpr uint32_t kSwizzle = X::kSpan == 128 ? 2 : 4, kGroup = 8 * X::kSpan;
    const uint32_t q_at = smem_addr(sm + X::kQ), p_at = smem_addr(sm + X::kP), ring = smem_addr(sm + X::kRing);
    int k = 0, segments = 0;
    bool alive = true;
    auto scores = [&](int i) {
      alive = __all_sync(kAll, wait(full + i % X::kStages, (i / X::kStages) & 1, status));
      if (!alive) return;
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t keys = ring + (i % X::kStages) * X::kStageBytes, d = tmem + (i & 1) * X::kCols;
#pragma unroll
        for (int st = 0; st < D / 32; ++st) {
          const int h = st * 32 / X::kSpan, at = st * 32 % X::kSpan;
          mma_f8(d, smem_desc(keys + h * kTile * X::kSpan + at, 16, kGroup, kSwizzle),
                 smem_desc(q_at + h * X::kCols * X::kSpan + at, 16, kGroup, kSwizzle), idesc_f8(X::kCols, false), st > 0);
        }
        tc_commit(s_full + (i & 1));
      }
      __syncwarp();
    };
    Segment<kMode, X::kRows> s = s_first;
    for (long long x = start; alive;) {
      if (s.begin < s.end) {
        alive = __all_sync(kAll, wait(q_ready, segments++ & 1, status));
        if (alive) scores(k);
      }
      for (int tile = s.begin; tile < s.end && alive; ++tile, ++k) {
        // The next tile's scores ahead of this one's output, unless its keys are still on their way.
        const bool more = tile + 1 < s.end;
        const bool early = more && __all_sync(kAll, mbar_test(full + (k + 1) % X::kStages, ((k + 1) / X::kStages) & 1));
        if (early) scores(k + 1);
        alive = alive && __all_sync(kAll, wait(p_ready, k & 1, status));
        if (X::kWideners) alive = alive && __all_sync(kAll, wait(v_ready + (k & 1), (k >> 1) & 1, status));
        if (!alive) break;
        tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t vals = ring + (k % X::kStages) * X::kStageBytes;
#pragma unroll
          for (int h = 0; h < X::kHalves; ++h)
#pragma unroll
            for (int st = 0; st < kTile / 16; ++st)
              mma_bf16(tmem_o + h * X::kCols, smem_desc(vals + 2 * h * kValueHalf + st * 2048, kNext, 1024, 2),
                       smem_desc(p_at + st / 4 * (X::kCols * 128) + st % 4 * 32, 16, 1024, 2),
                       idesc_bf16(X::kCols, true), tile > s.begin || st > 0);
          tc_commit(empty + k % X::kStages);
          tc_commit(o_full);
        }
        __syncwarp();
        if (more && !early) scores(k + 1);
      }
      x += s.length;
      if (x >= stop) break;
      s.next(a, prefix, shift, x, stop);
    }
    if (lane == 0) {
      tc_commit(drained);
      wait(drained, 0, status);
    }
    __syncwarp();
  } else if (X::kWideners && warp >= kWidenWarp) {
    const int at = tid - 32 * kWidenWarp;
    const uint32_t inverse = inverse_of(a.group);
    int k = 0, segments = 0;
    bool alive = true;
    Segment<kMode, X::kRows> s = s_first;
    for (long long x = start; alive;) {
      const Sight<kMode> sight(a, s, inverse);
      if (s.begin < s.end) alive = __all_sync(kAll, wait(q_ready, segments++ & 1, status));
      for (int tile = s.begin; tile < s.end && alive; ++tile, ++k) {
        const int stage = k % X::kStages;
        alive = __all_sync(kAll, wait(full + stage, (k / X::kStages) & 1, status));
        alive = alive && __all_sync(kAll, wait(s_full + (k & 1), (k >> 1) & 1, status));
        if (!alive) break;
        const uint32_t* mt = meta + stage * (kMaxPages + 1);
        const int base = (s.q.tile0 + tile) * kTile;
        const Widener<kMode, D / 32> widener(sight, mt[at >> shift], sight.edge(base) || mt[kMaxPages] == 0, base + at,
                                      reinterpret_cast<uint32_t*>(sm + X::kNan), &s_nans);
        widen_values<kMode, D, RT>(widener, sm + X::kRing + stage * X::kStageBytes, at);
        fence_proxy_async_shared();
        mbar_arrive(v_ready + (k & 1));
      }
      x += s.length;
      if (x >= stop) break;
      s.next(a, prefix, shift, x, stop);
    }
  } else {
    float* red = reinterpret_cast<float*>(sm + X::kRed);
    float* refs = reinterpret_cast<float*>(sm + X::kRef) + warp * X::kRows;
    float* row_f = reinterpret_cast<float*>(sm + X::kRowF);
    int* row_lo = reinterpret_cast<int*>(sm + X::kRowLo);
    int* row_hi = reinterpret_cast<int*>(sm + X::kRowHi);
    long long* row_dst = reinterpret_cast<long long*>(sm + X::kRowDst);
    uint32_t* nans = reinterpret_cast<uint32_t*>(sm + X::kNan);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21), lanes_o = tmem_o + (static_cast<uint32_t>(warp) << 21);
    int k = 0;
    bool failed = false, dead = false;  // a wait of this thread's ran out; one of any thread's did, all agreed
    if (tid == 0) {
      s_unit = start;
      s_segment = s_first;
    }
    compute_sync();
    const Segment<kMode, X::kRows>& s = s_segment;
    const uint32_t inverse = inverse_of(a.group);
    for (;;) {
      const Request<kMode>& rq = s.q;
      const Sight<kMode> sight(a, s, inverse);
      const int rows = sight.rows;
      float l[X::kRows];                 // sums of this thread's tokens' weights against the references
      float m = -INFINITY;               // reference of row `lane`
#pragma unroll
      for (int i = 0; i < X::kRows; ++i) l[i] = 0.0f;
      bool blank = false;  // some row has seen no token yet
      if (tid < X::kRows) {
        const int in_tile = per_group(s.within + tid, inverse), tok = s.token + in_tile, last = tid < rows ? sight.last(tid) : -1;
        row_hi[tid] = last;
        row_lo[tid] = tid < rows ? sight.first(last) : 0;
        row_dst[tid] = static_cast<long long>(rq.first + tok) * a.q_heads + s.head * a.group + s.within + tid - in_tile * a.group;
      }
      if (s.begin < s.end) {
        // Queries: hi rows, then lo rows, scaled by a power of two so that each row's largest magnitude lies in [128, 256).
        constexpr int kChunks = D / 8;
#pragma unroll
        for (int base = 0; base < X::kRows * kChunks; base += kCompute) {
          const int i = base + tid;
          const int row = i / kChunks, c = i % kChunks, tok = per_group(s.within + row, inverse);
          const bool used = row < rows;
          uint4 w = make_uint4(0, 0, 0, 0);
          if (used)
            w = *reinterpret_cast<const uint4*>(a.q + (rq.first + s.token + tok) * a.q_token_stride +
                                                (s.head * a.group + s.within + row - tok * a.group) * a.q_head_stride + c * 8);
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7FFFu, (v[j] >> 16) & 0x7FFFu));
#pragma unroll
          for (int d = 1; d < kChunks; d <<= 1) top = max(top, __shfl_xor_sync(kAll, top, d));
          const int e = max(static_cast<int>(top >> 7) - 127 - 7, -120);
          const float down = top == 0 ? 1.0f : pow2f(-e);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            split2(__uint_as_float(v[j] << 16) * down, __uint_as_float(v[j] & 0xFFFF0000u) * down, hi[j], lo[j]);
          if (row >= X::kRows) continue;  // whole warps, past the loop's shuffles
          const int span = c * 8 / X::kSpan, in = c * 8 % X::kSpan;
          uint8_t* dst = sm + X::kQ + span * (X::kCols * X::kSpan) + in % 16;
          *reinterpret_cast<uint2*>(dst + chunk_at<X::kSpan>(row, in / 16)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(dst + chunk_at<X::kSpan>(X::kRows + row, in / 16)) =
              make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          if (c == 0) row_f[row] = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : top == 0 ? 0.0f : a.scale * kLog2e * pow2f(e);
        }
        for (int i = tid; i < X::kRows * D / 32; i += kCompute) nans[i] = 0;
        if (tid == 0) s_nans = 0;
        fence_proxy_async_shared();
        mbar_arrive(q_ready);
        compute_sync();
      }
      for (int tile = s.begin; tile < s.end; ++tile, ++k) {
        const int stage = k % X::kStages;
        failed |= !wait(s_full + (k & 1), (k >> 1) & 1, status);
        failed |= !wait(full + stage, (k / X::kStages) & 1, status);  // complete before the scores: for what it makes visible
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t* mt = meta + stage * (kMaxPages + 1);
        const uint32_t entry = mt[tid >> shift];
        const int base = (rq.tile0 + tile) * kTile, token = base + tid;
        const bool edge = sight.edge(base) || mt[kMaxPages] == 0;
        if (!X::kWideners)
          widen_values<kMode, D, RT>(Widener<kMode, D / 32>(sight, entry, edge, token, nans, &s_nans), sm + X::kRing + stage * X::kStageBytes, tid);
        const float ks = scale_of(entry & 0xFFu);
        bool find = tile == s.begin;
        if (edge || blank)  // a row's first token
          find |= __any_sync(kAll, lane < X::kRows && m == -INFINITY && row_hi[min(lane, X::kRows - 1)] >= base &&
                                       row_lo[min(lane, X::kRows - 1)] - base < kTile);
        for (int tries = 0;; ++tries) {
          // Scores of this token, times log2 e.
          float sc[X::kRows];
#pragma unroll
          for (int part = 0; part < X::kRows; part += 8) {
            float u[8], w[8];  // hi columns, lo columns
            tmem_load_8_async(lanes + (k & 1) * X::kCols + part, u);
            tmem_load_8_async(lanes + (k & 1) * X::kCols + X::kRows + part, w);
            tmem_wait_8(u);
            tmem_wait_8(w);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              const float4 f = *reinterpret_cast<const float4*>(row_f + part + j);
              const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[part + j + e] = fmaf(w[j + e], kLo, u[j + e]) * (fs[e] * ks);
            }
          }
          if (edge) {
#pragma unroll
            for (int i = 0; i < X::kRows; ++i)
              if (token < row_lo[i] || token > row_hi[i] || !(entry >> 16)) sc[i] = -INFINITY;
          }
          if (find) {
            // The references are raised to each row's largest score; what is there already follows.
            float top = -INFINITY;  // of row `lane`
#pragma unroll
            for (int i = 0; i < X::kRows; ++i) {
              const float v = warp_max(sc[i]);
              if (lane == i) top = v;
            }
            if (lane < X::kRows) red[lane * 4 + warp] = top;
            dead = compute_any(failed);
            if (dead) break;
            float keep = 1.0f;
            if (lane < X::kRows) {
              const float4 v = *reinterpret_cast<const float4*>(red + lane * 4);
              top = fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
              keep = m > -INFINITY ? exp2_fast(m - top) : 0.0f;
              m = top;
            }
            blank = __any_sync(kAll, lane < rows && m == -INFINITY);
            if (lane < X::kRows) refs[lane] = m > -INFINITY ? m : 0.0f;
            __syncwarp();
            if (tile > s.begin) {
              float keeps[X::kRows];
#pragma unroll
              for (int i = 0; i < X::kRows; ++i) {
                keeps[i] = __shfl_sync(kAll, keep, i);
                l[i] *= keeps[i];
              }
              failed |= !wait(o_full, (k - 1) & 1, status);
              __syncwarp();
              tc_fence_after_sync();
#pragma unroll
              for (int h = 0; h < X::kHalves; ++h)
#pragma unroll
                for (int part = 0; part < X::kCols; part += 8) {
                  float o[8];
                  tmem_load_8_async(lanes_o + h * X::kCols + part, o);
                  tmem_wait_8(o);
#pragma unroll
                  for (int j = 0; j < 8; ++j) o[j] *= keeps[(part + j) % X::kRows];
                  tmem_store_8(lanes_o + h * X::kCols + part, o);
                }
              tmem_wait_stores();
            }
          }
          // Less their reference.
          float high = -INFINITY;
#pragma unroll
          for (int i = 0; i < X::kRows; i += 4) {
            const float4 r = *reinterpret_cast<const float4*>(refs + i);
            sc[i] -= r.x;
            sc[i + 1] -= r.y;
            sc[i + 2] -= r.z;
            sc[i + 3] -= r.w;
            high = fmaxf(high, fmaxf(fmaxf(sc[i], sc[i + 1]), fmaxf(sc[i + 2], sc[i + 3])));
          }
          // Every thread's weights are held against the same references: another round for all if one outgrew its own.
          // (Or a wait of its ran out: the other round agrees on that.)
          find = compute_any(high > kHighest || failed);
          if (find && tries == 0) continue;
          if (tile > s.begin) failed |= !wait(o_full, (k - 1) & 1, status);  // the last tile's weights have been used
          uint8_t* prow = sm + X::kP + tid / 64 * (X::kCols * 128) + tid % 8 * 2;
          const int chunk = tid % 64 / 8;
          auto put = [&](int row, uint32_t v) { *reinterpret_cast<uint16_t*>(prow + chunk_at<128>(row, chunk)) = static_cast<uint16_t>(v); };
#pragma unroll
          for (int i = 0; i < X::kRows; i += 2) {
            const float p0 = exp2_fast(sc[i]), p1 = exp2_fast(sc[i + 1]);
            l[i] += p0;
            l[i + 1] += p1;
            uint32_t hi, lo;
            split2_bf16(p0, p1, hi, lo);
            put(i, hi);
            put(i + 1, hi >> 16);
            put(X::kRows + i, lo);
            put(X::kRows + i + 1, lo >> 16);
          }
          break;
        }
        if (dead) break;
        fence_proxy_async_shared();
        tc_fence_before_sync();
        mbar_arrive(p_ready);
      }
      // The output: this thread's dimension of each row.
      float acc[X::kHalves][X::kRows];
      if (s.begin < s.end && !failed) {
        failed = !wait(o_full, (k - 1) & 1, status);
        if (X::kWideners) failed |= !wait(v_ready + ((k - 1) & 1), ((k - 1) >> 1) & 1, status);  // (for what they noted)
      }
      failed = compute_any(failed);  // agreed on before whole warps read TMEM: a wait may run out for some lanes only
      if (failed) break;
      if (s.begin < s.end) {
        tc_fence_after_sync();
#pragma unroll
        for (int h = 0; h < X::kHalves; ++h)
#pragma unroll
          for (int part = 0; part < X::kRows; part += 8) {
            float o[8], u[8];  // hi columns, lo columns
            tmem_load_8_async(lanes_o + h * X::kCols + part, o);
            tmem_load_8_async(lanes_o + h * X::kCols + X::kRows + part, u);
            tmem_wait_8(o);
            tmem_wait_8(u);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[h][part + j] = o[j] + u[j];
          }
        tc_fence_before_sync();
      } else {
#pragma unroll
        for (int h = 0; h < X::kHalves; ++h)
#pragma unroll
          for (int i = 0; i < X::kRows; ++i) acc[h][i] = 0.0f;
      }

      // The segment's sums over the tokens, and its rows.
      row_sums<X::kRows>(l, red, lane, warp);
      compute_sync();
      float sum = 0.0f;  // of row `lane`
      if (lane < X::kRows) {
        const float4 v = *reinterpret_cast<const float4*>(red + lane * 4);
        sum = (v.x + v.y) + (v.z + v.w);
      }
      if (s.begin < s.end && s_nans) {
#pragma unroll
        for (int h = 0; h < X::kHalves; ++h)
#pragma unroll
          for (int i = 0; i < X::kRows; ++i) {
            const int dim = h * 128 + tid;
            if (dim < D && (nans[i * (D / 32) + dim / 32] >> (dim % 32) & 1)) acc[h][i] = __uint_as_float(0x7FC00000u);
          }
      }
      const bool holds = D >= 128 || tid < D;  // this thread's dimension (D = 64: the upper lanes repeat the lower)
      auto store_row = [&](int i, float v0, float v1, float inv, float lse) {
        const int64_t dst = row_dst[i];
        if (kMode == kSuffix && s.shared()) {
          if (holds) {
            a.partial[dst * D + tid] = v0 * inv;
            if (X::kHalves == 2) a.partial[dst * D + 128 + tid] = v1 * inv;
          }
          if (tid == 0) a.partial_lse[dst] = lse;
          return;
        }
        if (holds) {
          a.out[dst * D + tid] = __bfloat16_as_ushort(__float2bfloat16(v0 * inv));
          if (X::kHalves == 2) a.out[dst * D + 128 + tid] = __bfloat16_as_ushort(__float2bfloat16(v1 * inv));
        }
        if (a.lse != nullptr && tid == 0) a.lse[dst] = lse;
      };
      if (s.whole) {
        if constexpr (kMode == kPrefix) {
          grid_dependency_wait();  // the requests' own parts are done
          const Joined j(m, sum, lane < rows ? __ldcg(a.partial_lse + row_dst[lane]) : -INFINITY);
          m = j.top;
          sum = j.sum;
#pragma unroll
          for (int i = 0; i < X::kRows; ++i) {
            const float own = __shfl_sync(kAll, j.own, i), other = __shfl_sync(kAll, j.other, i);
            if (i >= rows) continue;
#pragma unroll
            for (int h = 0; h < X::kHalves; ++h)
              acc[h][i] = acc[h][i] * own + (holds ? __ldcg(a.partial + row_dst[i] * D + h * 128 + tid) : 0.0f) * other;
          }
        }
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
        const float lse = sum == 0.0f ? -INFINITY : kMode == kSuffix && s.shared() ? m + log2f(sum) : (m + log2f(sum)) * kLn2;
#pragma unroll
        for (int i = 0; i < X::kRows; ++i) {
          const float f = __shfl_sync(kAll, inv, i), e = __shfl_sync(kAll, lse, i);
          if (i < rows) store_row(i, acc[0][i], acc[X::kHalves - 1][i], f, e);
        }
      } else {
        // A piece of an item: slot 0 where the item began before this CTA's run, slot 1 where it goes on after it.
        float* mine = partials + static_cast<int64_t>(blockIdx.x * 2 + (s.first ? 1 : 0)) * X::kPartialFloats;
        if (holds) {
#pragma unroll
          for (int i = 0; i < X::kRows; ++i)
#pragma unroll
            for (int h = 0; h < X::kHalves; ++h) mine[i * D + h * 128 + tid] = acc[h][i];
        }
        if (tid < X::kRows) {
          mine[X::kRows * D + tid] = m;
          mine[X::kRows * D + X::kRows + tid] = sum;
        }
        join_item<kMode, X::kRows, D, kCompute, 1>(a, s, row_dst, rows, ctas, total, tid, &s_last);
      }
      compute_sync();  // red, the rows' limits, the join word and the segment are free again
      if (tid == 0) {
        s_unit += s_segment.length;
        if (s_unit < stop) s_segment.next(a, prefix, shift, s_unit, stop);
      }
      compute_sync();
      if (s_unit >= stop) break;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, X::kTmem);
  }
  if (kMode == kPrefix && blockIdx.x == 0) grid_dependency_wait();
}

// CTAs of a call in row tiles of 8 * tile rows: as many as are resident together.
inline int decode_ctas(int head_dim, int tile, int sms) {
  int per_sm = 0;
  switch (head_dim * 8 + tile) {
    case 64 * 8 + 1: per_sm = Shape<64, 1>::kCtasPerSm; break;
    case 64 * 8 + 2: per_sm = Shape<64, 2>::kCtasPerSm; break;
    case 64 * 8 + 3: per_sm = Shape<64, 3>::kCtasPerSm; break;
    case 64 * 8 + 4: per_sm = Shape<64, 4>::kCtasPerSm; break;
    case 128 * 8 + 1: per_sm = Shape<128, 1>::kCtasPerSm; break;
    case 128 * 8 + 2: per_sm = Shape<128, 2>::kCtasPerSm; break;
    case 128 * 8 + 3: per_sm = Shape<128, 3>::kCtasPerSm; break;
    case 128 * 8 + 4: per_sm = Shape<128, 4>::kCtasPerSm; break;
    default: per_sm = 1;
  }
  return sms * per_sm < kMaxCtas ? sms * per_sm : kMaxCtas;
}
static_assert(Shape<256, 1>::kCtasPerSm == 1 && Shape<256, 2>::kCtasPerSm == 1, "heads of 256");

template <int kMode, int D, int RT>
cudaError_t launch_shape(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream) {
  const int smem = Shape<D, RT>::smem(a.b.requests);
  const cudaError_t e =
      cudaFuncSetAttribute(kv_attend_kernel<kMode, D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shape<D, RT>::smem(MOE_KV_MAX_REQUESTS));
  if (e != cudaSuccess) return e;
  return launch_chained(kv_attend_kernel<kMode, D, RT>, decode_ctas(D, RT, sms), Shape<D, RT>::kThreads, smem,
                        kMode != kWhole, stream, a, maps, shift);
}

// The form of row tiles of 8 * tile rows (heads of 256: of 16 at most).
template <int kMode>
cudaError_t launch_decode(const AttendArgs& a, const AttendMaps& maps, int tile, int shift, int sms, cudaStream_t stream) {
  switch (a.c.head_dim * 8 + tile) {
    case 64 * 8 + 1: return launch_shape<kMode, 64, 1>(a, maps, shift, sms, stream);
    case 64 * 8 + 2: return launch_shape<kMode, 64, 2>(a, maps, shift, sms, stream);
    case 64 * 8 + 3: return launch_shape<kMode, 64, 3>(a, maps, shift, sms, stream);
    case 64 * 8 + 4: return launch_shape<kMode, 64, 4>(a, maps, shift, sms, stream);
    case 128 * 8 + 1: return launch_shape<kMode, 128, 1>(a, maps, shift, sms, stream);
    case 128 * 8 + 2: return launch_shape<kMode, 128, 2>(a, maps, shift, sms, stream);
    case 128 * 8 + 3: return launch_shape<kMode, 128, 3>(a, maps, shift, sms, stream);
    case 128 * 8 + 4: return launch_shape<kMode, 128, 4>(a, maps, shift, sms, stream);
    case 256 * 8 + 1: return launch_shape<kMode, 256, 1>(a, maps, shift, sms, stream);
    default: return launch_shape<kMode, 256, 2>(a, maps, shift, sms, stream);
  }
}

}  // namespace
}  // namespace moe
