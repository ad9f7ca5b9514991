// Causal attention of new tokens over the paged 8-bit cache (moe_kv_attend in
// include/moe.h).
//
// The work is cut into tiles of 32 cache tokens of one item: a request, a
// cache head and 8 * RT of its query rows (token-major, the head's query heads
// within a token). All tiles in a row, [request][row tile][head][tile], are
// dealt to the CTAs in equal runs, so a long context is split over many CTAs
// and short ones share one. Within a CTA every warp streams its own tiles by
// TMA through its own ring and keeps a running maximum, sum and output; a
// segment (one item's tiles in this CTA) is joined in shared memory, and an item
// that spans CTAs by the last of them to finish, in CTA order.
//
// Both products run on the 8-bit tensor path, so the codes go from the cache to
// the matrix unit as they are. A query value is split into two e4m3 numbers,
// hi + lo / 16: together they hold the 8 significant bits of a BF16 exactly
// down to 2^-14 of the row's largest magnitude, and below that within 2^-22 of
// it. Rows 0-7 of the m16n8k32 product carry hi, rows 8-15 lo, and the two
// halves of the accumulator are added: one product serves 8 rows. The weights
// are split the same way: p = exp2(s - max over the tile) in [0, 1], times
// 256, within 2^-9 of p or 2^-22 of the tile's largest weight; their sum is
// taken of the unsplit values. Each tile's product joins the running output
// in FP32, with the tile's own maximum and value scale, so neither a dominant
// token nor an uneven page scale costs the others' precision.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kTile = 32;        // cache tokens of a tile
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;       // tiles of a warp's ring
constexpr int kItemTiles = 6;    // what starting and joining an item costs, in tiles
constexpr int kMaxCtas = 512;
constexpr int kCtasPerSm = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLo = 1.0f / 16.0f;  // lo parts are held 16 times as large
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kWaitNs = 2000000000ull;

// Workspace: the status word, one arrival counter for each CTA (zero between
// calls), two partial results for each CTA.
constexpr int kCounterOffset = 256;
constexpr int kPartialOffset = 4096;
static_assert(kCounterOffset + kMaxCtas * 4 <= kPartialOffset, "counters fit");

template <int D, int RT>
struct Shape {
  static constexpr int kRows = 8 * RT;
  static constexpr int kSteps = D / 32;                 // k32 steps of a score
  static constexpr int kCols = D / 8;                   // n8 columns of an output row
  static constexpr int kTileBytes = kTile * D;          // keys or values of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kHalves = D >= 128 ? D / 128 : 1;  // 128-byte spans of a row
  static constexpr int kSpan = D >= 128 ? 128 : 64;       // bytes of a row in one box
  static constexpr int kJoinStride = D + 4;
  static constexpr int kPartialFloats = kRows * (D + 2);  // rows, then maxima, then sums
  static constexpr int kRing = 0;
  static constexpr int kJoin = kRing + kWarps * kStages * kStageBytes;
  static constexpr int kStats = kJoin + kWarps * kRows * kJoinStride * 4;  // [warp][row] max, sum
  static constexpr int kMeta = kStats + kWarps * kRows * 8;
  static constexpr int kBars = kMeta + kWarps * kStages * 8;
  static constexpr int kPrefix = kBars + kWarps * kStages * 8;
  static constexpr int smem(int requests) { return kPrefix + (requests + 1) * 8 + 1024; }
  static_assert(kPartialOffset + 2ll * kMaxCtas * kPartialFloats * 4 <= MOE_KV_WORKSPACE_BYTES, "workspace");
};

__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma_e4m3_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// 2^x; what underflows FP32's normal range is zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(b - 127) of an E8M0 byte.
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack2(uint32_t codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
}

// hi and lo e4m3 words of four values of magnitude up to 256: v = hi + lo / 16.
__device__ __forceinline__ void split4(float v0, float v1, float v2, float v3, uint32_t& hi, uint32_t& lo) {
  const uint32_t h0 = pack2(v0, v1), h1 = pack2(v2, v3);
  const float2 f0 = unpack2(h0), f1 = unpack2(h1);
  hi = h0 | h1 << 16;
  lo = pack2((v0 - f0.x) * 16.0f, (v1 - f0.y) * 16.0f) | pack2((v2 - f1.x) * 16.0f, (v3 - f1.y) * 16.0f) << 16;
}

// r[i] = byte i of a, b, c, d.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&r)[4]) {
  const uint32_t ab = __byte_perm(a, b, 0x5140), cd = __byte_perm(c, d, 0x5140);
  const uint32_t ab2 = __byte_perm(a, b, 0x7362), cd2 = __byte_perm(c, d, 0x7362);
  r[0] = __byte_perm(ab, cd, 0x5410);
  r[1] = __byte_perm(ab, cd, 0x7632);
  r[2] = __byte_perm(ab2, cd2, 0x5410);
  r[3] = __byte_perm(ab2, cd2, 0x7632);
}

__device__ __forceinline__ uint32_t nan_code(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// Byte offset of 16-byte chunk c of row n in a tile's 128-byte (64-byte) spans,
// as the 128-byte (64-byte) TMA swizzle places it.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int n, int half, int c) {
  if (D >= 128) return half * (kTile * 128) + n * 128 + ((c ^ (n & 7)) << 4);
  return n * 64 + ((c ^ ((n >> 1) & 3)) << 4);
}

// A request's share of the work.
struct Request {
  int first, n, seq;       // first query row's token, query tokens, visible length
  int tile0, tiles;        // first tile that some query sees, their number (one at least)
  int row_tiles;
  __device__ Request(const AttendArgs& a, int shift, int r, int rows) {
    first = min(max(a.b.query_start[r], 0), a.b.tokens);
    n = min(max(a.b.query_start[r + 1], first), a.b.tokens) - first;
    seq = a.b.seq_lens[r];
    const long long room = static_cast<long long>(a.b.table_width) << shift;
    const int end = static_cast<int>(min(static_cast<long long>(max(seq, 0)), room));
    tile0 = a.window > 0 ? min(max(0, seq - n - a.window + 1), end) / kTile : 0;
    tiles = max(1, (end + kTile - 1) / kTile - tile0);
    row_tiles = (static_cast<int>(min(static_cast<long long>(n) * a.group, 0x7FFFFF00ll)) + rows - 1) / rows;
  }
  __device__ long long work(int heads) const { return static_cast<long long>(heads) * row_tiles * (tiles + kItemTiles); }
};

// A run of one item's tiles in this CTA (none, where the run covers only what the item's start counts).
struct Segment {
  int r, head, row_tile;
  int begin, end;          // tiles of the request, from tile0 on
  int length;              // in the units that the work is dealt in: kItemTiles for the item, then its tiles
  bool first, whole;       // the item starts here; and ends here too
  long long item;          // the item's first unit among all
  __device__ void find(const AttendArgs& a, const long long* prefix, int shift, int rows, long long x, long long stop) {
    int lo = 0, hi = a.b.requests;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= x) lo = mid;
      else hi = mid;
    }
    r = lo;
    const Request q(a, shift, r, rows);
    const int units = q.tiles + kItemTiles;
    const long long local = x - prefix[lo], index = local / units;
    const int from = static_cast<int>(local - index * units);
    const int to = static_cast<int>(min(static_cast<long long>(units), from + (stop - x)));
    item = x - from;
    length = to - from;
    whole = length == units;
    first = from == 0;
    begin = max(0, from - kItemTiles);
    end = max(0, to - kItemTiles);
    row_tile = static_cast<int>(index / a.c.kv_heads);
    head = static_cast<int>(index - static_cast<long long>(row_tile) * a.c.kv_heads);
  }
};

struct Maps {
  CUtensorMap k, v;  // [pages * heads][page_tokens][head_dim]
};

// A warp's stream of tiles over the CTA's segments, a ring ahead of their use.
template <int D, int RT>
struct Producer {
  using X = Shape<D, RT>;
  long long x, stop;
  Segment s;
  int tile, batch, slot;   // next tile, its place in the batch of 32 looked up together
  int pages[2];            // lane l: pages of the batch's tile l (two where a page holds 16 tokens)
  uint32_t scales;         // their key and value scales: k0, v0, k1, v1
  bool more;
  int tile0, end_token;

  __device__ void segment(const AttendArgs& a, const long long* prefix, int shift, int warp) {
    while (x < stop) {
      s.find(a, prefix, shift, X::kRows, x, stop);
      x += s.length;
      tile = s.begin + warp;
      batch = 0;
      if (tile < s.end) {
        const Request q(a, shift, s.r, X::kRows);
        tile0 = q.tile0;
        end_token = static_cast<int>(min(static_cast<long long>(max(q.seq, 0)), static_cast<long long>(a.b.table_width) << shift));
        return;
      }
    }
    more = false;
  }

  __device__ void look_up(const AttendArgs& a, int shift, int lane) {
    scales = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = tile + lane * kWarps;
      const long long token = static_cast<long long>(tile0 + t) * kTile + 16 * i;
      int page = -1;
      if (t < s.end && token < end_token && (i == 0 || shift == 4))
        page = a.b.block_table[s.r * a.b.table_stride + (token >> shift)];
      if (page >= a.c.pages) page = -1;
      if (page >= 0) {
        const long long at = static_cast<long long>(page) * a.c.kv_heads + s.head;
        scales |= (a.c.k_scale[at] | static_cast<uint32_t>(a.c.v_scale[at]) << 8) << (16 * i);
      }
      pages[i] = page;
    }
  }

  // Start the copies of the next tile into the ring's next slot.
  __device__ void issue(const AttendArgs& a, const Maps& maps, const long long* prefix, int shift, int warp, int lane,
                        uint8_t* ring, uint64_t* bars, uint2* meta, uint64_t policy) {
    if (!more) return;
    if (batch == 0) look_up(a, shift, lane);
    const int p0 = __shfl_sync(kAll, pages[0], batch), p1 = __shfl_sync(kAll, pages[1], batch);
    const uint32_t sc = __shfl_sync(kAll, scales, batch);
    // Lane 0 announces the bytes; then one lane for each box: keys and values, page halves, 128-byte spans.
    constexpr int kBoxes = 4 * X::kHalves;
    uint8_t* dst = ring + slot * X::kStageBytes;
    uint64_t* bar = bars + slot;
    if (lane == 0) {
      meta[slot] = make_uint2(sc, shift == 4 ? (p0 >= 0) | (p1 >= 0) << 1 : (p0 >= 0 ? 3u : 0u));
      const uint32_t bytes = shift == 4 ? X::kStageBytes / 2 : X::kStageBytes;
      if (p0 >= 0 || p1 >= 0) mbar_arrive_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * bytes);
      else mbar_arrive(bar);
    }
    __syncwarp();
    const int second = (lane >> 1) & 1, half = lane >> 2, p = second ? p1 : p0;
    if (lane < kBoxes && p >= 0)
      tma_load_3d(dst + (lane & 1) * X::kTileBytes + half * (kTile * X::kSpan) + second * (16 * X::kSpan),
                  lane & 1 ? &maps.v : &maps.k, half * X::kSpan, ((tile0 + tile) * kTile) & (a.c.page_tokens - 1),
                  p * a.c.kv_heads + s.head, bar, policy);
    slot = slot + 1 == kStages ? 0 : slot + 1;
    batch = (batch + 1) & 31;
    tile += kWarps;
    if (tile >= s.end) segment(a, prefix, shift, warp);
  }
};

// Bounded wait for a tile's copies. Once one has run out the call's outputs are void, and later waits, which
// see the status word set, give up at once.
__device__ __noinline__ void wait_slot(uint64_t* bar, uint32_t parity, int32_t* status) {
  const uint64_t began = global_timer_ns();
  while (!mbar_wait_hint(bar, parity, 20000)) {
    if (global_timer_ns() - began > kWaitNs || *reinterpret_cast<volatile int32_t*>(status) != 0) {
      report(status, MOE_ERR_DEVICE_TIMEOUT);
      return;
    }
  }
}

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2) kv_attend_kernel(const AttendArgs a, const __grid_constant__ Maps maps,
                                                             int shift) {
  using X = Shape<D, RT>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = sm + X::kRing + warp * kStages * X::kStageBytes;
  float* join = reinterpret_cast<float*>(sm + X::kJoin);
  float* stats = reinterpret_cast<float*>(sm + X::kStats);
  uint2* meta = reinterpret_cast<uint2*>(sm + X::kMeta) + warp * kStages;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + X::kBars) + warp * kStages;
  long long* prefix = reinterpret_cast<long long*>(sm + X::kPrefix);
  __shared__ long long s_sum[kWarps];
  __shared__ int s_last;
  int32_t* status = reinterpret_cast<int32_t*>(a.workspace);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace + kCounterOffset);
  float* partials = reinterpret_cast<float*>(a.workspace + kPartialOffset);

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars + i, 1);
    fence_mbar_init();
  }
  // Prefix sums of the requests' work.
  {
    const int per = (a.b.requests + kThreads - 1) / kThreads;
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r < a.b.requests) sum += Request(a, shift, r, X::kRows).work(a.c.kv_heads);
    }
    long long in = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(kAll, in, d);
      if (lane >= d) in += u;
    }
    if (lane == 31) s_sum[warp] = in;
    __syncthreads();
    long long at = in - sum;
    for (int w = 0; w < warp; ++w) at += s_sum[w];
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r < a.b.requests) {
        prefix[r] = at;
        at += Request(a, shift, r, X::kRows).work(a.c.kv_heads);
        if (r == a.b.requests - 1) prefix[r + 1] = at;
      }
    }
    __syncthreads();
  }
  const long long total = prefix[a.b.requests];
  // Each CTA gets at least an item's start and a tile for each of its warps.
  constexpr int kLeast = kItemTiles + kWarps;
  const long long ctas = min(static_cast<long long>(gridDim.x), (total + kLeast - 1) / kLeast);
  if (blockIdx.x >= ctas) return;
  const long long start = total * blockIdx.x / ctas, stop = total * (blockIdx.x + 1) / ctas;

  const uint64_t policy = policy_evict_first();
  Producer<D, RT> p;
  p.x = start;
  p.stop = stop;
  p.more = true;
  p.slot = 0;
  p.segment(a, prefix, shift, warp);
  for (int i = 0; i < kStages; ++i) p.issue(a, maps, prefix, shift, warp, lane, ring, bars, meta, policy);

  int slot = 0;
  uint32_t phase = 0;
  for (long long x = start; x < stop;) {
    Segment s;
    s.find(a, prefix, shift, X::kRows, x, stop);
    const Request rq(a, shift, s.r, X::kRows);
    const int rows = rq.n * a.group - s.row_tile * X::kRows;  // of this item, if under kRows
    // The lane's query rows: limits, factor, hi and lo words.
    uint32_t qa[RT][X::kSteps][4];
    float factor[RT];
    int lo[RT], hi[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int i = rt * 8 + g, row = s.row_tile * X::kRows + i;
      const bool used = i < rows;
      const int tok = row / a.group, h = s.head * a.group + row - tok * a.group;
      hi[rt] = used ? rq.seq - rq.n + tok : -1;
      lo[rt] = used && a.window > 0 ? max(0, hi[rt] - a.window + 1) : 0;
      const uint16_t* src = a.q + (rq.first + (used ? tok : 0)) * a.q_token_stride + h * a.q_head_stride;
      uint32_t top = 0;
      uint4 w[X::kSteps];
#pragma unroll
      for (int st = 0; st < X::kSteps; ++st) {
        const int dim = D >= 128 ? (st / 4) * 128 + t4 * 32 + (st % 4) * 8 : t4 * 16 + st * 8;
        w[st] = used ? *reinterpret_cast<const uint4*>(src + dim) : make_uint4(0, 0, 0, 0);
        const uint32_t e[4] = {w[st].x, w[st].y, w[st].z, w[st].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(e[j] & 0x7FFFu, (e[j] >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(kAll, top, 1));
      top = max(top, __shfl_xor_sync(kAll, top, 2));
      // Scaled by a power of two so that the row's largest magnitude lies in [128, 256).
      int e = static_cast<int>(top >> 7) - 127 - 7;
      if (e < -120) e = -120;
      const float down = top == 0 ? 1.0f : pow2f(-e);
      factor[rt] = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : top == 0 ? 0.0f : a.scale * kLog2e * pow2f(e);
#pragma unroll
      for (int st = 0; st < X::kSteps; ++st) {
        const uint32_t v[4] = {w[st].x, w[st].y, w[st].z, w[st].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = __uint_as_float(v[j] << 16) * down;
          f[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u) * down;
        }
        split4(f[0], f[1], f[2], f[3], qa[rt][st][0], qa[rt][st][1]);
        split4(f[4], f[5], f[6], f[7], qa[rt][st][2], qa[rt][st][3]);
      }
    }
    // Over the item's rows: tokens that any of them sees, and that all see.
    int any_lo = 0x7FFFFFFF, any_hi = -1, all_lo = 0, all_hi = 0x7FFFFFFF;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const bool used = rt * 8 + g < rows;
      any_lo = min(any_lo, used ? lo[rt] : 0x7FFFFFFF);
      any_hi = max(any_hi, hi[rt]);
      all_lo = max(all_lo, lo[rt]);
      all_hi = min(all_hi, used ? hi[rt] : 0x7FFFFFFF);
    }
    any_lo = __reduce_min_sync(kAll, any_lo);
    any_hi = __reduce_max_sync(kAll, any_hi);
    all_lo = __reduce_max_sync(kAll, all_lo);
    all_hi = __reduce_min_sync(kAll, all_hi);

    float acc[RT][X::kCols][2], m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY;
      l[rt] = 0.0f;
#pragma unroll
      for (int i = 0; i < X::kCols; ++i) acc[rt][i][0] = acc[rt][i][1] = 0.0f;
    }

    for (int tile = s.begin + warp; tile < s.end; tile += kWarps) {
      if (!mbar_test(bars + slot, phase)) wait_slot(bars + slot, phase, status);
      __syncwarp();
      const uint2 info = meta[slot];
      const uint8_t* keys = ring + slot * X::kStageBytes;
      const uint8_t* vals = keys + X::kTileBytes;
      const int base = (rq.tile0 + tile) * kTile;
      const bool edge = info.y != 3u || base < all_lo || base + kTile - 1 > all_hi;

      const float ks0 = scale_of(info.x & 0xFFu), ks1 = shift == 4 ? scale_of((info.x >> 16) & 0xFFu) : ks0;
      // Scores of 32 tokens: lane (g, t4) holds row g's of tokens 8 q + 2 t4 + {0, 1}.
      float sc[RT][4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float c[RT][4];
#pragma unroll
        for (int j = 0; j < X::kSteps / 2; ++j) {  // 16 bytes of a key: two steps
          const int half = D >= 128 ? j / 2 : 0, c16 = D >= 128 ? t4 * 2 + j % 2 : t4;
          const uint4 k = *reinterpret_cast<const uint4*>(keys + chunk_at<D>(8 * q + g, half, c16));
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if (j == 0) mma_e4m3_first(c[rt], qa[rt][0], k.x, k.y);
            else mma_e4m3(c[rt], qa[rt][2 * j], k.x, k.y);
            mma_e4m3(c[rt], qa[rt][2 * j + 1], k.z, k.w);
          }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float f = factor[rt] * (q < 2 ? ks0 : ks1);
          sc[rt][q][0] = fmaf(c[rt][2], kLo, c[rt][0]) * f;
          sc[rt][q][1] = fmaf(c[rt][3], kLo, c[rt][1]) * f;
        }
      }
      if (edge) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = base + 8 * q + 2 * t4 + e;
              if (j < lo[rt] || j > hi[rt] || !(info.y >> (q >> 1) & 1)) sc[rt][q][e] = -INFINITY;
            }
      }
      // Weights against the tile's own maximum, split for the second product.
      const int vb0 = (info.x >> 8) & 0xFF;
      float up0 = 256.0f, up1 = 256.0f, vs = scale_of(vb0) * (1.0f / 256.0f);
      if (shift == 4) {  // two pages: to the larger of their scales
        const int vb1 = info.x >> 24, vb = max(vb0, vb1);
        up0 *= pow2f(max(vb0 - vb, -126));
        up1 *= pow2f(max(vb1 - vb, -126));
        vs = scale_of(vb) * (1.0f / 256.0f);
      }
      uint32_t pa[RT][4];
      float into[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = fmaxf(sc[rt][0][0], sc[rt][0][1]);
#pragma unroll
        for (int q = 1; q < 4; ++q) top = fmaxf(top, fmaxf(sc[rt][q][0], sc[rt][q][1]));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
        const float ref = top == -INFINITY ? 0.0f : top;
        float w[4][2], sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            w[q][e] = exp2_fast(sc[rt][q][e] - ref);
            sum += w[q][e];
            w[q][e] *= q < 2 ? up0 : up1;
          }
        split4(w[0][0], w[0][1], w[1][0], w[1][1], pa[rt][0], pa[rt][1]);
        split4(w[2][0], w[2][1], w[3][0], w[3][1], pa[rt][2], pa[rt][3]);
        const float mn = fmaxf(m[rt], top);
        const float safe = mn == -INFINITY ? 0.0f : mn;
        const float keep = exp2_fast(m[rt] - safe), add = exp2_fast(top - safe);
        l[rt] = l[rt] * keep + sum * add;
        into[rt] = add * vs;
        m[rt] = mn;
        if (__any_sync(kAll, keep != 1.0f)) {
#pragma unroll
          for (int i = 0; i < X::kCols; ++i) {
            acc[rt][i][0] *= keep;
            acc[rt][i][1] *= keep;
          }
        }
      }
      // Output += weights x values. Values that no row sees are dropped; where rows see different
      // tokens and one of them holds a NaN, each row takes a pass of its own.
      int passes = 1;
      if (edge && (any_hi != all_hi || any_lo != all_lo)) {
        uint32_t nan = 0;
        for (int i = lane; i < X::kTileBytes / 16; i += 32) {
          const uint4 w = *reinterpret_cast<const uint4*>(vals + 16 * i);
          nan |= nan_code(w.x) | nan_code(w.y) | nan_code(w.z) | nan_code(w.w);
        }
        if (__any_sync(kAll, nan != 0)) passes = X::kRows;
      }
      for (int pass = 0; pass < passes; ++pass) {
        int from = any_lo, to = any_hi;
        if (passes > 1) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const int f = __shfl_sync(kAll, lo[rt], (pass & 7) * 4), u = __shfl_sync(kAll, hi[rt], (pass & 7) * 4);
            if (rt == pass >> 3) {
              from = f;
              to = u;
            }
          }
        }
#pragma unroll
        for (int half = 0; half < X::kHalves; ++half) {
          constexpr int kWords = D >= 128 ? 4 : 2;  // of the lane's values of a token, in this span
          uint32_t v[8][kWords];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int n = 8 * (i >> 1) + 2 * t4 + (i & 1);
            if (D >= 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(vals + chunk_at<D>(n, half, g));
              v[i][0] = w.x;
              v[i][1] = w.y;
              v[i][2 % kWords] = w.z;
              v[i][3 % kWords] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(vals + chunk_at<D>(n, half, g >> 1) + (g & 1) * 8);
              v[i][0] = w.x;
              v[i][1] = w.y;
            }
            if (edge) {
              const int j = base + n;
              if (j < from || j > to || !(info.y >> (i >> 2) & 1)) {
#pragma unroll
                for (int k = 0; k < kWords; ++k) v[i][k] = 0;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < kWords; ++k) {
            uint32_t b0[4], b1[4];
            transpose4(v[0][k], v[1][k], v[2][k], v[3][k], b0);
            transpose4(v[4][k], v[5][k], v[6][k], v[7][k], b1);
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                float c[4];
                mma_e4m3_first(c, pa[rt], b0[b], b1[b]);
                const int i = half * 16 + 4 * k + b;
                if (passes == 1 || (pass & 7) == g && rt == pass >> 3) {
                  acc[rt][i][0] += fmaf(c[2], kLo, c[0]) * into[rt];
                  acc[rt][i][1] += fmaf(c[3], kLo, c[1]) * into[rt];
                }
              }
          }
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      p.issue(a, maps, prefix, shift, warp, lane, ring, bars, meta, policy);
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
    }

    // Join the warps: the lane holds columns 32 t4 .. + 31 of each 128 of its row (16 t4 .. + 15 of 64).
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] += __shfl_xor_sync(kAll, l[rt], 1);
      l[rt] += __shfl_xor_sync(kAll, l[rt], 2);
      if (t4 == 0) {
        stats[(warp * X::kRows + rt * 8 + g) * 2] = m[rt];
        stats[(warp * X::kRows + rt * 8 + g) * 2 + 1] = l[rt];
      }
      float* row = join + (warp * X::kRows + rt * 8 + g) * X::kJoinStride;
#pragma unroll
      for (int half = 0; half < X::kHalves; ++half) {
        constexpr int kPer = D >= 128 ? 16 : 8;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < kPer; i += 4)
            *reinterpret_cast<float4*>(row + half * 128 + (2 * t4 + e) * kPer + i) =
                make_float4(acc[rt][half * 16 + i][e], acc[rt][half * 16 + i + 1][e], acc[rt][half * 16 + i + 2][e],
                            acc[rt][half * 16 + i + 3][e]);
      }
    }
    __syncthreads();
    const int part = s.first ? 1 : 0;  // an item that began before this CTA's run, or goes on after it
    float* mine = partials + static_cast<int64_t>(blockIdx.x * 2 + part) * X::kPartialFloats;
    for (int i = tid; i < X::kRows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), c = (i % (D / 4)) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[(w * X::kRows + row) * 2]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(stats[(w * X::kRows + row) * 2] - ref);
        sum += stats[(w * X::kRows + row) * 2 + 1] * f;
        const float4 u = *reinterpret_cast<const float4*>(join + (w * X::kRows + row) * X::kJoinStride + c);
        o.x += u.x * f;
        o.y += u.y * f;
        o.z += u.z * f;
        o.w += u.w * f;
      }
      if (!s.whole) {
        *reinterpret_cast<float4*>(mine + row * D + c) = o;
        if (c == 0) {
          mine[X::kRows * D + row] = top;
          mine[X::kRows * D + X::kRows + row] = sum;
        }
      } else if (row < rows) {
        const int at = s.row_tile * X::kRows + row, tok = at / a.group;
        const int64_t dst = static_cast<int64_t>(rq.first + tok) * a.q_heads + s.head * a.group + at - tok * a.group;
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
        __nv_bfloat162 u[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
        *reinterpret_cast<uint2*>(a.out + dst * D + c) = *reinterpret_cast<uint2*>(u);
        if (a.lse != nullptr && c == 0) a.lse[dst] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
    }
    if (!s.whole) {
      // The CTAs of this item: first .. last, by their runs' bounds.
      const long long item_end = s.item + rq.tiles + kItemTiles - 1;
      const int c0 = static_cast<int>(((s.item + 1) * ctas - 1) / total);
      const int c1 = static_cast<int>(((item_end + 1) * ctas - 1) / total);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t before = atom_add_acq_rel_gpu(counters + c0, 1);
        s_last = before == static_cast<uint32_t>(c1 - c0);
        if (s_last) counters[c0] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int i = tid; i < X::kRows * (D / 4); i += kThreads) {
          const int row = i / (D / 4), c = (i % (D / 4)) * 4;
          if (row >= rows) continue;
          float top = -INFINITY, sum = 0.0f;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int cta = c0; cta <= c1; ++cta) {
            const float* from = partials + static_cast<int64_t>(cta * 2 + (cta == c0)) * X::kPartialFloats;
            const float pm = __ldcg(from + X::kRows * D + row), pl = __ldcg(from + X::kRows * D + X::kRows + row);
            const float4 u = __ldcg(reinterpret_cast<const float4*>(from + row * D + c));
            const float mn = fmaxf(top, pm), ref = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2f(top - ref), h = exp2f(pm - ref);
            o.x = o.x * f + u.x * h;
            o.y = o.y * f + u.y * h;
            o.z = o.z * f + u.z * h;
            o.w = o.w * f + u.w * h;
            sum = sum * f + pl * h;
            top = mn;
          }
          const int at = s.row_tile * X::kRows + row, tok = at / a.group;
          const int64_t dst = static_cast<int64_t>(rq.first + tok) * a.q_heads + s.head * a.group + at - tok * a.group;
          const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
          __nv_bfloat162 u[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
          *reinterpret_cast<uint2*>(a.out + dst * D + c) = *reinterpret_cast<uint2*>(u);
          if (a.lse != nullptr && c == 0) a.lse[dst] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
      }
    }
    __syncthreads();  // the join buffers are free again
    x += s.length;
  }
}

cudaError_t encode_map(CUtensorMap* map, const uint8_t* data, const moe_kv_cache_t& c) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> entry{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 encode = entry.load(std::memory_order_acquire);
  if (encode == nullptr) {
    cudaDriverEntryPointQueryResult found{};
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", reinterpret_cast<void**>(&encode),
                                                           12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (encode == nullptr || found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    entry.store(encode, std::memory_order_release);
  }
  const cuuint64_t D = c.head_dim, P = c.page_tokens;
  const cuuint64_t dims[3] = {D, P, static_cast<cuuint64_t>(c.pages) * c.kv_heads};
  const cuuint64_t strides[2] = {D, D * P};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(D < 128 ? D : 128), static_cast<cuuint32_t>(P < kTile ? P : kTile), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(data), dims, strides, box, elem,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int RT>
cudaError_t launch_shape(const AttendArgs& a, const Maps& maps, int shift, cudaStream_t stream) {
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  const int smem = Shape<D, RT>::smem(a.b.requests);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv_attend_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shape<D, RT>::smem(MOE_KV_MAX_REQUESTS));
  if (e != cudaSuccess) return e;
  const int grid = sms * kCtasPerSm < kMaxCtas ? sms * kCtasPerSm : kMaxCtas;
  kv_attend_kernel<D, RT><<<grid, kThreads, smem, stream>>>(a, maps, shift);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const AttendArgs& a, const Maps& maps, int shift, cudaStream_t stream) {
  // One row tile of 8 where a request has no more rows on average.
  const long long rows = static_cast<long long>(a.b.tokens) * a.group;
  if (rows <= 8ll * a.b.requests) return launch_shape<D, 1>(a, maps, shift, stream);
  return launch_shape<D, 2>(a, maps, shift, stream);
}

}  // namespace

cudaError_t launch_kv_attend(const AttendArgs& a, cudaStream_t stream) {
  int shift = 4;
  while ((1 << shift) < a.c.page_tokens) ++shift;
  Maps maps;
  cudaError_t e = encode_map(&maps.k, a.c.k, a.c);
  if (e == cudaSuccess) e = encode_map(&maps.v, a.c.v, a.c);
  if (e != cudaSuccess) return e;
  if (a.c.head_dim == 64) return launch_dim<64>(a, maps, shift, stream);
  if (a.c.head_dim == 128) return launch_dim<128>(a, maps, shift, stream);
  return launch_dim<256>(a, maps, shift, stream);
}

}  // namespace moe
