// Building blocks of the attention kernels over the paged 8-bit cache
// (kv_attend.cu, kv_attend_rows.cu): the work split, the tile stream, the
// tensor-core and numeric primitives, the join of an item's pieces. Each
// translation unit that includes it gets its own copy (internal linkage).
//
// An item is a request, a cache head and a run of its query rows (token-major,
// the head's query heads within a token). Its cache tokens are cut into tiles
// of 128; all tiles in a row, [request][row tile][head][tile], are dealt to the
// CTAs in equal runs, so a long context is split over many CTAs and short ones
// share one. Results are sums over pieces in CTA order, whoever adds them.
#pragma once

#include <cuda_fp16.h>

#include "decode.h"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kTile = 128;        // cache tokens of a tile
constexpr int kCompute = 128;     // threads of a compute warpgroup
constexpr int kMaxPages = 8;      // pages of a tile
constexpr int kMaxCtas = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHighest = 8.0f;       // a weight may grow to 2^8 times its reference's: room for sums of large values
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kWaitNs = 2000000000ull;

// Workspace: the status word, arrival counters (zero between calls: for the
// runs of pieces that start with an item, for its other runs, for the item;
// each under the CTA of the first piece), two partial results for each CTA.
constexpr int kCounterOffset = 256;
constexpr int kPartialOffset = MOE_KV_WORKSPACE_HEADER;
static_assert(kCounterOffset + 3 * kMaxCtas * 4 <= kPartialOffset, "counters fit");


// ---------------------------------------------------------------- tensor core
// D[tmem] (+)= A[smem] x B[smem], e4m3 operands, FP32 accumulation; K = 32.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// M = 128 rows of A, N columns of B, FP32 accumulator; either transposed (its rows contiguous); B e4m3, A e4m3 or e5m2.
__host__ __device__ constexpr uint32_t idesc_f8(int n, bool a_transposed, bool b_transposed = false, bool a_e5m2 = false) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((a_transposed ? 1u : 0u) << 15) |
         ((b_transposed ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

// The same with BF16 operands; K = 16.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A in TMEM, a row to a lane, two values to a column.
__device__ __forceinline__ void mma_bf16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool a_transposed, bool b_transposed = false) {
  return idesc_f8(n, a_transposed, b_transposed) | (1u << 7) | (1u << 10);
}

__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// ------------------------------------------------------------------- numerics
// 2^x; what underflows FP32's normal range is zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(b - 127) of an E8M0 byte.
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// Warp maximum (NaN loses).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack2(uint32_t codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
}

// Codes of two values of magnitude up to 448: e4m3 hi and lo, v = hi + lo / 16.
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack2(v0, v1);
  const float2 f = unpack2(hi);
  lo = pack2((v0 - f.x) * 16.0f, (v1 - f.y) * 16.0f);
}

// Two weights as BF16 hi and lo: 16 bits of each, whatever its magnitude.
__device__ __forceinline__ void split2_bf16(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(v0 - __uint_as_float(hi << 16), v1 - __uint_as_float(hi & 0xFFFF0000u));
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Codes of two values: e4m3 hi and e5m2 lo, v = hi + lo.
__device__ __forceinline__ void split2_wide(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack2(v0, v1);
  const float2 f = unpack2(hi);
  lo = __nv_cvt_float2_to_fp8x2(make_float2(v0 - f.x, v1 - f.y), __NV_SATFINITE, __NV_E5M2);
}

// Values in BF16 are the code times its page's scale, exact. What leaves BF16's range (scales of 2^120 and more) or is a
// NaN is not finite there, and a weight of zero would not drop it: codes from a limit on, in magnitude. finite_limit is
// what takes each byte's magnitude to 128 from there on.
__device__ __forceinline__ uint32_t finite_limit(uint32_t scale) {
  return (scale < 247 ? 1u : scale == 255 ? 128u : 8 + 8 * (scale - 247)) * 0x01010101u;
}
__device__ __forceinline__ uint32_t not_finite(uint32_t codes, uint32_t limit) {
  return ((codes & 0x7F7F7F7Fu) + limit) & 0x80808080u;
}
__device__ __forceinline__ bool any_not_finite(const uint4& codes, uint32_t limit) {
  return (not_finite(codes.x, limit) | not_finite(codes.y, limit) | not_finite(codes.z, limit) | not_finite(codes.w, limit)) != 0;
}

// 2^(b - 127) of an E8M0 byte, twice.
__device__ __forceinline__ __nv_bfloat162 scale2_of(uint32_t b) {
  const uint32_t one = b ? b << 7 : 0x0040u, both = one | one << 16;
  return *reinterpret_cast<const __nv_bfloat162*>(&both);
}

// Four codes -> four values times `scale`.
__device__ __forceinline__ uint2 widen(uint32_t codes, __nv_bfloat162 scale) {
  const float2 a = unpack2(codes & 0xFFFFu), b = unpack2(codes >> 16);
  const __nv_bfloat162 v0 = __hmul2(__floats2bfloat162_rn(a.x, a.y), scale), v1 = __hmul2(__floats2bfloat162_rn(b.x, b.y), scale);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
}

// Takes the codes that are not finite out of a chunk of 16; their places as bits.
__device__ __forceinline__ uint32_t take_out(uint4& codes, uint32_t limit) {
  uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w}, places = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bad = not_finite(w[i], limit) >> 7;
    w[i] &= ~(bad * 0xFFu);
    places |= ((bad & 1u) | (bad >> 7 & 2u) | (bad >> 14 & 4u) | (bad >> 21 & 8u)) << (4 * i);
  }
  codes = make_uint4(w[0], w[1], w[2], w[3]);
  return places;
}

// Byte offset of 16-byte chunk c of row n in an image of kSpan-byte rows, as the swizzle of that width places it.
template <int kSpan>
__device__ __forceinline__ uint32_t chunk_at(int n, int c) {
  return kSpan == 128 ? n * 128 + ((c ^ (n & 7)) << 4) : n * 64 + ((c ^ ((n >> 1) & 3)) << 4);
}

// x / group for rows x of a row tile (from its first token's first row on, so below 2048): `inverse` is 2^32 / group,
// rounded up, or 0 for a group of one.
__device__ __forceinline__ uint32_t inverse_of(int group) { return group > 1 ? 0xFFFFFFFFu / group + 1 : 0; }
__device__ __forceinline__ int per_group(int x, uint32_t inverse) {
  return inverse ? static_cast<int>(__umulhi(x, inverse)) : x;
}

// ----------------------------------------------------------------------- work
// a / b of numbers that mostly fit 32 bits, where the division is far shorter.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A request's share of the work.
struct Request {
  int first, n, seq;       // first query row's token, query tokens, visible length
  int end;                 // tokens that the table has room for
  int tile0, tiles;        // first tile that some query sees, their number (one at least)
  int row_tiles;
  Request() = default;
  __device__ Request(const AttendArgs& a, int shift, int r, int rows) {
    first = min(max(a.b.query_start[r], 0), a.b.tokens);
    n = min(max(a.b.query_start[r + 1], first), a.b.tokens) - first;
    seq = a.b.seq_lens[r];
    const long long room = static_cast<long long>(a.b.table_width) << shift;
    end = static_cast<int>(min(static_cast<long long>(max(seq, 0)), room));
    tile0 = a.window > 0 ? static_cast<int>(min(max(0ll, static_cast<long long>(seq) - n - a.window + 1), static_cast<long long>(end))) / kTile : 0;
    tiles = max(1, (end + kTile - 1) / kTile - tile0);
    row_tiles = static_cast<int>((static_cast<long long>(n) * a.group + rows - 1) / rows);
  }
  __device__ long long items(int heads) const { return static_cast<long long>(heads) * row_tiles; }
};

// The tiles that each row tile of a request sees. In the 128-row form, which prompts take, they are counted exactly: a
// row tile's 128 rows advance the visible tokens by 128 / group, so row tile j sees the tiles from max(0, low + j) / group
// to before (high + j) / group. In the decode form, whose row tiles differ by a few tokens, each counts them all.
template <int kRows>
struct RowTiles {
  long long low = 0, high = 0;
  int group;
  __device__ __forceinline__ RowTiles(const AttendArgs& a, const Request& q) : group(a.group) {
    if constexpr (kRows != kTile) return;
    const long long before = max(0, q.seq - q.n);
    high = (before * group + kTile + kTile * group - 1) >> 7;
    low = a.window > 0 ? (before - a.window + 1) * group >> 7 : -(1ll << 40);
  }
  // The sum of i / group over 0 <= i < x.
  __device__ __forceinline__ long long sum(long long x) const {
    if (x <= group) return 0;
    const long long n = divide(x, group);
    return n * (n - 1) / 2 * group + n * (x - n * group);
  }
  // The tiles of the row tiles before j (j < row_tiles).
  __device__ __forceinline__ long long before(const Request& q, int j) const {
    if constexpr (kRows != kTile) return static_cast<long long>(j) * q.tiles;
    return sum(high + j) - sum(high) - (sum(low + j) - sum(low));
  }
  __device__ __forceinline__ int first(const Request& q, int j) const {
    if constexpr (kRows != kTile) return q.tile0;
    return static_cast<int>(divide(max(0ll, low + j), group));
  }
  __device__ __forceinline__ int count(const Request& q, int j) const {
    if constexpr (kRows != kTile) return q.tiles;
    const int from = first(q, j), to = static_cast<int>(divide(high + j, group));
    return max(1, (j + 1 == q.row_tiles ? min(to, q.tile0 + q.tiles) : to) - from);
  }
  __device__ __forceinline__ long long all(const Request& q) const {
    return q.row_tiles == 0 ? 0 : before(q, q.row_tiles - 1) + count(q, q.row_tiles - 1);
  }
};
static_assert(kTile == 128, "RowTiles' shifts");

// A run of one item's tiles in this CTA (none, where the run covers only what the item's start counts).
template <int kRows>
struct Segment {
  Request q;
  int r, head, row_tile;
  int token, within;       // the row tile's first query token, its first row among that token's
  int tile_first, units;   // the item's first tile, from q.tile0 on; its length in the units of the work
  int begin, end;          // tiles of the request, from q.tile0 on
  int weight;              // what starting and joining an item counts as, in tiles
  int length;              // in the units that the work is dealt in: `weight` for the item, then its tiles
  bool first, whole;       // the item starts here; and ends here too
  long long item;          // the item's first unit among all

  // The item's tiles from unit `from` on, as far as the run goes and this row tile's queries see.
  __device__ __forceinline__ void cut(const AttendArgs& a, long long x, long long stop, int from) {
    const int to = static_cast<int>(min(static_cast<long long>(units), from + (stop - x)));
    item = x - from;
    length = to - from;
    whole = length == units;
    first = from == 0;
    begin = tile_first + max(0, from - weight);
    end = tile_first + max(0, to - weight);
    const int before = q.seq - q.n;  // position of the request's first query
    const int last = min(q.n - 1, static_cast<int>((static_cast<long long>(row_tile + 1) * kRows - 1) / a.group));
    end = min(end, (min(q.end, max(0, before + last + 1)) + kTile - 1) / kTile - q.tile0);
    if (a.window > 0) {
      const long long from_token = static_cast<long long>(before) + static_cast<long long>(row_tile) * kRows / a.group - a.window + 1;
      begin = max(begin, static_cast<int>(max(from_token, 0ll) / kTile) - q.tile0);
    }
    if (begin >= end) begin = end = 0;
  }

  __device__ __forceinline__ void take(const RowTiles<kRows>& t) {
    const long long row0 = static_cast<long long>(row_tile) * kRows;
    token = static_cast<int>(divide(row0, t.group));
    within = static_cast<int>(row0 - static_cast<long long>(token) * t.group);
    tile_first = t.first(q, row_tile) - q.tile0;
    units = t.count(q, row_tile) + weight;
  }

  // The segment at unit x of a run that ends at `stop`.
  __device__ void find(const AttendArgs& a, const long long* prefix, int item_weight, int shift, long long x,
                       long long stop) {
    weight = item_weight;
    int lo = 0, hi = a.b.requests;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= x) lo = mid;
      else hi = mid;
    }
    r = lo;
    q = Request(a, shift, r, kRows);
    const RowTiles<kRows> t(a, q);
    const long long local = x - prefix[lo];
    lo = 0;
    hi = q.row_tiles;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((t.before(q, mid) + static_cast<long long>(mid) * weight) * a.c.kv_heads <= local) lo = mid;
      else hi = mid;
    }
    row_tile = lo;
    take(t);
    const long long in_row_tile = local - (t.before(q, lo) + static_cast<long long>(lo) * weight) * a.c.kv_heads;
    head = static_cast<int>(divide(in_row_tile, units));
    cut(a, x, stop, static_cast<int>(in_row_tile - static_cast<long long>(head) * units));
  }

  // The one after it, at unit x < stop: an item's start.
  __device__ __forceinline__ void next(const AttendArgs& a, const long long* prefix, int shift, long long x, long long stop) {
    if (++head == a.c.kv_heads) {
      head = 0;
      if (++row_tile == q.row_tiles) {
        row_tile = 0;
        do ++r;
        while (prefix[r + 1] == x);  // requests without rows
        q = Request(a, shift, r, kRows);
      }
      take(RowTiles<kRows>(a, q));
    }
    cut(a, x, stop, 0);
  }
};

// What a row tile's rows see: the tokens that any of them sees and those that all see. Rows of later tokens see later ones.
struct Sight {
  int any_lo, any_hi, all_lo, all_hi;
  int rows;      // of the row tile
  bool mixed;    // its rows see different tokens
  int within, window;
  uint32_t inverse;
  template <int kRows>
  __device__ __forceinline__ Sight(const AttendArgs& a, const Segment<kRows>& s, uint32_t inverse)
      : within(s.within), window(a.window), inverse(inverse) {
    rows = static_cast<int>(min(static_cast<long long>(s.q.n - s.token) * a.group - s.within, static_cast<long long>(kRows)));
    all_hi = s.q.seq - s.q.n + s.token;
    any_hi = last(rows - 1);
    any_lo = first(all_hi);
    all_lo = first(any_hi);
    mixed = any_lo != all_lo || any_hi != all_hi;
  }
  // The last token that row i sees, and the first that a row with this last one sees.
  __device__ __forceinline__ int last(int i) const { return all_hi + per_group(within + i, inverse); }
  __device__ __forceinline__ int first(int last) const {  // (in 64 bits: the window may be any, `last` below 0)
    return window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(last) - window + 1)) : 0;
  }
  // Some row does not see some token of the tile from `base` on.
  __device__ __forceinline__ bool edge(int base) const { return base < all_lo || base + kTile - 1 > all_hi; }
  __device__ __forceinline__ bool any(int token) const { return token >= any_lo && token <= any_hi; }
  __device__ __forceinline__ bool sees(int i, int token) const {
    const int end = last(i);
    return token <= end && token >= first(end);
  }
};

// Widens one token's value codes to BF16 rows of 64 dimensions. Values that no row sees are dropped, whatever they hold;
// what is not finite and only some rows see is taken out and noted for those, in `nans` ([row][kWords]).
template <int kWords>
struct Widener {
  const Sight& sight;
  uint32_t* nans;
  int* any_nans;
  int token;
  bool dropped, careful;
  uint32_t limit;
  __nv_bfloat162 factor;
  __device__ __forceinline__ Widener(const Sight& sight, uint32_t entry, bool edge, int token, uint32_t* nans, int* any_nans)
      : sight(sight), nans(nans), any_nans(any_nans), token(token) {
    uint32_t scale = (entry >> 8) & 0xFFu;
    limit = finite_limit(scale);
    dropped = edge && (!sight.any(token) || !(entry >> 16));
    careful = edge && sight.mixed;
    if (dropped || (careful && scale == 255)) scale = 0;  // (all taken out)
    factor = scale2_of(scale);
  }
  // Chunk c of 16 dimensions, into row `row` of an image.
  __device__ __forceinline__ void operator()(uint4 codes, int c, int row, uint8_t* image) const {
    if (dropped) {
      codes = make_uint4(0, 0, 0, 0);
    } else if (careful && any_not_finite(codes, limit)) {
      const uint32_t places = take_out(codes, limit) << (c % 2 * 16);
      *any_nans = 1;
#pragma unroll 1
      for (int i = 0; i < sight.rows; ++i)
        if (sight.sees(i, token)) atomicOr(nans + i * kWords + c / 2, places);
    }
    uint8_t* dst = image + c / 4 * (kTile * 128);
    const uint2 v0 = widen(codes.x, factor), v1 = widen(codes.y, factor), v2 = widen(codes.z, factor), v3 = widen(codes.w, factor);
    *reinterpret_cast<uint4*>(dst + chunk_at<128>(row, c % 4 * 2)) = make_uint4(v0.x, v0.y, v1.x, v1.y);
    *reinterpret_cast<uint4*>(dst + chunk_at<128>(row, c % 4 * 2 + 1)) = make_uint4(v2.x, v2.y, v3.x, v3.y);
  }
};

// The workspace header's first words.
struct Header {
  int32_t status;
  int32_t withhold;      // test hook: the CTA (from 1) whose first tile is never copied
  uint64_t timeout_ns;   // of one wait; 0: the default
};

// Bounded wait for a barrier's phase: false, and the error reported, when it runs out. A role that sees that issues
// nothing more, waits (bounded again) for what it has in flight, and goes to the CTA's end.
__device__ __forceinline__ bool wait_more(uint64_t* bar, uint32_t parity, int32_t* status) {
  const uint64_t began = global_timer_ns(), set = reinterpret_cast<const volatile Header*>(status)->timeout_ns;
  const uint64_t limit = set ? set : kWaitNs;
  while (!mbar_wait_hint(bar, parity, 20000)) {
    if (global_timer_ns() - began > limit) {
      report(status, MOE_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return mbar_test(bar, parity) || wait_more(bar, parity, status);
}

// Prefix sums of the requests' work, by the whole CTA of kThreads threads; returns what an item counts as: nothing
// while there are no more tiles than CTAs, so that each gets one, else kItemTiles.
template <int kThreads, int kRows, int kItemTiles>
__device__ int sum_work(const AttendArgs& a, int shift, long long* prefix, long long (*s_sum)[2]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.b.requests + kThreads - 1) / kThreads;
  long long tiles = 0, items = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < a.b.requests) {
      const Request q(a, shift, r, kRows);
      items += q.items(a.c.kv_heads);
      tiles += RowTiles<kRows>(a, q).all(q) * a.c.kv_heads;
    }
  }
  long long tiles_in = tiles, items_in = items;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(kAll, tiles_in, d), v = __shfl_up_sync(kAll, items_in, d);
    if (lane >= d) {
      tiles_in += u;
      items_in += v;
    }
  }
  if (lane == 31) {
    s_sum[warp][0] = tiles_in;
    s_sum[warp][1] = items_in;
  }
  __syncthreads();
  long long all = 0, tiles_at = tiles_in - tiles, items_at = items_in - items;
  for (int w = 0; w < kThreads / 32; ++w) {
    all += s_sum[w][0];
    if (w < warp) {
      tiles_at += s_sum[w][0];
      items_at += s_sum[w][1];
    }
  }
  const int weight = all > gridDim.x ? kItemTiles : 0;
  long long at = tiles_at + items_at * weight;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < a.b.requests) {
      prefix[r] = at;
      const Request q(a, shift, r, kRows);
      at += (RowTiles<kRows>(a, q).all(q) + static_cast<long long>(q.row_tiles) * weight) * a.c.kv_heads;
      if (r == a.b.requests - 1) prefix[r + 1] = at;
    }
  }
  __syncthreads();
  return weight;
}

// A producer warp: looks up the pages of the CTA's tiles and streams their keys (kWhich 1), values (2) or both (3)
// through the ring. With the values go the pages' entries: key scale, value scale << 8, present << 16; and after a
// tile's, whether every page is there.
template <class X, int D, int kWhich>
__device__ void produce(const AttendArgs& a, const AttendMaps& maps, const long long* prefix, int weight, int shift,
                        long long start, long long stop, uint8_t* sm, uint32_t* meta, uint64_t* full, uint64_t* empty, int32_t* status) {
  constexpr int kStages = kWhich == 1 ? X::kKeyStages : X::kStages;
  const int lane = threadIdx.x & 31;
  const uint64_t policy = policy_evict_first();
  const int per_tile = kTile >> shift, in_tile = lane & (per_tile - 1);  // pages of a tile; this lane's
  const int batch_tiles = 32 / per_tile;                                 // tiles looked up at once
  int k = 0;
  bool alive = reinterpret_cast<const volatile Header*>(status)->withhold != static_cast<int>(blockIdx.x) + 1;
  Segment<X::kRows> s;
  s.find(a, prefix, weight, shift, start, stop);
  for (long long x = start; alive;) {
    const Request& q = s.q;
    int page = -1;
    uint32_t entry = 0;
    bool fresh = false;  // a batch whose scales are not read yet
    for (int tile = s.begin; tile < s.end; ++tile, ++k) {
      const int batch = (tile - s.begin) & (batch_tiles - 1);
      if (batch == 0) {
        const long long token = static_cast<long long>(q.tile0 + tile) * kTile + (lane << shift);
        page = -1;
        if (token < q.end && tile + lane / per_tile < s.end) page = a.b.block_table[s.r * a.b.table_stride + (token >> shift)];
        if (page >= a.c.pages) page = -1;
        fresh = true;
      }
      const int stage = k % kStages;
      if (k >= kStages) alive = __all_sync(kAll, wait(empty + stage, (k / kStages - 1) & 1, status));
      if (!alive) break;
      // The copies first; the barrier's phase stays open until lane 0 arrives.
      const bool mine = lane / per_tile == batch;
      const int boxes = __popc(__ballot_sync(kAll, mine && page >= 0));
      if (mine && page >= 0) {
        uint8_t* keys = sm + X::kRing + stage * X::kKeyStride + (in_tile << shift) * X::kSpan;
        uint8_t* vals = sm + X::kRing + X::kValuesAt + stage * X::kValueStride + (in_tile << shift) * X::kSpan;
        const int row = page * a.c.kv_heads + s.head;
#pragma unroll
        for (int h = 0; h < X::kHalves; ++h) {
          if (kWhich & 1) tma_load_3d(keys + h * (kTile * X::kSpan), &maps.k, h * X::kSpan, 0, row, full + stage, policy);
          if (kWhich & 2) tma_load_3d(vals + h * (kTile * X::kSpan), &maps.v, h * X::kSpan, 0, row, full + stage, policy);
        }
      }
      if ((kWhich & 2) && fresh) {
        fresh = false;
        entry = 0;
        if (page >= 0) {
          const long long at = static_cast<long long>(page) * a.c.kv_heads + s.head;
          entry = a.c.k_scale[at] | static_cast<uint32_t>(a.c.v_scale[at]) << 8 | 1u << 16;
        }
      }
      if (kWhich & 2) {
        uint32_t* m = meta + stage * (kMaxPages + 1);
        if (mine) {
          m[in_tile] = entry;
          if (in_tile == 0) m[kMaxPages] = boxes == per_tile;
        }
        __syncwarp();  // the entries are written before lane 0 arrives
      }
      if (lane == 0) {
        if (boxes) mbar_arrive_expect_tx(full + stage, boxes * ((kWhich == 3 ? 2 : 1) * D << shift));
        else mbar_arrive(full + stage);
      }
    }
    x += s.length;
    if (x >= stop) break;
    s.next(a, prefix, shift, x, stop);
  }
  // The copies in flight land before the CTA ends (at once, unless another role gave up).
  for (int i = max(0, k - kStages); i < k; ++i) wait(full + i % kStages, (i / kStages) & 1, status);
}

// A piece of an item has been stored: joins the item's pieces once they are all there. By kThreads threads, whose barrier
// is kBarrier. row_dst: the rows' places among the outputs' rows.
template <int kRows, int D, int kThreads, int kBarrier>
__device__ void join_item(const AttendArgs& a, const Segment<kRows>& s, const long long* row_dst, int rows, long long ctas, long long total,
                          int tid, int* s_last) {
  constexpr int kPartialFloats = kRows * (D + 2);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace + kCounterOffset);
  float* partials = reinterpret_cast<float*>(a.workspace + kPartialOffset);
  auto sync = [] { asm volatile("bar.sync %0, %1;" ::"n"(kBarrier), "n"(kThreads) : "memory"); };
  // The CTAs of this item: c0 .. c1, by the bounds of their runs.
  const int c0 = static_cast<int>(divide((s.item + 1) * ctas - 1, total));
  const int c1 = static_cast<int>(divide((s.item + s.units) * ctas - 1, total));
  // The pieces are joined in two steps, by about the square root of their number at a time: by the last CTA of
  // each run of `width` pieces, then by the last of those, so no CTA reads more than a few dozen pieces.
  float* piece1 = partials + static_cast<int64_t>(c0 * 2 + 1) * kPartialFloats;  // the first piece
  float* piece0 = partials + static_cast<int64_t>(c0 * 2) * kPartialFloats;      // piece i: 2 i slots on
  auto piece = [&](int i) { return i == 0 ? piece1 : piece0 + static_cast<int64_t>(i) * 2 * kPartialFloats; };
  const int pieces = c1 - c0 + 1;
  int width = 8;
  while (width * width < pieces) ++width;
  int from = (static_cast<int>(blockIdx.x) - c0) / width * width, stride = 1, count = min(width, pieces - from);
  uint32_t* counter = from == 0 ? counters + c0 : counters + kMaxCtas + c0 + from;
  for (;;) {
    sync();
    if (tid == 0) {
      // Releases the CTA's stores (ordered before it by the barrier), acquires the other pieces'.
      const uint32_t before = atom_add_acq_rel_gpu(counter, 1);
      *s_last = before == static_cast<uint32_t>(count - 1);
      if (*s_last) *counter = 0;
    }
    sync();
    if (!*s_last) break;
    // A thread joins four dimensions of some rows, several pieces' loads in flight together.
    constexpr int kQuads = D / 4, kAllUnits = kRows * kQuads / kThreads, kUnits = kAllUnits % 4 == 0 ? 4 : kAllUnits % 2 == 0 ? 2 : 1;
    constexpr int kBatch = 8 / kUnits;
    const bool last = stride > 1 || count == pieces;
    for (int group = 0; group < kAllUnits; group += kUnits) {
      float4 o[kUnits];
      float top[kUnits], total_l[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        o[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        top[u] = -INFINITY;
        total_l[u] = 0.0f;
      }
      for (int c = 0; c < count; c += kBatch) {
        float pm[kBatch][kUnits], pl[kBatch][kUnits];
        float4 pv[kBatch][kUnits];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const bool in = c + e < count;
          const float* src = piece(from + (in ? c + e : c) * stride);
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            const int i = ((group + u) * kThreads + tid) / kQuads, c4 = ((group + u) * kThreads + tid) % kQuads * 4;
            pm[e][u] = __ldcg(src + kRows * D + i);
            pl[e][u] = __ldcg(src + kRows * D + kRows + i);
            pv[e][u] = __ldcg(reinterpret_cast<const float4*>(src + i * D + c4));
            if (!in) pm[e][u] = -INFINITY;
          }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          float mn = top[u];
#pragma unroll
          for (int e = 0; e < kBatch; ++e) mn = fmaxf(mn, pm[e][u]);
          const float ref = mn > -INFINITY ? mn : 0.0f, f = exp2_fast(top[u] - ref);
          total_l[u] *= f;
          o[u].x *= f;
          o[u].y *= f;
          o[u].z *= f;
          o[u].w *= f;
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            if (e > 0 && c + e >= count) continue;
            const float g = exp2_fast(pm[e][u] - ref);
            total_l[u] = fmaf(pl[e][u], g, total_l[u]);
            o[u].x = fmaf(pv[e][u].x, g, o[u].x);
            o[u].y = fmaf(pv[e][u].y, g, o[u].y);
            o[u].z = fmaf(pv[e][u].z, g, o[u].z);
            o[u].w = fmaf(pv[e][u].w, g, o[u].w);
          }
          top[u] = mn;
        }
      }
      if (!last) sync();  // the first piece of the run has been read everywhere: the run's result takes its place
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int i = ((group + u) * kThreads + tid) / kQuads, c4 = ((group + u) * kThreads + tid) % kQuads * 4;
        if (!last) {
          float* dst = piece(from);
          *reinterpret_cast<float4*>(dst + i * D + c4) = o[u];
          if (c4 == 0) {
            dst[kRows * D + i] = top[u];
            dst[kRows * D + kRows + i] = total_l[u];
          }
          continue;
        }
        if (i >= rows) continue;
        const float inv = total_l[u] == 0.0f ? 0.0f : __fdiv_rn(1.0f, total_l[u]);
        const int64_t dst = row_dst[i];
        __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o[u].x * inv, o[u].y * inv), __floats2bfloat162_rn(o[u].z * inv, o[u].w * inv)};
        *reinterpret_cast<uint2*>(a.out + dst * D + c4) = *reinterpret_cast<uint2*>(w);
        if (a.lse != nullptr && c4 == 0) a.lse[dst] = total_l[u] == 0.0f ? -INFINITY : (top[u] + log2f(total_l[u])) * kLn2;
      }
    }
    if (last) break;
    from = 0;
    stride = width;
    count = (pieces + width - 1) / width;
    counter = counters + 2 * kMaxCtas + c0;
  }
}

}  // namespace
}  // namespace moe
