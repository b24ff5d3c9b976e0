// What the cached attention's two kernels share: the call's parameters, the
// checks of a sequence's numbers, and how its work is cut into tiles.
//
// A sequence's n rows form blocks of N; a block's keys are the 128-token
// tiles [0, tiles) of its cache, up to the last position that one of its rows
// sees.  An item is a (block, head).  All items' tiles in a line, ordered by
// sequence, block, head and tile, are cut into parts of equal cost, one a CTA; a
// CTA's part of an item is a piece, and leaves one FP32 sum [N][d] in the
// workspace at slot item + CTA (no two pieces share one: every further piece
// crosses the border of an item, of a CTA, or both).  So a long cache with one
// row fills the machine as well as many users do, and the sums are added in the
// same order every time.
#pragma once

#include "hstu_fp4.cuh"
#include "hstu_internal.h"

namespace hstu {

constexpr int kCachedTile = 128;

struct CachedParams {
  const int64_t* off;
  const int32_t* lens;
  const int32_t* nt;
  const int32_t* table;
  const int64_t* times;       // NULL: no time bias
  const float* rab_pos;
  const float* rab_time;      // NULL without times
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* u;
  __nv_bfloat16* o;
  __nv_bfloat16* y;
  const uint8_t* pages;
  const int64_t* page_times;
  float* part;                // [slots][N][d]
  int4* rows;                 // [T] where a row's sums lie (row_record)
  int* hdr;
  int64_t T, slots;           // rows, sums that part has room for
  uint64_t wait_ns;           // limit of a wait
  int B, H, page_size, page_log, num_pages, max_pages, max_rows, max_n, P, Tb, norm;
  int withhold;               // test only: CTA 0 prepares no piece
  float alpha, inv_n, eps;
  float k_scale;              // 2^k_exp
  float o_scale;              // 2^v_exp / 16 / N of a tensor-core sum
};

// header words of the cached attention's workspace (beside WS_ERR)
enum : int { WS_CA_QUOTA = 16 };   // cost a CTA, -1 where the batch was refused or a wait ran out

struct CachedSeq {
  int64_t row0;   // first row
  int n, m, L;    // rows, candidates among them, cached tokens
};

// Loads sequence b; false where its numbers do not fit together.
__device__ __forceinline__ bool load_seq(const CachedParams& p, int b, CachedSeq& s) {
  const int64_t o0 = p.off[b], n = p.off[b + 1] - o0;
  s.row0 = o0;
  s.m = p.nt ? p.nt[b] : 0;
  s.L = p.lens[b];
  s.n = (int)n;
  return o0 >= 0 && n >= 0 && o0 + n <= p.T && n <= p.max_rows && s.m >= 0 && s.m <= n && s.L >= n - s.m &&
         (int64_t)s.L + s.m <= p.max_n && s.L <= (int64_t)p.max_pages * p.page_size;
}

// What a tile costs, by the ways the tensor-memory kernel scores it: near
// tiles, where a block's rows differ in position bucket or mask, take 5.0 us
// with 128 rows, the others 1.9.  Where a batch has near tiles the work is cut
// by these costs, else by tiles: first passes of 4 histories of 900 to 2,100 rows
// by tiles 65.8 us (the CTAs at the sequences' beginnings end after 51 us, the
// others after 30), by costs 52.6.  In halves of a far tile's cost: sums over 12
// batches of first passes of 100 to 6,000 rows (128 rows a block) 4: 955 us, 5:
// 925, 6: 887, 7: 893, 8: 905; 32 users' new rows and candidates (32 rows a block)
// 5: 19.2 us, 6: 20.1; 12 batches of up to 64 rows (64 rows a block) 5: 247.8, 6: 248.2.
constexpr int kFarCost = 2, kMostTileCost = 6;
__device__ __forceinline__ int near_cost(int N) { return N == 128 ? 6 : 5; }

// Tiles of a block of rows: far ones, then near ones.  near_c: what a near one
// costs, or 0 where every tile counts 1.
struct BlockTiles {
  int far, near;
  __device__ __forceinline__ int all() const { return far + near; }
  __device__ __forceinline__ int cost(int near_c) const { return near_c ? kFarCost * far + near_c * near : far + near; }
  // cost of the tiles before tile t, and the first tile with at least `c` before it
  __device__ __forceinline__ int before(int t, int near_c) const {
    return near_c ? kFarCost * min(t, far) + near_c * max(t - far, 0) : t;
  }
  __device__ __forceinline__ int tile_at(int c, int near_c) const {
    if (!near_c) return c;
    const int rest = c - kFarCost * far;
    return rest <= 0 ? (c + kFarCost - 1) / kFarCost : far + (near_c == 6 ? (rest + 5) / 6 : (rest + 4) / 5);
  }
};
__device__ __forceinline__ BlockTiles block_tiles(const CachedParams& p, const CachedSeq& s, int qb, int N) {
  const int first = qb * N, last = min(s.n, first + N) - 1, hist = s.n - s.m;
  const int seen = last >= hist ? s.L : s.L - hist + last + 1;
  const int tiles = (seen + kCachedTile - 1) / kCachedTile;
  // blocks of several rows, history rows among them: tiles within the position buckets' reach of the first row
  const int reach = p.rab_pos ? p.P : 1;
  const int far = N > 8 && first < hist && last > first ? min(max(s.L - hist + first - reach + 2, 0) / kCachedTile, tiles) : tiles;
  return {far, tiles - far};
}

// Where a CTA's part of the work begins.
struct Start {
  CachedSeq s;        // the sequence it begins in
  int b, rem;         // its number, and the cost of its tiles that belong to CTAs before
  int items;          // items before the sequence
  int total, quota;   // cost in all (0 where the batch is refused), cost a CTA
  int near_c;         // what a near tile costs, or 0: cut by tiles
};

// A row's record for the finishing kernel: the cost of the tiles before its
// block's first item, that item, an item's cost, and its place in the block with,
// from bit 16 on, the last tile's cost and, in bit 30, whether it is a candidate.
__device__ __forceinline__ int4 row_record(int line, int item0, int cost, int place, int last, bool candidate) {
  return make_int4(line, item0, cost, place | (last << 16) | (candidate ? 1 << 30 : 0));
}

// A row's sums of head h: the slot of the first and their number, 0 where the
// record does not lead to slots that exist.  A CTA whose wait ran out leaves the
// records of its blocks unwritten; whatever the workspace held there, nothing
// outside it is read.
struct RowPieces {
  int64_t slot;
  int64_t n;
};
__host__ __device__ __forceinline__ RowPieces row_pieces(int4 rec, int h, int quota, int N, int64_t slots) {
  RowPieces r{0, 0};
  if (rec.z <= 0 || rec.y < 0 || (rec.w & 0xffff) >= N) return r;
  const uint32_t at = (uint32_t)rec.x + (uint32_t)h * (uint32_t)rec.z, last = (uint32_t)(rec.w >> 16) & 0xffu;
  const uint32_t c0 = at / (uint32_t)quota, c1 = (at + (uint32_t)rec.z - last) / (uint32_t)quota;
  r.slot = (int64_t)rec.y + h + c0;
  if (c1 >= c0 && r.slot + (c1 - c0) < slots) r.n = (int64_t)(c1 - c0) + 1;
  return r;
}

// Every CTA counts all sequences' tiles and finds its own beginning.  The rows'
// records are written by the CTA that begins their block (write_records), those
// of a sequence without cached tokens here.  A thread takes `per` neighbouring
// sequences (one, unless there are more of them than threads: then nothing is
// read twice).  scan: 3 x 32 ints in shared memory; the caller synchronises
// before it reads start.
template <int THREADS>
__device__ __forceinline__ void cut_work(const CachedParams& p, int N, int* scan, Start* start) {
  constexpr int WARPS = THREADS / 32;
  static_assert(WARPS <= 32, "the warps' sums are added by one warp");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.B + THREADS - 1) / THREADS;
  const int lo = min((int)threadIdx.x * per, p.B), hi = min(lo + per, p.B);
  bool bad = threadIdx.x == THREADS - 1 && (p.off[0] != 0 || p.off[p.B] > p.T);
  CachedSeq s{};
  // far and near tiles of all heads, items
  auto count = [&](int b, int (&n)[3]) -> bool {
    if (!load_seq(p, b, s)) return false;
    const int blocks = (s.n + N - 1) / N;
    n[0] = n[1] = 0;
    for (int qb = 0; qb < blocks; ++qb) {
      const BlockTiles t = block_tiles(p, s, qb, N);
      n[0] += t.far;
      n[1] += t.near;
    }
    n[0] *= p.H;
    n[1] *= p.H;
    n[2] = blocks * p.H;
    return true;
  };
  int own[3] = {};
  for (int b = lo; b < hi; ++b) {
    int n[3];
    if (!count(b, n)) {
      bad = true;
      set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, b);
      break;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) own[i] += n[i];
  }
  if (bad) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
  auto scan_warp = [&](int (&x)[3]) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int a = __shfl_up_sync(0xffffffffu, x[i], o);
        if (lane >= o) x[i] += a;
      }
    }
  };
  int before[3] = {own[0], own[1], own[2]};
  scan_warp(before);
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < 3; ++i) scan[32 * i + warp] = before[i];
  }
  const int any_bad = __syncthreads_or(bad);
  // every warp adds the warps' sums up for itself
  int all[3], sum[2];
#pragma unroll
  for (int i = 0; i < 3; ++i) all[i] = lane < WARPS ? scan[32 * i + lane] : 0;
  scan_warp(all);
#pragma unroll
  for (int i = 0; i < 2; ++i) sum[i] = __shfl_sync(0xffffffffu, all[i], 31);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int others = __shfl_sync(0xffffffffu, all[i], max(warp - 1, 0));
    before[i] += (warp > 0 ? others : 0) - own[i];
  }
  const int near_c = sum[1] > 0 ? near_cost(N) : 0;
  auto cost = [&](const int (&n)[3]) { return BlockTiles{n[0], n[1]}.cost(near_c); };
  const int total = any_bad ? 0 : BlockTiles{sum[0], sum[1]}.cost(near_c);
  // a CTA's share holds a tile's beginning: no CTA between an item's first and last goes without a tile of it
  const int quota = max((total + (int)gridDim.x - 1) / (int)gridDim.x, max(near_c, 1));
  const int first = (int)blockIdx.x * quota;
  if (threadIdx.x == 0) {
    start->total = total;
    start->quota = quota;
    start->near_c = near_c;
    if (blockIdx.x == 0) p.hdr[WS_CA_QUOTA] = any_bad ? -1 : quota;
  }
  if (any_bad) return;
  int at = cost(before);
  const bool mine = first < total && at <= first && first < at + cost(own);
  if (per == 1) {
    if (mine) {
      start->s = s;
      start->b = lo;
      start->rem = first - at;
      start->items = before[2];
    }
    // a warp's sequences that are this CTA's to write, one after the other
    unsigned m = __ballot_sync(0xffffffffu, lo < hi && lo % (int)gridDim.x == (int)blockIdx.x && s.n > 0 && s.L == 0);
    for (; m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int64_t row0 = __shfl_sync(0xffffffffu, s.row0, src);
      const int n = __shfl_sync(0xffffffffu, s.n, src);
      for (int r = lane; r < n; r += 32) p.rows[row0 + r] = row_record(0, 0, 0, 0, 0, true);
    }
  } else {
    int items = before[2];
    for (int b = lo; b < hi; ++b) {
      int n[3];
      count(b, n);
      if (mine && first >= at && first < at + cost(n)) {
        start->s = s;
        start->b = b;
        start->rem = first - at;
        start->items = items;
      }
      if (s.L == 0 && b % (int)gridDim.x == (int)blockIdx.x)
        for (int r = 0; r < s.n; ++r) p.rows[s.row0 + r] = row_record(0, 0, 0, 0, 0, true);
      at += cost(n);
      items += n[2];
    }
  }
}

// A CTA's walk over its pieces: every thread that calls it sees the same.  All
// items' tiles in a line, each as long as it costs: a CTA takes the tiles that
// begin in its part of the line.
struct Walk {
  CachedSeq s;
  BlockTiles tiles;
  int b, qb, h, tile, items;
  int line, end;      // where the item begins in the line, and the CTA's part ends
  int near_c;
  bool more;

  __device__ __forceinline__ void begin(const CachedParams& p, const Start& st, int N) {
    const int first = (int)blockIdx.x * st.quota;
    near_c = st.near_c;
    end = min(first + st.quota, st.total);
    more = first < st.total;
    b = st.b; items = st.items; qb = 0; h = 0; tile = 0; line = first; tiles = {0, 0};
    if (!more) return;
    s = st.s;
    int rem = st.rem;
    tiles = block_tiles(p, s, qb, N);
    while (rem >= tiles.cost(near_c) * p.H) {
      rem -= tiles.cost(near_c) * p.H;
      ++qb;
      tiles = block_tiles(p, s, qb, N);
    }
    const int cost = tiles.cost(near_c);
    h = rem / cost;
    rem -= h * cost;
    line = first - rem;
    tile = tiles.tile_at(rem, near_c);
    if (tile >= tiles.all()) next_item(p, N);   // the item's last tile began before
  }
  // the piece at hand: tiles [tile, tile + take())
  __device__ __forceinline__ int take() const {
    const int room = end - line;
    return (room >= tiles.cost(near_c) ? tiles.all() : min(tiles.tile_at(room, near_c), tiles.all())) - tile;
  }
  __device__ __forceinline__ int slot(const CachedParams& p) const { return items + qb * p.H + h + (int)blockIdx.x; }
  // the records of a block's rows, with its first piece; a warp
  __device__ __forceinline__ void write_records(const CachedParams& p, int N, int lane) const {
    if (h > 0 || tile > 0) return;
    const int r0 = qb * N, rows = min(N, s.n - r0), cost = tiles.cost(near_c);
    const int last = cost - tiles.before(tiles.all() - 1, near_c);
    for (int r = lane; r < rows; r += 32)
      p.rows[s.row0 + r0 + r] = row_record(line, items + qb * p.H, cost, r, last, r0 + r >= s.n - s.m);
  }
  __device__ __forceinline__ void next(const CachedParams& p, int N) {
    if (tile + take() < tiles.all()) more = false;
    else next_item(p, N);
  }

 private:
  __device__ __forceinline__ void next_item(const CachedParams& p, int N) {
    line += tiles.cost(near_c);
    tile = 0;
    more = line < end;
    if (!more || ++h < p.H) return;
    h = 0;
    do {
      ++qb;
      if (qb * N >= s.n) {
        items += ((s.n + N - 1) / N) * p.H;
        qb = 0;
        s.n = 0;                 // some later sequence has tiles: the line goes on
        while (s.n == 0 && ++b < p.B) load_seq(p, b, s);
        if (s.n == 0) {
          more = false;
          return;
        }
      }
      tiles = block_tiles(p, s, qb, N);
    } while (tiles.all() == 0);
  }
};

// --------------------------------------------------------------- arithmetic
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPScale = 16.f;   // on the scores, against FP16's range

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// the FP16 pair (a, b), a in the low half
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// 16 SiLU(z) of two scores given as w = -log2(e) z: w c / (1 + 2^w) with
// c = -16 / log2(e).  Far below zero 2^w is infinity and the value a zero; the
// biases are kept below kMostBias so that w itself is not (0 x infinity).
__device__ __forceinline__ uint32_t silu_pair(float2 w) {
  const float c = -kPScale / kLog2e;
  const float2 d = __fadd2_rn(make_float2(ex2_approx(w.x), ex2_approx(w.y)), make_float2(1.f, 1.f));
  const float2 x = __fmul2_rn(__fmul2_rn(w, make_float2(c, c)), make_float2(rcp_approx(d.x), rcp_approx(d.y)));
  return pack_f16(x.x, x.y);
}
// A bias as the kernels use it: times -log2(e), and cut where it mutes for good.
constexpr float kMostBias = 1e30f;
__device__ __forceinline__ float scaled_bias(float b) { return min_nan(-kLog2e * b, kMostBias); }

// The power of two that brings a q row whose largest magnitude has the bits
// `top` (FP32) to [2^14, 2^15), and its inverse; rows below 2^-100 take
// what 2^-100 takes.  FP16 then holds the BF16 row exactly down to 2^-28 of
// its largest feature.
__device__ __forceinline__ float row_scale(uint32_t top, float& down) {
  const int ex = max((int)(top >> 23), 27);
  down = __uint_as_float((uint32_t)(ex - 14) << 23);
  return __uint_as_float((uint32_t)(127 + 14 + 127 - ex) << 23);
}

__device__ __forceinline__ uint32_t mul_half2(__half2 a, __half2 b) {
  const __half2 r = __hmul2(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 8 codes (32 bits) times their scale: 8 FP16 values
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 s) {
  return make_uint4(mul_half2(e2m1x2_half2<0>(w), s), mul_half2(e2m1x2_half2<1>(w), s),
                    mul_half2(e2m1x2_half2<2>(w), s), mul_half2(e2m1x2_half2<3>(w), s));
}

// Number of binary digits of |a - b|: the time bucket before it is cut to Tb - 1.
__device__ __forceinline__ int bit_length(int64_t a, int64_t b) {
  const uint64_t d = a >= b ? (uint64_t)a - (uint64_t)b : (uint64_t)b - (uint64_t)a;
  return 64 - __clzll((long long)d);
}
constexpr int kTimeSlots = 65;   // bit lengths 0 .. 64

// A head's biases as the kernels use them: by time bucket, then the last
// position bucket's.  A warp; the loads are under way together.
__device__ __forceinline__ void store_time_biases(const CachedParams& p, int h, float* to, int lane) {
  constexpr int EACH = (kTimeSlots + 31) / 32;
  float b[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) b[i] = p.rab_time ? p.rab_time[h * p.Tb + min(lane + 32 * i, p.Tb - 1)] : 0.f;
  const float far = p.rab_pos ? p.rab_pos[h * p.P + p.P - 1] : 0.f;
#pragma unroll
  for (int i = 0; i < EACH; ++i)
    if (lane + 32 * i < kTimeSlots) to[lane + 32 * i] = scaled_bias(b[i]);
  if (lane == 0) to[kTimeSlots] = scaled_bias(far);
}

// Rows of a block: as few as the longest sequence asks for.  Up to 8 rows go
// through the streaming kernel, more through the tensor-memory one.  Single
// calls for 32 users over some 160,000 cached tokens, four heads of 128, by
// candidates a user: 1: 40.6 us (with 32 rows a block through tensor memory
// 55.9), 8: 46.7 (58.0), 32: 58.0 (with 128 rows a block 78.5), 64: 65 (79.5),
// 128: 87.
inline int cached_block_rows(int max_rows) {
  return max_rows <= 8 ? 8 : (max_rows <= 32 ? 32 : (max_rows <= 64 ? 64 : 128));
}
cudaError_t launch_stream_cached(const CachedParams& p, int d, int ctas, cudaStream_t st);
cudaError_t launch_tc_cached(const CachedParams& p, int d, int N, int ctas, cudaStream_t st);

}  // namespace hstu
