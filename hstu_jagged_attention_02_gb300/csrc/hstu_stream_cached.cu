// The attention over the paged 4-bit cache for few rows (hstu_attn_fwd_cached
// with at most 8 rows a sequence: decode steps, a handful of candidates).
//
// With few rows the work is the bytes of the cache: 9/16 byte a feature, read
// once.  So a warp decodes packed rows in registers, in the shape in which its
// matrix instruction (m16n8k16, FP16 -> FP32) takes them; a decoded tile is
// not written to shared memory and read again as in the tensor-memory kernel,
// whose 128 KB of traffic for 18 KB of cache would bound few rows by the shared
// memory's rate.  A warp takes 16 tokens at a time:
//
//   S^T [16 tokens x 8 rows] = K Q^T      lane (g, t), g = lane / 4, t = lane % 4, holds tokens tok(g), tok(g) + 8,
//                                         features [t d/4, (t + 1) d/4): the products' inner index runs over the
//                                         features in any order, as long as q is held in the same one
//   P = 16 SiLU(z)                        in the accumulator's places, to FP16, turned by movmatrix
//   O^T [d x 8 rows] += V^T P             lane (g, t) holds tokens tok(2t), tok(2t + 1) and those + 8, features
//                                         [g d/8, (g + 1) d/8), pairs of tokens put together by byte permutes
//
// tok(r) = 0, 2, 4, 6, 1, 3, 5, 7: neighbouring t then read rows of both
// parities, half as many bank conflicts.  q stays in registers (FP16, scaled
// per row by a power of two: hstu_cached.cuh), so does O.
//
// One warp copies pages, whole (page, head) blocks by cp.async.bulk, into a
// ring of NR tiles of 128 tokens; the other warps, 8 to a tile, deal the tiles
// among themselves and add their sums up in shared memory at a piece's end.
// Every wait is bounded.
#include "hstu_cached.cuh"
#include "tc_ptx.cuh"

namespace hstu {

namespace {

using namespace tc;

constexpr int kRows = 8;       // of a block

// A piece of an item, as the copying warp hands it to the others.
template <int D>
struct __align__(16) SPiece {
  uint2 q[D / 16][32];         // the products' right operands, a lane's two registers an inner step
  int64_t tq[kRows], tmin, tmax;   // the rows' times and their range
  float ka[kRows];             // score factors
  int valid;                   // 0: no more pieces
  int h, rows, hist;           // head; rows of the block, history rows among them
  int pos0, L;                 // position of its first row, cached tokens
  int tile0, tile1, slot;
};

template <int D>
struct SCfg {
  static constexpr int GROUPS = 3;                  // of 8 warps: 25 warps, 7 a sub-partition
  static constexpr int REGS = 72;
  static constexpr int WARPS = 8 * GROUPS, THREADS = (WARPS + 1) * 32;
  static constexpr int TILE_BYTES = 2 * kCachedTile * (D / 2 + D / 16);
  static constexpr int NR = D == 128 ? 5 : 8;
  static constexpr int SUM_OFF = NR * TILE_BYTES;                     // float [WARPS][kRows][D]: the warps' sums
  static constexpr int TS_OFF = SUM_OFF + WARPS * kRows * D * 4;      // int64 [NR][128]
  static constexpr int PIECE_OFF = TS_OFF + NR * kCachedTile * 8;     // SPiece [2]
  static constexpr int BAR_OFF = PIECE_OFF + 2 * (int)sizeof(SPiece<D>);   // full, empty [NR], pieces full, empty [2]
  static constexpr int BYTES = BAR_OFF + (2 * NR + 4) * 8;
  static_assert(BYTES <= (int)kMaxSmemPerCta - 1024, "one CTA's shared memory");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x; w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// The token of row r (0 .. 7) of a matrix instruction.
__device__ __forceinline__ int token_of(int r) { return ((r & 3) << 1) | (r >> 2); }

// Where a lane's parts of a step lie in a (page, head) block.
template <int D>
struct LaneOffsets {
  int k, ks, v[2], vs[2];
  __device__ __forceinline__ LaneOffsets(const PageLayout& lay, int lane) {
    const int g = lane >> 2, t = lane & 3;
    k = token_of(g) * (D / 2) + t * (D / 8);
    ks = lay.scales() + token_of(g) * (D / 16) + t * (D / 64);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] = lay.half() + token_of(2 * t + i) * (D / 2) + g * (D / 16);
      vs[i] = lay.half() + lay.scales() + token_of(2 * t + i) * (D / 16) + (g * (D / 8)) / 16;
    }
  }
};

// Writes the record of the walk's piece: the block's rows to FP16 in the
// matrix instruction's shape (lane (g, t): row g, features [t D/4, (t + 1) D/4)), their
// factors and times.  A whole warp.
template <int D>
__device__ __forceinline__ void write_piece(const CachedParams& p, const Walk& w, SPiece<D>& out) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = w.qb * kRows, rows = min(kRows, w.s.n - r0), hist = w.s.n - w.s.m;
  const int64_t row0 = w.s.row0 + r0;
  uint32_t x[D / 8];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (g < rows) v = *reinterpret_cast<const uint4*>(p.q + ((row0 + g) * p.H + w.h) * D + t * (D / 4) + e * 8);
    x[4 * e] = v.x; x[4 * e + 1] = v.y; x[4 * e + 2] = v.z; x[4 * e + 3] = v.w;
  }
  int64_t tq = 0, tmin = INT64_MAX, tmax = INT64_MIN;
  if (p.times && lane < rows) tq = tmin = tmax = p.times[row0 + lane];
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < D / 8; ++e) top = max(top, max((x[e] << 16) & 0x7fff0000u, x[e] & 0x7fff0000u));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  float down;
  const float up = row_scale(top, down);
#pragma unroll
  for (int e = 0; e < D / 16; ++e)
    out.q[e][lane] = make_uint2(
        pack_f16(__uint_as_float(x[2 * e] << 16) * up, __uint_as_float(x[2 * e] & 0xFFFF0000u) * up),
        pack_f16(__uint_as_float(x[2 * e + 1] << 16) * up, __uint_as_float(x[2 * e + 1] & 0xFFFF0000u) * up));
  if (t == 0) out.ka[g] = -kLog2e * p.alpha * p.k_scale * down;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const int64_t a = __shfl_xor_sync(0xffffffffu, tmin, o), b = __shfl_xor_sync(0xffffffffu, tmax, o);
    tmin = a < tmin ? a : tmin;
    tmax = b > tmax ? b : tmax;
  }
  if (lane < kRows) out.tq[lane] = tq;
  if (lane == 0) {
    out.tmin = tmin;
    out.tmax = tmax;
    out.valid = 1;
    out.h = w.h;
    out.rows = rows;
    out.hist = max(0, min(hist - r0, rows));
    out.pos0 = w.s.L - hist + r0;
    out.L = w.s.L;
    out.tile0 = w.tile;
    out.tile1 = w.tile + w.take();
    out.slot = w.slot(p);
  }
  __syncwarp();
}

template <int D>
__global__ void __maxnreg__(SCfg<D>::REGS) cached_stream_kernel(const __grid_constant__ CachedParams p) {
  using C = SCfg<D>;
  constexpr int MT = D / 16;             // 16-feature tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int scan[2 * (C::WARPS + 1)];
  __shared__ Start start;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t smem0 = smem_u32(smem);
  auto full = [&](uint32_t i) -> uint32_t { return smem0 + C::BAR_OFF + 8 * i; };
  auto empty = [&](uint32_t i) -> uint32_t { return smem0 + C::BAR_OFF + 8 * (C::NR + i); };
  auto piece_full = [&](uint32_t i) -> uint32_t { return smem0 + C::BAR_OFF + 8 * (2 * C::NR + i); };
  auto piece_empty = [&](uint32_t i) -> uint32_t { return smem0 + C::BAR_OFF + 8 * (2 * C::NR + 2 + i); };
  SPiece<D>* pieces = reinterpret_cast<SPiece<D>*>(smem + C::PIECE_OFF);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NR; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(piece_full(i), 1);
      mbar_init(piece_empty(i), C::WARPS);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();   // the finishing kernel waits for this grid's end itself
  cut_work<C::THREADS>(p, kRows, scan, &start);
  __syncthreads();
  Watchdog wd;
  wd.abort = &abort_flag;
  wd.err = p.hdr + WS_ERR;
  wd.err_info = p.hdr + WS_ERR_INFO;
  wd.limit_ns = 2000000000ull;
  const PageLayout lay(p.page_size, D);
  uint32_t rs = 0, ring = 0;             // stage of the ring, and the parity of its round
  uint32_t np = 0;                       // pieces so far

  if (warp == C::WARPS) {
    // ------------------------------------------------- pieces, page copies
    Walk w;
    w.begin(p, start, kRows);
    const int ppt_log = 7 - p.page_log, ppt = 1 << ppt_log;
    uint32_t used = 0;                   // stages used at all
    bool ok = true;
    while (ok) {
      if (lane == 0) ok = mbar_wait(piece_empty(np & 1), ((np >> 1) & 1) ^ 1, wd, 91);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      SPiece<D>& pc = pieces[np & 1];
      const bool some = w.left > 0;
      if (some) write_piece<D>(p, w, pc);
      else if (lane == 0) pc.valid = 0;
      if (lane == 0) mbar_arrive(piece_full(np & 1));
      ++np;
      if (!some) break;
      const int t1 = w.tile + w.take();
      // the block table's entries, 32 at a time: lane i holds entry e0 + i
      const int32_t* row = p.table + (int64_t)w.b * p.max_pages;
      const int npages = (w.s.L + p.page_size - 1) >> p.page_log;
      int e0 = w.tile << ppt_log;
      int32_t entry = e0 + lane < npages ? row[e0 + lane] : -1;
      int32_t next = e0 + 32 + lane < npages ? row[e0 + 32 + lane] : -1;
      for (int tile = w.tile; tile < t1; ++tile) {
        const int e = tile << ppt_log;
        if (e >= e0 + 32) {
          e0 += 32;
          entry = next;
          next = e0 + 32 + lane < npages ? row[e0 + 32 + lane] : -1;
        }
        // lanes 0 .. ppt - 1: a page's block each; the next ppt lanes: its times
        const int pg = lane & (ppt - 1);
        const int id = __shfl_sync(0xffffffffu, entry, (e - e0 + pg) & 31);
        const bool there = lane < 2 * ppt && e + pg < npages;
        const bool good = there && id >= 0 && id < p.num_pages;
        if (there && !good) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, w.b);
        const int n = __popc(__ballot_sync(0xffffffffu, good && lane < ppt));
        if (lane == 0) {
          ok = mbar_wait(empty(rs), ring ^ 1, wd, 92);
          if (ok) mbar_arrive_expect_tx(full(rs), (uint32_t)(n * (lay.bytes() + (p.times ? p.page_size * 8 : 0))));
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (good && lane < ppt)
          bulk_load(smem0 + rs * C::TILE_BYTES + pg * lay.bytes(), p.pages + ((int64_t)id * p.H + w.h) * lay.bytes(),
                    (uint32_t)lay.bytes(), full(rs));
        else if (good && p.times)
          bulk_load(smem0 + C::TS_OFF + rs * (kCachedTile * 8) + pg * p.page_size * 8,
                    p.page_times + ((int64_t)id << p.page_log), (uint32_t)(p.page_size * 8), full(rs));
        if (used < (uint32_t)C::NR) ++used;
        if (++rs == C::NR) {
          rs = 0;
          ring ^= 1;
        }
      }
      w.next(p, kRows);
    }
    // no copy may land in shared memory after the CTA's end: the last round of every stage
    if (lane == 0) {
      for (uint32_t i = 0; i < used; ++i) {
        const uint32_t parity = i < rs ? ring : ring ^ 1;
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(full(i), parity))
          if (globaltimer() - t0 > 200000000ull) break;
      }
    }
    return;
  }

  const int group = warp >> 3, local = (warp & 7) * 16;    // of the tiles; this warp's tokens in a tile
  int turn = 0;                                            // the group whose turn the next tile is
  const LaneOffsets<D> at(lay, lane);
  const int in_tile = (local >> p.page_log) * lay.bytes();
  const int place = local & (p.page_size - 1);
  const uint32_t code0 = in_tile + place * (D / 2), scale0 = in_tile + place * (D / 16);
  float* sums = reinterpret_cast<float*>(smem + C::SUM_OFF);
  bool ok = true;
  for (;; ++np) {
    ok = mbar_wait(piece_full(np & 1), (np >> 1) & 1, wd, 93);
    const SPiece<D>& pc = pieces[np & 1];
    const bool some = ok && pc.valid;
    const int rows = some ? pc.rows : 0, slot = pc.slot;
    float o[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
    if (some) {
      const int len = pc.L, pos0 = pc.pos0, nh = pc.hist;  // (rows behind the history rows are at len)
      const int pmin = nh > 0 ? pos0 : len, pmax = nh == rows ? pos0 + rows - 1 : len;
      const bool one_bias = pmin == pmax && pc.tmin == pc.tmax;    // all rows at one place and time
      const float* rp = p.rab_pos ? p.rab_pos + pc.h * p.P : nullptr;
      const float* rt = p.rab_time ? p.rab_time + pc.h * p.Tb : nullptr;
      const int t1 = pc.tile1;
#pragma unroll 1
      for (int tile = pc.tile0; tile < t1; ++tile) {
        const uint32_t stage = rs, parity = ring;
        if (++rs == C::NR) {
          rs = 0;
          ring ^= 1;
        }
        const bool mine = turn == group;
        if (++turn == C::GROUPS) turn = 0;
        if (!mine) continue;
        ok = mbar_wait(full(stage), parity, wd, 94);
        if (!ok) break;
        const int j16 = tile * kCachedTile + local;        // first token of the step
        if (j16 < len) {
          const uint8_t *codes = smem + stage * C::TILE_BYTES + code0, *scales = smem + stage * C::TILE_BYTES + scale0;
          float c[2][4] = {};     // two chains of products, added at their end
          {
            uint32_t k0[D / 32], k1[D / 32];
            load_words<D / 32>(codes + at.k, k0);
            load_words<D / 32>(codes + at.k + 8 * (D / 2), k1);
            const uint8_t* ks = scales + at.ks;
            const __half2 s0 = e4m3x2_half2(D == 128 ? *reinterpret_cast<const uint16_t*>(ks) : *ks);
            const __half2 s1 = e4m3x2_half2(D == 128 ? *reinterpret_cast<const uint16_t*>(ks + 8 * (D / 16)) : ks[8 * (D / 16)]);
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {             // 8 features at a time: two inner steps
              const bool hi = D == 128 && x >= 2;
              const uint4 a = decode8(k0[x], hi ? __high2half2(s0) : __low2half2(s0));
              const uint4 b = decode8(k1[x], hi ? __high2half2(s1) : __low2half2(s1));
              const uint2 q0 = pc.q[2 * x][lane], q1 = pc.q[2 * x + 1][lane];
              mma16816(c[0], a.x, b.x, a.y, b.y, q0.x, q0.y);
              mma16816(c[1], a.z, b.z, a.w, b.w, q1.x, q1.y);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) c[0][e] += c[1][e];
          }
          // a lane looks up the bias of token lane % 16 towards the block's rows, if they share it
          const int jl = j16 + (lane & 15);
          int64_t tl = 0;
          if (p.times) tl = reinterpret_cast<const int64_t*>(smem + C::TS_OFF + stage * (kCachedTile * 8))[local + (lane & 15)];
          bool same = jl <= pmin;
          float bl = 0.f;
          if (rp) {
            const int a = min(max(pmin - jl, 0), p.P - 1);
            bl = __ldg(rp + a);
            if (!one_bias) same = same && a == min(max(pmax - jl, 0), p.P - 1);
          }
          if (rt) {
            const int64_t tmin = pc.tmin;
            const int a = time_bucket(tmin, tl, p.Tb);
            bl += __ldg(rt + a);
            if (!one_bias) {
              const int64_t tmax = pc.tmax;
              same = same && a == time_bucket(tmax, tl, p.Tb) && (tl <= tmin || tl >= tmax);
            }
          }
          bl *= -kLog2e;
          // scores of tokens j0 (c[0], c[1]) and j0 + 8 (c[2], c[3]) for rows 2t, 2t + 1
          const int j0 = j16 + token_of(g);
          uint32_t pr[2];
          const float2 k2 = *reinterpret_cast<const float2*>(pc.ka + 2 * t);
          if (__all_sync(0xffffffffu, same || jl >= len)) {
            const float b0 = __shfl_sync(0xffffffffu, bl, token_of(g)), b1 = __shfl_sync(0xffffffffu, bl, token_of(g) + 8);
            pr[0] = silu_pair(__ffma2_rn(make_float2(c[0][0], c[0][1]), k2, make_float2(b0, b0)));
            pr[1] = silu_pair(__ffma2_rn(make_float2(c[0][2], c[0][3]), k2, make_float2(b1, b1)));
          } else {
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
              const int j = j0 + 8 * e;
              const int64_t tj = __shfl_sync(0xffffffffu, tl, token_of(g) + 8 * e);
              float b[2];
              uint32_t keep = 0;
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const int r = 2 * t + f, pos = r < nh ? pos0 + r : len;
                b[f] = 0.f;
                if (rp) b[f] = rp[min(max(pos - j, 0), p.P - 1)];
                if (rt) b[f] += rt[time_bucket(pc.tq[r], tj, p.Tb)];
                b[f] *= -kLog2e;
                keep |= j <= pos ? 0xffffu << (16 * f) : 0u;
              }
              const float2 cc = e ? make_float2(c[0][2], c[0][3]) : make_float2(c[0][0], c[0][1]);
              const uint32_t v = silu_pair(__ffma2_rn(cc, k2, make_float2(b[0], b[1]))) & keep;
              if (e) pr[1] = v;
              else pr[0] = v;
            }
          }
          uint32_t vs[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) vs[e] = scales[at.vs[e & 1] + 8 * (e >> 1) * (D / 16)];
          if (j16 + 16 > len) {                            // tokens behind the cache's end: neither scores nor values
#pragma unroll
            for (int e = 0; e < 2; ++e) pr[e] = j0 + 8 * e < len ? pr[e] : 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j16 + token_of(2 * t + (e & 1)) + 8 * (e >> 1) >= len) vs[e] = 0;
          }
          const uint32_t b0 = transpose8x8(pr[0]), b1 = transpose8x8(pr[1]);
          // values: a code of each of two tokens to a byte, so that the decoded pairs are pairs of tokens
          const __half2 s01 = e4m3x2_half2(vs[0] | (vs[1] << 8)), s23 = e4m3x2_half2(vs[2] | (vs[3] << 8));
          uint32_t v[4][D / 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) load_words<D / 64>(codes + at.v[e & 1] + 8 * (e >> 1) * (D / 2), v[e]);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {               // 8 features of the lane's D / 8
            auto even = [](uint32_t a, uint32_t b) { return (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u); };
            auto odd = [](uint32_t a, uint32_t b) { return ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u); };
            const uint4 e0 = decode8(even(v[0][x], v[1][x]), s01), o0 = decode8(odd(v[0][x], v[1][x]), s01);
            const uint4 e1 = decode8(even(v[2][x], v[3][x]), s23), o1 = decode8(odd(v[2][x], v[3][x]), s23);
            mma16816(o[4 * x], e0.x, o0.x, e1.x, o1.x, b0, b1);
            mma16816(o[4 * x + 1], e0.y, o0.y, e1.y, o1.y, b0, b1);
            mma16816(o[4 * x + 2], e0.z, o0.z, e1.z, o1.z, b0, b1);
            mma16816(o[4 * x + 3], e0.w, o0.w, e1.w, o1.w, b0, b1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(stage));
      }
    }
    // the warps' sums: o[m] holds features g D/8 + 2m, + 1 of rows 2t, 2t + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * t + e;
      if (r < rows) {
        float* dst = sums + (warp * kRows + r) * D + g * (D / 8);
#pragma unroll
        for (int m = 0; m < MT; ++m) *reinterpret_cast<float2*>(dst + 2 * m) = make_float2(o[m][e], o[m][2 + e]);
      }
    }
    // the warps meet; at the end, or if one of them has given up, all leave
    uint32_t leave;
    asm volatile("{\n\t.reg .pred q, r;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred r, 1, %2, q;\n\tselp.u32 %0, 1, 0, r;\n\t}"
                 : "=r"(leave)
                 : "r"(ok && some ? 0u : 1u), "n"(C::WARPS * 32)
                 : "memory");
    if (leave) break;
    if (lane == 0) mbar_arrive(piece_empty(np & 1));
    float* part = p.part + (int64_t)slot * (kRows * D);
    for (int e = threadIdx.x; e < rows * D; e += C::WARPS * 32) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < C::WARPS; ++k) x += sums[k * kRows * D + e];
      part[e] = x;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(C::WARPS * 32) : "memory");
  }
}

template <int D>
cudaError_t launch_t(const CachedParams& p, int ctas, cudaStream_t st) {
  using C = SCfg<D>;
  auto kern = cached_stream_kernel<D>;
  const void* fn = reinterpret_cast<const void*>(kern);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(C::THREADS), C::BYTES, st, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_launch_detail(e, "cached_stream_kernel", fn, C::THREADS, C::BYTES);
  }
  return e;
}

}  // namespace

cudaError_t launch_stream_cached(const CachedParams& p, int d, int ctas, cudaStream_t st) {
  return d == 128 ? launch_t<128>(p, ctas, st) : launch_t<64>(p, ctas, st);
}

}  // namespace hstu
