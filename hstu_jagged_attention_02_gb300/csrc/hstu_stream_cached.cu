// The attention over the paged 4-bit cache for few rows (hstu_attn_fwd_cached
// with at most 8 rows a sequence: decode steps, a handful of candidates).
//
// With few rows the work is the bytes of the cache: 9/16 byte a feature, read
// once.  So a warp decodes packed rows in registers, in the shape in which its
// matrix instruction (m16n8k16, FP16 -> FP32) takes them; a decoded tile is
// not written to shared memory and read again as in the tensor-memory kernel,
// whose 128 KB of traffic for 18 KB of cache would bound few rows by the shared
// memory's rate.  A warp takes 32 tokens at a time, in two halves of 16:
//
//   S^T [16 tokens x 8 rows] = K Q^T      lane (g, t), g = lane / 4, t = lane % 4, holds tokens tok(g), tok(g) + 8,
//                                         features [t d/4, (t + 1) d/4): the products' inner index runs over the
//                                         features in any order, as long as q is held in the same one
//   P = 16 SiLU(z)                        in the accumulator's places, to FP16, turned by movmatrix
//   O^T [d x 8 rows] += V^T P             lane (g, t) holds tokens tok(2t), tok(2t + 1) and those + 8, features
//                                         [g d/8, (g + 1) d/8), pairs of tokens put together by byte permutes
//
// tok(r) = 0, 2, 4, 6, 1, 3, 5, 7: neighbouring t then read rows of both
// parities, half as many bank conflicts.  O stays in registers; q (FP16, scaled
// per row by a power of two: hstu_cached.cuh) comes from shared memory, once
// for both halves.  A lane looks up the bias of one token, once for all rows
// where they share it.
//
// A piece's steps are dealt to the warps in turn.  Each warp copies its own
// steps ahead (cp.async, two or three in flight) into a ring of its own, so that
// no warp waits for another; one warp that copied for all of them took 1,650
// cycles a tile to issue the copies, twice what the others take to use them.
// One more warp walks the CTA's pieces and prepares their records (the rows in
// FP16, their factors, the head's time biases) a few pieces ahead.  At a piece's
// end each warp leaves its sum in shared memory and goes on; the last one adds
// them up, in the warps' order.  Every wait on a barrier is bounded.
//
// What bounds it: instructions, 790 for 32 tokens of 128 features, at 1.9 a
// cycle with the four warps a sub-partition that the registers allow, and 4 us
// of lookups before the first product.  32 users with one row each over some
// 162,000 cached tokens, four heads of 128: 32.9 us with the finishing kernel,
// 2.9 TB/s of cache (of 6.8 measured for a copy).  Steps of 16 tokens took 1.6 us
// more (the lookups and the copies' addresses twice as often), but 0.5 us less
// for a single row over 300 tokens, which takes 9.2.
#include "hstu_cached.cuh"
#include "tc_ptx.cuh"

namespace hstu {

namespace {

using namespace tc;

constexpr int kRows = 8;       // of a block

// A piece of an item, as its record goes to the warps.
template <int D>
struct __align__(16) SPiece {
  uint2 q[D / 16][32];         // the products' right operands, a lane's two registers an inner step
  int64_t tq[kRows], tmin, tmax;   // the rows' times and their range
  float ka[kRows];             // score factors
  float time_bias[kTimeSlots + 1];   // of the head by bucket, then its last position bucket's, times -log2(e)
  const int32_t* table;        // the sequence's pages
  int valid;                   // 0: no more pieces
  int b, h, rows, hist;        // sequence, head; rows of the block, history rows among them
  int pos0, L;                 // position of its first row, cached tokens
  int step0, step1, slot;      // 32-token steps; where the sum goes
};

template <int D>
struct SCfg {
  static constexpr int WARPS = 16, THREADS = (WARPS + 1) * 32;        // 17 warps, 5 a sub-partition
  static constexpr int REGS = 96;
  static constexpr int TOKENS = 32;                                   // of a step: two matrix instructions' M
  static constexpr int DEPTH = D == 128 ? 2 : 3;                      // steps in flight a warp
  static constexpr int PIECES = DEPTH + 1;   // records: a warp's copies run up to DEPTH pieces ahead of its work
  // a step: K codes, V codes, K scales, V scales, times
  static constexpr int CODES = TOKENS * (D / 2), SCALES = TOKENS * (D / 16);
  static constexpr int STEP_V = CODES, STEP_KS = 2 * CODES, STEP_VS = STEP_KS + SCALES, STEP_T = STEP_VS + SCALES;
  static constexpr int STEP = STEP_T + TOKENS * 8;
  static constexpr int SUM_OFF = WARPS * DEPTH * STEP;                // float [WARPS][kRows][D], or of half the rows twice
  static constexpr int PIECE_OFF = SUM_OFF + WARPS * kRows * D * 4;   // SPiece [PIECES]
  static constexpr int BAR_OFF = PIECE_OFF + PIECES * (int)sizeof(SPiece<D>);   // records full, empty; sums free [2]
  static constexpr int BYTES = BAR_OFF + (2 * PIECES + 2) * 8;
  static_assert(BYTES <= (int)kMaxSmemPerCta - 1024, "one CTA's shared memory");
  static_assert(STEP % 128 == 0, "a warp's ring keeps its alignment");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// Where a lane's parts of a step lie in its ring slot.
template <int D>
struct LaneOffsets {
  using C = SCfg<D>;
  int k, ks, v[2], vs[2];
  __device__ __forceinline__ explicit LaneOffsets(int lane) {
    const int g = lane >> 2, t = lane & 3;
    k = token_of(g) * (D / 2) + t * (D / 8);
    ks = C::STEP_KS + token_of(g) * (D / 16) + t * (D / 64);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] = C::STEP_V + token_of(2 * t + i) * (D / 2) + g * (D / 16);
      vs[i] = C::STEP_VS + token_of(2 * t + i) * (D / 16) + (g * (D / 8)) / 16;
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
  store_time_biases(p, w.h, out.time_bias, lane);
  if (lane == 0) {
    out.tmin = tmin;
    out.tmax = tmax;
    out.valid = 1;
    out.h = w.h;
    out.rows = rows;
    out.hist = max(0, min(hist - r0, rows));
    out.pos0 = w.s.L - hist + r0;
    out.L = w.s.L;
    out.b = w.b;
    out.table = p.table + (int64_t)w.b * p.max_pages;
    out.step0 = w.tile * (kCachedTile / SCfg<D>::TOKENS);
    out.step1 = min((w.tile + w.take()) * (kCachedTile / SCfg<D>::TOKENS), (w.s.L + SCfg<D>::TOKENS - 1) / SCfg<D>::TOKENS);
    out.slot = w.slot(p);
  }
  __syncwarp();
}

template <int D>
__global__ void __maxnreg__(SCfg<D>::REGS) cached_stream_kernel(const __grid_constant__ CachedParams p) {
  using C = SCfg<D>;
  constexpr int MT = D / 16;             // 16-feature tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int scan[96];
  __shared__ Start start;
  __shared__ int abort_flag, left_sums[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t smem0 = smem_u32(smem);
  auto piece_full = [&](uint32_t i) -> uint32_t { return smem0 + C::BAR_OFF + 8 * i; };
  auto piece_empty = [&](uint32_t i) -> uint32_t { return smem0 + C::BAR_OFF + 8 * (C::PIECES + i); };
  auto sum_free = [&](uint32_t i) -> uint32_t { return smem0 + C::BAR_OFF + 8 * (2 * C::PIECES + i); };
  SPiece<D>* pieces = reinterpret_cast<SPiece<D>*>(smem + C::PIECE_OFF);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::PIECES; ++i) {
      mbar_init(piece_full(i), 1);
      mbar_init(piece_empty(i), C::WARPS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sum_free(i), 1);
      left_sums[i] = 0;
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
  wd.limit_ns = p.wait_ns;

  if (warp == C::WARPS) {
    // ------------------------------------------------------------- records
    Walk w;
    w.begin(p, start, kRows);
    bool ok = !(p.withhold && blockIdx.x == 0);
    for (uint32_t np = 0; ok; ++np) {
      const uint32_t at = np % C::PIECES;
      if (lane == 0) ok = mbar_wait(piece_empty(at), ((np / C::PIECES) & 1) ^ 1, wd, 91);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      const bool some = w.more;
      if (some) write_piece<D>(p, w, pieces[at]);
      else if (lane == 0) pieces[at].valid = 0;
      if (lane == 0) mbar_arrive(piece_full(at));
      if (!some) break;
      w.write_records(p, kRows, lane);
      w.next(p, kRows);
    }
    if (!ok) p.hdr[WS_CA_QUOTA] = -1;    // records are missing: the finishing kernel leaves everything as it is
    return;
  }

  const LaneOffsets<D> at(lane);
  float* sums = reinterpret_cast<float*>(smem + C::SUM_OFF);
  const uint8_t* ring = smem + warp * (C::DEPTH * C::STEP);
  const uint32_t ring0 = smem0 + warp * (C::DEPTH * C::STEP);
  const int spp_log = p.page_log - 5;    // steps of a page
  bool ok = true, wide = false;          // wide: the last piece's sums took the whole space

  // The copies run ahead of the work: `issued` and `worked` steps of this warp
  // so far; the next one to copy, if it is known yet (have), is ist of piece
  // ip - 1, its page on its way.  Looking for it never waits: a record that is not there yet
  // may be waiting for this warp's work on an older piece.
  uint32_t issued = 0, worked = 0, ip = 0;
  int ist = 0, ilast = 0, ifirst = warp, ipage = 0, ih = 0, ib = 0;
  const int32_t* itable = nullptr;
  bool have = false;
  const PageLayout lay(p.page_size, D);
  auto look = [&]() -> bool {
    while (!have) {
      if (!__all_sync(0xffffffffu, mbar_test_wait(piece_full(ip % C::PIECES), (ip / C::PIECES) & 1))) return false;
      const SPiece<D>& pc = pieces[ip % C::PIECES];
      if (!pc.valid) return false;
      ist = pc.step0 + ifirst;
      ilast = pc.step1;
      ++ip;
      have = ist < ilast;
      if (have) {
        itable = pc.table;
        ih = pc.h;
        ib = pc.b;
        ipage = __ldg(itable + (ist >> spp_log));
      } else {
        ifirst = ist - ilast;
      }
    }
    return true;
  };
  auto fill = [&]() {
    while (issued - worked < (uint32_t)C::DEPTH && look()) {
      if (ipage >= 0 && ipage < p.num_pages) {
        const int place = (ist & ((1 << spp_log) - 1)) * C::TOKENS;
        const uint8_t* block = p.pages + ((int64_t)ipage * p.H + ih) * lay.bytes();
        const uint8_t* codes = block + place * (D / 2) + lane * 16;
        const uint32_t dst = ring0 + (issued % C::DEPTH) * C::STEP + lane * 16;
#pragma unroll
        for (int i = 0; i < C::CODES / 512; ++i) {
          copy16(dst + 512 * i, codes + 512 * i);
          copy16(dst + C::STEP_V + 512 * i, codes + lay.half() + 512 * i);
        }
        constexpr int NS = C::SCALES / 16;   // lanes that copy K scales, V scales
        const uint8_t* scales = block + lay.scales() + place * (D / 16) + lane * 16;
        if (lane < NS) copy16(dst + C::STEP_KS, scales);
        else if (lane < 2 * NS) copy16(dst + C::STEP_KS, scales + lay.half() - C::SCALES);
        if (p.times && lane >= 16)           // and the times
          copy16(dst - 256 + C::STEP_T, reinterpret_cast<const uint8_t*>(p.page_times + ((int64_t)ipage << p.page_log) + place) +
                                            (lane - 16) * 16);
      } else if (lane == 0) {
        set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, ib);
      }
      copy_commit();
      ++issued;
      ist += C::WARPS;
      have = ist < ilast;
      if (have) ipage = __ldg(itable + (ist >> spp_log));
      else ifirst = ist - ilast;
    }
  };

  int first = warp;                      // steps of the next piece before this warp's first
  for (uint32_t np = 0;; ++np) {
    ok = mbar_wait(piece_full(np % C::PIECES), (np / C::PIECES) & 1, wd, 93);
    const SPiece<D>& pc = pieces[np % C::PIECES];
    if (!ok || !pc.valid) break;
    __syncwarp();
    const int rows = pc.rows, slot = pc.slot;
    if (!have && ip <= np) {             // (pieces in between had no step for this warp)
      ip = np;
      ifirst = first;
    }
    fill();
    float o[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
    {
      const int len = pc.L, pos0 = pc.pos0, nh = pc.hist;  // (rows behind the history rows are at len)
      const int pmin = nh > 0 ? pos0 : len, pmax = nh == rows ? pos0 + rows - 1 : len;
      const bool one_time = !p.rab_time || pc.tmin == pc.tmax;
      const float far_bias = pc.time_bias[kTimeSlots];
      const float* rp = p.rab_pos ? p.rab_pos + pc.h * p.P : nullptr;
      const int step1 = pc.step1;
      int step = pc.step0 + first;
#pragma unroll 1
      for (; step < step1; step += C::WARPS) {
        // the oldest of DEPTH copies; with fewer under way, all of them
        if (issued - worked == (uint32_t)C::DEPTH) copy_wait<C::DEPTH - 1>();
        else copy_wait<0>();
        __syncwarp();
        const uint8_t* part = ring + (worked % C::DEPTH) * C::STEP;
        const int js = step * C::TOKENS;                   // first token of the step
        {
          float c[2][4] = {};     // scores of its two halves
          {
            uint32_t k[4][D / 32];
            uint32_t ks[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {                  // tokens token_of(g) + 8 i
              load_words<D / 32>(part + at.k + 8 * i * (D / 2), k[i]);
              const uint8_t* sp = part + at.ks + 8 * i * (D / 16);
              ks[i] = D == 128 ? *reinterpret_cast<const uint16_t*>(sp) : *sp;
            }
            __half2 sc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[i] = e4m3x2_half2(ks[i]);
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {             // 8 features at a time: two inner steps
              const bool hi = D == 128 && x >= 2;
              const uint2 q0 = pc.q[2 * x][lane], q1 = pc.q[2 * x + 1][lane];
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const __half2 s0 = sc[2 * half], s1 = sc[2 * half + 1];
                const uint4 a = decode8(k[2 * half][x], hi ? __high2half2(s0) : __low2half2(s0));
                const uint4 b = decode8(k[2 * half + 1][x], hi ? __high2half2(s1) : __low2half2(s1));
                mma16816(c[half], a.x, b.x, a.y, b.y, q0.x, q0.y);
                mma16816(c[half], a.z, b.z, a.w, b.w, q1.x, q1.y);
              }
            }
          }
          // a lane looks up the bias of its token towards the block's rows, if they share it
          const int jl = js + lane;
          int64_t tl = 0;
          if (p.times) tl = reinterpret_cast<const int64_t*>(part + C::STEP_T)[lane];
          bool same = jl <= pmin;
          float bl = far_bias;
          if (pmin - (js + C::TOKENS - 1) < p.P - 1 && rp) {   // near tokens: their buckets' own biases, from global memory
            const int a = min(max(pmin - jl, 0), p.P - 1);
            bl = scaled_bias(__ldg(rp + a));
            same = same && a == min(max(pmax - jl, 0), p.P - 1);
          }
          {
            const int a = bit_length(pc.tmin, tl);
            bl += pc.time_bias[a];
            if (!one_time) {
              const int64_t tmin = pc.tmin, tmax = pc.tmax;
              same = same && min(a, p.Tb - 1) == min(bit_length(tmax, tl), p.Tb - 1) && (tl <= tmin || tl >= tmax);
            }
          }
          // scores of tokens token_of(g) + 8 i (c[i / 2][2 (i % 2)], and the next) for rows 2t, 2t + 1
          const int j0 = js + token_of(g);
          uint32_t pr[4];
          const float2 k2 = *reinterpret_cast<const float2*>(pc.ka + 2 * t);
          if (__all_sync(0xffffffffu, same || jl >= len)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float b = __shfl_sync(0xffffffffu, bl, token_of(g) + 8 * i);
              pr[i] = silu_pair(__ffma2_rn(make_float2(c[i >> 1][2 * (i & 1)], c[i >> 1][2 * (i & 1) + 1]), k2,
                                           make_float2(b, b)));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 8 * i;
              const int64_t tj = __shfl_sync(0xffffffffu, tl, token_of(g) + 8 * i);
              float b[2];
              uint32_t keep = 0;
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const int r = 2 * t + f, pos = r < nh ? pos0 + r : len;
                b[f] = pc.time_bias[bit_length(pc.tq[r], tj)];
                if (rp) b[f] += scaled_bias(rp[min(max(pos - j, 0), p.P - 1)]);
                keep |= j <= pos ? 0xffffu << (16 * f) : 0u;
              }
              pr[i] = silu_pair(__ffma2_rn(make_float2(c[i >> 1][2 * (i & 1)], c[i >> 1][2 * (i & 1) + 1]), k2,
                                           make_float2(b[0], b[1]))) & keep;
            }
          }
          const bool tail = js + C::TOKENS > len;          // tokens behind the cache's end: neither scores nor values
          if (tail) {
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] = j0 + 8 * i < len ? pr[i] : 0u;
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t vs[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) vs[e] = part[at.vs[e & 1] + (16 * half + 8 * (e >> 1)) * (D / 16)];
            if (tail) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (js + token_of(2 * t + (e & 1)) + 16 * half + 8 * (e >> 1) >= len) vs[e] = 0;
            }
            const uint32_t b0 = transpose8x8(pr[2 * half]), b1 = transpose8x8(pr[2 * half + 1]);
            // values: a code of each of two tokens to a byte, so that the decoded pairs are pairs of tokens
            const __half2 s01 = e4m3x2_half2(vs[0] | (vs[1] << 8)), s23 = e4m3x2_half2(vs[2] | (vs[3] << 8));
            uint32_t v[4][D / 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) load_words<D / 64>(part + at.v[e & 1] + (16 * half + 8 * (e >> 1)) * (D / 2), v[e]);
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {             // 8 features of the lane's D / 8
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
        }
        __syncwarp();
        ++worked;
        fill();
      }
      first = step - step1;
    }
    // the piece's record is free once every warp has read it
    __syncwarp();
    if (lane == 0) mbar_arrive(piece_empty(np % C::PIECES));
    // the warps' sums: o[m] holds features g D/8 + 2m, + 1 of rows 2t, 2t + 1.  Up to 4 rows leave room for two
    // pieces' sums, so that a warp goes on to the next piece while others finish this one; the last warp to leave
    // its sum adds them all up.
    const uint32_t nbuf = rows <= kRows / 2 ? 2u : 1u;
    float* mine = sums + (nbuf == 2 ? (np & 1) * (C::WARPS * (kRows / 2) * D) : 0);
    // the buffer's previous piece, np - 2 (or the one before this, with more rows), has been added up
    ok = mbar_wait(sum_free(np & 1), ((np >> 1) & 1) ^ 1, wd, 95) &&
         (nbuf == 2 && !wide ? true : np == 0 || mbar_wait(sum_free((np - 1) & 1), ((np - 1) >> 1) & 1, wd, 96));
    if (!ok) break;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * t + e;
      if (r < rows) {
        float* dst = mine + (warp * rows + r) * D + g * (D / 8);
#pragma unroll
        for (int m = 0; m < MT; ++m) *reinterpret_cast<float2*>(dst + 2 * m) = make_float2(o[m][e], o[m][2 + e]);
      }
    }
    wide = nbuf == 1;
    __threadfence_block();
    __syncwarp();
    int done = 0;
    if (lane == 0) done = atomicAdd(&left_sums[np & 1], 1);
    done = __shfl_sync(0xffffffffu, done, 0);
    if (done == C::WARPS - 1) {
      __threadfence_block();
      float* part = p.part + (int64_t)slot * (kRows * D);
      for (int e = lane * 4; e < rows * D; e += 128) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < C::WARPS; ++k) {
          const float4 y = *reinterpret_cast<const float4*>(mine + k * rows * D + e);
          x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        *reinterpret_cast<float4*>(part + e) = x;
      }
      if (lane == 0) left_sums[np & 1] = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(sum_free(np & 1));
    }
  }
  copy_wait<0>();
  if (!ok) p.hdr[WS_CA_QUOTA] = -1;
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
