// Tensor-core kernel of the attention over the paged 4-bit cache
// (hstu_attn_fwd_cached): for a block of up to N rows of one head, over tiles
// of 128 cached tokens,
//
//   S^T [128 x N] = K Q^T          tcgen05.mma, FP16 x FP16 -> FP32 in TMEM
//   P   = 16 SiLU(z), rounded once to FP16, 0 where a row does not see a token
//   O^T [d x N] += V^T P           tcgen05.mma, accumulator in TMEM
//
// The cached tokens are the M side of the first product and the features that
// of the second, so the tensor core's fixed 128 is filled however few rows
// there are, and N follows the rows (32, 64 or 128; up to 8 rows have a kernel
// of their own).  A thread of the score step holds one cached token, whose
// position and time biases are the same for every candidate of a request: one
// table lookup a token where the block's rows share the position and time
// buckets towards it, as they do for candidates and for tokens far back (the
// decoding warps make it, while they wait for a tile buffer); a time lookup a
// score where only a time bucket's border lies inside the block; otherwise (rows
// near the tokens) both lookups a score.
//
// The pages reach shared memory as they are (cp.async.bulk, 9/16 byte a
// feature) and are decoded there to FP16, where code x scale is exact.  q is
// FP16 too: a BF16 row times the power of two that brings its largest feature
// to 2^14 is exact down to 2^-28 of that feature; the power goes back in with
// alpha.
//
// Roles (27 warps): 0-15 scores (warp w: TMEM lanes 32 (w % 4), columns quarter
// w / 4 of the tile), 16-23 decoding, q and the tokens' biases, 24 page copies and
// the CTA's list of pieces, 25 S products and TMEM, 26 PV products.  Two tile buffers {K, V}; P
// takes K's place once the tile's S is complete.  Work is dealt evenly
// (hstu_cached.cuh).  Every wait is bounded.
//
// What bounds it: a tile buffer's round of decoding K (1,000 cycles), the S
// product (1,100), the scores (2,450), the PV product (1,300) and back, which two
// buffers share: 3,200 cycles a tile of 128 tokens x 128 rows, where the tensor
// core itself needs 1,000.  A third buffer does not fit beside the packed tiles.
// 32 users x 128 candidates over some 158,000 cached tokens, four heads of 128:
// 80 us with the finishing kernel, 520 TFLOP/s.  Scores by 16 warps on one tile or
// by two groups of 8 on a tile each take the same time with 128 rows; with fewer
// rows or the near tokens' lookups the 16 were ahead (27 against 30 us, 75 against
// 78 us, before other steps).  One reciprocal for two scores, or Newton steps in
// its place, bought nothing: without any SiLU at all the kernel took 9% less.  Gaps
// in 32 bits where they fit took first passes from 74 to 65 us.  Biases found by
// the decoding warps instead of every score warp: new rows and candidates of 32
// users 20.7 -> 19.2 us, 128 candidates 81.4 -> 80.0, first passes 51.6 -> 53.5.
#include "hstu_cached.cuh"
#include "tc_ptx.cuh"

namespace hstu {

namespace {

using namespace tc;

constexpr int TILE = kCachedTile;
constexpr int kEpiWarps = 16, kDecWarps = 8;    // score warps, decoding warps
constexpr int kDecWarp0 = kEpiWarps, kCopyWarp = kDecWarp0 + kDecWarps, kSWarp = kCopyWarp + 1, kPvWarp = kSWarp + 1;
constexpr int kThreads = (kPvWarp + 1) * 32;     // 27 warps, 7 a sub-partition: 72 registers

template <int D, int N>
struct Cfg {
  static constexpr int NCH = D / 64;                       // 128-byte column chunks of a decoded row
  static constexpr int CHUNK = TILE * 128;
  static constexpr int KV_BYTES = NCH * CHUNK;
  static constexpr int P_BYTES = TILE * N * 2;
  static constexpr int KP_BYTES = KV_BYTES > P_BYTES ? KV_BYTES : P_BYTES;
  static constexpr int P_ROW = N >= 64 ? 128 : N * 2;      // bytes of a row of a P chunk
  static constexpr int QB = N == 128 ? 1 : 2;              // q buffers
  static constexpr int Q_BYTES = N * D * 2;
  static constexpr int ITEMS = N == 128 ? 2 : 3;           // piece records in flight
  static constexpr int NR = D == 64 ? 6 : (N >= 64 ? 3 : 4);   // packed tiles in flight
  static constexpr int NT = NR + (N == 32 ? 1 : 2);                        // their times live until the scores are done
  static constexpr int RAW_BYTES = 2 * TILE * (D / 2 + D / 16);   // the tile's pages' blocks, as they are
  // shared memory
  static constexpr int KP_OFF = 0;
  static constexpr int V_OFF = KP_OFF + 2 * KP_BYTES;
  static constexpr int Q_OFF = V_OFF + 2 * KV_BYTES;
  static constexpr int RAW_OFF = Q_OFF + QB * Q_BYTES;
  static constexpr int TS_OFF = RAW_OFF + NR * RAW_BYTES;
  static constexpr int QT_OFF = TS_OFF + NT * TILE * 8;    // int64 [ITEMS][N] row times
  static constexpr int QT32_OFF = QT_OFF + ITEMS * N * 8;  // int32 [ITEMS][N], from the earliest row's
  static constexpr int KA_OFF = QT32_OFF + ITEMS * N * 4;    // float [ITEMS][N] score factors
  static constexpr int TB_OFF = KA_OFF + ITEMS * N * 4;    // float [ITEMS][kTimeSlots + 1] time biases, the far position's
  static constexpr int BIAS_OFF = TB_OFF + ITEMS * (kTimeSlots + 1) * 4;   // float [2][TILE] of a tile's tokens, where rows share them
  static constexpr int MODE_OFF = BIAS_OFF + 2 * TILE * 4;                 // int [2][4] how 32 tokens are scored
  static constexpr int SLOT_OFF = (MODE_OFF + 32 + 15) / 16 * 16;
  // barriers
  static constexpr int RAWFULL = 0, RAWEMPTY = RAWFULL + NR, TSFULL = RAWEMPTY + NR, TSEMPTY = TSFULL + NT,
                       ITEMFULL = TSEMPTY + NT, ITEMEMPTY = ITEMFULL + ITEMS, QTFULL = ITEMEMPTY + ITEMS,
                       QFULL = QTFULL + ITEMS, QEMPTY = QFULL + QB, KREADY = QEMPTY + QB, VREADY = KREADY + 2,
                       STEMPTY = VREADY + 2, SFULL = STEMPTY + 2, PREADY = SFULL + 2, OFULL = PREADY + 2,
                       OEMPTY = OFULL + 2, DRAIN = OEMPTY + 2, NBAR = DRAIN + 1;
  static constexpr int BAR_OFF = SLOT_OFF + ITEMS * 96;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int BYTES = MISC_OFF + 512;
  static_assert(16 + sizeof(Start) <= 128, "the start's place");
  static constexpr uint32_t TMEM_COLS = 4 * N;             // S 0, 1 and O 0, 1
  static_assert(BYTES + 1024 <= (int)kMaxSmemPerCta, "one CTA's shared memory");
};

// A piece of an item, as the copy warp hands it to the other roles.
struct __align__(16) Piece {
  int64_t row0;       // first row of the block
  int64_t tmin, tmax; // of the block's rows (written by the decode warps)
  int valid;          // 0: no more pieces
  int b, h, rows;     // rows of the block that exist
  int L, pos0, hist;  // cached tokens; position of the block's first row; its history rows (the others are at L)
  int tile0, tile1;   // tiles of the piece
  int slot;           // of its sum
};
static_assert(sizeof(Piece) <= 96, "a slot holds a piece");

// How 32 tokens of a tile are scored: one bias a token for all rows; all tokens exist; gaps of 32 bits; the last
// position bucket.
enum : int { kFast = 1, kWhole = 2, kNarrow = 4, kFar = 8 };
// Binary digits of a gap to the block's earliest row: two such gaps differ by less than 2^31.
constexpr int kNarrowBits = 30;
static_assert(kNarrowTsSpan == (int64_t)1 << kNarrowBits, "as in the other kernels");

__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > 200000000ull) break;
  }
}

// The place of 16-byte column chunk c of row r in a swizzled chunk whose rows are ROW bytes.
template <int ROW>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  constexpr int SH = ROW == 128 ? 0 : (ROW == 64 ? 1 : 2), M = ROW / 16 - 1;
  return (uint32_t)(r * ROW + ((c ^ ((r >> SH) & M)) << 4));
}

// Where a decoding thread's parts of a tile lie: it takes 32 features of a row
// at a time.  With 4 threads a row (D = 128) 8 neighbouring threads take
// 4 rows x 2 segments: their stores then hit 8 different 16-byte banks, their
// loads 4 (the loads are a quarter of the stores).
template <int D>
struct DecodePlan {
  static constexpr int SEGS = D / 32, RPW = 32 / SEGS, STEPS = TILE / (kDecWarps * RPW);   // rows a warp takes at a time
  int row0;                 // row of step 0; a step is kDecWarps * RPW rows on
  int code[STEPS], scale[STEPS];   // in the packed tile: blocks of a page, codes and scales of K (V: half a block on)
  uint32_t out[4];          // of the four 16-byte chunks in the decoded tile, at step 0
  __device__ __forceinline__ DecodePlan(const PageLayout& lay, int page_log, int dw, int lane) {
    const int seg = D == 128 ? (lane & 1) + 2 * (lane >> 4) : lane & 1, sub = D == 128 ? (lane >> 1) & 7 : lane >> 1;
    row0 = dw * RPW + sub;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = row0 + i * kDecWarps * RPW, at = r & ((1 << page_log) - 1), block = (r >> page_log) * lay.bytes();
      code[i] = block + at * (D / 2) + seg * 16;
      scale[i] = block + lay.scales() + at * (D / 16) + seg * 2;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) out[c] = (seg / 2) * (TILE * 128) + swz<128>(row0, (seg & 1) * 4 + c);
  }
  // part: the packed K or V; rows from `rows` on become zeros
  __device__ __forceinline__ void decode(const uint8_t* part, uint8_t* to, int rows) const {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      uint4 w = *reinterpret_cast<const uint4*>(part + code[i]);
      uint32_t sc = *reinterpret_cast<const uint16_t*>(part + scale[i]);
      if (rows < TILE && row0 + i * kDecWarps * RPW >= rows) {
        w = make_uint4(0, 0, 0, 0);
        sc = 0;
      }
      const __half2 s = e4m3x2_half2(sc);
      const __half2 s0 = __low2half2(s), s1 = __high2half2(s);
      uint8_t* base = to + i * (kDecWarps * RPW * 128);   // a multiple of 8 rows on: the same swizzle
      *reinterpret_cast<uint4*>(base + out[0]) = decode8(w.x, s0);
      *reinterpret_cast<uint4*>(base + out[1]) = decode8(w.y, s0);
      *reinterpret_cast<uint4*>(base + out[2]) = decode8(w.z, s1);
      *reinterpret_cast<uint4*>(base + out[3]) = decode8(w.w, s1);
    }
  }
};

template <int D, int N>
__global__ void __maxnreg__(72) cached_tc_kernel(const __grid_constant__ CachedParams p) {
  using L = Cfg<D, N>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  auto bar = [&](int i) -> uint32_t { return base_u32 + L::BAR_OFF + 8u * (uint32_t)i; };
  auto piece_at = [&](uint32_t i) -> Piece& { return *reinterpret_cast<Piece*>(base + L::SLOT_OFF + 96 * (int)i); };
  int64_t* qt = reinterpret_cast<int64_t*>(base + L::QT_OFF);
  int32_t* qt32 = reinterpret_cast<int32_t*>(base + L::QT32_OFF);
  float* kA = reinterpret_cast<float*>(base + L::KA_OFF);
  float* tb = reinterpret_cast<float*>(base + L::TB_OFF);
  float* token_bias = reinterpret_cast<float*>(base + L::BIAS_OFF);
  int* modes = reinterpret_cast<int*>(base + L::MODE_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + L::MISC_OFF + 4);
  Start* start = reinterpret_cast<Start*>(base + L::MISC_OFF + 16);
  int* scan = reinterpret_cast<int*>(base + L::MISC_OFF + 128);   // [3][32] warp sums

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NBAR; ++i) {
      int n = 1;
      if ((i >= L::RAWEMPTY && i < L::TSFULL) || (i >= L::QTFULL && i < L::QEMPTY) || (i >= L::KREADY && i < L::STEMPTY))
        n = kDecWarps;
      else if ((i >= L::TSEMPTY && i < L::ITEMFULL) || (i >= L::PREADY && i < L::OFULL) || (i >= L::OEMPTY && i < L::DRAIN))
        n = kEpiWarps;
      else if (i >= L::ITEMEMPTY && i < L::QTFULL)
        n = kDecWarps + kEpiWarps + 2;
      else if (i == L::DRAIN)
        n = 2;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kSWarp) {
    tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();               // what came before in the stream may have written anything read below
  pdl_launch_dependents();  // the finishing kernel waits for this grid's end itself

  cut_work<kThreads>(p, N, scan, start);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  Watchdog wd;
  wd.abort = abort_flag;
  wd.err = p.hdr + WS_ERR;
  wd.err_info = p.hdr + WS_ERR_INFO;
  wd.limit_ns = p.wait_ns;
  const bool timed = p.times != nullptr;

  if (warp == kCopyWarp) {
    // -------------------------------------------------- pieces, page copies
    uint32_t it = 0, tk = 0;     // pieces, tiles so far
    bool ok = !(p.withhold && blockIdx.x == 0);
    const int ppt = TILE / p.page_size;
    const PageLayout lay(p.page_size, D);
    Walk w;
    w.begin(p, *start, N);
    while (ok && w.more) {
      const int take = w.take(), tile = w.tile, b = w.b, h = w.h;
      const CachedSeq s = w.s;
      const uint32_t sl = it % L::ITEMS;
      if (lane == 0) ok = mbar_wait(bar(L::ITEMEMPTY + sl), ((it / L::ITEMS) & 1) ^ 1, wd, 61);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (lane == 0) {
        Piece& pc = piece_at(sl);
        const int r0 = w.qb * N, hist = s.n - s.m;
        pc.row0 = s.row0 + r0;
        pc.valid = 1;
        pc.b = b; pc.h = h; pc.rows = min(N, s.n - r0); pc.L = s.L;
        pc.hist = max(0, min(hist - r0, pc.rows));
        pc.pos0 = s.L - hist + r0;
        pc.tile0 = tile; pc.tile1 = tile + take;
        pc.slot = w.slot(p);
        mbar_arrive(bar(L::ITEMFULL + sl));
      }
      __syncwarp();
      ++it;
      w.write_records(p, N, lane);
      // the block table's entries, 32 at a time: lane i holds entry e0 + i
      const int32_t* row = p.table + (int64_t)b * p.max_pages;
      const int npages = (s.L + p.page_size - 1) / p.page_size;
      int e0 = tile * ppt;
      int32_t entry = e0 + lane < npages ? row[e0 + lane] : -1;
      int32_t next = e0 + 32 + lane < npages ? row[e0 + 32 + lane] : -1;
      for (int t = tile; ok && t < tile + take; ++t, ++tk) {
        const int e = t * ppt;
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
        if (there && !good) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, b);
        const int n = __popc(__ballot_sync(0xffffffffu, good && lane < ppt));
        const uint32_t rs = tk % L::NR, ts = tk % L::NT;
        if (lane == 0) {
          ok = mbar_wait(bar(L::RAWEMPTY + rs), ((tk / L::NR) & 1) ^ 1, wd, 62) &&
               (!timed || mbar_wait(bar(L::TSEMPTY + ts), ((tk / L::NT) & 1) ^ 1, wd, 63));
          if (ok) {
            mbar_arrive_expect_tx(bar(L::RAWFULL + rs), (uint32_t)(n * lay.bytes()));
            if (timed) mbar_arrive_expect_tx(bar(L::TSFULL + ts), (uint32_t)(n * p.page_size * 8));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (good && lane < ppt)
          bulk_load(base_u32 + L::RAW_OFF + rs * L::RAW_BYTES + pg * lay.bytes(), p.pages + ((int64_t)id * p.H + h) * lay.bytes(),
                    (uint32_t)lay.bytes(), bar(L::RAWFULL + rs));
        else if (good && timed)
          bulk_load(base_u32 + L::TS_OFF + ts * (TILE * 8) + pg * p.page_size * 8, p.page_times + ((int64_t)id << p.page_log),
                    (uint32_t)(p.page_size * 8), bar(L::TSFULL + ts));
      }
      if (!ok) break;
      w.next(p, N);
    }
    if (ok && lane == 0) {
      const uint32_t sl = it % L::ITEMS;
      if (mbar_wait(bar(L::ITEMEMPTY + sl), ((it / L::ITEMS) & 1) ^ 1, wd, 64)) {
        piece_at(sl).valid = 0;
        mbar_arrive(bar(L::ITEMFULL + sl));
      }
    }
    // no copy may land in shared memory after the CTA's end
    if (lane == 0) {
      for (uint32_t i = 0; i < (uint32_t)L::NR; ++i)
        if (tk > i) drain(bar(L::RAWFULL + i), ((tk - 1 - i) / L::NR) & 1);
      for (uint32_t i = 0; timed && i < (uint32_t)L::NT; ++i)
        if (tk > i) drain(bar(L::TSFULL + i), ((tk - 1 - i) / L::NT) & 1);
    }
  } else if (warp >= kDecWarp0 && warp < kDecWarp0 + kDecWarps) {
    // --------------------------------------------------------- decoding, q
    const int dw = warp - kDecWarp0;
    const PageLayout lay(p.page_size, D);
    const DecodePlan<D> plan(lay, p.page_log, dw, lane);
    const int half_block = lay.half();
    uint32_t it = 0, tk = 0;
    bool ok = true;
    while (ok) {
      const uint32_t sl = it % L::ITEMS, qbuf = it % L::QB;
      ok = mbar_wait(bar(L::ITEMFULL + sl), (it / L::ITEMS) & 1, wd, 65);
      if (!ok) break;
      Piece& pc = piece_at(sl);
      if (!pc.valid) break;
      {
        // q rows: D / 8 lanes a row, 8 features each
        constexpr int LR = D / 8, RPP = kDecWarps * 32 / LR, PASSES = (N + RPP - 1) / RPP;
        const int64_t row0 = pc.row0;
        const int rows = pc.rows, h = pc.h;
        const int sub = dw * 32 + lane, c = sub % LR;
        uint4 x[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int r = i * RPP + sub / LR;
          x[i] = make_uint4(0, 0, 0, 0);
          if (r < rows) x[i] = *reinterpret_cast<const uint4*>(p.q + ((row0 + r) * p.H + h) * D + c * 8);
        }
        if (dw == 1) store_time_biases(p, h, tb + sl * (kTimeSlots + 1), lane);
        if (dw == 0) {   // the rows' times, and their range
          int64_t row_time[N / 32], mn = timed ? INT64_MAX : 0, mx = timed ? INT64_MIN : 0;
#pragma unroll
          for (int i = 0; i < N / 32; ++i) row_time[i] = timed && lane + 32 * i < rows ? p.times[row0 + lane + 32 * i] : 0;
#pragma unroll
          for (int i = 0; i < N / 32; ++i) {
            if (timed && lane + 32 * i < rows) {
              mn = row_time[i] < mn ? row_time[i] : mn;
              mx = row_time[i] > mx ? row_time[i] : mx;
            }
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const int64_t a = __shfl_xor_sync(0xffffffffu, mn, o), b2 = __shfl_xor_sync(0xffffffffu, mx, o);
            mn = a < mn ? a : mn;
            mx = b2 > mx ? b2 : mx;
          }
          if (lane == 0) {
            pc.tmin = mn;
            pc.tmax = mx;
          }
#pragma unroll
          for (int i = 0; i < N / 32; ++i) {
            qt[sl * N + lane + 32 * i] = row_time[i];
            qt32[sl * N + lane + 32 * i] = (int32_t)(row_time[i] - mn);   // used where it fits
          }
        }
        ok = mbar_wait(bar(L::QEMPTY + qbuf), ((it / L::QB) & 1) ^ 1, wd, 66);
        if (!ok) break;
        uint8_t* qs = base + L::Q_OFF + qbuf * L::Q_BYTES;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int r = i * RPP + sub / LR;
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t top = 0;    // largest magnitude's bits (BF16 in the high half of FP32)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7fff0000u, w[e] & 0x7fff0000u));
#pragma unroll
          for (int o = LR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          float down;
          const float up = row_scale(top, down);
          uint32_t f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = pack_f16(bf16_lo_f(w[e]) * up, bf16_hi_f(w[e]) * up);
          if (N % RPP == 0 || r < N) {
            *reinterpret_cast<uint4*>(qs + (c / 8) * (N * 128) + swz<128>(r, c % 8)) = make_uint4(f[0], f[1], f[2], f[3]);
            if (c == 0) kA[sl * N + r] = -kLog2e * p.alpha * p.k_scale * down;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(L::QFULL + qbuf));
          mbar_arrive(bar(L::QTFULL + sl));
        }
      }
      const int t0 = pc.tile0, t1 = pc.tile1, len = pc.L;
      const float* tbl = tb + sl * (kTimeSlots + 1);
      if (dw < 4) {      // the first four warps also find the tokens' biases, from the rows' range of times
        ok = mbar_wait(bar(L::QTFULL + sl), (it / L::ITEMS) & 1, wd, 81);
        if (!ok) break;
      }
      const int64_t tmin = pc.tmin, tmax = pc.tmax;
      const int pmin = pc.hist > 0 ? pc.pos0 : len, pmax = pc.hist == pc.rows ? pc.pos0 + pc.rows - 1 : len;
      const float* rp = p.rab_pos ? p.rab_pos + pc.h * p.P : nullptr;
      const bool one_time = !p.rab_time || tmin == tmax, one_span = bit_length(tmin, tmax) <= kNarrowBits;
      for (int t = t0; t < t1; ++t, ++tk) {
        const uint32_t rs = tk % L::NR, st = tk & 1;
        ok = mbar_wait(bar(L::RAWFULL + rs), (tk / L::NR) & 1, wd, 67);
        if (!ok) break;
        float bias = 0.f;
        int mode = 0;
        if (dw < 4) {    // while the tile buffer is still in use
          const uint32_t ts = tk % L::NT;
          const int r = dw * 32 + lane, j = t * TILE + r;
          int64_t tj = 0;
          if (timed) {
            ok = mbar_wait(bar(L::TSFULL + ts), (tk / L::NT) & 1, wd, 79);
            if (!ok) break;
            tj = *reinterpret_cast<const int64_t*>(base + L::TS_OFF + ts * (TILE * 8) + r * 8);
          }
          // one bias for all of the block's rows?
          bool same = j <= pmin;
          bias = tbl[kTimeSlots];                            // far tokens share the last position bucket
          const bool far = pmin - (t * TILE + dw * 32 + 31) >= p.P - 1;
          if (!far && rp) {
            const int a = min(max(pmin - j, 0), p.P - 1);
            same = same && a == min(max(pmax - j, 0), p.P - 1);
            bias = scaled_bias(__ldg(rp + a));
          }
          const int a = bit_length(tmin, tj);
          bias += tbl[a];
          if (!one_time) same = same && min(a, p.Tb - 1) == min(bit_length(tmax, tj), p.Tb - 1) && (tj <= tmin || tj >= tmax);
          const bool fast = __all_sync(0xffffffffu, same || j >= len);
          const bool whole = __all_sync(0xffffffffu, j < len);
          // else gaps of 32 bits where they fit (their lengths say so whatever the times are; differences may wrap)
          const bool narrow = __all_sync(0xffffffffu, j >= len || a <= kNarrowBits) && one_span;
          mode = (fast ? kFast : 0) | (whole ? kWhole : 0) | (narrow ? kNarrow : 0) | (far ? kFar : 0);
        }
        ok = mbar_wait(bar(L::STEMPTY + st), ((tk >> 1) & 1) ^ 1, wd, 68);
        if (!ok) break;
        if (dw < 4) {
          token_bias[st * TILE + dw * 32 + lane] = bias;
          if (lane == 0) modes[st * 4 + dw] = mode;
        }
        const uint8_t* raw = base + L::RAW_OFF + rs * L::RAW_BYTES;
        const int rows = len - t * TILE;
        plan.decode(raw, base + L::KP_OFF + st * L::KP_BYTES, rows);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::KREADY + st));
        plan.decode(raw + half_block, base + L::V_OFF + st * L::KV_BYTES, rows);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(L::VREADY + st));
          mbar_arrive(bar(L::RAWEMPTY + rs));
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::ITEMEMPTY + sl));
      ++it;
    }
  } else if (warp == kSWarp) {
    // ---------------------------------------------------------- S^T = K Q^T
    {   // the whole warp walks, so that the operands are uniform values; one elected lane issues
      auto wait = [](bool done) { return (bool)__all_sync(0xffffffffu, done); };   // one answer for the warp
      constexpr uint32_t IDESC = idesc_f16(TILE, N, false, false);
      uint32_t it = 0, tk = 0;
      bool ok = true;
      while (ok) {
        const uint32_t sl = it % L::ITEMS, qbuf = it % L::QB;
        ok = wait(mbar_wait(bar(L::ITEMFULL + sl), (it / L::ITEMS) & 1, wd, 69));
        if (!ok) break;
        const Piece& pc = piece_at(sl);
        if (!pc.valid) break;
        const int nt = pc.tile1 - pc.tile0;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::ITEMEMPTY + sl));
        ok = wait(mbar_wait(bar(L::QFULL + qbuf), (it / L::QB) & 1, wd, 70));
        if (!ok) break;
        ++it;
        const SDesc dq = sdesc_w(base_u32 + L::Q_OFF + qbuf * L::Q_BYTES, 16, 1024);
        for (int t = 0; t < nt; ++t, ++tk) {
          const uint32_t st = tk & 1;
          // the S buffer of tile tk - 2 was read before its PV, which freed the tile buffer
          ok = wait(mbar_wait(bar(L::KREADY + st), (tk >> 1) & 1, wd, 71));
          if (!ok) break;
          fence_after_sync();
          const SDesc dk = sdesc_w(base_u32 + L::KP_OFF + st * L::KP_BYTES, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_e(tmem + st * N, dk + ((kk >> 2) * L::CHUNK + (kk & 3) * 32), dq + ((kk >> 2) * (N * 128) + (kk & 3) * 32),
                     IDESC, kk > 0 ? 1u : 0u);
          mma_commit_e(bar(L::SFULL + st));
        }
        if (!ok) break;
        mma_commit_e(bar(L::QEMPTY + qbuf));
      }
      mma_commit_e(bar(L::DRAIN));
      drain(bar(L::DRAIN), 0);
    }
  } else if (warp == kPvWarp) {
    // --------------------------------------------------------- O^T += V^T P
    {
      auto wait = [](bool done) { return (bool)__all_sync(0xffffffffu, done); };
      constexpr uint32_t IDESC = idesc_f16(128, N, true, true);
      uint32_t it = 0, tk = 0;
      bool ok = true;
      while (ok) {
        const uint32_t sl = it % L::ITEMS, ob = it & 1;
        ok = wait(mbar_wait(bar(L::ITEMFULL + sl), (it / L::ITEMS) & 1, wd, 72));
        if (!ok) break;
        const Piece& pc = piece_at(sl);
        if (!pc.valid) break;
        const int nt = pc.tile1 - pc.tile0;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::ITEMEMPTY + sl));
        ok = wait(mbar_wait(bar(L::OEMPTY + ob), ((it >> 1) & 1) ^ 1, wd, 73));
        if (!ok) break;
        ++it;
        for (int t = 0; t < nt; ++t, ++tk) {
          const uint32_t st = tk & 1;
          ok = wait(mbar_wait(bar(L::VREADY + st), (tk >> 1) & 1, wd, 74) &&
                    mbar_wait(bar(L::PREADY + st), (tk >> 1) & 1, wd, 75));
          if (!ok) break;
          fence_after_sync();
          // with 64 features the upper half of M reads the same features again; its rows are not used
          const SDesc dv = sdesc_w(base_u32 + L::V_OFF + st * L::KV_BYTES, D == 128 ? L::CHUNK : 0, 1024);
          const SDesc dp = sdesc_rows<L::P_ROW>(base_u32 + L::KP_OFF + st * L::KP_BYTES, N == 128 ? L::CHUNK : 16, 8 * L::P_ROW);
#pragma unroll
          for (int kk = 0; kk < TILE / 16; ++kk)
            mma_ss_e(tmem + (2 + ob) * N, dv + kk * 2048, dp + kk * (16 * L::P_ROW), IDESC, (t > 0 || kk > 0) ? 1u : 0u);
          mma_commit_e(bar(L::STEMPTY + st));
        }
        if (!ok) break;
        mma_commit_e(bar(L::OFULL + ob));
      }
      mma_commit_e(bar(L::DRAIN));
      drain(bar(L::DRAIN), 0);
    }
  } else {
    // -------------------------------------------------------------- scores
    constexpr int COLS = N / 4;                    // columns of a warp
    constexpr int CH = COLS < 16 ? COLS : 16;      // columns in registers at a time
    const int wq = warp & 3, col0 = (warp >> 2) * COLS;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16) + col0;
    const int r = wq * 32 + lane;                  // this thread's token in a tile, and feature in O
    uint32_t it = 0, tk = 0;
    bool ok = true;
    // a piece's sum is written out after the next piece's first scores
    bool pend = false;
    uint32_t pend_it = 0;
    int pend_slot = 0, pend_rows = 0;
    auto load_cols = [&](uint32_t addr, uint32_t (&v)[CH]) {
      if constexpr (CH == 16) tmem_ld16(addr, v);
      else tmem_ld8(addr, v);
    };
    auto write_sum = [&]() -> bool {
      const uint32_t ob = pend_it & 1;
      if (!mbar_wait(bar(L::OFULL + ob), (pend_it >> 1) & 1, wd, 76)) return false;
      fence_after_sync();
      float* dst = p.part + (int64_t)pend_slot * (N * D) + r;
#pragma unroll 1
      for (int c0 = 0; c0 < COLS; c0 += CH) {
        uint32_t v[CH];
        load_cols(lane_base + (2 + ob) * N + c0, v);
        tmem_wait_ld();
        if (D == 128 || wq < 2) {
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (col0 + c0 + c < pend_rows) dst[(col0 + c0 + c) * D] = __uint_as_float(v[c]);
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::OEMPTY + ob));
      pend = false;
      return true;
    };
    while (ok) {
      const uint32_t sl = it % L::ITEMS;
      ok = mbar_wait(bar(L::ITEMFULL + sl), (it / L::ITEMS) & 1, wd, 77);
      if (!ok) break;
      const Piece& pc = piece_at(sl);
      if (!pc.valid) break;
      ok = mbar_wait(bar(L::QTFULL + sl), (it / L::ITEMS) & 1, wd, 78);
      if (!ok) break;
      const int len = pc.L, pos0 = pc.pos0, hist = pc.hist, rows = pc.rows, t0 = pc.tile0, t1 = pc.tile1, slot = pc.slot;
      const int64_t tmin = pc.tmin;
      const float* rp = p.rab_pos ? p.rab_pos + pc.h * p.P : nullptr;
      const float* tbl = tb + sl * (kTimeSlots + 1);
      const float* ka = kA + sl * N + col0;
      const int64_t* tq = qt + sl * N + col0;
      const int32_t* tq32 = qt32 + sl * N + col0;
      for (int t = t0; t < t1; ++t, ++tk) {
        const uint32_t st = tk & 1, ts = tk % L::NT;
        const int j = t * TILE + r;
        ok = mbar_wait(bar(L::KREADY + st), (tk >> 1) & 1, wd, 82);   // the tokens' biases come with K
        if (!ok) break;
        const int mode = modes[st * 4 + wq];
        const float bias = token_bias[st * TILE + r];
        const bool fast = mode & kFast, whole = mode & kWhole, narrow = mode & kNarrow, far = mode & kFar;
        int64_t tj = 0;
        if (!fast && timed) {
          ok = mbar_wait(bar(L::TSFULL + ts), (tk / L::NT) & 1, wd, 83);
          if (!ok) break;
          tj = *reinterpret_cast<const int64_t*>(base + L::TS_OFF + ts * (TILE * 8) + r * 8);
        }
        const int rel32 = (int)(tj - tmin);      // used where it fits
        ok = mbar_wait(bar(L::SFULL + st), (tk >> 1) & 1, wd, 80);
        if (!ok) break;
        fence_after_sync();
        uint8_t* ps = base + L::KP_OFF + st * L::KP_BYTES;
        // P over K: row = token, 16-byte chunks of 8 columns
        auto put = [&](int c0, const uint32_t (&h2)[CH / 2]) {
#pragma unroll
          for (int c = 0; c < CH / 8; ++c) {
            const int col = col0 + c0 + c * 8;
            const uint32_t at = N >= 64 ? (col / 64) * L::CHUNK + swz<L::P_ROW>(r, (col % 64) / 8) : swz<L::P_ROW>(r, col / 8);
            *reinterpret_cast<uint4*>(ps + at) = make_uint4(h2[4 * c], h2[4 * c + 1], h2[4 * c + 2], h2[4 * c + 3]);
          }
        };
        if (fast) {   // the warp's columns all at once: their loads' latency is paid once
          uint32_t v[COLS / CH][CH];
#pragma unroll
          for (int i = 0; i < COLS / CH; ++i) load_cols(lane_base + st * N + i * CH, v[i]);
          tmem_wait_ld();
          const float2 b2 = make_float2(bias, bias);
#pragma unroll
          for (int i = 0; i < COLS / CH; ++i) {
            uint32_t h2[CH / 2];
#pragma unroll
            for (int c = 0; c < CH; c += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(ka + i * CH + c);
              h2[c / 2] = silu_pair(__ffma2_rn(make_float2(__uint_as_float(v[i][c]), __uint_as_float(v[i][c + 1])),
                                               make_float2(k4.x, k4.y), b2));
              h2[c / 2 + 1] = silu_pair(__ffma2_rn(make_float2(__uint_as_float(v[i][c + 2]), __uint_as_float(v[i][c + 3])),
                                                   make_float2(k4.z, k4.w), b2));
            }
            if (!whole) {
#pragma unroll
              for (int c = 0; c < CH / 2; ++c) h2[c] = j < len ? h2[c] : 0u;
            }
            put(i * CH, h2);
          }
        } else {
#pragma unroll 1
          for (int c0 = 0; c0 < COLS; c0 += CH) {
            uint32_t v[CH];
            load_cols(lane_base + st * N + c0, v);
            tmem_wait_ld();
            uint32_t h2[CH / 2];
            if (narrow && far) {
              const float fb = tbl[kTimeSlots];
#pragma unroll
              for (int c = 0; c < CH; c += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(ka + c0 + c);
                const int4 q4 = *reinterpret_cast<const int4*>(tq32 + c0 + c);
                const float2 b01 = make_float2(tbl[32 - __clz(abs(q4.x - rel32))] + fb, tbl[32 - __clz(abs(q4.y - rel32))] + fb);
                const float2 b23 = make_float2(tbl[32 - __clz(abs(q4.z - rel32))] + fb, tbl[32 - __clz(abs(q4.w - rel32))] + fb);
                h2[c / 2] = silu_pair(__ffma2_rn(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                                 make_float2(k4.x, k4.y), b01));
                h2[c / 2 + 1] = silu_pair(__ffma2_rn(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                                                     make_float2(k4.z, k4.w), b23));
              }
            } else if (narrow) {
              const int base_gap = pos0 - j, cand_gap = len - j;   // a row's distance, less its column
#pragma unroll
              for (int c = 0; c < CH; c += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(ka + c0 + c);
                const int4 q4 = *reinterpret_cast<const int4*>(tq32 + c0 + c);
                const float kf[4] = {k4.x, k4.y, k4.z, k4.w};
                const int qf[4] = {q4.x, q4.y, q4.z, q4.w};
                float w[4];
                uint32_t keep[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int col = col0 + c0 + c + e, gap = col < hist ? base_gap + col : cand_gap;
                  float bb = tbl[32 - __clz(abs(qf[e] - rel32))];
                  if (rp) bb += scaled_bias(__ldg(rp + min(max(gap, 0), p.P - 1)));
                  w[e] = fmaf(__uint_as_float(v[c + e]), kf[e], bb);
                  keep[e >> 1] |= gap >= 0 ? 0xffffu << (16 * (e & 1)) : 0u;
                }
                h2[c / 2] = silu_pair(make_float2(w[0], w[1])) & keep[0];
                h2[c / 2 + 1] = silu_pair(make_float2(w[2], w[3])) & keep[1];
              }
              if (!whole) {
#pragma unroll
                for (int c = 0; c < CH / 2; ++c) h2[c] = j < len ? h2[c] : 0u;
              }
            } else {
#pragma unroll
              for (int c = 0; c < CH; c += 2) {
                float w[2];
                uint32_t keep = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int col = col0 + c0 + c + e;
                  const int pos = col < hist ? pos0 + col : len;
                  float bb = tbl[bit_length(tq[c0 + c + e], tj)];
                  if (rp) bb += scaled_bias(rp[min(max(pos - j, 0), p.P - 1)]);
                  w[e] = fmaf(__uint_as_float(v[c + e]), ka[c0 + c + e], bb);
                  keep |= (j <= pos && j < len) ? 0xffffu << (16 * e) : 0u;
                }
                h2[c / 2] = silu_pair(make_float2(w[0], w[1])) & keep;
              }
            }
            put(c0, h2);
          }
        }
        fence_before_sync();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(L::PREADY + st));
          if (timed) mbar_arrive(bar(L::TSEMPTY + ts));
        }
        if (pend) {
          ok = write_sum();
          if (!ok) break;
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::ITEMEMPTY + sl));
      pend = true;
      pend_it = it;
      pend_slot = slot;
      pend_rows = rows;
      ++it;
    }
    if (ok && pend) write_sum();
  }

  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (threadIdx.x == 0 && *abort_flag) p.hdr[WS_CA_QUOTA] = -1;   // records and sums are missing: nothing is finished
  if (warp == kSWarp) tmem_dealloc(tmem, L::TMEM_COLS);
}

template <int D, int N>
cudaError_t launch_t(const CachedParams& p, int ctas, cudaStream_t st) {
  const size_t smem = Cfg<D, N>::BYTES + 1024;
  auto kern = cached_tc_kernel<D, N>;
  const void* fn = reinterpret_cast<const void*>(kern);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, st, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_launch_detail(e, "cached_tc_kernel", fn, kThreads, smem);
  }
  return e;
}

}  // namespace

cudaError_t launch_tc_cached(const CachedParams& p, int d, int N, int ctas, cudaStream_t st) {
  if (d == 128)
    return N == 32 ? launch_t<128, 32>(p, ctas, st) : N == 64 ? launch_t<128, 64>(p, ctas, st) : launch_t<128, 128>(p, ctas, st);
  return N == 32 ? launch_t<64, 32>(p, ctas, st) : N == 64 ? launch_t<64, 64>(p, ctas, st) : launch_t<64, 128>(p, ctas, st);
}

}  // namespace hstu
