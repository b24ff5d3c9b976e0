// Products of ragged groups of rows with a weight matrix each: y = x W[g]
// and dx = dy W[g]^T (hstu_group_fwd, the dx of hstu_group_bwd), and the C calls.
//
// Transposed: the tensor core's rows are output features, its columns the group's rows.  A
// group's last tile so costs what it has rows (in 16s or 32s), not 128, and a group of one row
// costs a load of its weights.  D[f, r] = sum_k W[k, f] x[r, k]:
//   A = 128 features x 64 k of W[g] a CTA (features contiguous: MN-major; for dx k is the
//   contiguous side: K-major), from a 3-D map [g][K][N], so that a tile's edge never
//   reads the next group's weights;
//   B = up to 256 rows x 64 k of x (K-major).  Rows of the next group that a load brings
//   along give columns that nobody stores.
// What bounded large batches was the way from L2 to the SMs (12 TB/s measured: single CTAs that
// load A and B for each 128 x 256 tile took 324 us for 161,293 rows, 512 -> 2048, whatever the tensor core had
// to do).  So CTAs work in pairs (cta_group::2: 256 features, each CTA holds half of A and half of
// B), and walk neighbouring tiles, which have the same rows: where the depth allows (512),
// B stays in shared memory from one tile to the next and A alone streams: 250-260 us (cuBLAS's product of one group of that
// size 231-249; the board is at its power limit).  What is left there: the storing warps, 5,000 cycles for a pair's
// 256 x 256 against 4,096 of the tensor core at a depth of 512, waits of 50 cycles each on barriers that are there
// already, commits (75 each).  At dx's depth of 2,048 both stream: a stage is 32 KB a CTA, 780 cycles at an SM's
// share of L2 (42 bytes a cycle) for 512 of the tensor core, which is what dx takes (31 us for 16,410 rows, 2 tiles of 32
// stages each; 236-257 us for 161,293; cuBLAS 26 and 188-204).  The loading and issuing warps run their loops as one with
// an elected lane, so that operands are uniform values (800 cycles a stage where they are not: one issuing thread, or an
// accumulator's place that changes inside the loop over the stages).
// Two accumulators in TMEM, so that a tile is stored while the next one is computed.
//
// Precision: as in hstu_group_dw.cu, the tensor core's sums lose a little at every addition, always towards zero.
// Beyond a depth of 1,024 (DEEP) an accumulator so is read after 1,024 of it and added up in the storing warps'
// registers, while the other one takes the next 1,024: FP32 results are at most 1.0e-6 off whatever the depth, where one
// accumulator is 2.1e-6 off at 2,048 and 7.6e-5 at 65,536 (a plain FP32 product 0.2e-6 and 0.4e-6); dx of 161,288 rows
// with a depth of 2,048 takes 257 us for 254, of 16,410 31.0 for 29.6.  Every 512 it would be 0.5e-6 and 274 us.
//
// Roles (352 threads): warps 0-7 store, warp 8 loads A, warp 10 B, warp 9 issues (the pair's first CTA) and
// owns TMEM.  Every wait is bounded.
#include "hstu_group.cuh"

namespace hstu {

namespace {

using namespace grp;

constexpr int kStagesMax = 8, kSlotsMax = 8;
constexpr int kRowsWarp = 10, kRowsThreads = 11 * 32;
constexpr int kABytes = 128 * 64 * 2;
enum : int { B_AFULL = 0, B_AEMPTY = B_AFULL + kStagesMax, B_BFULL = B_AEMPTY + kStagesMax, B_BEMPTY = B_BFULL + kSlotsMax,
             B_DFULL = B_BEMPTY + kSlotsMax, B_DEMPTY = B_DFULL + 2, B_DRAIN = B_DEMPTY + 2, B_COUNT };

// a 32 x 32 buffer of each storing warp
constexpr int staging_bytes(int element) { return kEpiWarps * 1024 * element; }

// 16 lanes x 32 columns: registers 4 j, 4 j + 1 are columns 8 j + 2 (t % 4) + {0, 1} of lane t / 4, the next two
// those of lane t / 4 + 8
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// four 8 x 8 matrices of 16-bit elements, transposed: lane l gives the address of row l % 8 of matrix l / 8
__device__ __forceinline__ void stmatrix_trans(uint32_t at, const uint32_t (&m)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(m[0]), "r"(m[1]),
               "r"(m[2]), "r"(m[3])
               : "memory");
}

// Walks a CTA's (a pair's) share [t, end) of the tiles: t = row block x feature blocks + feature block.
struct Tiles {
  const int* start;
  const int* first;
  int fb, rb, wide, e, row0, rows, f0, t, end, begin, blk;
  __device__ __forceinline__ Tiles(const int* start_, const int* first_, int E, int fblocks, int row_block, int width, int share,
                                   int shares, bool good)
      : start(start_), first(first_), fb(fblocks), rb(row_block), wide(width), e(0), t(0), end(0), begin(0), blk(0) {
    if (!good) return;
    const int total = start[E] * fblocks, each = total / shares, more = total - each * shares;
    t = begin = each * share + min(share, more);
    end = begin + each + (share < more ? 1 : 0);
    if (t >= end) return;
    blk = t / fb;
    int lo = 0, hi = E;   // the last group that begins at or below blk, and has rows
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= blk) lo = mid;
      else hi = mid;
    }
    e = lo;
    set();
  }
  __device__ __forceinline__ void set() {
    const int in = (blk - start[e]) * rb;
    row0 = first[e] + in;
    rows = min(rb, first[e + 1] - row0);
    f0 = (t - blk * fb) * wide;
  }
  __device__ __forceinline__ bool more() const { return t < end; }
  // whether the tile's rows are new to this share, and needed no more by the next tile
  __device__ __forceinline__ bool fresh() const { return t == begin || f0 == 0; }
  __device__ __forceinline__ bool last() const { return t + 1 == end || t + 1 == (blk + 1) * fb; }
  __device__ __forceinline__ void next() {
    if (++t >= end) return;
    if (t == (blk + 1) * fb) {
      ++blk;
      while (start[e + 1] <= blk) ++e;
    }
    set();
  }
};

// KMAJOR: W is read with k contiguous (dx), else with features contiguous (forward); CG: CTAs that work together;
// DEEP: a tile takes more than one accumulator
template <int CG, bool KMAJOR, bool DEEP, typename TO>
__global__ void __launch_bounds__(kRowsThreads, 1)
group_rows_kernel(const __grid_constant__ GroupParams p, const __grid_constant__ CUtensorMap tmw,
                  const __grid_constant__ CUtensorMap tmr, const __grid_constant__ CUtensorMap tmo) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B_COUNT];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t raw_u32 = smem_u32(smem_raw), base = (raw_u32 + 1023u) & ~1023u;
  // a ring of A, a ring (or the whole depth) of B, the storing warps' buffers, the lists of groups
  const int slot_bytes = p.row_block / CG * 128;
  const uint32_t a_at = base, b_at = a_at + p.stages * kABytes, stg_at = b_at + p.slots * slot_bytes;
  int* start = reinterpret_cast<int*>(smem_raw + (stg_at - raw_u32) + staging_bytes(sizeof(TO)));
  int* first = start + p.E + 1;
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars) + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0u : cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStagesMax; ++s) {
      mbar_init(bar(B_AFULL + s), 1);
      mbar_init(bar(B_AEMPTY + s), 1);
    }
    for (int s = 0; s < kSlotsMax; ++s) {
      mbar_init(bar(B_BFULL + s), 1);
      mbar_init(bar(B_BEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_DFULL + s), 1);
      mbar_init(bar(B_DEMPTY + s), CG * kEpiWarps);
    }
    mbar_init(bar(B_DRAIN), 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) alloc_tmem<CG>(smem_u32(&tmem_slot));
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmw);
    tma_prefetch_desc(&tmr);
    tma_prefetch_desc(&tmo);
  }
  pdl_wait();
  if (p.counters && blockIdx.x == 0) clear_counters(p.counters, threadIdx.x, kRowsThreads);
  const int rb = p.row_block;
  const bool good = scan_groups<kRowsThreads>(p, start, first, [&](int n) { return (n + rb - 1) / rb; });
  fence_before_sync();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();   // the peer's barriers are there before anything arrives on them
  fence_after_sync();
  const uint32_t tmem = tmem_slot;

  Watchdog wd;
  wd.abort = &abort_word;
  wd.err = p.hdr + WS_ERR;
  wd.err_info = p.hdr + WS_ERR_INFO;
  wd.limit_ns = p.test_timeout ? 1000000ull : 2000000000ull;
  const int wide = 128 * CG, fblocks = (p.features + wide - 1) / wide, kblocks = (p.depth + 63) / 64;
  const bool resident = p.slots >= kblocks;   // B stays for all of a row block's tiles
  Tiles w(start, first, p.E, fblocks, rb, wide, blockIdx.x / CG, gridDim.x / CG, good);
  // columns of a product: the tile's rows in 16s, in 32s for a pair, whose CTAs hold half of them each
  auto columns = [&]() { return CG == 1 ? (w.rows + 15) & ~15 : (w.rows + 31) & ~31; };

  if (warp == kLoadWarp) {
    // ------------------------------------------------- A
    int stage = 0;
    uint32_t phase = 0, loads = 0;
    const uint32_t there = CG == 1 ? bar(B_AFULL) : in_cta(bar(B_AFULL), 0);   // the pair's barriers
    bool ok = true, withhold = p.test_timeout && rank == 0 && w.more() && w.begin == 0;
    for (; ok && w.more(); w.next()) {
      const int f = w.f0 + (int)rank * 128;
      for (int kb = 0; kb < kblocks; ++kb) {
        if (loads >= (uint32_t)p.stages) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_AEMPTY) + stage * 8, phase ^ 1, wd, 61)) != 0;
        if (!ok) break;
        ++loads;
        if (withhold) {   // test only: this copy never comes
          withhold = false;
        } else {
          const uint32_t dst = a_at + stage * kABytes, full = there + stage * 8;
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(B_AFULL) + stage * 8, CG * kABytes);
          __syncwarp();
          if (KMAJOR) {
            load_3d<CG == 2>(dst, &tmw, full, kb * 64, f, w.e);
          } else if (p.one_w) {
            load_3d<CG == 2>(dst, &tmw, full, 0, w.e * p.depth + kb * 64, f >> 6);
          } else {
            load_3d<CG == 2>(dst, &tmw, full, f, kb * 64, w.e);
            load_3d<CG == 2>(dst + kABytes / 2, &tmw, full, f + 64, kb * 64, w.e);
          }
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) tail<CG>(bar, B_AEMPTY, B_AFULL, p.stages, stage, phase, loads, rank, ok, wd, 67);
    __syncwarp();
  } else if (warp == kRowsWarp) {
    // ------------------------------------------------- B
    int slot = 0;
    uint32_t phase = 0, loads = 0;
    bool ok = true;
    const int ring = resident ? kblocks : p.slots;
    const uint32_t there = CG == 1 ? bar(B_BFULL) : in_cta(bar(B_BFULL), 0);
    for (; ok && w.more(); w.next()) {
      if (resident && !w.fresh()) continue;
      const int row = w.row0 + (int)rank * (columns() / CG);
      for (int kb = 0; kb < kblocks; ++kb) {
        if (loads >= (uint32_t)ring) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_BEMPTY) + slot * 8, phase ^ 1, wd, 65)) != 0;
        if (!ok) break;
        ++loads;
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(B_BFULL) + slot * 8, CG * slot_bytes);
        __syncwarp();
        load_2d<CG == 2>(b_at + slot * slot_bytes, &tmr, there + slot * 8, kb * 64, row);
        if (++slot == ring) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) tail<CG>(bar, B_BEMPTY, B_BFULL, ring, slot, phase, loads, rank, ok, wd, 68);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      int stage = 0, slot = 0;
      uint32_t phase = 0, slot_phase = 0, n = 0;
      const SDesc da0 = KMAJOR ? sdesc_w(a_at, 16, 1024) : sdesc_w(a_at, kABytes / 2, 1024), db0 = sdesc_w(b_at, 16, 1024);
      const int ring = resident ? kblocks : p.slots;
      auto wait = [&](uint32_t at, uint32_t parity, int site) { return __all_sync(0xffffffffu, mbar_wait(at, parity, wd, site)) != 0; };
      bool ok = true;
      for (; ok && w.more(); w.next()) {
        const uint32_t idesc = idesc_bf16(wide, columns(), !KMAJOR, false);
        const bool fresh = !resident || w.fresh(), release = !resident || w.last();
        // an accumulator after the other, each of at most kRun blocks of the depth
        for (int k0 = 0; ok && k0 < kblocks; k0 += DEEP ? kRun : kblocks, ++n) {
          const int end = DEEP ? min(kblocks, k0 + kRun) : kblocks;
          const uint32_t d = tmem + (n & 1) * 256;
          ok = wait(bar(B_DEMPTY) + (n & 1) * 8, ((n >> 1) & 1) ^ 1, 62);
          if (!ok) break;
          for (int kb = k0; kb < end; ++kb) {
            if (fresh) {
              ok = wait(bar(B_BFULL) + slot * 8, slot_phase, 66);
              if (!ok) break;
            }
            ok = wait(bar(B_AFULL) + stage * 8, phase, 63);
            if (!ok) break;
            fence_after_sync();
            const SDesc da = da0 + stage * kABytes, db = db0 + slot * slot_bytes;
            mma<CG>(d, da, db, idesc, kb > k0 ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < 4; ++kk) mma<CG>(d, da + (KMAJOR ? kk * 32 : kk * 2048), db + kk * 32, idesc, 1u);
            commit<CG>(bar(B_AEMPTY) + stage * 8);
            if (release) commit<CG>(bar(B_BEMPTY) + slot * 8);
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1;
            }
            if (++slot == ring) {
              slot = 0;
              if (release) slot_phase ^= 1;
            }
          }
          if (ok) commit<CG>(bar(B_DFULL) + (n & 1) * 8);
        }
      }
      __syncwarp();
      commit_here<CG>(bar(B_DRAIN));
      if (lane == 0) drain(bar(B_DRAIN), 0);
      __syncwarp();
    }
  } else {
    // a warp stores 32 features of 32 rows at a time, through its staging buffer [row][feature]
    const int wq = warp & 3, half = warp >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    constexpr int kBuf = 1024 * sizeof(TO);
    const uint32_t to = stg_at + warp * kBuf;
    const uint8_t* from = smem_raw + (to - raw_u32);
    TO* out = static_cast<TO*>(p.out);
    // where this lane's row of an 8 x 8 matrix goes: matrix l / 8 of 4 has features 8 (m % 2).. and rows 8 (m / 2)..
    const uint32_t lane_row = (lane >> 4) * 8 + (lane & 7), lane_chunk = (lane >> 3 & 1) ^ (lane >> 1 & 3);
    // 32 columns of an accumulator from c on.  FP32: lanes are features, a register a row.  BF16: 16 features x 32 rows
    // a load, whose registers are 8 x 8 matrices [feature][row].
    auto read16 = [&](uint32_t d, int c, int h, uint32_t (&v)[16]) {
      if constexpr (sizeof(TO) == 4) tmem_ld16(lane_base + d * 256 + c + 16 * h, v);
      else tmem_ld_16x256b_x4(lane_base + ((uint32_t)(16 * h) << 16) + d * 256 + c, v);
    };
    // stores the tile's rows from c on, 32 at most: v[h] is what read16 gives for h
    auto store = [&](int f, int c, const uint32_t (&v)[2][16]) {
      if (lane == 0) bulk_wait_read<0>();   // the buffer's last store has read it
      __syncwarp();
      if constexpr (sizeof(TO) == 4) {
        // a row at a time, 32 neighbouring words
#pragma unroll
        for (int r = 0; r < 32; ++r)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + r * 128 + lane * 4), "r"(v[r >> 4][r & 15]) : "memory");
      } else {
        // transposed, 16-byte chunk k of row r at k ^ (r / 2 % 4)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            uint32_t m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = 4 * (j + (k >> 1)) + 2 * (k & 1);
              m[k] = pack_bf16(__uint_as_float(v[h][at]), __uint_as_float(v[h][at + 1]));
            }
            stmatrix_trans(to + (lane_row + 8 * j) * 64 + ((lane_chunk ^ (2 * h)) << 4), m);
          }
      }
      const int live = w.rows - c;
      if (live >= 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (f < p.features) tma_store_2d(&tmo, to, f, w.row0 + c);
          bulk_commit();
        }
      } else {
        // the group's last rows: a tile store would go on into the next group's
        __syncwarp();
        constexpr int kChunks = 32 * sizeof(TO) / 16, kRows = 32 / kChunks;
        const int chunk = lane % kChunks, col = f + chunk * (16 / (int)sizeof(TO));
#pragma unroll
        for (int r = lane / kChunks; r < 32; r += kRows) {
          const int place = sizeof(TO) == 2 ? chunk ^ (r >> 1 & 3) : chunk;
          const uint4 x = *reinterpret_cast<const uint4*>(from + r * (32 * sizeof(TO)) + place * 16);
          if (r < live && col < p.features)
            *reinterpret_cast<uint4*>(out + (int64_t)(w.row0 + c + r) * p.out_stride + col) = x;
        }
        __syncwarp();
      }
    };
    auto release = [&](uint32_t d) {
      fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1) mbar_arrive(bar(B_DEMPTY + d));
        else arrive_in_cluster(in_cta(bar(B_DEMPTY + d), 0));
      }
    };
    uint32_t n = 0;
    bool ok = true;
    for (; ok && w.more(); w.next()) {
      const int f = w.f0 + (int)rank * 128 + wq * 32;
      if constexpr (!DEEP) {
        const uint32_t d = n & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_DFULL + d), (n >> 1) & 1, wd, 64)) != 0;
        if (!ok) break;
        fence_after_sync();
#pragma unroll 1
        for (int c = half * 32; c < w.rows; c += 64) {
          uint32_t v[2][16];
          read16(d, c, 0, v[0]);
          read16(d, c, 1, v[1]);
          tmem_wait_ld();
          store(f, c, v);
        }
        release(d);
        ++n;
      } else {
        float acc[4][2][16];   // columns 64 i + 32 half..
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[i][e >> 4][e & 15] = 0.f;
        for (int kb = 0; kb < kblocks; kb += kRun, ++n) {
          const uint32_t d = n & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(B_DFULL + d), (n >> 1) & 1, wd, 64)) != 0;
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = half * 32 + 64 * i;
            if (c < w.rows) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t v[16];
                read16(d, c, h, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][h][e] += __uint_as_float(v[e]);
              }
            }
          }
          release(d);
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = half * 32 + 64 * i;
          if (c < w.rows) {
            uint32_t v[2][16];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e >> 4][e & 15] = __float_as_uint(acc[i][e >> 4][e & 15]);
            store(f, c, v);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  fence_before_sync();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();   // nothing of the pair is under way in either CTA
  fence_after_sync();
  if (warp == kMmaWarp) free_tmem<CG>(tmem);
}

template <int CG, bool KMAJOR, bool DEEP, typename TO>
cudaError_t launch_t(GroupParams p, const void* rows, int64_t row_stride, const void* w, int K, int N, int sms,
                     cudaStream_t st) {
  CUtensorMap mw, mr, mo;
  p.box_rows = p.row_block / CG;
  // [features / 64][g K + k][64]: a stage's two boxes in one copy, where no box of k goes on into the next group's
  p.one_w = !KMAJOR && N % 64 == 0 && K % 64 == 0;
  const uint64_t wd1[3] = {64, (uint64_t)K * p.E, (uint64_t)N / 64}, ws1[2] = {(uint64_t)N * 2, 128};
  const uint32_t wbox1[3] = {64, 64, 2};
  const uint64_t wd[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)p.E}, ws[2] = {(uint64_t)N * 2, (uint64_t)N * K * 2};
  const uint32_t wbox[3] = {64, KMAJOR ? 128u : 64u, 1};
  const uint64_t rd[2] = {(uint64_t)p.depth, (uint64_t)p.rows}, rs[1] = {(uint64_t)row_stride * 2};
  const uint32_t rbox[2] = {64, (uint32_t)p.box_rows}, obox[2] = {32, 32};
  const uint64_t od[2] = {(uint64_t)p.features, (uint64_t)p.rows}, os[1] = {(uint64_t)p.out_stride * sizeof(TO)};
  if (!make_tmap_tile(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, w, p.one_w ? wd1 : wd, p.one_w ? ws1 : ws,
                      p.one_w ? wbox1 : wbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_tile(&mr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, rd, rs, rbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_tile(&mo, sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.out,
                      od, os, obox, sizeof(TO) == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  // B for the whole depth where that leaves three stages of A, else as many slots as stages
  const int64_t kblocks = (p.depth + 63) / 64;
  const size_t fixed = 1024 + staging_bytes(sizeof(TO)) + 8 * ((size_t)p.E + 1), slot = (size_t)p.row_block / CG * 128;
  const size_t room = kMaxDynamic - fixed;
  if (kblocks <= kSlotsMax && kblocks * slot + 3 * (size_t)kABytes <= room) {
    p.slots = (int)kblocks;
    p.stages = (int)((room - kblocks * slot) / kABytes);
  } else {
    p.stages = (int)(room / (kABytes + slot));
    if (p.stages >= kblocks) p.stages = (int)kblocks - 1;   // (fewer slots than k-blocks: a ring)
    if (p.stages > kSlotsMax) p.stages = kSlotsMax;
    p.slots = p.stages;
  }
  if (p.stages > kStagesMax) p.stages = kStagesMax;
  const size_t smem = fixed + p.stages * (size_t)kABytes + p.slots * slot;
  auto kern = group_rows_kernel<CG, KMAJOR, DEEP, TO>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDynamic);
  if (e != cudaSuccess) return e;
  const int64_t most = (p.rows / p.row_block + p.E) * (int64_t)((p.features + 128 * CG - 1) / (128 * CG));
  const unsigned grid = (unsigned)(most < sms / CG ? most : sms / CG) * CG;
  return launch_cluster<CG>(kern, grid, kRowsThreads, smem, st, p, mw, mr, mo);
}

template <bool KMAJOR, typename TO>
cudaError_t launch_shape(const GroupParams& p, const void* rows, int64_t row_stride, const void* w, int K, int N, int sms,
                         cudaStream_t st) {
  if (p.depth > 64 * kRun)
    return p.pair ? launch_t<2, KMAJOR, true, TO>(p, rows, row_stride, w, K, N, sms, st)
                  : launch_t<1, KMAJOR, true, TO>(p, rows, row_stride, w, K, N, sms, st);
  return p.pair ? launch_t<2, KMAJOR, false, TO>(p, rows, row_stride, w, K, N, sms, st)
                : launch_t<1, KMAJOR, false, TO>(p, rows, row_stride, w, K, N, sms, st);
}

hstu_status_t check_desc(const hstu_group_desc* d) {
  if (!d || d->struct_size != sizeof(hstu_group_desc) || d->reserved != 0 || (d->flags & ~HSTU_FLAG_TEST_TIMEOUT))
    return HSTU_ERR_INVALID_ARG;
  for (int t : {d->y_dtype, d->dx_dtype})
    if (t != HSTU_BF16 && t != HSTU_FP32) return HSTU_ERR_INVALID_ARG;
  if (d->groups < 1 || d->K < 1 || d->N < 1 || d->rows < 0) return HSTU_ERR_INVALID_ARG;
  if (d->groups > kMaxGroups || d->K % 8 || d->N % 8 || d->K > 65536 || d->N > 65536 || d->rows > (1 << 30))
    return HSTU_ERR_UNSUPPORTED;
  // tiles are counted in 32 bits
  const int64_t wide = (d->K > d->N ? d->K : d->N);
  if ((d->rows / 32 + d->groups) * ((wide + 127) / 128) > 0x7fffffff) return HSTU_ERR_UNSUPPORTED;
  if ((int64_t)((d->K + 127) / 128) * ((d->N + 255) / 256) * (d->rows / 64 + 2 * (int64_t)d->groups) > 0x7fffffff)
    return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// a stride of rows of 2-byte elements that tile loads take
bool stride_ok(int64_t stride, int width, int64_t rows) {
  return rows <= 1 || (stride >= width && stride % 8 == 0 && stride < ((int64_t)1 << 38));
}

hstu_status_t device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) return HSTU_OK;
  (void)cudaGetLastError();
  set_error_detail(e, "reading the number of SMs");
  return HSTU_ERR_CUDA;
}

size_t bwd_bytes(const hstu_group_desc* d) {
  return kWsHeaderBytes + group_dw_bytes(d->rows, d->groups, d->K, d->N);
}

// A tile's rows, and whether CTAs work in pairs.  What a choice costs: rounds of tiles over the
// CTAs, a tile taking for each 64 of the depth the longer of its products (2 cycles a row) and of
// its loads (128 bytes a row of A and B at 42 bytes a cycle, an SM's share of L2's 12 TB/s),
// and some 1,500 cycles at its ends.  Single CTAs against pairs, 512 -> 2,048: 8 x 8 rows 6.5 us against 8.0, 4 x 1,500
// 18.4 against 14.9, 16 x 1,000 37.6 against 32.7; dx of the same 13.9 against 15.5, 16.8 against 17.7 (taken), 46.5
// against 30.9; 256 -> 256, 8 x 12,500 rows 18.6 against 24.3.  It errs by 12% at 4 x 1,000 rows of 1,024 -> 1,024 (pairs
// 12.0, single 10.6) and at dx of 4 x 600 rows of 512 and 2,048 (16.5, 14.8).
void set_tile(GroupParams& p, int sms) {
  const int64_t kblocks = (p.depth + 63) / 64, groups = p.rows < p.E ? p.rows : p.E;
  int64_t best = -1;
  for (int cg = 1; cg <= 2; ++cg) {   // (pairs where they are ahead)
    if (cg == 2 && p.features <= 128) continue;
    for (int rb = 32 * cg; rb <= 256; rb *= 2) {   // (short tiles leave more stages to the weights)
      const int64_t tiles = (p.rows / rb + groups) * ((p.features + 128 * cg - 1) / (128 * cg));
      const int64_t rounds = (tiles + sms / cg - 1) / (sms / cg);
      const bool stays = kblocks <= kSlotsMax && kblocks * (rb / cg) <= 1024;   // B for the whole depth in 128 KB
      const int64_t loads = 3 * (128 + (stays ? 0 : rb / cg)), products = 2 * rb;
      const int64_t cost = rounds * (kblocks * (loads > products ? loads : products) + 1500);
      if (best < 0 || cost < best) {
        best = cost;
        p.row_block = rb;
        p.pair = cg == 2;
      }
    }
  }
}

}  // namespace

cudaError_t launch_group_rows(const GroupParams& p, bool transposed, int out_dtype, const void* rows, int64_t row_stride,
                              const void* w, int K, int N, int sms, cudaStream_t st) {
  if (transposed)
    return out_dtype == HSTU_BF16 ? launch_shape<true, __nv_bfloat16>(p, rows, row_stride, w, K, N, sms, st)
                                  : launch_shape<true, float>(p, rows, row_stride, w, K, N, sms, st);
  return out_dtype == HSTU_BF16 ? launch_shape<false, __nv_bfloat16>(p, rows, row_stride, w, K, N, sms, st)
                                : launch_shape<false, float>(p, rows, row_stride, w, K, N, sms, st);
}

}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_group_workspace_size(const hstu_group_desc* desc, size_t* fwd, size_t* bwd, size_t* zero) {
  const hstu_status_t s = check_desc(desc);
  if (s != HSTU_OK) return s;
  if (zero) *zero = kWsHeaderBytes + kDwCounterBytes;
  if (fwd) *fwd = kWsHeaderBytes;
  if (bwd) *bwd = bwd_bytes(desc);
  return HSTU_OK;
}

hstu_status_t hstu_group_fwd(const hstu_group_desc* d, const hstu_group_fwd_args* a, void* workspace, size_t workspace_bytes,
                             hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  if (s != HSTU_OK) return s;
  if (!a || !a->group_offsets || (d->rows > 0 && (!a->x || !a->w || !a->y))) return HSTU_ERR_INVALID_ARG;
  if (!aligned16(a->x) || !aligned16(a->w) || !aligned16(a->y) || !stride_ok(d->x_stride, d->K, d->rows) ||
      !stride_ok(d->y_stride, d->N, d->rows))
    return HSTU_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) || workspace_bytes < kWsHeaderBytes)
    return HSTU_ERR_WORKSPACE;
  reset_launches();
  if (d->rows == 0) return HSTU_OK;
  int sms = 0;
  if ((s = device_sms(&sms)) != HSTU_OK) return s;
  GroupParams p{};
  p.off = a->group_offsets; p.hdr = static_cast<int*>(workspace);
  p.rows = d->rows; p.E = d->groups; p.features = d->N; p.depth = d->K;
  p.out = a->y; p.out_stride = d->rows == 1 ? d->N : d->y_stride;
  p.test_timeout = (d->flags & HSTU_FLAG_TEST_TIMEOUT) ? 1 : 0;
  set_tile(p, sms);
  const int64_t xs = d->rows == 1 ? d->K : d->x_stride;
  const cudaError_t e = launch_group_rows(p, false, d->y_dtype, a->x, xs, a->w, d->K, d->N, sms,
                                          reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_error_detail(e, "launching group_rows_kernel");
    return HSTU_ERR_CUDA;
  }
  note_launches(1);
  return HSTU_OK;
}

hstu_status_t hstu_group_bwd(const hstu_group_desc* d, const hstu_group_bwd_args* a, void* workspace, size_t workspace_bytes,
                             hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  if (s != HSTU_OK) return s;
  if (d->flags) return HSTU_ERR_UNSUPPORTED;   // the test mode is of the forward
  if (!a || !a->group_offsets || (!a->dx && !a->dw)) return HSTU_ERR_INVALID_ARG;
  if (d->rows > 0 && (!a->dy || (a->dx && !a->w) || (a->dw && !a->x))) return HSTU_ERR_INVALID_ARG;
  for (const void* ptr : {a->x, a->w, a->dy, (const void*)a->dx, (const void*)a->dw})
    if (!aligned16(ptr)) return HSTU_ERR_INVALID_ARG;
  if (!stride_ok(d->y_stride, d->N, d->rows) || (a->dw && !stride_ok(d->x_stride, d->K, d->rows)) ||
      (a->dx && !stride_ok(d->dx_stride, d->K, d->rows)))
    return HSTU_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) || workspace_bytes < bwd_bytes(d))
    return HSTU_ERR_WORKSPACE;
  reset_launches();
  int sms = 0;
  if ((s = device_sms(&sms)) != HSTU_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  GroupParams p{};
  p.off = a->group_offsets; p.hdr = static_cast<int*>(workspace);
  p.rows = d->rows; p.E = d->groups;
  const int64_t ys = d->rows <= 1 ? d->N : d->y_stride, xs = d->rows <= 1 ? d->K : d->x_stride;
  cudaError_t e = cudaSuccess;
  int launches = 0;
  if (a->dw && d->rows > 0) p.counters = reinterpret_cast<int*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  if (a->dx && d->rows > 0) {
    p.features = d->K; p.depth = d->N;
    p.out = a->dx; p.out_stride = d->rows == 1 ? d->K : d->dx_stride;
    set_tile(p, sms);
    e = launch_group_rows(p, true, d->dx_dtype, a->dy, ys, a->w, d->K, d->N, sms, st);
    launches = 1;
  }
  if (e == cudaSuccess && a->dw) {
    if (d->rows == 0) {
      e = cudaMemsetAsync(a->dw, 0, sizeof(float) * (size_t)d->groups * d->K * d->N, st);
    } else {
      p.dw = a->dw;
      if (!a->dx) {
        e = launch_group_dw_clear(p.counters, st);
        ++launches;
      }
      if (e == cudaSuccess) e = launch_group_dw(p, a->x, xs, a->dy, ys, d->K, d->N, sms, st);
      ++launches;
    }
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_error_detail(e, "launching the group gradients' kernels");
    return HSTU_ERR_CUDA;
  }
  note_launches(launches);
  return HSTU_OK;
}

}  // extern "C"
