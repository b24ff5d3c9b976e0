// Weight gradients of ragged groups: dW[g] = sum over the group's rows r of
// x[r]^T dy[r] (the dw of hstu_group_bwd).
//
// Tiles of a dW[g] of 128 features of x a CTA by 256 of dy, summed over the group's rows in
// 64s: both operands are read with features contiguous (MN-major).  CTAs work in pairs (cta_group::2,
// 256 x 256; each holds half of both operands) where there is work for all of them: for large batches single CTAs
// come to the 12 TB/s at which the SMs read L2 (161,293 rows, 512 x 2048: 308 us against 248).
//
// What bounds a pair is its loads from L2: a stage (4 products of 128 tensor-core cycles) is 32 KB a CTA, 780 cycles at an SM's
// share (42 bytes a cycle).  161,293 rows are 531 blocks a pair: 230 us at 1.8 GHz by that, 231-250 measured (by the
// clock: the board is at its power limit then); cuBLAS's product of one group of that size 200-211 us.  For that, what the
// loading and issuing warps do for a stage has to be less: a copy an operand where the width is a multiple of 64 (a 3-D map,
// 64 features innermost), both warps run their loops as one with an elected lane (uniform operands); 293 us with a copy for
// each 64 features and single threads.  Stages: 267 us with 4, 248 with 5, 246 with 6.  Two pairs side by side that share
// x by multicast were no faster (252 us), which was tried before the loops were made uniform.
//
// Rows of the next group (or past the end) in a group's last 64 are cleared in shared memory
// before the tensor core reads them, in both operands, since 0 x infinity is no zero.  Such a block
// counts on each CTA's own barrier, is cleared by its MMA warp, and taken when both CTAs are through.
//
// Precision: the tensor core's sums lose a little at every addition, always towards zero.  The
// accumulator so is read after 16 blocks (1,024 rows) and added up in registers (128 a thread), while
// the second accumulator takes the next 16: 2.5e-6 of dW at 6,415 rows in one accumulator, 0.9e-6 so, against 0.6e-6 of a
// plain FP32 product.
//
// Groups of many rows are cut into pieces of about equal length, so that one large group fills
// the GPU as many small ones do; pieces are dealt out longest first, back and forth.  A
// piece that is a whole tile is stored; of others each storing warp leaves its sums in the workspace, and the warp
// that comes last (a counter) adds up all of them, in the order of the pieces: equal inputs give equal bits.  (A second
// kernel for that took 11 us of 58 with a heavy-tailed batch.)  A group without rows gets zeros.  The counters lie at the
// same place for every shape and are cleared by the call (by dx's kernel, or by one of its own), so that a workspace
// may have served other shapes and operators before.
//
// Roles as in hstu_group_rows.cu (one warp loads both operands).
#include "hstu_group.cuh"

namespace hstu {

namespace {

using namespace grp;

constexpr int kStagesMax = 8;
constexpr int kBox = 64 * 64 * 2;                 // 64 rows x 64 features
constexpr int kStaging = kEpiWarps * 4096;        // a 32 x 32 FP32 buffer of each storing warp
constexpr int kRanked = kThreads;                 // groups up to which they are sorted by the length of their pieces
enum : int { B_FULL = 0, B_EMPTY = B_FULL + kStagesMax, B_DFULL = B_EMPTY + kStagesMax, B_DEMPTY = B_DFULL + 2,
             B_CLEAR = B_DEMPTY + 2, B_DRAIN = B_CLEAR + kStagesMax, B_COUNT };

template <int CG> constexpr int boxes_of() { return CG == 1 ? 6 : 4; }   // of a stage: 2 of x, the others of dy

// pieces of a group of n rows
__device__ __forceinline__ int pieces(int n, int kper) {
  const int blocks = (n + 63) / 64;
  return blocks <= kper ? 1 : (blocks + kper - 1) / kper;
}

// The lists of a call: in the order of work, order[i] the group and start[i] the pieces before it; first[e] as ever.
struct Lists {
  int* start;
  int* first;
  int* order;
};
__device__ __forceinline__ Lists lists_at(void* at, int E) {
  int* p = static_cast<int*>(at);
  return Lists{p, p + E + 1, p + 2 * (E + 1)};
}
constexpr size_t lists_bytes(int E) { return 4 * 3 * ((size_t)E + 1); }

__device__ __forceinline__ bool make_lists(const GroupParams& p, const Lists& l) {
  if (!scan_groups<kThreads>(p, l.start, l.first, [&](int n) { return pieces(n, p.kper); })) return false;
  const int tid = threadIdx.x;
  if (p.E <= kRanked) {
    // longest pieces first
    int np = 1, mine = 0;
    if (tid < p.E) {
      np = l.start[tid + 1] - l.start[tid];
      mine = (l.first[tid + 1] - l.first[tid]) / np;
      l.order[tid] = mine;
    }
    __syncthreads();
    int rank = 0, before = 0;
    if (tid < p.E) {
#pragma unroll 4
      for (int e = 0; e < p.E; ++e) {
        const int other = l.order[e], others = l.start[e + 1] - l.start[e];
        const bool ahead = other > mine || (other == mine && e < tid);
        rank += ahead ? 1 : 0;
        before += ahead ? others : 0;
      }
    }
    __syncthreads();
    if (tid < p.E) {
      l.order[rank] = tid;
      l.start[rank] = before;   // start[E] stays
    }
  } else {
    for (int e = tid; e < p.E; e += kThreads) l.order[e] = e;
  }
  __syncthreads();
  return true;
}

// A CTA's (a pair's) share of the work, piece after piece, tiles fastest (neighbours share their rows): items
// q, 2 P - 1 - q, 2 P + q, .. of P shares.
struct Pieces {
  Lists l;
  int tpg, nt, wide, at_group, e, total, share, shares, k, t, slots, splits;   // slots, cut tiles before at_group
  int k0, n0, row0, rows, blocks;
  int np, piece, slot, split;   // np > 1: the tile's first slot and its place among cut tiles
  __device__ __forceinline__ Pieces(const Lists& l_, const GroupParams& p, int width, int share_, int shares_, bool good)
      : l(l_), tpg(p.kt * p.nt), nt(p.nt), wide(width), at_group(0), e(0), total(good ? l_.start[p.E] * p.kt * p.nt : 0),
        share(share_), shares(shares_), k(0), t(share_), slots(0), splits(0) {}
  __device__ __forceinline__ bool more() {
    if (t >= total) return false;
    while (l.start[at_group + 1] * tpg <= t) {
      const int n = l.start[at_group + 1] - l.start[at_group];
      slots += n > 1 ? n * tpg : 0;
      splits += n > 1 ? tpg : 0;
      ++at_group;
    }
    e = l.order[at_group];
    np = l.start[at_group + 1] - l.start[at_group];
    const int in = t - l.start[at_group] * tpg;
    piece = in / tpg;
    const int tile = in - piece * tpg;
    const int n = l.first[e + 1] - l.first[e], all = (n + 63) / 64;
    // pieces as even as whole blocks allow
    const int b0 = (int)((int64_t)all * piece / np), b1 = (int)((int64_t)all * (piece + 1) / np);
    k0 = tile / nt * wide;
    n0 = tile % nt * 256;
    row0 = l.first[e] + b0 * 64;
    blocks = b1 - b0;
    rows = min(n - b0 * 64, blocks * 64);
    slot = slots + tile * np;
    split = splits + tile;
    return true;
  }
  __device__ __forceinline__ void next() {
    ++k;
    t = k * shares + (k & 1 ? shares - 1 - share : share);
  }
};

// 16-byte chunk c of row r of a 32 x 32 FP32 buffer lies at chunk c ^ (r % 8)
__device__ __forceinline__ void stage_f32(uint8_t* buf, int lane, const float* a) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_float4(a[4 * c], a[4 * c + 1], a[4 * c + 2], a[4 * c + 3]);
}

// CG: CTAs that work together
template <int CG>
__global__ void __launch_bounds__(kThreads, 1)
group_dw_kernel(const __grid_constant__ GroupParams p, const __grid_constant__ CUtensorMap tmx,
                const __grid_constant__ CUtensorMap tmg, const __grid_constant__ CUtensorMap tmo) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B_COUNT];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  constexpr int BOXES = boxes_of<CG>(), kStage = BOXES * kBox;
  const uint32_t raw_u32 = smem_u32(smem_raw), base = (raw_u32 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_u32);
  uint8_t* staging = smem + p.stages * kStage;
  const Lists lists = lists_at(staging + kStaging, p.E);
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars) + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0u : cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStagesMax; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_DFULL + s), 1);
      mbar_init(bar(B_DEMPTY + s), CG * kEpiWarps);
    }
    for (int s = 0; s < kStagesMax; ++s) mbar_init(bar(B_CLEAR + s), 1);
    mbar_init(bar(B_DRAIN), 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) alloc_tmem<CG>(smem_u32(&tmem_slot));
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmx);
    tma_prefetch_desc(&tmg);
    tma_prefetch_desc(&tmo);
  }
  pdl_wait();
  const bool good = make_lists(p, lists);
  fence_before_sync();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;

  Watchdog wd;
  wd.abort = &abort_word;
  wd.err = p.hdr + WS_ERR;
  wd.err_info = p.hdr + WS_ERR_INFO;
  wd.limit_ns = 2000000000ull;
  Pieces w(lists, p, 128 * CG, blockIdx.x / CG, gridDim.x / CG, good);

  if (warp == kLoadWarp) {
    int stage = 0;
    uint32_t phase = 0, loads = 0;
    bool ok = true;
    const uint32_t there = CG == 1 ? bar(B_FULL) : in_cta(bar(B_FULL), 0);   // the pair's barriers
    auto copies = [&](uint32_t dst, const CUtensorMap* map, int boxes, bool one, uint32_t full, bool here, int x, int row) {
      if (one) {
        if (CG == 1 || here) load_3d<false>(dst, map, full, 0, row, x >> 6);
        else load_3d<true>(dst, map, full, 0, row, x >> 6);
      } else {
#pragma unroll
        for (int c = 0; c < boxes; ++c) {
          if (CG == 1 || here) load_2d<false>(dst + c * kBox, map, full, x + c * 64, row);
          else load_2d<true>(dst + c * kBox, map, full, x + c * 64, row);
        }
      }
    };
    for (; ok && w.more(); w.next()) {
      const int k0 = w.k0 + (int)rank * 128, n0 = w.n0 + (int)rank * 128;
      int row = w.row0;
      for (int left = w.rows; left > 0; left -= 64, row += 64) {
        if (loads >= (uint32_t)p.stages) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_EMPTY) + stage * 8, phase ^ 1, wd, 71)) != 0;
        if (!ok) break;
        ++loads;
        const uint32_t s = base + stage * kStage, mine = bar(B_FULL) + stage * 8;
        const bool cut = CG == 2 && left < 64;   // the group ends inside: each CTA's copies count on its own barrier
        const uint32_t full = cut ? mine : there + 8u * (uint32_t)stage;
        if (lane == 0 && (cut || rank == 0)) mbar_arrive_expect_tx(mine, cut || CG == 1 ? kStage : 2 * kStage);
        __syncwarp();
        copies(s, &tmx, 2, p.one_x, full, cut, k0, row);
        copies(s + 2 * kBox, &tmg, BOXES - 2, p.one_dy, full, cut, n0, row);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) tail<CG>(bar, B_EMPTY, B_FULL, p.stages, stage, phase, loads, rank, ok, wd, 75);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t IDESC = idesc_bf16(128 * CG, 256, true, true);
    int stage = 0;
    uint32_t phase = 0, n = 0, cuts = 0;
    bool ok = true;
    auto wait = [&](uint32_t at, uint32_t parity, int site) { return __all_sync(0xffffffffu, mbar_wait(at, parity, wd, site)) != 0; };
    const SDesc da0 = sdesc_w(base, kBox, 1024), db0 = sdesc_w(base + 2 * kBox, kBox, 1024);
    // a block's products and their arrivals
    auto products = [&](uint32_t first, bool last) {
      fence_after_sync();
      const uint32_t d = tmem + (n & 1) * 256;
      const SDesc da = da0 + stage * kStage, db = db0 + stage * kStage;
      mma<CG>(d, da, db, IDESC, first ? 0u : 1u);
#pragma unroll
      for (int kk = 1; kk < 4; ++kk) mma<CG>(d, da + kk * 2048, db + kk * 2048, IDESC, 1u);
      commit<CG>(bar(B_EMPTY) + stage * 8);
      if (last) commit<CG>(bar(B_DFULL) + (n & 1) * 8);
    };
    auto next = [&]() {
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    };
    for (; ok && w.more(); w.next()) {
      const int whole = w.rows >> 6;
      if (rank == 0) {
        for (int kb = 0; kb < whole; ++kb) {
          const bool first = kb % kRun == 0, last = kb % kRun == kRun - 1 || kb == w.blocks - 1;
          if (first) ok = wait(bar(B_DEMPTY) + (n & 1) * 8, ((n >> 1) & 1) ^ 1, 72);
          if (ok) ok = wait(bar(B_FULL) + stage * 8, phase, 73);
          if (!ok) break;
          products(first, last);
          n += last ? 1u : 0u;
          next();
        }
      } else {
        phase ^= (uint32_t)((stage + whole) / p.stages) & 1u;
        stage = (stage + whole) % p.stages;
      }
      if (!ok) break;
      if (whole == w.blocks) continue;
      // a block in which the group ends
      const bool first = whole % kRun == 0;
      if (rank == 0 && first) ok = wait(bar(B_DEMPTY) + (n & 1) * 8, ((n >> 1) & 1) ^ 1, 72);
      // (the second CTA's barriers have no other phases than those of such blocks)
      if (ok) ok = wait(bar(B_FULL) + stage * 8, rank == 0 ? phase : cuts >> stage & 1, 73);
      if (!ok) break;
      // rows of the next group: cleared (a row is 128 bytes of each box, whatever the swizzle)
      uint8_t* s = smem + stage * kStage;
      for (int c = 0; c < BOXES; ++c)
        for (int i = (w.rows & 63) * 8 + lane; i < 64 * 8; i += 32)
          *reinterpret_cast<uint4*>(s + c * kBox + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      if (CG == 2 && rank != 0 && lane == 0) arrive_in_cluster(in_cta(bar(B_CLEAR + stage), 0));
      if (CG == 2 && rank == 0) ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar(B_CLEAR + stage), cuts >> stage & 1, wd, 77));
      if (!ok) break;
      cuts ^= 1u << stage;
      if (rank == 0) products(first, true);
      ++n;
      next();
    }
    if (rank == 0) {
      __syncwarp();
      commit_here<CG>(bar(B_DRAIN));
      if (lane == 0) drain(bar(B_DRAIN), 0);
    }
    __syncwarp();
  } else {
    const int wq = warp & 3, half = warp >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16) + half * 128;
    uint8_t* stg = staging + warp * 4096;
    const uint32_t stg_u32 = smem_u32(stg);
    uint32_t n = 0;
    bool ok = true;
    for (; ok && w.more(); w.next()) {
      float acc[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c][i] = 0.f;
      for (int kb = 0; kb < w.blocks; kb += kRun, ++n) {
        const uint32_t d = n & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_DFULL + d), (n >> 1) & 1, wd, 74));
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t v[16];
          tmem_ld16(lane_base + d * 256 + c * 16, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c / 2][c % 2 * 16 + i] += __uint_as_float(v[i]);
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) mbar_arrive(bar(B_DEMPTY + d));
          else arrive_in_cluster(in_cta(bar(B_DEMPTY + d), 0));
        }
      }
      if (!ok) break;
      if (w.np > 1) {
        // this warp's 32 x 128 of a tile's pieces lie side by side, a float4 a lane
        constexpr size_t kPart = 32 * 128;
        const size_t per = kPart * kEpiWarps * CG;
        float4* parts = reinterpret_cast<float4*>(p.partial + (size_t)w.slot * per +
                                                  ((size_t)rank * kEpiWarps + warp) * kPart) + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            parts[(size_t)w.piece * (per / 4) + (c * 8 + q) * 32] =
                make_float4(acc[c][4 * q], acc[c][4 * q + 1], acc[c][4 * q + 2], acc[c][4 * q + 3]);
        __threadfence();
        __syncwarp();
        int* counter = p.counters + ((size_t)w.split * CG + rank) * kEpiWarps + warp;
        int there = 0;
        if (lane == 0) there = atomicAdd(counter, 1);
        there = __shfl_sync(0xffffffffu, there, 0);
        if (there != w.np - 1) continue;
        __threadfence();
        // in the order of the pieces; a warp's own sums stay where they are if they are the first or second
        const bool keeps = w.piece <= 1;
        if (!keeps) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int q = 0; q < 32; ++q) acc[c][q] = 0.f;
        }
#pragma unroll 1
        for (int k = 0; k < w.np; ++k) {
          if (keeps && k == w.piece) continue;
          const float4* part = parts + (size_t)k * (per / 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = __ldcg(part + (c * 8 + q) * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              float* a = &acc[c][4 * q];
              a[0] += v[q].x;
              a[1] += v[q].y;
              a[2] += v[q].z;
              a[3] += v[q].w;
            }
          }
        }
      }
      const int k0 = w.k0 + (int)rank * 128 + wq * 32, n0 = w.n0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = half * 128 + c * 32;
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        stage_f32(stg, lane, acc[c]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (n0 + col < p.features && k0 < p.depth) tma_store_3d(&tmo, stg_u32, n0 + col, k0, w.e);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  fence_before_sync();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();
  fence_after_sync();
  if (warp == kMmaWarp) free_tmem<CG>(tmem);
}

// The shape of a call on a whole GB300 (its SMs set the size of the workspace).
constexpr int64_t kSms = 152;
struct DwShape {
  int cg, kt, nt, kper;   // tiles of 128 cg x 256
  int64_t slots;                 // of as many sums
};
DwShape dw_shape(int64_t rows, int E, int K, int N) {
  DwShape s;
  const int64_t blocks = rows / 64 + (rows < E ? rows : E);   // of all groups, at most
  const int nt = (N + 255) / 256;
  // pairs where each has 46 blocks of a tile's rows to do, and K does not leave many of their tiles half empty.  Groups of
  // equal size, single CTAs against pairs: 4 x 600 rows of 512 and 2,048 11.6 us against 13.0, 4 x 3,000 36.3 against 37.8 (40
  // blocks a pair), 4 x 4,000 43.7 against 41.5 (53); of 512 and 512: 4 x 10,000 34.0 against 36.5 (33), 4 x 15,000 44.8
  // against 43.5 (50), 4 x 30,000 98 against 91
  const int halves = (K + 127) / 128, pairs = (halves + 1) / 2;
  s.cg = blocks * pairs * nt >= kSms / 2 * 46 && (halves % 2 == 0 || halves >= 5) ? 2 : 1;
  s.nt = nt;
  s.kt = (K + 128 * s.cg - 1) / (128 * s.cg);
  // A piece: what a CTA (a pair) has to do on average, and not so little that adding up the pieces (2 to 3 us each, one
  // after the other) takes longer than they do (0.6 us a block): at least 2 sqrt(blocks); of one group, whose pieces are all alike, the
  // length of two rounds at most that ends first, a cut tile's sums counted as 8 blocks (written, read)
  const int64_t tiles = (int64_t)s.kt * s.nt, shares = kSms / s.cg, all = (rows + 63) / 64, each = (all * tiles + shares - 1) / shares;
  int64_t least = 8;
  while (least * least < 4 * all) ++least;
  int64_t kper = each < least ? least : each;
  if (E == 1) {
    int64_t best = -1;
    for (int64_t np = 1; np * tiles <= 2 * shares && np <= all; ++np) {
      const int64_t len = (all + np - 1) / np, cost = (np * tiles + shares - 1) / shares * (len + (np > 1 ? 8 : 0));
      if (len >= least && (best < 0 || cost < best)) {
        best = cost;
        kper = len;
      }
    }
  }
  s.kper = (int)kper;
  // a group of b > kper blocks has at most (b + kper - 1) / kper < 2 b / kper pieces a tile; such groups have more than
  // 64 kper rows, so there are fewer than all / kper of them, and fewer than all tiles / kper <= shares cut tiles (of one
  // group at most tiles, where np >= 2: no more than shares)
  s.slots = all <= kper ? 0 : 2 * (blocks / kper + 1) * tiles;
  return s;
}

template <int CG>
cudaError_t launch_t(GroupParams p, const void* x, int64_t x_stride, const void* dy, int64_t dy_stride, int sms,
                     cudaStream_t st) {
  const int K = p.depth, N = p.features;
  CUtensorMap mx, mg, mo;
  const uint64_t xd[2] = {(uint64_t)K, (uint64_t)p.rows}, xs[1] = {(uint64_t)x_stride * 2};
  const uint64_t gd[2] = {(uint64_t)N, (uint64_t)p.rows}, gs[1] = {(uint64_t)dy_stride * 2};
  const uint64_t od[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)p.E}, os[2] = {(uint64_t)N * 4, (uint64_t)N * K * 4};
  const uint32_t ibox[2] = {64, 64}, obox[3] = {32, 32, 1};
  // [features / 64][rows][64]: a stage's boxes side by side in one copy
  p.one_x = K % 64 == 0;
  p.one_dy = N % 64 == 0;
  const uint64_t xd3[3] = {64, (uint64_t)p.rows, (uint64_t)K / 64}, xs3[2] = {(uint64_t)x_stride * 2, 128};
  const uint64_t gd3[3] = {64, (uint64_t)p.rows, (uint64_t)N / 64}, gs3[2] = {(uint64_t)dy_stride * 2, 128};
  const uint32_t xbox[3] = {64, 64, 2}, gbox[3] = {64, 64, boxes_of<CG>() - 2};
  auto side = [](CUtensorMap* m, bool one, const void* at, const uint64_t* d2, const uint64_t* s2, const uint32_t* b2,
                 const uint64_t* d3, const uint64_t* s3, const uint32_t* b3) {
    return one ? make_tmap_tile(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, at, d3, s3, b3, CU_TENSOR_MAP_SWIZZLE_128B)
               : make_tmap_tile(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, at, d2, s2, b2, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!side(&mx, p.one_x, x, xd, xs, ibox, xd3, xs3, xbox) || !side(&mg, p.one_dy, dy, gd, gs, ibox, gd3, gs3, gbox) ||
      !make_tmap_tile(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p.dw, od, os, obox, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const size_t fixed = 1024 + kStaging + lists_bytes(p.E), stage = (size_t)boxes_of<CG>() * kBox;
  p.stages = (int)((kMaxDynamic - fixed) / stage);
  if (p.stages > kStagesMax) p.stages = kStagesMax;
  const size_t smem = fixed + p.stages * stage;
  auto kern = group_dw_kernel<CG>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDynamic);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)p.kt * p.nt * (p.E + p.rows / 64 / p.kper + 1);
  const unsigned grid = (unsigned)(most < sms / CG ? most : sms / CG) * CG;
  return launch_cluster<CG>(kern, grid, kThreads, smem, st, p, mx, mg, mo);
}

}  // namespace

// counters, a warp of a cut tile each (at most kSms / cg cut tiles of cg CTAs), then the slots
static_assert(kSms * kEpiWarps <= kDwCounters && kDwCounterBytes % kWsAlign == 0, "counters of cut tiles");
size_t group_dw_bytes(int64_t rows, int E, int K, int N) {
  const DwShape s = dw_shape(rows, E, K, N);
  return kDwCounterBytes + (size_t)s.slots * 128 * s.cg * 256 * sizeof(float);
}

__global__ void __launch_bounds__(256) group_clear_kernel(int* counters) {
  pdl_wait();
  clear_counters(counters, threadIdx.x, 256);
}

cudaError_t launch_group_dw_clear(int* counters, cudaStream_t st) {
  return launch_pdl(group_clear_kernel, dim3(1), dim3(256), 0, st, counters);
}

cudaError_t launch_group_dw(const GroupParams& q, const void* x, int64_t x_stride, const void* dy, int64_t dy_stride, int K,
                            int N, int sms, cudaStream_t st) {
  const DwShape s = dw_shape(q.rows, q.E, K, N);
  GroupParams p = q;
  p.features = N; p.depth = K;
  p.kt = s.kt; p.nt = s.nt; p.kper = s.kper;
  p.partial = reinterpret_cast<float*>(reinterpret_cast<char*>(q.counters) + kDwCounterBytes);
  return s.cg == 2 ? launch_t<2>(p, x, x_stride, dy, dy_stride, sms, st) : launch_t<1>(p, x, x_stride, dy, dy_stride, sms, st);
}

}  // namespace hstu
