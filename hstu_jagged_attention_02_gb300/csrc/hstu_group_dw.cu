// Weight gradients of ragged groups: dW[g] = sum over the group's rows r of
// x[r]^T dy[r] (the dw of hstu_group_bwd).
//
// Tiles of 128 (K) x 256 (N) of a dW[g], summed over the group's rows in 64s: both
// operands are read with features contiguous (MN-major).  Rows of the next group (or
// past the end) in a group's last 64 are cleared in shared memory before the tensor core
// reads them, in both operands, since 0 x infinity is no zero.
//
// Groups of many rows are cut into pieces of about equal length, so that one large group fills
// the GPU as many small ones do.  A piece that is a whole tile is stored; others leave
// their sums in the workspace, which a second kernel adds up in the order of the pieces:
// equal inputs give equal bits.  A group without rows gets zeros.
//
// Roles as in hstu_group_rows.cu.
#include "hstu_group.cuh"

namespace hstu {

namespace {

using namespace grp;

constexpr int kStagesMax = 3;
constexpr int kBox = 64 * 64 * 2;                 // 64 rows x 64 features
constexpr int kABytes = 2 * kBox, kBBytes = 4 * kBox, kStage = kABytes + kBBytes;
constexpr int kStaging = kEpiWarps * 2 * 4096;    // two 32 x 32 FP32 buffers a storing warp
constexpr int kTile = 128 * 256;
enum : int { B_FULL = 0, B_EMPTY = B_FULL + kStagesMax, B_AFULL = B_EMPTY + kStagesMax, B_AEMPTY = B_AFULL + 2,
             B_DRAIN = B_AEMPTY + 2, B_COUNT };

// pieces of a group of n rows
__device__ __forceinline__ int pieces(int n, int kper) {
  const int blocks = (n + 63) / 64;
  return blocks <= kper ? 1 : (blocks + kper - 1) / kper;
}

// The work blockIdx.x, blockIdx.x + gridDim.x, ..: group, piece, tile (in this order, tiles fastest, so that
// neighbours share their rows), and the slots of partial sums below the group.
struct Pieces {
  const int* start;
  const int* first;
  int tpg, nt, kper, e, t, slots;
  int k0, n0, row0, rows, blocks, slot;   // slot < 0: stored whole
  __device__ __forceinline__ Pieces(const int* start_, const int* first_, int kt_, int nt_, int kper_)
      : start(start_), first(first_), tpg(kt_ * nt_), nt(nt_), kper(kper_), e(0), t(blockIdx.x), slots(0) {}
  __device__ __forceinline__ bool at(int total) {
    if (t >= total) return false;
    while (start[e + 1] * tpg <= t) {
      const int np = start[e + 1] - start[e];
      slots += np > 1 ? np * tpg : 0;
      ++e;
    }
    const int np = start[e + 1] - start[e], in = t - start[e] * tpg, piece = in / tpg, tile = in - piece * tpg;
    const int n = first[e + 1] - first[e], all = (n + 63) / 64;
    // pieces as even as whole blocks allow
    const int b0 = (int)((int64_t)all * piece / np), b1 = (int)((int64_t)all * (piece + 1) / np);
    k0 = tile / nt * 128;
    n0 = tile % nt * 256;
    row0 = first[e] + b0 * 64;
    blocks = b1 - b0;
    rows = min(n - b0 * 64, blocks * 64);
    slot = np > 1 ? slots + tile * np + piece : -1;
    return true;
  }
  __device__ __forceinline__ void next() { t += gridDim.x; }
};

// 16-byte chunk c of row r of a 32 x 32 FP32 buffer lies at chunk c ^ (r % 8)
__device__ __forceinline__ void stage_f32(uint8_t* buf, int lane, const uint32_t (&a)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(a[4 * c], a[4 * c + 1], a[4 * c + 2], a[4 * c + 3]);
}

__global__ void __launch_bounds__(kThreads, 1)
group_dw_kernel(const __grid_constant__ GroupParams p, const __grid_constant__ CUtensorMap tmx,
                const __grid_constant__ CUtensorMap tmg, const __grid_constant__ CUtensorMap tmo,
                const __grid_constant__ CUtensorMap tmp) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B_COUNT];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t raw_u32 = smem_u32(smem_raw), base = (raw_u32 + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_u32);
  uint8_t* staging = smem + p.stages * kStage;
  int* start = reinterpret_cast<int*>(staging + kStaging);
  int* first = start + p.E + 1;
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars) + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_AFULL + s), 1);
      mbar_init(bar(B_AEMPTY + s), kEpiWarps);
    }
    mbar_init(bar(B_DRAIN), 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmx);
    tma_prefetch_desc(&tmg);
  }
  pdl_wait();
  const bool good = scan_groups<kThreads>(p, start, first, [&](int n) { return pieces(n, p.kper); });
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;

  Watchdog wd;
  wd.abort = &abort_word;
  wd.err = p.hdr + WS_ERR;
  wd.err_info = p.hdr + WS_ERR_INFO;
  wd.limit_ns = 2000000000ull;
  const int total = good ? start[p.E] * p.kt * p.nt : 0;
  Pieces w(start, first, p.kt, p.nt, p.kper);

  if (warp == kLoadWarp) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, used = 0;
      uint32_t last[kStagesMax];
      bool ok = true;
      for (; ok && w.at(total); w.next()) {
        for (int kb = 0; kb < w.blocks; ++kb) {
          ok = mbar_wait(bar(B_EMPTY + stage), phase ^ 1, wd, 71);
          if (!ok) break;
          const uint32_t sA = base + stage * kStage, sB = sA + kABytes, full = bar(B_FULL + stage);
          mbar_arrive_expect_tx(full, kStage);
          const int row = w.row0 + kb * 64;
          for (int c = 0; c < 2; ++c) tma_load_2d(sA + c * kBox, &tmx, full, w.k0 + c * 64, row);
          for (int c = 0; c < 4; ++c) tma_load_2d(sB + c * kBox, &tmg, full, w.n0 + c * 64, row);
          used |= 1u << stage;
#pragma unroll
          for (int s = 0; s < kStagesMax; ++s)
            if (s == stage) last[s] = phase;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
#pragma unroll
      for (int s = 0; s < kStagesMax; ++s)
        if (used >> s & 1) drain(bar(B_FULL + s), last[s]);
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t IDESC = idesc_bf16(128, 256, true, true);
    int stage = 0;
    uint32_t phase = 0, n = 0;
    bool ok = true;
    for (; ok && w.at(total); w.next()) {
      if (w.blocks == 0) continue;
      const uint32_t ab = n & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(B_AEMPTY + ab), ((n >> 1) & 1) ^ 1, wd, 72));
      if (!ok) break;
      fence_after_sync();
      for (int kb = 0; kb < w.blocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_FULL + stage), phase, wd, 73));
        if (!ok) break;
        const int live = w.rows - kb * 64;
        if (live < 64) {   // rows of the next group: cleared (a row is 128 bytes of each box, whatever the swizzle)
          uint8_t* s = smem + stage * kStage;
          for (int c = 0; c < 6; ++c)
            for (int i = live * 8 + lane; i < 64 * 8; i += 32)
              *reinterpret_cast<uint4*>(s + c * kBox + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        fence_after_sync();
        if (lane == 0) {
          const uint32_t sA = base + stage * kStage, sB = sA + kABytes;
          const SDesc da = sdesc_w(sA, kBox, 1024), db = sdesc_w(sB, kBox, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_w(tmem + ab * 256, da + kk * 2048, db + kk * 2048, IDESC, kb > 0 || kk > 0 ? 1u : 0u);
          mma_commit(bar(B_EMPTY + stage));
        }
        __syncwarp();
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok && lane == 0) mma_commit(bar(B_AFULL + ab));
      ++n;
    }
    if (lane == 0) {
      mma_commit(bar(B_DRAIN));
      drain(bar(B_DRAIN), 0);
    }
    __syncwarp();
  } else {
    const int wq = warp & 3, half = warp >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    uint8_t* stg = staging + warp * 8192;
    const uint32_t stg_u32 = smem_u32(stg);
    uint32_t n = 0, sc = 0;
    for (; w.at(total); w.next()) {
      const uint32_t ab = n & 1;
      if (w.blocks > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(B_AFULL + ab), (n >> 1) & 1, wd, 74))) break;
        fence_after_sync();
      }
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        const int col = half * 128 + cc * 32;
        uint32_t v[32];
        if (w.blocks > 0) {
          tmem_ld32(lane_base + ab * 256 + col, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        const uint32_t at = (sc & 1) * 4096;
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        stage_f32(stg + at, lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (w.slot >= 0) tma_store_2d(&tmp, stg_u32 + at, col, w.slot * 128 + wq * 32);
          else if (w.n0 + col < p.features && w.k0 + wq * 32 < p.depth)
            tma_store_3d(&tmo, stg_u32 + at, w.n0 + col, w.k0 + wq * 32, w.e);
          bulk_commit();
        }
        ++sc;
      }
      if (w.blocks > 0) {
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_AEMPTY + ab));
        ++n;
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Sums of the pieces' partial sums, in their order: 16 rows of a tile at a time.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) group_dw_sum_kernel(const __grid_constant__ GroupParams p) {
  extern __shared__ int lists[];
  int* start = lists;
  int* first = lists + p.E + 1;
  pdl_wait();
  if (!scan_groups<kSumThreads>(p, start, first, [&](int n) { return pieces(n, p.kper); })) return;
  const int tpg = p.kt * p.nt;
  int e = 0, slots = 0, below = 0;   // below: split tiles of the groups below e
  const int c4 = threadIdx.x % 64 * 4, r0 = threadIdx.x / 64;
  for (int u = blockIdx.x;; u += gridDim.x) {
    const int split = u / 8, r = u % 8 * 16 + r0;
    while (e < p.E) {
      const int np = start[e + 1] - start[e];
      if (np > 1 && split < below + tpg) break;
      if (np > 1) {
        below += tpg;
        slots += np * tpg;
      }
      ++e;
    }
    if (e == p.E) return;
    const int np = start[e + 1] - start[e], tile = split - below;
    const int k0 = tile / p.nt * 128, n = tile % p.nt * 256 + c4;
    const float* src = p.partial + (size_t)(slots + tile * np) * kTile;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r + 4 * i;
      if (k0 + row >= p.depth || n >= p.features) continue;
      float4 s = __ldcg(reinterpret_cast<const float4*>(src + row * 256 + c4));
      for (int k = 1; k < np; ++k) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(src + (size_t)k * kTile + row * 256 + c4));
        s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
      }
      *reinterpret_cast<float4*>(p.dw + ((size_t)e * p.depth + k0 + row) * p.features + n) = s;
    }
  }
}

}  // namespace

// 64-row blocks of a piece: what an SM has to do on average, at least 8.
int group_dw_blocks(int64_t rows, int E, int K, int N, int sms) {
  const int64_t tpg = (int64_t)((K + 127) / 128) * ((N + 255) / 256);
  const int64_t b = ((rows + 63) / 64 * tpg + sms - 1) / sms;
  return (int)(b < 8 ? 8 : b);
}

// Slots that any offsets may need: a group of b > kper blocks has at most
// (b + kper - 1) / kper pieces a tile, b summing to at most rows / 64 + groups.
int64_t group_dw_slots(int64_t rows, int E, int K, int N, int sms) {
  const int64_t tpg = (int64_t)((K + 127) / 128) * ((N + 255) / 256);
  const int64_t kper = group_dw_blocks(rows, E, K, N, sms);
  const int64_t blocks = rows / 64 + (rows < E ? rows : E);
  if ((rows + 63) / 64 <= kper) return 0;   // no group is long enough
  return 2 * (blocks / kper + 1) * tpg;   // a split group has fewer than 2 b / kper pieces
}

cudaError_t launch_group_dw(const GroupParams& q, const void* x, int64_t x_stride, const void* dy, int64_t dy_stride, int K,
                            int N, int sms, cudaStream_t st, int* launches) {
  GroupParams p = q;
  p.features = N; p.depth = K;
  p.kt = (K + 127) / 128; p.nt = (N + 255) / 256;
  p.kper = group_dw_blocks(p.rows, p.E, K, N, 152);
  const int64_t slots = group_dw_slots(p.rows, p.E, K, N, 152);
  CUtensorMap mx, mg, mo, mp;
  const uint64_t xd[2] = {(uint64_t)K, (uint64_t)p.rows}, xs[1] = {(uint64_t)x_stride * 2};
  const uint64_t gd[2] = {(uint64_t)N, (uint64_t)p.rows}, gs[1] = {(uint64_t)dy_stride * 2};
  const uint64_t od[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)p.E}, os[2] = {(uint64_t)N * 4, (uint64_t)N * K * 4};
  const uint64_t pd[2] = {256, (uint64_t)(slots > 0 ? slots : 1) * 128}, ps[1] = {1024};
  const uint32_t ibox[2] = {64, 64}, obox[3] = {32, 32, 1};
  if (!make_tmap_tile(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, xd, xs, ibox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_tile(&mg, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dy, gd, gs, ibox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_tile(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p.dw, od, os, obox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_tile(&mp, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.partial, pd, ps, obox, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const size_t lists = 8 * ((size_t)p.E + 1);
  p.stages = 1024 + 3 * (size_t)kStage + kStaging + lists + 1024 <= kMaxSmemPerCta ? 3 : 2;
  const size_t smem = 1024 + (size_t)p.stages * kStage + kStaging + lists;
  cudaError_t e = cudaFuncSetAttribute(group_dw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)p.kt * p.nt * (p.E + p.rows / 64 / p.kper + 1);
  e = launch_pdl(group_dw_kernel, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads), smem, st, p, mx, mg, mo, mp);
  ++*launches;
  if (e != cudaSuccess || slots == 0) return e;
  e = launch_pdl(group_dw_sum_kernel, dim3((unsigned)(4 * sms)), dim3(kSumThreads), lists, st, p);
  ++*launches;
  return e;
}

}  // namespace hstu
