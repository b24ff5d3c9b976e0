// Products of ragged groups of rows with a weight matrix each: y = x W[g]
// and dx = dy W[g]^T (hstu_group_fwd, the dx of hstu_group_bwd), and the C calls.
//
// Transposed: the tensor core's 128 rows are output features, its columns
// the group's rows.  A group's last tile so costs what it has rows (in 16s), not 128,
// and a group of one row costs a load of its weights.  D[f, r] = sum_k W[k, f] x[r, k]:
//   A = 128 features x 64 k of W[g] (features contiguous: MN-major; for dx k is the
//   contiguous side: K-major), from a 3-D map [g][K][N], so that a tile's edge never
//   reads the next group's weights;
//   B = up to 256 rows x 64 k of x (K-major).  Rows of the next group that a load brings
//   along give columns that nobody stores.
// One persistent CTA an SM, 128 x row_block tiles, a ring of loads, two accumulators in
// TMEM, so that a tile is stored while the next one is computed.  The tiles of a row block
// are neighbours in the order of work: its rows and the group's weights come from L2.
//
// Roles (320 threads): warps 0-7 store, warp 8 loads, warp 9 issues and owns TMEM.  Every
// wait is bounded.
#include "hstu_group.cuh"

namespace hstu {

namespace {

using namespace grp;

constexpr int kStagesMax = 9;
constexpr int kABytes = 128 * 64 * 2;
enum : int { B_FULL = 0, B_EMPTY = B_FULL + kStagesMax, B_AFULL = B_EMPTY + kStagesMax, B_AEMPTY = B_AFULL + 2,
             B_DRAIN = B_AEMPTY + 2, B_COUNT };

// two 32 x 32 buffers a storing warp
constexpr int staging_bytes(int element) { return kEpiWarps * 2 * 1024 * element; }

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

// Walks the tiles blockIdx.x, blockIdx.x + gridDim.x, ..: t = row block x feature blocks + feature block.
struct Tiles {
  const int* start;
  const int* first;
  int fb, rb, e, row0, rows, f0, t;
  __device__ __forceinline__ Tiles(const int* start_, const int* first_, int fblocks, int row_block)
      : start(start_), first(first_), fb(fblocks), rb(row_block), e(0), t(blockIdx.x) {}
  __device__ __forceinline__ bool at(int total) {
    if (t >= total) return false;
    const int blk = t / fb;
    while (start[e + 1] <= blk) ++e;
    const int in = (blk - start[e]) * rb;
    row0 = first[e] + in;
    rows = min(rb, first[e + 1] - row0);
    f0 = (t - blk * fb) * 128;
    return true;
  }
  __device__ __forceinline__ void next() { t += gridDim.x; }
};

// KMAJOR: W is read with k contiguous (dx), else with features contiguous (forward)
template <bool KMAJOR, typename TO>
__global__ void __launch_bounds__(kThreads, 1)
group_rows_kernel(const __grid_constant__ GroupParams p, const __grid_constant__ CUtensorMap tmw,
                  const __grid_constant__ CUtensorMap tmr, const __grid_constant__ CUtensorMap tmo) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[B_COUNT];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t raw_u32 = smem_u32(smem_raw), base = (raw_u32 + 1023u) & ~1023u;
  const int stage_bytes = kABytes + p.row_block * 128;
  int* start = reinterpret_cast<int*>(smem_raw + (base - raw_u32) + p.stages * stage_bytes + staging_bytes(sizeof(TO)));
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
    tma_prefetch_desc(&tmw);
    tma_prefetch_desc(&tmr);
  }
  pdl_wait();
  const int rb = p.row_block;
  const bool good = scan_groups<kThreads>(p, start, first, [&](int n) { return (n + rb - 1) / rb; });
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;

  Watchdog wd;
  wd.abort = &abort_word;
  wd.err = p.hdr + WS_ERR;
  wd.err_info = p.hdr + WS_ERR_INFO;
  wd.limit_ns = p.test_timeout ? 1000000ull : 2000000000ull;
  const int fblocks = (p.features + 127) / 128, kblocks = (p.depth + 63) / 64;
  const int total = good ? start[p.E] * fblocks : 0;
  Tiles w(start, first, fblocks, rb);

  if (warp == kLoadWarp) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, used = 0;   // used: stages whose barrier was armed
      bool ok = true, withhold = p.test_timeout && blockIdx.x == 0;
      uint32_t last[kStagesMax];
      for (; ok && w.at(total); w.next()) {
        const int boxes = (w.rows + p.box_rows - 1) / p.box_rows;
        const uint32_t box_bytes = (uint32_t)p.box_rows * 128u, bytes = kABytes + boxes * box_bytes;
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = mbar_wait(bar(B_EMPTY + stage), phase ^ 1, wd, 61);
          if (!ok) break;
          if (withhold) {   // test only: this copy never comes
            withhold = false;
          } else {
            const uint32_t sA = base + stage * stage_bytes, sB = sA + kABytes, full = bar(B_FULL + stage);
            mbar_arrive_expect_tx(full, bytes);
            if (KMAJOR) {
              tma_load_3d(sA, &tmw, full, kb * 64, w.f0, w.e);
            } else {
              tma_load_3d(sA, &tmw, full, w.f0, kb * 64, w.e);
              tma_load_3d(sA + kABytes / 2, &tmw, full, w.f0 + 64, kb * 64, w.e);
            }
            for (int b = 0; b < boxes; ++b) tma_load_2d(sB + b * box_bytes, &tmr, full, kb * 64, w.row0 + b * p.box_rows);
            used |= 1u << stage;
#pragma unroll
            for (int s = 0; s < kStagesMax; ++s)
              if (s == stage) last[s] = phase;
          }
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
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, n = 0;
      bool ok = true;
      for (; ok && w.at(total); w.next(), ++n) {
        const uint32_t ab = n & 1;
        ok = mbar_wait(bar(B_AEMPTY + ab), ((n >> 1) & 1) ^ 1, wd, 62);
        if (!ok) break;
        fence_after_sync();
        // as many columns as there are rows, in 16s
        const uint32_t idesc = idesc_bf16(128, (w.rows + 15) & ~15, !KMAJOR, false);
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = mbar_wait(bar(B_FULL + stage), phase, wd, 63);
          if (!ok) break;
          fence_after_sync();
          const uint32_t sA = base + stage * stage_bytes, sB = sA + kABytes;
          const SDesc da = KMAJOR ? sdesc_w(sA, 16, 1024) : sdesc_w(sA, kABytes / 2, 1024);
          const SDesc db = sdesc_w(sB, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_w(tmem + ab * 256, da + (KMAJOR ? kk * 32 : kk * 2048), db + kk * 32, idesc, kb > 0 || kk > 0 ? 1u : 0u);
          mma_commit(bar(B_EMPTY + stage));
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok) mma_commit(bar(B_AFULL + ab));
      }
      mma_commit(bar(B_DRAIN));
      drain(bar(B_DRAIN), 0);
    }
  } else {
    // a warp stores 32 features of 32 rows at a time, through its two staging buffers [row][feature]
    const int wq = warp & 3, half = warp >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    constexpr int kBuf = 1024 * sizeof(TO);
    const uint32_t stg = base + p.stages * stage_bytes + warp * 2 * kBuf;
    const uint8_t* stg_ptr = smem_raw + (stg - raw_u32);
    TO* out = static_cast<TO*>(p.out);
    // where this lane's row of an 8 x 8 matrix goes: matrix l / 8 of 4 has features 8 (m % 2).. and rows 8 (m / 2)..
    const uint32_t lane_row = (lane >> 4) * 8 + (lane & 7), lane_chunk = (lane >> 3 & 1) ^ (lane >> 1 & 3);
    uint32_t n = 0, buf = 0;
    for (; w.at(total); w.next(), ++n) {
      const uint32_t ab = n & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_AFULL + ab), (n >> 1) & 1, wd, 64))) break;
      fence_after_sync();
      const int f = w.f0 + wq * 32;
#pragma unroll 1
      for (int c = half * 32; c < w.rows; c += 64) {
        const uint32_t to = stg + buf * kBuf;
        const uint8_t* from = stg_ptr + buf * kBuf;
        if (lane == 0) bulk_wait_read<1>();   // the buffer's last store has read it
        __syncwarp();
        if constexpr (sizeof(TO) == 4) {
          // lanes are features: a row at a time, 32 neighbouring words
          uint32_t v[32];
          tmem_ld32(lane_base + ab * 256 + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < 32; ++r)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + r * 128 + lane * 4), "r"(v[r]) : "memory");
        } else {
          // 16 features x 32 rows a load, whose registers are 8 x 8 matrices [feature][row]; stored transposed,
          // 16-byte chunk k of row r at k ^ (r / 2 % 4)
          uint32_t v[2][16];
          tmem_ld_16x256b_x4(lane_base + ab * 256 + c, v[0]);
          tmem_ld_16x256b_x4(lane_base + (16u << 16) + ab * 256 + c, v[1]);
          tmem_wait_ld();
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
          if (lane == 0) bulk_commit();   // an empty group, so that a buffer's group is always the last but one
        }
        buf ^= 1;
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_AEMPTY + ab));
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <bool KMAJOR, typename TO>
cudaError_t launch_t(GroupParams p, const void* rows, int64_t row_stride, const void* w, int K, int N, int sms,
                     cudaStream_t st) {
  CUtensorMap mw, mr, mo;
  const uint64_t wd[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)p.E}, ws[2] = {(uint64_t)N * 2, (uint64_t)N * K * 2};
  const uint32_t wbox[3] = {64, KMAJOR ? 128u : 64u, 1};
  const uint64_t rd[2] = {(uint64_t)p.depth, (uint64_t)p.rows}, rs[1] = {(uint64_t)row_stride * 2};
  const uint32_t rbox[2] = {64, (uint32_t)p.box_rows}, obox[2] = {32, 32};
  const uint64_t od[2] = {(uint64_t)p.features, (uint64_t)p.rows}, os[1] = {(uint64_t)p.out_stride * sizeof(TO)};
  if (!make_tmap_tile(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, w, wd, ws, wbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_tile(&mr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, rd, rs, rbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_tile(&mo, sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.out,
                      od, os, obox, sizeof(TO) == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const size_t fixed = 1024 + staging_bytes(sizeof(TO)) + 8 * ((size_t)p.E + 1), stage = kABytes + p.row_block * 128;
  p.stages = (int)((kMaxSmemPerCta - 1024 - fixed) / stage);   // (the rest: barriers and the scan's sums)
  if (p.stages > kStagesMax) p.stages = kStagesMax;
  const size_t smem = fixed + p.stages * stage;
  auto kern = group_rows_kernel<KMAJOR, TO>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t most = (p.rows / p.row_block + p.E) * (int64_t)((p.features + 127) / 128);
  return launch_pdl(kern, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads), smem, st, p, mw, mr, mo);
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

// The workspace has to hold for any GPU of this kind: sized for the SMs of a whole GB300.
constexpr int kSizeSms = 152;

size_t bwd_bytes(const hstu_group_desc* d) {
  return kWsHeaderBytes + sizeof(float) * 128 * 256 * (size_t)group_dw_slots(d->rows, d->groups, d->K, d->N, kSizeSms);
}

void set_tile(GroupParams& p, int sms) {
  p.row_block = group_row_block(p.rows, p.E, p.features, sms);
  p.box_rows = p.row_block < 64 ? 32 : 64;
}

}  // namespace

// The tile's rows.  Cost of a choice: waves of tiles over the SMs, a tile costing its rows and
// about 64 more for its weights' loads and its ends.
int group_row_block(int64_t rows, int E, int features, int sms) {
  const int64_t fb = (features + 127) / 128;
  int64_t best = -1;
  int take = 256;
  for (int rb = 256; rb >= 32; rb >>= 1) {
    const int64_t full = rows / rb + (rows < E ? rows : E), waves = (full * fb + sms - 1) / sms;
    const int64_t cost = waves * (rb + 64);
    if (best < 0 || cost < best) {
      best = cost;
      take = rb;
    }
  }
  return take;
}

cudaError_t launch_group_rows(const GroupParams& p, bool transposed, int out_dtype, const void* rows, int64_t row_stride,
                              const void* w, int K, int N, int sms, cudaStream_t st) {
  if (transposed)
    return out_dtype == HSTU_BF16 ? launch_t<true, __nv_bfloat16>(p, rows, row_stride, w, K, N, sms, st)
                                  : launch_t<true, float>(p, rows, row_stride, w, K, N, sms, st);
  return out_dtype == HSTU_BF16 ? launch_t<false, __nv_bfloat16>(p, rows, row_stride, w, K, N, sms, st)
                                : launch_t<false, float>(p, rows, row_stride, w, K, N, sms, st);
}

}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_group_workspace_size(const hstu_group_desc* desc, size_t* fwd, size_t* bwd) {
  const hstu_status_t s = check_desc(desc);
  if (s != HSTU_OK) return s;
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
  if (sms > kSizeSms) sms = kSizeSms;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  GroupParams p{};
  p.off = a->group_offsets; p.hdr = static_cast<int*>(workspace);
  p.rows = d->rows; p.E = d->groups;
  const int64_t ys = d->rows <= 1 ? d->N : d->y_stride, xs = d->rows <= 1 ? d->K : d->x_stride;
  cudaError_t e = cudaSuccess;
  int launches = 0;
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
      p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeaderBytes);
      e = launch_group_dw(p, a->x, xs, a->dy, ys, d->K, d->N, sms, st, &launches);
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
