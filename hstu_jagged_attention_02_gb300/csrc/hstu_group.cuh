// Products of ragged groups of rows (hstu_group_fwd, hstu_group_bwd): what the
// row products (hstu_group_rows.cu: y = x W, dx = dy W^T) and the weight
// gradients (hstu_group_dw.cu) share.
//
// The groups' sizes are on the device only.  Every CTA reads the offsets and
// makes its own list of work from them: a scan of the groups' counts of
// row blocks (or of pieces of work) into shared memory, of which each role
// walks its share with a cursor.
#pragma once
#include "hstu_internal.h"
#include "tc_ptx.cuh"

namespace hstu {
namespace grp {

using namespace tc;

constexpr int kMaxGroups = 4096;
constexpr size_t kMaxDynamic = kMaxSmemPerCta - 512;   // (512: barriers and the scan's sums)
constexpr int kThreads = 10 * 32;   // 8 warps read accumulators, one loads, one issues the products
constexpr int kRun = 16;            // blocks of 64 summed in one accumulator
constexpr int kEpiWarps = 8, kLoadWarp = 8, kMmaWarp = 9;

// Counters of the weight gradients' cut tiles, at the same place of the workspace for every shape.
constexpr int kDwCounters = 152 * kEpiWarps;
constexpr size_t kDwCounterBytes = kDwCounters * sizeof(int);
__device__ __forceinline__ void clear_counters(int* at, int thread, int threads) {
  for (int i = thread; i < kDwCounters; i += threads) at[i] = 0;
}

struct GroupParams {
  const int64_t* off;
  int* hdr;
  int64_t rows;
  int E;
  int features;      // of the output: N (forward), K (dx)
  int depth;         // features summed over: K (forward), N (dx)
  int row_block;     // rows of a tile, 32, 64, 128 or 256
  int pair;          // CTAs work in pairs
  int box_rows;      // rows of a load box
  int one_w;         // a stage's part of W comes in one copy
  int stages;        // of the ring of loads (of A, where B has slots of its own)
  int slots;         // of B
  void* out;
  int64_t out_stride;
  int test_timeout;
  // weight gradients: tiles of 128 x 256 of [K, N], pieces of at most kper 64-row blocks
  int kt, nt, kper;
  int one_x, one_dy; // a stage's part of x (dy) comes in one copy
  float* dw;
  int* counters;     // of cut tiles, a storing warp each; row products: cleared for the weight gradients behind them, or NULL
  float* partial;    // [slots][CTAs of a tile][warps][32 x 128]
};

// mbar_wait for what threads of the other CTA of a pair have written and fenced
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, const Watchdog& wd, int site) {
  if (!mbar_wait(bar, parity, wd, site)) return false;
  uint32_t ok;   // complete by now: once more with the cluster's scope
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// After a wait ran out: until the phase completes, or 0.2 s.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > 200000000ull) break;
  }
}

// ---- what a pair of CTAs needs beside tc_ptx.cuh
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// the address of the same place in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tile loads (x innermost, a multiple of 16 bytes) by one elected lane of a converged warp, whose operands are uniform so;
// PAIR: into this CTA, counted on a barrier of the pair.
template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
  }
}
template <bool PAIR>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  }
}
template <int CG> __device__ __forceinline__ void alloc_tmem(uint32_t dst) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, 512);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG> __device__ __forceinline__ void free_tmem(uint32_t taddr) {
  if constexpr (CG == 1) tmem_dealloc(taddr, 512);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(512) : "memory");
}
// Issued by one elected lane of a converged warp, which runs the loop around them as one, so that operands are
// uniform values (an issuing thread alone took 800 cycles for a stage's four products, which take the tensor core 512).
template <int CG> __device__ __forceinline__ void mma(uint32_t d, SDesc a, SDesc b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1) {
    mma_ss_e(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\telect.sync _|e, 0xffffffff;\n\tmov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// arrives on the barrier (of both CTAs of a pair) when every tcgen05 operation so far has completed
template <int CG> __device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1) mma_commit_e(bar);
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// the same, on the issuing CTA's barrier alone
template <int CG> __device__ __forceinline__ void commit_here(uint32_t bar) {
  if constexpr (CG == 1) mma_commit_e(bar);
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// A loading thread's end; (stage, phase) is the next to be loaded, `loads` the loads so far.  Every stage is waited for once
// more by both CTAs of a pair: the products' arrivals come from the
// pair's first CTA on their own time, and one that came after this CTA's end would count on a barrier of its successor.
// After a wait that ran out: until the copies under way are there.
template <int CG, typename Bar>
__device__ __forceinline__ void tail(Bar bar, int empty, int full, int ring, int stage, uint32_t phase, uint32_t loads,
                                     uint32_t rank, bool ok, const Watchdog& wd, int site) {
  int s = stage;
  uint32_t ph = phase;
  for (int i = 0; CG == 2 && ok && i < ring; ++i) {
    if (loads >= (uint32_t)ring || s < stage) ok = mbar_wait(bar(empty + s), ph ^ 1, wd, site);
    if (++s == ring) {
      s = 0;
      ph ^= 1;
    }
  }
  if (ok) return;
  if (rank == 0) {   // the barriers count both CTAs' copies
    for (s = 0; s < ring; ++s)
      if (s < stage) drain(bar(full + s), phase);
      else if (loads >= (uint32_t)ring) drain(bar(full + s), phase ^ 1);
  } else {   // the other CTA's copies are not counted here
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {}
  }
}

// start[e] = sum of count(rows of the groups below e), e <= E, and first[e] =
// first row of group e, by all threads of the CTA.  False (for all threads), and the error recorded by CTA 0, where
// the offsets are not in order.
template <int THREADS, typename F>
__device__ __forceinline__ bool scan_groups(const GroupParams& p, int* start, int* first, F count) {
  __shared__ int warp_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.E + THREADS - 1) / THREADS, lo = min(p.E, tid * per), hi = min(p.E, lo + per);
  int sum = 0;
  bool bad = tid == 0 && p.off[0] != 0;
  if (lo < hi) {
    int64_t a = p.off[lo];
    for (int e = lo; e < hi; ++e) {
      const int64_t b = p.off[e + 1];
      const bool wrong = a < 0 || b < a || b > p.rows;
      bad |= wrong;
      first[e] = wrong ? 0 : (int)a;
      const int c = wrong ? 0 : count((int)(b - a));
      start[e] = c;
      sum += c;
      a = b;
    }
    if (hi == p.E) first[p.E] = bad ? 0 : (int)a;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && tid == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return false;
  }
  int base = incl - sum;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  for (int e = lo; e < hi; ++e) {
    const int c = start[e];
    start[e] = base;
    base += c;
  }
  if (lo < hi && hi == p.E) start[p.E] = base;
  __syncthreads();
  return true;
}

// A launch as launch_pdl makes it, in clusters of CG CTAs.
template <int CG, typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, int threads, size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace grp

cudaError_t launch_group_rows(const grp::GroupParams& p, bool transposed, int out_dtype, const void* rows, int64_t row_stride,
                              const void* w, int K, int N, int sms, cudaStream_t st);
// p.counters: group_dw_bytes of room, whose counters launch_group_rows or launch_group_dw_clear has cleared
cudaError_t launch_group_dw(const grp::GroupParams& p, const void* x, int64_t x_stride, const void* dy, int64_t dy_stride,
                            int K, int N, int sms, cudaStream_t st);
cudaError_t launch_group_dw_clear(int* counters, cudaStream_t st);
size_t group_dw_bytes(int64_t rows, int E, int K, int N);

}  // namespace hstu
