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
constexpr int kThreads = 10 * 32;   // 8 warps read accumulators, one loads, one issues the products
constexpr int kEpiWarps = 8, kLoadWarp = 8, kMmaWarp = 9;

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
  int stages;        // of the ring of loads (of A, where B has slots of its own)
  int slots;         // of B
  void* out;
  int64_t out_stride;
  int test_timeout;
  // weight gradients: tiles of 128 x 256 of [K, N], pieces of at most kper 64-row blocks
  int kt, nt, kper;
  float* dw;
  float* partial;    // [slots][128][256]
};

// 3-D tile load (x innermost, a multiple of 16 bytes)
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// After a wait ran out: until the phase completes, or 0.2 s.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > 200000000ull) break;
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

}  // namespace grp

cudaError_t launch_group_rows(const grp::GroupParams& p, bool transposed, int out_dtype, const void* rows, int64_t row_stride,
                              const void* w, int K, int N, int sms, cudaStream_t st);
cudaError_t launch_group_dw(const grp::GroupParams& p, const void* x, int64_t x_stride, const void* dy, int64_t dy_stride,
                            int K, int N, int sms, cudaStream_t st, int* launches);
// 64-row blocks of a piece, and slots of partial sums
int group_dw_blocks(int64_t rows, int E, int K, int N, int sms);
int64_t group_dw_slots(int64_t rows, int E, int K, int N, int sms);

}  // namespace hstu
