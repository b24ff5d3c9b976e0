// The attention over the paged 4-bit cache for few rows (hstu_attn_fwd_cached
// with at most 16 rows a sequence: decode steps, a handful of candidates).
//
// With few rows the work is the bytes of the cache: 9/16 byte a feature, read
// once.  So the packed rows go from global memory straight to registers, in
// the shape in which a warp's matrix instruction (m16n8k16, FP16 -> FP32)
// takes them, and are decoded there; nothing is staged in shared memory, whose
// bandwidth bounds the tensor-memory kernel at few rows (a decoded tile is
// written once and read once, 128 KB for 18 KB of cache).  A warp takes 16
// tokens at a time:
//
//   S^T [16 tokens x 8 rows] = K Q^T      lane (g, t), g = lane / 4, t = lane % 4, holds tokens g and g + 8, features
//                                         [t d/4, (t + 1) d/4): the products' inner index runs over the features in
//                                         any order, as long as q is held in the same one
//   P = 16 SiLU(z)                        in the accumulator's places, to FP16, turned by movmatrix
//   O^T [d x 8 rows] += V^T P             lane (g, t) holds tokens 2t, 2t + 1, 2t + 8, 2t + 9, features
//                                         [g d/8, (g + 1) d/8), pairs of tokens put together by byte permutes
//
// q stays in registers (FP16, scaled per row by a power of two: hstu_cached.cuh),
// so does O.  The CTA's warps deal a piece's 16-token steps among themselves
// and add their sums up in shared memory at the piece's end.  The loads of the next step are
// issued before the current one is worked on.
#include "hstu_cached.cuh"

namespace hstu {

namespace {

template <int D, int QT>
struct SCfg {
  static constexpr int WARPS = QT == 1 ? 16 : 12;   // 128 and 168 registers a thread
  static constexpr int THREADS = WARPS * 32;
  static constexpr int N = 8 * QT;
  static constexpr int SMEM = WARPS * N * D * 4;    // the warps' sums at a piece's end
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

// A lane's packed part of 16 tokens.
template <int D>
struct Step {
  static constexpr int KW = D / 32, VW = D / 64;   // 32-bit words of codes: a K token's, a V token's
  uint32_t k[2][KW], ks[2], v[4][VW], vs[4];
  int64_t t[2];
};

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (W == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x; w[1] = x.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

template <int D>
__device__ __forceinline__ void load_step(const CachedParams& p, const PageLayout& lay, int page, int h, int place, int lane,
                                          Step<D>& s) {
  const int g = lane >> 2, t = lane & 3;
  const uint8_t* kp = p.pages + ((int64_t)page * p.H + h) * lay.bytes();
  const uint8_t* vp = kp + lay.half();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = place + g + 8 * i;
    load_words<D / 32>(kp + tok * (D / 2) + t * (D / 8), s.k[i]);
    const uint8_t* sp = kp + lay.scales() + tok * (D / 16) + t * (D / 64);
    s.ks[i] = D == 128 ? __ldg(reinterpret_cast<const uint16_t*>(sp)) : __ldg(sp);
    s.t[i] = p.times ? __ldg(p.page_times + (int64_t)page * p.page_size + tok) : 0;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = place + 2 * t + (i & 1) + 8 * (i >> 1);
    load_words<D / 64>(vp + tok * (D / 2) + g * (D / 16), s.v[i]);
    s.vs[i] = __ldg(vp + lay.scales() + tok * (D / 16) + (g * (D / 8)) / 16);
  }
}

template <int D, int QT>
__global__ void __launch_bounds__(SCfg<D, QT>::THREADS, 1) cached_stream_kernel(const __grid_constant__ CachedParams p) {
  using C = SCfg<D, QT>;
  constexpr int N = C::N, KS = D / 16, MT = D / 16;   // inner steps of S, 16-feature tiles of O
  extern __shared__ __align__(16) float sums[];
  __shared__ int scan[2 * C::WARPS];
  __shared__ Start start;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();   // the finishing kernel waits for this grid's end itself
  cut_work<C::THREADS>(p, N, scan, &start);
  __syncthreads();
  Walk w;
  w.begin(p, start, N);
  const PageLayout lay(p.page_size, D);
  while (w.left > 0) {
    const CachedSeq s = w.s;
    const int h = w.h, r0 = w.qb * N, rows = min(N, s.n - r0), hist = s.n - s.m;
    const int pos0 = s.L - hist + r0;                      // position of the block's first row
    const int nh = max(0, min(hist - r0, rows));           // its history rows; the others are at L
    const int64_t row0 = s.row0 + r0;
    // q: lane (g, t) holds row g (+ 8) and features [t D/4, (t + 1) D/4)
    uint32_t q[QT][KS][2];
    float ka[QT][2];
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int r = i * 8 + g;
      uint32_t x[D / 8];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows) v = *reinterpret_cast<const uint4*>(p.q + ((row0 + r) * p.H + h) * D + t * (D / 4) + e * 8);
        x[4 * e] = v.x; x[4 * e + 1] = v.y; x[4 * e + 2] = v.z; x[4 * e + 3] = v.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < D / 8; ++e) top = max(top, max((x[e] << 16) & 0x7fff0000u, x[e] & 0x7fff0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float down;
      const float up = row_scale(top, down);
#pragma unroll
      for (int e = 0; e < D / 8; ++e)
        q[i][e >> 1][e & 1] = pack_f16(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xFFFF0000u) * up);
      // the factor of this lane's score columns, rows 2t and 2t + 1
      const float f = -kLog2e * p.alpha * p.k_scale * down;
      ka[i][0] = __shfl_sync(0xffffffffu, f, 8 * t);
      ka[i][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
    // the rows' times, and their range
    int64_t tq = 0, tmin = INT64_MAX, tmax = INT64_MIN;
    if (p.times && lane < rows) tq = tmin = tmax = p.times[row0 + lane];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const int64_t a = __shfl_xor_sync(0xffffffffu, tmin, o), b = __shfl_xor_sync(0xffffffffu, tmax, o);
      tmin = a < tmin ? a : tmin;
      tmax = b > tmax ? b : tmax;
    }
    tmin = __shfl_sync(0xffffffffu, tmin, 0);
    tmax = __shfl_sync(0xffffffffu, tmax, 0);
    const int pmin = nh > 0 ? pos0 : s.L, pmax = nh == rows ? pos0 + rows - 1 : s.L;
    const float* rp = p.rab_pos ? p.rab_pos + h * p.P : nullptr;
    const float* rt = p.rab_time ? p.rab_time + h * p.Tb : nullptr;

    float o[QT][MT][4];
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) o[i][m][0] = o[i][m][1] = o[i][m][2] = o[i][m][3] = 0.f;

    // 16-token steps of the piece, dealt to the warps in turn
    const int last = min((w.tile + w.take()) * (kCachedTile / 16), (s.L + 15) / 16);
    const int32_t* table = p.table + (int64_t)w.b * p.max_pages;
    const int spp = p.page_size / 16;
    int st = w.tile * (kCachedTile / 16) + warp;
    auto page_of = [&](int step) -> int {
      const int id = step < last ? __ldg(table + step / spp) : 0;
      if (id >= 0 && id < p.num_pages) return id;
      set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, w.b);
      return 0;                                            // some page: the batch's result is undefined
    };
    Step<D> cur, nxt;
    int page = page_of(st), page1 = page_of(st + C::WARPS);
    if (st < last) load_step<D>(p, lay, page, h, (st % spp) * 16, lane, cur);
    for (; st < last; st += C::WARPS) {
      const int st1 = st + C::WARPS;
      if (st1 < last) {
        load_step<D>(p, lay, page1, h, (st1 % spp) * 16, lane, nxt);
        page1 = page_of(st1 + C::WARPS);
      }
      float c[QT][4];
#pragma unroll
      for (int i = 0; i < QT; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
      {
        const __half2 s0 = e4m3x2_half2(cur.ks[0]), s1 = e4m3x2_half2(cur.ks[1]);
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {                 // 8 features at a time: two inner steps
          const bool hi = D == 128 && x >= 2;
          const uint4 a = decode8(cur.k[0][x], hi ? __high2half2(s0) : __low2half2(s0));
          const uint4 b = decode8(cur.k[1][x], hi ? __high2half2(s1) : __low2half2(s1));
#pragma unroll
          for (int i = 0; i < QT; ++i) {
            mma16816(c[i], a.x, b.x, a.y, b.y, q[i][2 * x][0], q[i][2 * x][1]);
            mma16816(c[i], a.z, b.z, a.w, b.w, q[i][2 * x + 1][0], q[i][2 * x + 1][1]);
          }
        }
      }
      // scores of tokens j0 (c[0], c[1]) and j0 + 8 (c[2], c[3]) for rows 2t, 2t + 1
      const int j0 = st * 16 + g;
      uint32_t pr[QT][2];
      float bias[2];
      bool same = true;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + 8 * e;
        bool ok = j <= pmin;
        float b = 0.f;
        if (rp) {
          const int a = min(max(pmin - j, 0), p.P - 1), z = min(max(pmax - j, 0), p.P - 1);
          ok = ok && a == z;
          b = rp[a];
        }
        if (rt) {
          const int a = time_bucket(tmin, cur.t[e], p.Tb), z = time_bucket(tmax, cur.t[e], p.Tb);
          ok = ok && a == z && (cur.t[e] <= tmin || cur.t[e] >= tmax);
          b += rt[a];
        }
        bias[e] = -kLog2e * b;
        same = same && (ok || j >= s.L);
      }
      if (__all_sync(0xffffffffu, same)) {
#pragma unroll
        for (int i = 0; i < QT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            pr[i][e] = silu_pair(__ffma2_rn(make_float2(c[i][2 * e], c[i][2 * e + 1]), make_float2(ka[i][0], ka[i][1]),
                                            make_float2(bias[e], bias[e])));
      } else {
#pragma unroll
        for (int i = 0; i < QT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = j0 + 8 * e;
            float x[2];
            uint32_t keep = 0;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int r = i * 8 + 2 * t + f, pos = r < nh ? pos0 + r : s.L;
              const int64_t tr = __shfl_sync(0xffffffffu, tq, r);
              float b = 0.f;
              if (rp) b = rp[min(max(pos - j, 0), p.P - 1)];
              if (rt) b += rt[time_bucket(tr, cur.t[e], p.Tb)];
              x[f] = fmaf(c[i][2 * e + f], ka[i][f], -kLog2e * b);
              keep |= j <= pos ? 0xffffu << (16 * f) : 0u;
            }
            pr[i][e] = silu_pair(make_float2(x[0], x[1])) & keep;
          }
      }
      const bool whole = (st + 1) * 16 <= s.L;
      if (!whole) {                                        // tokens behind the cache's end: neither scores nor values
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < QT; ++i) pr[i][e] = j0 + 8 * e < s.L ? pr[i][e] : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (st * 16 + 2 * t + (e & 1) + 8 * (e >> 1) >= s.L) cur.vs[e] = 0;
      }
      uint32_t b[QT][2];
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) b[i][e] = transpose8x8(pr[i][e]);
      {
        const __half2 x01 = e4m3x2_half2(cur.vs[0] | (cur.vs[1] << 8)), x23 = e4m3x2_half2(cur.vs[2] | (cur.vs[3] << 8));
        const __half2 s0 = __low2half2(x01), s1 = __high2half2(x01), s2 = __low2half2(x23), s3 = __high2half2(x23);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {                 // 8 features of the lane's D / 8
          const uint4 v0 = decode8(cur.v[0][x], s0), v1 = decode8(cur.v[1][x], s1);
          const uint4 v2 = decode8(cur.v[2][x], s2), v3 = decode8(cur.v[3][x], s3);
          const uint32_t a0[4] = {v0.x, v0.y, v0.z, v0.w}, a1[4] = {v1.x, v1.y, v1.z, v1.w};
          const uint32_t a2[4] = {v2.x, v2.y, v2.z, v2.w}, a3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t r0_ = __byte_perm(a0[y], a1[y], 0x5410), r1_ = __byte_perm(a0[y], a1[y], 0x7632);
            const uint32_t r2_ = __byte_perm(a2[y], a3[y], 0x5410), r3_ = __byte_perm(a2[y], a3[y], 0x7632);
#pragma unroll
            for (int i = 0; i < QT; ++i) mma16816(o[i][4 * x + y], r0_, r1_, r2_, r3_, b[i][0], b[i][1]);
          }
        }
      }
      cur = nxt;
    }
    // the warps' sums: o[i][m] holds features g D/8 + 2m, + 1 of rows 8i + 2t, + 1
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = i * 8 + 2 * t + e;
        if (r < rows) {
          float* dst = sums + (warp * N + r) * D + g * (D / 8);
#pragma unroll
          for (int m = 0; m < MT; ++m) *reinterpret_cast<float2*>(dst + 2 * m) = make_float2(o[i][m][e], o[i][m][2 + e]);
        }
      }
    __syncthreads();
    float* part = p.part + (int64_t)w.slot(p) * (N * D);
    for (int e = threadIdx.x; e < rows * D; e += C::THREADS) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < C::WARPS; ++k) x += sums[k * N * D + e];
      part[e] = x;
    }
    __syncthreads();
    w.next(p, N);
  }
}

template <int D, int QT>
cudaError_t launch_t(const CachedParams& p, int ctas, cudaStream_t st) {
  using C = SCfg<D, QT>;
  auto kern = cached_stream_kernel<D, QT>;
  const void* fn = reinterpret_cast<const void*>(kern);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(C::THREADS), C::SMEM, st, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_launch_detail(e, "cached_stream_kernel", fn, C::THREADS, C::SMEM);
  }
  return e;
}

}  // namespace

cudaError_t launch_stream_cached(const CachedParams& p, int d, int N, int ctas, cudaStream_t st) {
  if (d == 128) return N == 8 ? launch_t<128, 1>(p, ctas, st) : launch_t<128, 2>(p, ctas, st);
  return N == 8 ? launch_t<64, 1>(p, ctas, st) : launch_t<64, 2>(p, ctas, st);
}

}  // namespace hstu
