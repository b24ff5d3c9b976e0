// Norm and rotation of queries and keys per head (hstu_qk_norm_rope_*).
//
//   r = 1 / sqrt(mean(x^2) + eps), w = x r gain, each pair of w turned by the
//   angle of the token's position; backward: the incoming gradient turned
//   back, e = dout R^T, then dgain += e x r and dx = r (e g - x r mean(e g x r)).
//
// HBM-bound: every row of d features is read once (backward: x and dout)
// and written once, so what counts is to spend few instructions a byte and to
// have many loads in flight.  d / 8 lanes hold a row, so that a warp's pass
// covers 256 features, the row's sum takes few shuffles, and both features of
// every pair lie in one lane (hstu_rows.cuh): the rotation exchanges nothing.
// A warp takes up to kPasses passes (heads) of one token, all loads first; the
// token's cosines and sines are loaded once for them.
//
// The backward's gain gradients are sums over all tokens and heads.  The
// CTAs walk tokens and keep per-lane FP32 partial sums; the CTAs' rows of
// partial sums land in the workspace and the CTA that finishes last (a
// counter in the workspace's header) adds them up in row order in FP64, so
// the result does not depend on the order in which CTAs finish.
#include "hstu_internal.h"
#include "hstu_rows.cuh"

namespace hstu {

namespace {

constexpr int kQkThreads = 256;
constexpr int kBwdThreads = 512;
constexpr int kPasses = 4;

struct QkParams {
  const int64_t* num_tokens;
  const int32_t* positions;
  const float* cos;
  const float* sin;
  const float* gain[2];
  const void* x[2];      // q, k
  const void* g[2];      // backward: incoming gradients
  void* out[2];          // forward: outputs; backward: dq, dk
  int64_t xs[2][2], gs[2][2], os[2][2];
  float* dgain[2];
  float* partial;        // [CTAs][2][d]
  int* hdr;
  int64_t T, max_pos;
  int H[2];
  int rot, interleaved, norm;
  float eps;
};

// The position's row in the tables; one outside them is recorded and row 0 taken.
__device__ __forceinline__ int64_t checked_position(const QkParams& p, int64_t t) {
  if (p.rot == 0) return 0;
  const int64_t pos = p.positions[t];
  if (pos >= 0 && pos < p.max_pos) return pos;
  set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, (int)(t & 0x7fffffff));
  return 0;
}

__device__ __forceinline__ int64_t live_tokens(const QkParams& p) {
  if (!p.num_tokens) return p.T;
  const int64_t n = *p.num_tokens;
  if (n > p.T || n < 0) {
    set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return 0;
  }
  return n;
}

// The lane's cosines and sines (dir -1: turned back, the backward).
__device__ __forceinline__ void load_angles(const QkParams& p, const Parts& pt, int64_t pos, int l, float dir, float (&c)[4],
                                            float (&s)[4]) {
  if (pt.turns) {
    const int64_t at = pos * (p.rot >> 1) + 4 * l;
    load4(p.cos + at, c);
    load4(p.sin + at, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] *= dir;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) { c[e] = 1.f; s[e] = 0.f; }
  }
}

// Pass i of a token: q's heads come first, PER = 256 / D heads a pass.
struct Pass {
  int w, head;   // 0: q, 1: k; this lane's head
  bool on;
  __device__ __forceinline__ Pass(const QkParams& p, int i, int pq, int per, int sub) {
    w = i >= pq;
    head = (i - (w ? pq : 0)) * per + sub;
    on = head < p.H[w];
  }
};

template <typename TI, int D>
__global__ void __launch_bounds__(kQkThreads) qk_fwd_kernel(const __grid_constant__ QkParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
  const int64_t t = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
  if (t >= live_tokens(p)) return;
  const int pq = (p.H[0] + PER - 1) / PER, pk = (p.H[1] + PER - 1) / PER, i0 = blockIdx.y * kPasses;
  const Parts pt(l, p.rot, p.interleaved);
  Raw4<TI> r0[kPasses], r1[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (i0 + i >= pq + pk) break;
    const Pass ps(p, i0 + i, pq, PER, sub);
    const TI* src = static_cast<const TI*>(p.x[ps.w]) + t * p.xs[ps.w][0] + (ps.on ? ps.head : 0) * p.xs[ps.w][1];
    r0[i] = fetch4(src + pt.f0);
    r1[i] = fetch4(src + pt.f1);
  }
  float c[4], s[4];
  load_angles(p, pt, checked_position(p, t), l, 1.f, c, s);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (i0 + i >= pq + pk) break;
    const Pass ps(p, i0 + i, pq, PER, sub);
    float x[4], y[4];
    unpack4(r0[i], x);
    unpack4(r1[i], y);
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
      const float rs = __frsqrt_rn(fmaf(row_sum<LANES>(ss), 1.f / D, p.eps));
#pragma unroll
      for (int e = 0; e < 4; ++e) { x[e] *= rs; y[e] *= rs; }
      if (p.gain[ps.w]) {
        float a[4], b[4];
        load4(p.gain[ps.w] + pt.f0, a);
        load4(p.gain[ps.w] + pt.f1, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[e] *= a[e]; y[e] *= b[e]; }
      }
    }
    if (pt.turns) turn_pairs(x, y, c, s, p.interleaved);
    if (ps.on) {
      TI* dst = static_cast<TI*>(p.out[ps.w]) + t * p.os[ps.w][0] + ps.head * p.os[ps.w][1];
      store4(dst + pt.f0, x);
      store4(dst + pt.f1, y);
    }
  }
}

template <typename TI, int D>
__global__ void __launch_bounds__(kBwdThreads) qk_bwd_kernel(const __grid_constant__ QkParams p, int chunks) {
  constexpr int LANES = D / 8, PER = 32 / LANES, WARPS = kBwdThreads / 32, PASSES = 2;
  __shared__ __align__(16) float red[WARPS][2][D];
  __shared__ int last;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LANES, sub = lane / LANES;
  const int pq = (p.H[0] + PER - 1) / PER, pk = (p.H[1] + PER - 1) / PER;
  const Parts pt(l, p.rot, p.interleaved);
  const int64_t T = live_tokens(p);
  float dg[2][2][4];        // [q, k][part]
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) dg[w][0][e] = dg[w][1][e] = 0.f;
  // a warp takes PASSES passes of a token at a time
  const int step = (int)gridDim.x * WARPS;
  int unit = (int)blockIdx.x * WARPS + warp;
  for (int64_t t = unit / chunks; t < T; unit += step, t = unit / chunks) {
    const int i0 = (unit - (int)t * chunks) * PASSES;
    Raw4<TI> x0[PASSES], x1[PASSES], g0[PASSES], g1[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if (i0 + i >= pq + pk) break;
      const Pass ps(p, i0 + i, pq, PER, sub);
      const int head = ps.on ? ps.head : 0;
      const TI* gs = static_cast<const TI*>(p.g[ps.w]) + t * p.gs[ps.w][0] + head * p.gs[ps.w][1];
      g0[i] = fetch4(gs + pt.f0);
      g1[i] = fetch4(gs + pt.f1);
      if (p.norm) {
        const TI* xs = static_cast<const TI*>(p.x[ps.w]) + t * p.xs[ps.w][0] + head * p.xs[ps.w][1];
        x0[i] = fetch4(xs + pt.f0);
        x1[i] = fetch4(xs + pt.f1);
      }
    }
    float c[4], s[4];
    load_angles(p, pt, checked_position(p, t), l, -1.f, c, s);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if (i0 + i >= pq + pk) break;
      const Pass ps(p, i0 + i, pq, PER, sub);
      float a[4], b[4];
      unpack4(g0[i], a);
      unpack4(g1[i], b);
      if (pt.turns) turn_pairs(a, b, c, s, p.interleaved);
      if (p.norm) {
        float x[4], y[4], ga[4] = {1.f, 1.f, 1.f, 1.f}, gb[4] = {1.f, 1.f, 1.f, 1.f};
        unpack4(x0[i], x);
        unpack4(x1[i], y);
        if (p.gain[ps.w]) {
          load4(p.gain[ps.w] + pt.f0, ga);
          load4(p.gain[ps.w] + pt.f1, gb);
        }
        float ss = 0.f, se = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
          se = fmaf(a[e] * ga[e], x[e], fmaf(b[e] * gb[e], y[e], se));
        }
        ss = row_sum<LANES>(ss);
        se = row_sum<LANES>(se);
        const float rs = __frsqrt_rn(fmaf(ss, 1.f / D, p.eps));
        const float m = se * rs * (1.f / D);      // mean(e gain x r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = x[e] * rs, v = y[e] * rs;
          const float du = ps.on ? a[e] * u : 0.f, dv = ps.on ? b[e] * v : 0.f;
          if (ps.w) { dg[1][0][e] += du; dg[1][1][e] += dv; }
          else { dg[0][0][e] += du; dg[0][1][e] += dv; }
          a[e] = rs * fmaf(-u, m, a[e] * ga[e]);
          b[e] = rs * fmaf(-v, m, b[e] * gb[e]);
        }
      }
      if (ps.on) {
        TI* dst = static_cast<TI*>(p.out[ps.w]) + t * p.os[ps.w][0] + ps.head * p.os[ps.w][1];
        store4(dst + pt.f0, a);
        store4(dst + pt.f1, b);
      }
    }
  }
  if (!p.norm || (!p.dgain[0] && !p.dgain[1])) return;
  // lane groups of a warp, then the warps of the CTA, then the CTAs, each in a fixed order
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) dg[w][h][e] += __shfl_xor_sync(0xffffffffu, dg[w][h][e], o);
        if (lane < LANES) red[warp][w][(h ? pt.f1 : pt.f0) + e] = dg[w][h][e];
      }
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    const int w = threadIdx.x / D, i = threadIdx.x % D;
    float s = 0.f;
    for (int k = 0; k < WARPS; ++k) s += red[k][w][i];
    p.partial[((size_t)blockIdx.x * 2 + w) * D + i] = s;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(p.hdr + WS_NEXT, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // 2 D columns, the rows dealt to kBwdThreads / (2 D) groups, each group's sum in FP64
  double* dred = reinterpret_cast<double*>(&red[0][0][0]);   // WARPS * 2 * D floats >= kBwdThreads doubles
  static_assert(WARPS * 2 * D >= 2 * kBwdThreads, "the FP64 sums share the FP32 ones' space");
  constexpr int GROUPS = kBwdThreads / (2 * D);
  const int col = threadIdx.x % (2 * D), grp = threadIdx.x / (2 * D);
  double s = 0.0;
#pragma unroll 8
  for (int b = grp; b < (int)gridDim.x; b += GROUPS) s += (double)__ldcg(p.partial + (size_t)b * 2 * D + col);
  __syncthreads();
  dred[threadIdx.x] = s;
  __syncthreads();
  if (grp == 0) {
    for (int k = 1; k < GROUPS; ++k) s += dred[k * 2 * D + col];
    float* dst = p.dgain[col / D];
    if (dst) dst[col % D] = (float)s;
  }
  if (threadIdx.x == 0) p.hdr[WS_NEXT] = 0;   // ready for the workspace's next call
}

// grid of the backward: one CTA an SM
constexpr int kMaxBwdCtas = 256;

hstu_status_t check_qk_desc(const hstu_qk_desc* d, bool bwd) {
  if (!d || d->struct_size != sizeof(hstu_qk_desc)) return HSTU_ERR_INVALID_ARG;
  if (d->dtype != HSTU_BF16 && d->dtype != HSTU_FP32) return HSTU_ERR_INVALID_ARG;
  if (d->Hq < 0 || d->Hk < 0 || d->Hq + (int64_t)d->Hk < 1 || d->total_tokens < 0 || d->reserved != 0)
    return HSTU_ERR_INVALID_ARG;
  if ((d->interleaved & ~1) || (d->norm & ~1)) return HSTU_ERR_INVALID_ARG;
  if (d->norm && !(d->eps >= 0.f && d->eps < 1e30f)) return HSTU_ERR_INVALID_ARG;
  if (d->rot_dim < 0 || d->rot_dim > d->d || (d->rot_dim > 0 && d->max_position < 1)) return HSTU_ERR_INVALID_ARG;
  if (d->d != 32 && d->d != 64 && d->d != 128) return HSTU_ERR_UNSUPPORTED;
  if (d->rot_dim % 8 != 0) return HSTU_ERR_UNSUPPORTED;
  // units of work (tokens x passes) are counted in 32 bits
  if (d->Hq + (int64_t)d->Hk > 4096 || d->total_tokens > ((int64_t)1 << 30) / (d->Hq + (int64_t)d->Hk))
    return HSTU_ERR_UNSUPPORTED;
  const int64_t per = d->dtype == HSTU_BF16 ? 8 : 4;   // elements of 16 bytes
  const int64_t* all[6] = {d->q_strides, d->k_strides, d->q_out_strides, d->k_out_strides, d->dq_strides, d->dk_strides};
  for (int i = 0; i < (bwd ? 6 : 4); ++i) {
    if ((i % 2 ? d->Hk : d->Hq) == 0) continue;
    if (all[i][0] % per || all[i][1] % per) return HSTU_ERR_INVALID_ARG;
  }
  return HSTU_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

size_t qk_bwd_bytes(const hstu_qk_desc* d) { return kWsHeaderBytes + sizeof(float) * kMaxBwdCtas * 2 * (size_t)d->d; }

template <typename TI, int D, bool BWD>
cudaError_t launch_qk(const QkParams& p, int sms, cudaStream_t st) {
  constexpr int PER = 256 / D;
  const int passes = (p.H[0] + PER - 1) / PER + (p.H[1] + PER - 1) / PER;
  if constexpr (!BWD) {
    const dim3 grid((unsigned)((p.T + kQkThreads / 32 - 1) / (kQkThreads / 32)), (unsigned)((passes + kPasses - 1) / kPasses));
    return launch_pdl(qk_fwd_kernel<TI, D>, grid, dim3(kQkThreads), 0, st, p);
  } else {
    const int chunks = (passes + 1) / 2;
    int64_t ctas = (p.T * chunks + kBwdThreads / 32 - 1) / (kBwdThreads / 32);
    const int64_t most = sms < kMaxBwdCtas ? sms : kMaxBwdCtas;
    if (ctas > most) ctas = most;
    if (ctas < 1) ctas = 1;
    return launch_pdl(qk_bwd_kernel<TI, D>, dim3((unsigned)ctas), dim3(kBwdThreads), 0, st, p, chunks);
  }
}

template <bool BWD>
hstu_status_t dispatch_qk(const hstu_qk_desc* d, const QkParams& p, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) {
    if (d->dtype == HSTU_BF16)
      e = d->d == 128 ? launch_qk<__nv_bfloat16, 128, BWD>(p, sms, st)
                      : (d->d == 64 ? launch_qk<__nv_bfloat16, 64, BWD>(p, sms, st)
                                    : launch_qk<__nv_bfloat16, 32, BWD>(p, sms, st));
    else
      e = d->d == 128 ? launch_qk<float, 128, BWD>(p, sms, st)
                      : (d->d == 64 ? launch_qk<float, 64, BWD>(p, sms, st) : launch_qk<float, 32, BWD>(p, sms, st));
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_error_detail(e, BWD ? "launching qk_bwd_kernel" : "launching qk_fwd_kernel");
    return HSTU_ERR_CUDA;
  }
  note_launches(1);
  return HSTU_OK;
}

void copy_strides(int64_t (&dst)[2], const int64_t (&src)[2]) {
  dst[0] = src[0];
  dst[1] = src[1];
}

template <typename A>
hstu_status_t fill_common(const hstu_qk_desc* d, const A* a, void* ws, size_t bytes, size_t need, QkParams& p) {
  if (d->rot_dim > 0 && d->total_tokens > 0 && (!a->positions || !a->cos || !a->sin)) return HSTU_ERR_INVALID_ARG;
  if (!d->norm && (a->q_gain || a->k_gain)) return HSTU_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)a->cos, (const void*)a->sin, (const void*)a->q_gain, (const void*)a->k_gain, a->q, a->k})
    if (ptr && !aligned16(ptr)) return HSTU_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) || bytes < need) return HSTU_ERR_WORKSPACE;
  p.num_tokens = a->num_tokens;
  p.positions = a->positions; p.cos = a->cos; p.sin = a->sin;
  p.gain[0] = a->q_gain; p.gain[1] = a->k_gain;
  p.x[0] = a->q; p.x[1] = a->k;
  copy_strides(p.xs[0], d->q_strides); copy_strides(p.xs[1], d->k_strides);
  p.hdr = static_cast<int*>(ws);
  p.T = d->total_tokens; p.max_pos = d->max_position;
  p.H[0] = d->Hq; p.H[1] = d->Hk;
  p.rot = d->rot_dim; p.interleaved = d->interleaved; p.norm = d->norm; p.eps = d->eps;
  return HSTU_OK;
}

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_qk_workspace_size(const hstu_qk_desc* desc, size_t* fwd_bytes, size_t* bwd_bytes) {
  const hstu_status_t s = check_qk_desc(desc, false);
  if (s != HSTU_OK) return s;
  if (fwd_bytes) *fwd_bytes = kWsHeaderBytes;
  if (bwd_bytes) *bwd_bytes = qk_bwd_bytes(desc);
  return HSTU_OK;
}

hstu_status_t hstu_qk_norm_rope_fwd(const hstu_qk_desc* d, const hstu_qk_fwd_args* a, void* workspace,
                                    size_t workspace_bytes, hstu_stream_t stream) {
  hstu_status_t s = check_qk_desc(d, false);
  if (s != HSTU_OK) return s;
  if (!a || (d->total_tokens > 0 && ((d->Hq > 0 && (!a->q || !a->q_out)) || (d->Hk > 0 && (!a->k || !a->k_out)))))
    return HSTU_ERR_INVALID_ARG;
  if ((a->q_out && !aligned16(a->q_out)) || (a->k_out && !aligned16(a->k_out))) return HSTU_ERR_INVALID_ARG;
  QkParams p{};
  if ((s = fill_common(d, a, workspace, workspace_bytes, kWsHeaderBytes, p)) != HSTU_OK) return s;
  p.out[0] = a->q_out; p.out[1] = a->k_out;
  copy_strides(p.os[0], d->q_out_strides); copy_strides(p.os[1], d->k_out_strides);
  reset_launches();
  if (d->total_tokens == 0) return HSTU_OK;
  return dispatch_qk<false>(d, p, reinterpret_cast<cudaStream_t>(stream));
}

hstu_status_t hstu_qk_norm_rope_bwd(const hstu_qk_desc* d, const hstu_qk_bwd_args* a, void* workspace,
                                    size_t workspace_bytes, hstu_stream_t stream) {
  hstu_status_t s = check_qk_desc(d, true);
  if (s != HSTU_OK) return s;
  // without the norm the gradient does not read q and k
  if (!a || (d->total_tokens > 0 &&
             ((d->Hq > 0 && (!a->dq_out || !a->dq || (d->norm && !a->q))) ||
              (d->Hk > 0 && (!a->dk_out || !a->dk || (d->norm && !a->k))))))
    return HSTU_ERR_INVALID_ARG;
  if (!d->norm && (a->d_q_gain || a->d_k_gain)) return HSTU_ERR_INVALID_ARG;
  for (const void* ptr : {a->dq_out, a->dk_out, (const void*)a->dq, (const void*)a->dk})
    if (ptr && !aligned16(ptr)) return HSTU_ERR_INVALID_ARG;
  QkParams p{};
  if ((s = fill_common(d, a, workspace, workspace_bytes, qk_bwd_bytes(d), p)) != HSTU_OK) return s;
  p.g[0] = a->dq_out; p.g[1] = a->dk_out;
  copy_strides(p.gs[0], d->q_out_strides); copy_strides(p.gs[1], d->k_out_strides);
  p.out[0] = a->dq; p.out[1] = a->dk;
  copy_strides(p.os[0], d->dq_strides); copy_strides(p.os[1], d->dk_strides);
  p.dgain[0] = a->d_q_gain; p.dgain[1] = a->d_k_gain;
  p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  reset_launches();
  if (d->total_tokens == 0 && !a->d_q_gain && !a->d_k_gain) return HSTU_OK;   // no token: the gains' gradients are zero
  return dispatch_qk<true>(d, p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
