// Norm and rotation of queries and keys per head (hstu_qk_norm_rope_*).
//
//   r = 1 / sqrt(mean(x^2) + eps), w = x r gain, each pair of w turned by the
//   angle of the token's position; backward: the incoming gradient turned
//   back, e = dout R^T, then dgain += e x r and dx = r (e g - x r mean(e g x r)).
//
// HBM-bound: every row of d features is read once (backward: twice, x and
// dout) and written once, in a handful of FP32 operations a feature.  So a
// lane holds 4 neighbouring features (8 bytes BF16, 16 bytes FP32), d / 4
// lanes hold a row, and a warp has kRows rows of one token in flight: the
// tables' 4 cosines and sines are loaded once for all of them.  The row's sum
// goes over d / 4 lanes by shuffles.  Pairs of halves sit rot_dim / 8 lanes
// apart (4 shuffles a row), neighbouring pairs in the lane itself.
//
// The backward's gain gradients are sums over all tokens and heads.  One CTA
// an SM walks tokens and keeps per-lane FP32 partial sums; the CTAs' rows of
// partial sums land in the workspace and the CTA that finishes last (a
// counter in the workspace's header) adds them up in row order in FP64, so
// the result does not depend on the order in which CTAs finish.
#include "hstu_internal.h"
#include "hstu_vec.cuh"

namespace hstu {

namespace {

constexpr int kQkThreads = 256;
constexpr int kBwdThreads = 512;

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

// The 4 cosines and sines of a lane's features [f, f + 4), already signed for
// the turn: out = w * c + partner * s.
struct Turn {
  float c[4], s[4];
};

// dir +1 turns by the position's angle, -1 back (the backward).
__device__ __forceinline__ Turn load_turn(const QkParams& p, int64_t pos, int f, float dir) {
  Turn t;
  if (f >= p.rot) {
#pragma unroll
    for (int e = 0; e < 4; ++e) { t.c[e] = 1.f; t.s[e] = 0.f; }
    return t;
  }
  const int half = p.rot >> 1;
  const float* cr = p.cos + pos * half;
  const float* sr = p.sin + pos * half;
  if (p.interleaved) {
    const float2 c = *reinterpret_cast<const float2*>(cr + (f >> 1));
    const float2 s = *reinterpret_cast<const float2*>(sr + (f >> 1));
    t.c[0] = t.c[1] = c.x; t.c[2] = t.c[3] = c.y;
    t.s[0] = -dir * s.x; t.s[1] = dir * s.x; t.s[2] = -dir * s.y; t.s[3] = dir * s.y;
  } else {
    const bool second = f >= half;
    const int i = second ? f - half : f;
    const float4 c = *reinterpret_cast<const float4*>(cr + i);
    const float4 s = *reinterpret_cast<const float4*>(sr + i);
    const float g = second ? dir : -dir;
    t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
    t.s[0] = g * s.x; t.s[1] = g * s.y; t.s[2] = g * s.z; t.s[3] = g * s.w;
  }
  return t;
}

// w turned in place; every lane of the warp takes part
__device__ __forceinline__ void turn(const Turn& t, bool interleaved, int partner, float (&w)[4]) {
  float o[4];
  if (interleaved) {
    o[0] = w[1]; o[1] = w[0]; o[2] = w[3]; o[3] = w[2];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(0xffffffffu, w[e], partner);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = fmaf(w[e], t.c[e], o[e] * t.s[e]);
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane that holds the other halves of this lane's pairs.
template <int LANES>
__device__ __forceinline__ int partner_lane(int lane, int rot) {
  const int l = lane % LANES, h = rot >> 3;   // 4 features a lane
  return lane - l + (l < h ? l + h : (l < 2 * h ? l - h : l));
}

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

// A warp takes kRows x (128 / D) heads of one token.
template <typename TI, int D, int kRows>
__global__ void __launch_bounds__(kQkThreads) qk_fwd_kernel(const __grid_constant__ QkParams p, int chunks) {
  constexpr int LANES = D / 4, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / chunks;
  const int first = (int)(unit - t * chunks) * kRows * PER;
  const int heads = p.H[0] + p.H[1];
  if (t >= live_tokens(p)) return;
  const int f = (lane % LANES) * 4;
  float x[kRows][4];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int hh = first + r * PER + lane / LANES;
    const int w = hh >= p.H[0];
    if (hh < heads)
      load4(static_cast<const TI*>(p.x[w]) + t * p.xs[w][0] + (int64_t)(hh - (w ? p.H[0] : 0)) * p.xs[w][1] + f, x[r]);
    else
      x[r][0] = x[r][1] = x[r][2] = x[r][3] = 0.f;
  }
  const Turn tn = load_turn(p, checked_position(p, t), f, 1.f);
  const int partner = partner_lane<LANES>(lane, p.rot);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int hh = first + r * PER + lane / LANES;
    const int w = hh >= p.H[0];
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(x[r][e], x[r][e], ss);
      const float rs = __frsqrt_rn(fmaf(lanes_sum<LANES>(ss), 1.f / D, p.eps));
      float g[4] = {1.f, 1.f, 1.f, 1.f};
      if (p.gain[w]) load4(p.gain[w] + f, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[r][e] = x[r][e] * rs * g[e];
    }
    if (p.rot) turn(tn, p.interleaved, partner, x[r]);
    if (hh < heads)
      store4(static_cast<TI*>(p.out[w]) + t * p.os[w][0] + (int64_t)(hh - (w ? p.H[0] : 0)) * p.os[w][1] + f, x[r]);
  }
}

template <typename TI, int D, int kRows>
__global__ void __launch_bounds__(kBwdThreads) qk_bwd_kernel(const __grid_constant__ QkParams p, int chunks) {
  constexpr int LANES = D / 4, PER = 32 / LANES, WARPS = kBwdThreads / 32;
  __shared__ __align__(16) float red[WARPS][2][D];
  __shared__ int last;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int f = (lane % LANES) * 4;
  const int heads = p.H[0] + p.H[1];
  const int partner = partner_lane<LANES>(lane, p.rot);
  const int64_t units = live_tokens(p) * chunks;
  float gain[2][4], dg[2][4];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) { gain[w][e] = 1.f; dg[w][e] = 0.f; }
    if (p.norm && p.gain[w]) load4(p.gain[w] + f, gain[w]);
  }
  for (int64_t unit = (int64_t)blockIdx.x * WARPS + warp; unit < units; unit += (int64_t)gridDim.x * WARPS) {
    const int64_t t = unit / chunks;
    const int first = (int)(unit - t * chunks) * kRows * PER;
    float x[kRows][4], g[kRows][4];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int hh = first + r * PER + lane / LANES;
      const int w = hh >= p.H[0], h = hh - (w ? p.H[0] : 0);
      if (hh < heads) {
        load4(static_cast<const TI*>(p.g[w]) + t * p.gs[w][0] + (int64_t)h * p.gs[w][1] + f, g[r]);
        if (p.norm) load4(static_cast<const TI*>(p.x[w]) + t * p.xs[w][0] + (int64_t)h * p.xs[w][1] + f, x[r]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[r][e] = g[r][e] = 0.f;
      }
    }
    const Turn tn = load_turn(p, checked_position(p, t), f, -1.f);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int hh = first + r * PER + lane / LANES;
      const int w = hh >= p.H[0];
      if (p.rot) turn(tn, p.interleaved, partner, g[r]);
      if (p.norm) {
        float ss = 0.f, se = 0.f;
        float eg[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          eg[e] = g[r][e] * (w ? gain[1][e] : gain[0][e]);
          ss = fmaf(x[r][e], x[r][e], ss);
          se = fmaf(eg[e], x[r][e], se);
        }
        ss = lanes_sum<LANES>(ss);
        se = lanes_sum<LANES>(se);
        const float rs = __frsqrt_rn(fmaf(ss, 1.f / D, p.eps));
        const float m = se * rs * (1.f / D);      // mean(e gain x r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float xr = x[r][e] * rs;
          const float add = g[r][e] * xr;
          dg[0][e] += w ? 0.f : add;
          dg[1][e] += w ? add : 0.f;
          g[r][e] = rs * fmaf(-xr, m, eg[e]);
        }
      }
      if (hh < heads)
        store4(static_cast<TI*>(p.out[w]) + t * p.os[w][0] + (int64_t)(hh - (w ? p.H[0] : 0)) * p.os[w][1] + f, g[r]);
    }
  }
  if (!p.norm || (!p.dgain[0] && !p.dgain[1])) return;
  // lane groups of a warp, then the warps of the CTA, then the CTAs, each in a fixed order
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) dg[w][e] += __shfl_xor_sync(0xffffffffu, dg[w][e], o);
      if (lane < LANES) red[warp][w][f + e] = dg[w][e];
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
  // the grid counts chunks of at least 4 rows, 8 a CTA
  if (d->Hq + (int64_t)d->Hk > 4096 || d->total_tokens > ((int64_t)1 << 32) ||
      d->total_tokens * (d->Hq + (int64_t)d->Hk) > ((int64_t)1 << 33))
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

// every kernel variant's launch: kRows rows of a token in flight a warp
template <typename TI, int D, bool BWD>
cudaError_t launch_qk(const QkParams& p, int sms, cudaStream_t st) {
  constexpr int PER = 128 / D;
  const int heads = p.H[0] + p.H[1];
  if constexpr (!BWD) {
    constexpr int R = 4;
    const int chunks = (heads + R * PER - 1) / (R * PER);
    const int64_t ctas = (p.T * chunks + kQkThreads / 32 - 1) / (kQkThreads / 32);
    return launch_pdl(qk_fwd_kernel<TI, D, R>, dim3((unsigned)ctas), dim3(kQkThreads), 0, st, p, chunks);
  } else {
    constexpr int R = 4;
    const int chunks = (heads + R * PER - 1) / (R * PER);
    int64_t ctas = (p.T * chunks + kBwdThreads / 32 - 1) / (kBwdThreads / 32);
    const int64_t most = sms < kMaxBwdCtas ? sms : kMaxBwdCtas;
    if (ctas > most) ctas = most;
    if (ctas < 1) ctas = 1;
    return launch_pdl(qk_bwd_kernel<TI, D, R>, dim3((unsigned)ctas), dim3(kBwdThreads), 0, st, p, chunks);
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
