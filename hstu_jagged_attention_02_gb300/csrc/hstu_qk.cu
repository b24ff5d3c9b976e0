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
// A warp takes a few passes of one token, all loads first; the token's cosines
// and sines are loaded once for them.  161,293 tokens, four heads of 128 of q and
// k, BF16: 114.8 us, 5.9 TB/s (87% of a copy's rate); 64 tokens: 3.3 us, a launch.
//
// The backward's gain gradients are sums over all tokens and heads.  The
// CTAs walk tokens and keep per-lane FP32 partial sums; the CTAs' rows of
// partial sums land in the workspace and the CTA that finishes last (a
// counter in the workspace's header) adds them up in row order, their rounding
// errors carried along, so the result does not depend on the order in which CTAs
// finish.  That last step takes 3 us of 31.5 for 16,410 tokens (3.3 TB/s); the walk
// waits for its loads and shuffles, 16 warps an SM at 126 registers, q's and k's
// rows side by side (one after the other: 35.5).  Copying rows ahead through
// shared memory, or 32 warps that hold either q or k, took 38 us.
#include <type_traits>

#include "hstu_internal.h"
#include "hstu_rows.cuh"

namespace hstu {

namespace {

constexpr int kQkThreads = 128;
constexpr int kBwdThreads = 512;
constexpr int kPasses = 2;   // 256 features each, of q and of k (161,293 tokens, single calls: 1 156 us, 2 119, 4 152)

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
__device__ __forceinline__ int checked_position(const QkParams& p, int64_t t) {
  const int pos = p.positions[t];
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

__device__ __forceinline__ Row8 load_gain(const float* gain, const Parts& pt) {
  Row8 g;
  if (gain) {
    g = Row8(fetch4(gain + pt.f0), fetch4(gain + pt.f1));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) g.v[e] = make_float2(1.f, 1.f);
  }
  return g;
}

// A warp takes one token, kPasses passes of q's heads and as many of k's.
template <typename TI, int D>
__global__ void __launch_bounds__(kQkThreads) qk_fwd_kernel(const __grid_constant__ QkParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
  const int64_t t = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
  if (t >= live_tokens(p)) return;
  const Parts pt(l, p.rot, p.interleaved);
  const int h0 = blockIdx.y * (kPasses * PER) + sub;
  int pos = 0;
  if (pt.turns) pos = checked_position(p, t);   // another load waits for it: first
  Raw4<TI> r0[2][kPasses], r1[2][kPasses];
  auto load = [&](auto W) {
    constexpr int w = decltype(W)::value;
    const TI* src = static_cast<const TI*>(p.x[w]) + t * p.xs[w][0];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (h0 + i * PER < p.H[w]) {
        const TI* row = src + (h0 + i * PER) * p.xs[w][1];
        r0[w][i] = fetch4(row + pt.f0);
        r1[w][i] = fetch4(row + pt.f1);
      }
    }
  };
  load(std::integral_constant<int, 0>());
  load(std::integral_constant<int, 1>());
  Angles an;
  if (pt.turns) {
    const int64_t at = (int64_t)pos * (p.rot >> 1) + 4 * l;
    an.load(p.cos + at, p.sin + at, 1.f);
  }
  auto work = [&](auto W) {
    constexpr int w = decltype(W)::value;
    if ((int)blockIdx.y * (kPasses * PER) >= p.H[w]) return;
    Row8 gain;
    if (p.norm) gain = load_gain(p.gain[w], pt);
    TI* dst = static_cast<TI*>(p.out[w]) + t * p.os[w][0];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if ((int)blockIdx.y * (kPasses * PER) + i * PER >= p.H[w]) break;
      Row8 x(r0[w][i], r1[w][i]);
      if (p.norm) {
        x.times(rsqrtf(fmaf(row_sum<LANES>(x.dot(x)), 1.f / D, p.eps)));
        x.times(gain);
      }
      if (pt.turns) an.turn(x, p.interleaved);
      if (h0 + i * PER < p.H[w]) {
        TI* row = dst + (h0 + i * PER) * p.os[w][1];
        store_part(row + pt.f0, x.v[0], x.v[1]);
        store_part(row + pt.f1, x.v[2], x.v[3]);
      }
    }
  };
  work(std::integral_constant<int, 0>());
  work(std::integral_constant<int, 1>());
}

// A warp takes one pass of q's heads and one of k's at a time.
template <typename TI, int D>
__global__ void __launch_bounds__(kBwdThreads) qk_bwd_kernel(const __grid_constant__ QkParams p, int chunks) {
  constexpr int LANES = D / 8, PER = 32 / LANES, WARPS = kBwdThreads / 32;
  // the warps' sums; at the end the groups' sums and errors
  constexpr int ROWS = 8 * kBwdThreads / (2 * D) > WARPS ? 8 * kBwdThreads / (2 * D) : WARPS;
  __shared__ __align__(16) float red[ROWS][2][D];
  __shared__ int last;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LANES, sub = lane / LANES;
  const Parts pt(l, p.rot, p.interleaved);
  const int64_t T = live_tokens(p);
  float2 dg[2][4];          // [q, k]: sums over this lane's features
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) dg[w][e] = make_float2(0.f, 0.f);
  // unit (t, r): pass r of token t
  const int step = (int)gridDim.x * WARPS, unit = (int)blockIdx.x * WARPS + warp;
  const int dt = step / chunks, dr = step - dt * chunks;
  int64_t t = unit / chunks;
  int r = unit - (int)t * chunks;
  while (t < T) {
    const int h = r * PER + sub;
    Raw4<TI> x0[2], x1[2], g0[2], g1[2];
    auto load = [&](auto W) {
      constexpr int w = decltype(W)::value;
      if (h < p.H[w]) {
        const TI* gs = static_cast<const TI*>(p.g[w]) + t * p.gs[w][0] + h * p.gs[w][1];
        g0[w] = fetch4(gs + pt.f0);
        g1[w] = fetch4(gs + pt.f1);
        if (p.norm) {
          const TI* xs = static_cast<const TI*>(p.x[w]) + t * p.xs[w][0] + h * p.xs[w][1];
          x0[w] = fetch4(xs + pt.f0);
          x1[w] = fetch4(xs + pt.f1);
        }
      }
    };
    load(std::integral_constant<int, 0>());
    load(std::integral_constant<int, 1>());
    Angles an;
    if (pt.turns) {
      const int64_t at = (int64_t)checked_position(p, t) * (p.rot >> 1) + 4 * l;
      an.load(p.cos + at, p.sin + at, -1.f);
    }
    // q's rows (1), k's (2) or both (3): side by side, so that their sums' shuffles overlap
    auto work = [&](auto WHICH) {
      constexpr int W0 = decltype(WHICH)::value == 2 ? 1 : 0, W1 = decltype(WHICH)::value == 1 ? 1 : 2;
      Row8 g[2];
#pragma unroll
      for (int w = W0; w < W1; ++w) {
        g[w] = Row8(g0[w], g1[w]);
        if (pt.turns) an.turn(g[w], p.interleaved);
      }
      if (p.norm) {
        Row8 x[2], e[2];
        float ss[2], se[2];
#pragma unroll
        for (int w = W0; w < W1; ++w) {
          x[w] = Row8(x0[w], x1[w]);
          e[w] = g[w];
          e[w].times(load_gain(p.gain[w], pt));
          ss[w] = x[w].dot(x[w]);
          se[w] = x[w].dot(e[w]);
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
          for (int w = W0; w < W1; ++w) {
            ss[w] += __shfl_xor_sync(0xffffffffu, ss[w], o);
            se[w] += __shfl_xor_sync(0xffffffffu, se[w], o);
          }
#pragma unroll
        for (int w = W0; w < W1; ++w) {
          const float rs = rsqrtf(fmaf(ss[w], 1.f / D, p.eps));
          const float m = -se[w] * rs * (1.f / D);      // - mean(e gain x r)
          const bool on = h < p.H[w];
          x[w].times(rs);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (on) dg[w][i] = __ffma2_rn(g[w].v[i], x[w].v[i], dg[w][i]);
            g[w].v[i] = __fmul2_rn(__ffma2_rn(x[w].v[i], make_float2(m, m), e[w].v[i]), make_float2(rs, rs));
          }
        }
      }
#pragma unroll
      for (int w = W0; w < W1; ++w) {
        if (h < p.H[w]) {
          TI* dst = static_cast<TI*>(p.out[w]) + t * p.os[w][0] + h * p.os[w][1];
          store_part(dst + pt.f0, g[w].v[0], g[w].v[1]);
          store_part(dst + pt.f1, g[w].v[2], g[w].v[3]);
        }
      }
    };
    if (r * PER < min(p.H[0], p.H[1])) work(std::integral_constant<int, 3>());
    else if (r * PER < p.H[0]) work(std::integral_constant<int, 1>());
    else work(std::integral_constant<int, 2>());
    t += dt;
    r += dr;
    if (r >= chunks) {
      r -= chunks;
      ++t;
    }
  }
  if (!p.norm || (!p.dgain[0] && !p.dgain[1])) return;
  // lane groups of a warp, then the warps of the CTA, then the CTAs, each in a fixed order
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) {
        dg[w][e].x += __shfl_xor_sync(0xffffffffu, dg[w][e].x, o);
        dg[w][e].y += __shfl_xor_sync(0xffffffffu, dg[w][e].y, o);
      }
      if (lane < LANES) *reinterpret_cast<float2*>(&red[warp][w][(e < 2 ? pt.f0 : pt.f1) + 2 * (e & 1)]) = dg[w][e];
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
  // 2 D columns, 4 a thread, the rows dealt to kBwdThreads / (D / 2) groups with
  // all of a group's loads under way together; every sum carries its rounding
  // errors along (two-sum), as FP64 has a 64th of the rate
  constexpr int QUADS = D / 2, GROUPS = kBwdThreads / QUADS, DEEP = D == 128 ? 20 : (D == 64 ? 10 : 5);
  const int quad = threadIdx.x % QUADS, grp = threadIdx.x / QUADS;
  auto add = [](float& sum, float& err, float v) {
    const float s = sum + v, back = s - sum;
    err += (sum - (s - back)) + (v - back);
    sum = s;
  };
  float sum[4] = {}, err[4] = {};
  for (int b0 = grp; b0 < (int)gridDim.x; b0 += GROUPS * DEEP) {
    float4 v[DEEP];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (b0 + i * GROUPS < (int)gridDim.x)
        v[i] = __ldcg(reinterpret_cast<const float4*>(p.partial + (size_t)(b0 + i * GROUPS) * 2 * D) + quad);
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      add(sum[0], err[0], v[i].x); add(sum[1], err[1], v[i].y); add(sum[2], err[2], v[i].z); add(sum[3], err[3], v[i].w);
    }
  }
  float* sums = &red[0][0][0];            // [GROUPS][2 D] sums, then as many errors
  __syncthreads();
  *reinterpret_cast<float4*>(sums + grp * 2 * D + 4 * quad) = make_float4(sum[0], sum[1], sum[2], sum[3]);
  *reinterpret_cast<float4*>(sums + 4 * kBwdThreads + grp * 2 * D + 4 * quad) = make_float4(err[0], err[1], err[2], err[3]);
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    const int col = threadIdx.x;
    float s = 0.f, e = 0.f;
    for (int k = 0; k < GROUPS; ++k) {
      add(s, e, sums[k * 2 * D + col]);
      e += sums[4 * kBwdThreads + k * 2 * D + col];
    }
    float* dst = p.dgain[col / D];
    // of a sum that is not finite the errors are NaN (infinity less infinity): it stands as it is
    if (dst) dst[col % D] = fabsf(s) <= 3.4028234663852886e38f ? s + e : s;
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
  const int heads = p.H[0] > p.H[1] ? p.H[0] : p.H[1], passes = (heads + PER - 1) / PER;
  if constexpr (!BWD) {
    const dim3 grid((unsigned)((p.T + kQkThreads / 32 - 1) / (kQkThreads / 32)), (unsigned)((passes + kPasses - 1) / kPasses));
    return launch_pdl(qk_fwd_kernel<TI, D>, grid, dim3(kQkThreads), 0, st, p);
  } else {
    int64_t ctas = (p.T * passes + kBwdThreads / 32 - 1) / (kBwdThreads / 32);
    const int64_t most = sms < kMaxBwdCtas ? sms : kMaxBwdCtas;
    if (ctas > most) ctas = most;
    if (ctas < 1) ctas = 1;
    return launch_pdl(qk_bwd_kernel<TI, D>, dim3((unsigned)ctas), dim3(kBwdThreads), 0, st, p, passes);
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
