// Layer norm with weight and bias, backward (hstu_ln_bwd).
//
//   h = (x - mean) rstd, e = dy weight
//   dx = rstd (e - mean(e) - h mean(e h)) [+ dres];  d_weight = sum dy h, d_bias = sum dy
//
// HBM-bound: x and dy are read once, dx written once.  Teams (warps, or CTAs
// for wide rows) walk the rows and keep each feature's two sums in registers; a CTA
// adds its warps' sums in shared memory and leaves a row of 2 D sums in the
// workspace, and a second kernel adds these rows, column by column, in their
// order.
#include "hstu_ln.cuh"

namespace hstu {

namespace {

using namespace ln;

template <typename TX, typename TY, int V, int L, int N>
__global__ void __launch_bounds__(L == 32 ? 32 * kWarpTeams : L) ln_bwd_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ float sums[];   // warps' teams: [warps][2][D]
  __shared__ float2 red[2][L / 32];
  constexpr int TEAMS = L == 32 ? kWarpTeams : 1;
  pdl_wait();
  const int team = L == 32 ? threadIdx.x >> 5 : 0, l = threadIdx.x % L;
  const int64_t rows = live_rows(p), step = (int64_t)gridDim.x * TEAMS;
  float sw[N][V], sb[N][V];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) sw[i][e] = sb[i][e] = 0.f;
  const float inv = 1.f / (float)p.D;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * TEAMS + team; r < rows; r += step) {
    const TX* x = static_cast<const TX*>(p.x) + r * p.xs;
    const TY* dy = static_cast<const TY*>(p.dy) + r * p.ys;
    Pack<TX, V> rx[N];
    Pack<TY, V> rg[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = (i * L + l) * V;
      if (f < p.D) {
        rx[i].load(x + f);
        rg[i].load(dy + f);
      }
    }
    const float mean = p.mean[r], rstd = p.rstd[r];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = (i * L + l) * V;
      if (f < p.D) {
        float h[V], g[V], w[V];
        rx[i].get(h);
        rg[i].get(g);
        if (p.weight) {
          Pack<float, V> c;
          c.load(p.weight + f);
          c.get(w);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          h[e] = (h[e] - mean) * rstd;
          sw[i][e] = fmaf(g[e], h[e], sw[i][e]);
          sb[i][e] += g[e];
          const float t = p.weight ? g[e] * w[e] : g[e];
          s.x += t;
          s.y = fmaf(t, h[e], s.y);
        }
      }
    }
    s = team_sum<L>(s, red[turn]);
    turn ^= 1;
    const float m0 = s.x * inv, m1 = s.y * inv;
    TX* dx = static_cast<TX*>(p.dx) + r * p.dxs;
    const TX* dres = static_cast<const TX*>(p.dres) + r * p.drs;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = (i * L + l) * V;
      if (f < p.D) {
        float h[V], g[V], w[V], a[V];
        rx[i].get(h);
        rg[i].get(g);
        if (p.weight) {
          Pack<float, V> c;
          c.load(p.weight + f);
          c.get(w);
        }
        if (p.dres) {
          Pack<TX, V> c;
          c.load(dres + f);
          c.get(a);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float t = p.weight ? g[e] * w[e] : g[e];
          g[e] = rstd * (t - m0 - (h[e] - mean) * rstd * m1);
          if (p.dres) g[e] += a[e];
        }
        put(dx + f, g);
      }
    }
  }
  if (!p.d_weight && !p.d_bias) return;
  float* out = p.partial + (size_t)blockIdx.x * 2 * p.D;
  if constexpr (L == 32) {
    float* mine = sums + (size_t)team * 2 * p.D;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = (i * L + l) * V;
      if (f < p.D) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          mine[f + e] = sw[i][e];
          mine[p.D + f + e] = sb[i][e];
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.D; c += 32 * kWarpTeams) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWarpTeams; ++w) t += sums[(size_t)w * 2 * p.D + c];
      out[c] = t;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = (i * L + l) * V;
      if (f < p.D) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          out[f + e] = sw[i][e];
          out[p.D + f + e] = sb[i][e];
        }
      }
    }
  }
}

// d_weight and d_bias from `rows` rows of 2 D sums: 32 columns a CTA, its 8
// warps take every 8th row.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps)
ln_sum_kernel(const float* __restrict__ partial, int rows, int D, float* d_weight, float* d_bias) {
  __shared__ float red[kSumWarps][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int r = warp; r < rows; r += kSumWarps) s += __ldcg(partial + (size_t)r * 2 * D + c);
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * D) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) s += red[w][lane];
    if (c < D) {
      if (d_weight) d_weight[c] = s;
    } else if (d_bias) {
      d_bias[c - D] = s;
    }
  }
}

template <typename TX, typename TY>
cudaError_t launch_t(const LnParams& p, bool wide, int sms, cudaStream_t st) {
  return dispatch_shape(p.D, wide, [&](auto S) {
    using Sh = decltype(S);
    constexpr int TEAMS = Sh::l == 32 ? kWarpTeams : 1;
    auto kern = ln_bwd_kernel<TX, TY, Sh::v, Sh::l, Sh::n>;
    int64_t ctas = (p.rows + TEAMS - 1) / TEAMS;
    const int64_t most = 2 * (int64_t)sms < kLnMaxBwdCtas ? 2 * (int64_t)sms : kLnMaxBwdCtas;
    if (ctas > most) ctas = most;
    if (ctas < 1) ctas = 1;
    const size_t smem = Sh::l == 32 ? sizeof(float) * kWarpTeams * 2 * (size_t)p.D : 0;
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_pdl(kern, dim3((unsigned)ctas), dim3(Sh::l == 32 ? 32 * kWarpTeams : Sh::l), smem, st, p);
    if (e != cudaSuccess || (!p.d_weight && !p.d_bias)) return e;
    return launch_pdl(ln_sum_kernel, dim3((unsigned)((2 * p.D + 31) / 32)), dim3(32 * kSumWarps), 0, st,
                      (const float*)p.partial, (int)ctas, p.D, p.d_weight, p.d_bias);
  });
}

}  // namespace

cudaError_t launch_ln_bwd(const LnParams& p, int x_dtype, int y_dtype, bool wide, int sms, cudaStream_t st) {
  if (x_dtype == HSTU_BF16)
    return y_dtype == HSTU_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(p, wide, sms, st)
                                : launch_t<__nv_bfloat16, float>(p, wide, sms, st);
  return y_dtype == HSTU_BF16 ? launch_t<float, __nv_bfloat16>(p, wide, sms, st) : launch_t<float, float>(p, wide, sms, st);
}

}  // namespace hstu
