// Layer norm with weight and bias, backward (hstu_ln_bwd).
//
//   h = (x - mean) rstd, e = dy weight
//   dx = rstd (e - mean(e) - h mean(e h)) [+ dres];  d_weight = sum dy h, d_bias = sum dy
//
// HBM-bound: x and dy are read once, dx written once.  Teams (a warp, or up to a CTA
// for wide rows) walk the rows and keep each feature's two sums in registers; a CTA
// adds its teams' sums in shared memory and leaves a row of 2 D sums in the
// workspace, and a second kernel adds these rows, column by column, in their
// order.
//
// 16,410 rows of 512, BF16: 14.2 us (floor 7.5), of which the second kernel takes 3: 16 warps an SM, whose lanes' sums
// and rows fill 128 registers, wait for loads (a third of the stalls) and shuffles.  4,099 FP32 rows of 301: 5.6 us, two launches.
// Teams of 64 lanes with half of the sums each were slower (20 us); narrow rows want more of them than a warp
// gives: 107,181 rows of 89 took 31 us with a warp a row, 12 us with 16 lanes.  Rows that are not 16-byte aligned hold 16
// single features a lane up to 8,192 (2,000 FP32 rows of 5,001 48 us, with 32 a lane 88 and more).
#include "hstu_ln.cuh"

namespace hstu {

namespace {

using namespace ln;

// A CTA an SM, cut into teams of 8 to 512 threads: 16 warps leave 128 registers a thread, of which a lane's sums
// take 2 N V.  Short rows are read one ahead of the row that is worked on, and keep the weight in registers.
constexpr int kBwdThreads = 512;

// Sums of two values over a team of L threads, which has the barrier team + 1 and red for itself.
template <int L>
__device__ __forceinline__ float2 team_sum_of(float2 v, float2* red, int team) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (L > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x % L >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(L) : "memory");
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < L / 32; ++w) {
      v.x += red[w].x;
      v.y += red[w].y;
    }
  }
  return v;
}

template <typename TX, typename TY, int V, int L, int N>
__global__ void __launch_bounds__(kBwdThreads, 1) ln_bwd_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ float sums[];   // [teams][2][D]
  constexpr int TEAMS = kBwdThreads / L, E = N * V;
  static_assert(E % 2 == 0, "features are worked on in pairs");
  __shared__ float2 red[2][L <= 32 ? 1 : TEAMS][L <= 32 ? 1 : L / 32];
  // registers of a row as it is read.  Up to 16 features a lane h, dy weight and the weight stay in registers beside the sums
  // (5 E), and the next row is read ahead where that leaves room for it; beyond, a row is computed twice
  constexpr int RAW = N * (V == 1 ? 2 : (int)(sizeof(TX) + sizeof(TY)) * 2);
  constexpr bool TWICE = E > 16, AHEAD = !TWICE && 5 * E + RAW <= 100;
  pdl_wait();
  const int team = threadIdx.x / L, l = threadIdx.x % L;
  const int64_t rows = live_rows(p), step = (int64_t)gridDim.x * TEAMS;
  auto at = [&](int i) { return (i * L + l) * V; };   // first of the lane's features in part i
  // features behind D count as zeros: of dy and of the weight
  float2 sw[E / 2], sb[E / 2], kept[TWICE ? 1 : E / 2];
#pragma unroll
  for (int k = 0; k < E / 2; ++k) sw[k] = sb[k] = make_float2(0.f, 0.f);
  auto weight = [&](float2 (&w)[E / 2]) {
    float a[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) a[i][e] = at(i) < p.D ? 1.f : 0.f;
      if (p.weight && at(i) < p.D) {
        Pack<float, V> c;
        c.load(p.weight + at(i));
        c.get(a[i]);
      }
    }
#pragma unroll
    for (int k = 0; k < E / 2; ++k) w[k] = make_float2(a[2 * k / V][2 * k % V], a[(2 * k + 1) / V][(2 * k + 1) % V]);
  };
  if constexpr (!TWICE) weight(kept);
  const float inv = 1.f / (float)p.D;
  int turn = 0;
  Pack<TX, V> rx[N];
  Pack<TY, V> rg[N];
  float mean = 0.f, rstd = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    rx[i] = Pack<TX, V>();
    rg[i] = Pack<TY, V>();
  }
  auto fetch = [&](int64_t r) {
    if (r >= rows) return;
    const TX* x = static_cast<const TX*>(p.x) + r * p.xs;
    const TY* dy = static_cast<const TY*>(p.dy) + r * p.ys;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (at(i) < p.D) {
        rx[i].load(x + at(i));
        rg[i].load(dy + at(i));
      }
    }
    mean = p.mean[r];
    rstd = p.rstd[r];
  };
  int64_t r = (int64_t)blockIdx.x * TEAMS + team;
  fetch(r);
  // (the teams of a warp go on together: one without a row has zeros for dy and stores nothing)
  const int ahead = L < 32 ? (threadIdx.x & 31) / L : 0;
  for (; r - ahead < rows; r += step) {
    const int D = L >= 32 || r < rows ? p.D : 0;
    if (L < 32 && D == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        rx[i] = Pack<TX, V>();
        rg[i] = Pack<TY, V>();
      }
      mean = rstd = 0.f;
    }
    TX* dx = static_cast<TX*>(p.dx) + r * p.dxs;
    const TX* dres = static_cast<const TX*>(p.dres) + r * p.drs;
    auto store = [&](int i, float (&o)[V]) {
      if (p.dres) {
        Pack<TX, V> c;
        float add[V];
        c.load(dres + at(i));
        c.get(add);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] += add[e];
      }
      put(dx + at(i), o);
    };
    const float mean_r = mean, rstd_r = rstd;
    // h = x rstd - mean rstd with that product in two parts: rounded to one it would leave 2^-24 of |mean| rstd where rows
    // lie far from zero (as near as (x - mean) rstd, and 140 us for 163 with 161,293 rows of 512, FP32 and BF16)
    const float sh = -mean_r * rstd_r, sl = fmaf(-mean_r, rstd_r, -sh);
    const float2 scale = make_float2(rstd_r, rstd_r), shift = make_float2(sh, sh), low = make_float2(sl, sl);
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
    if constexpr (!TWICE) {
      float2 h[E / 2], t[E / 2];   // x, dy; then h and t = dy weight
      {
        float x[N][V], g[N][V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          rx[i].get(x[i]);
          rg[i].get(g[i]);
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          h[k] = make_float2(x[2 * k / V][2 * k % V], x[(2 * k + 1) / V][(2 * k + 1) % V]);
          t[k] = make_float2(g[2 * k / V][2 * k % V], g[(2 * k + 1) / V][(2 * k + 1) % V]);
        }
      }
      if constexpr (AHEAD) fetch(r + step);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        h[k] = __fadd2_rn(__ffma2_rn(h[k], scale, shift), low);
        sw[k] = __ffma2_rn(t[k], h[k], sw[k]);
        sb[k] = __fadd2_rn(sb[k], t[k]);
        t[k] = __fmul2_rn(t[k], kept[k]);
        s0 = __fadd2_rn(s0, t[k]);
        s1 = __ffma2_rn(t[k], h[k], s1);
      }
      const float2 s = team_sum_of<L>(make_float2(s0.x + s0.y, s1.x + s1.y), red[turn][L <= 32 ? 0 : team], team);
      // dx = rstd (t - m0 - h m1)
      const float a1 = -s.y * inv * rstd_r, b1 = -s.x * inv * rstd_r;
      const float2 a = make_float2(a1, a1), b = make_float2(b1, b1);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) t[k] = __ffma2_rn(t[k], scale, __ffma2_rn(h[k], a, b));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (at(i) < D) {
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = (i * V + e) % 2 ? t[(i * V + e) / 2].y : t[(i * V + e) / 2].x;
          store(i, o);
        }
      }
    } else {
      // rows whose sums fill the registers: h and t are computed twice from what was read (single features behind D as
      // zeros of the weight, without a branch, and read-only loads, so that the weight's go together and before stores)
      auto part = [&](int i, float (&h)[V], float (&g)[V], float (&t)[V]) {
        rx[i].get(h);
        rg[i].get(g);
        if constexpr (V == 1) {
          t[0] = p.weight && at(i) < D ? __ldg(p.weight + at(i)) : 0.f;
        } else if (p.weight) {
          Pack<float, V> c;
          c.load(p.weight + at(i));
          c.get(t);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          h[e] = (h[e] - mean_r) * rstd_r;
          t[e] = p.weight ? g[e] * t[e] : g[e];
        }
      };
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (V == 1 || at(i) < D) {
          float h[V], g[V], t[V];
          part(i, h, g, t);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const int k = (i * V + e) / 2;
            float& cw = (i * V + e) % 2 ? sw[k].y : sw[k].x;
            float& cb = (i * V + e) % 2 ? sb[k].y : sb[k].x;
            cw = fmaf(g[e], h[e], cw);
            cb += g[e];
            s.x += t[e];
            s.y = fmaf(t[e], h[e], s.y);
          }
        }
      }
      s = team_sum_of<L>(s, red[turn][L <= 32 ? 0 : team], team);
      const float a = -s.y * inv * rstd_r, b = -s.x * inv * rstd_r;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (at(i) < D) {
          float h[V], g[V], t[V];
          part(i, h, g, t);
#pragma unroll
          for (int e = 0; e < V; ++e) t[e] = fmaf(t[e], rstd_r, fmaf(h[e], a, b));
          store(i, t);
        }
      }
    }
    turn ^= 1;
    if constexpr (!AHEAD) fetch(r + step);
  }
  if (!p.d_weight && !p.d_bias) return;
  float* out = p.partial + (size_t)blockIdx.x * 2 * p.D;
  float* mine = TEAMS > 1 ? sums + (size_t)team * 2 * p.D : out;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int f = (i * L + l) * V;
    if (f < p.D) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 a = sw[(i * V + e) / 2], b = sb[(i * V + e) / 2];
        mine[f + e] = (i * V + e) % 2 ? a.y : a.x;
        mine[p.D + f + e] = (i * V + e) % 2 ? b.y : b.x;
      }
    }
  }
  if constexpr (TEAMS > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.D; c += kBwdThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < TEAMS; ++w) t += sums[(size_t)w * 2 * p.D + c];
      out[c] = t;
    }
  }
}

// d_weight and d_bias from `rows` (at most kLnMaxBwdCtas) rows of 2 D sums: 32 columns a CTA,
// its 16 warps take every 16th row, all of a warp's loads under way together.
constexpr int kSumWarps = 16, kSumDeep = (kLnMaxBwdCtas + kSumWarps - 1) / kSumWarps;
__global__ void __launch_bounds__(32 * kSumWarps)
ln_sum_kernel(const float* __restrict__ partial, int rows, int D, float* d_weight, float* d_bias) {
  __shared__ float red[kSumWarps][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v[kSumDeep];
#pragma unroll
  for (int i = 0; i < kSumDeep; ++i) {
    const int r = warp + i * kSumWarps;
    v[i] = r < rows && c < 2 * D ? __ldcg(partial + (size_t)r * 2 * D + c) : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumDeep; ++i) s += v[i];
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

// SHORT (both sides BF16): a row's 16 features a lane leave room for the next row's, and smaller teams have more rows under
// way (16,000 rows of 1,024 22.3 us against 26.5, of 2,048 38.9 against 47.6; 8,000 of 4,096 40.1 against 52.4).  With
// an FP32 side there is none, and 8 features a lane are ahead (8,000 FP32 rows of 4,096 73.4 us against 84.1).
template <bool SHORT, typename F>
auto dispatch_bwd_shape(int D, bool wide, F&& go) {
  if (wide) {
    if (D <= 64) return go(Shape<8, 8, 1>());
    if (D <= 128) return go(Shape<8, 16, 1>());
    if (D <= 256) return go(Shape<8, 32, 1>());
    if (D <= 512) return go(Shape<8, 32, 2>());
    if constexpr (SHORT) {
      if (D <= 1024) return go(Shape<8, 64, 2>());
      if (D <= 2048) return go(Shape<8, 128, 2>());
      if (D <= 4096) return go(Shape<8, 256, 2>());
    } else {
      if (D <= 1024) return go(Shape<8, 128, 1>());
      if (D <= 2048) return go(Shape<8, 256, 1>());
      if (D <= 4096) return go(Shape<8, 512, 1>());
    }
    if (D <= 8192) return go(Shape<8, 512, 2>());
    return go(Shape<8, 512, 4>());
  }
  if (D <= 32) return go(Shape<1, 8, 4>());
  if (D <= 128) return go(Shape<1, 16, 8>());
  if (D <= 320) return go(Shape<1, 32, 10>());
  if (D <= 1024) return go(Shape<1, 128, 8>());
  if (D <= 4096) return go(Shape<1, 512, 8>());
  if (D <= 8192) return go(Shape<1, 512, 16>());
  return go(Shape<1, 512, 32>());
}

template <typename TX, typename TY>
cudaError_t launch_t(const LnParams& p, bool wide, int sms, cudaStream_t st) {
  return dispatch_bwd_shape<sizeof(TX) + sizeof(TY) == 4>(p.D, wide, [&](auto S) {
    using Sh = decltype(S);
    constexpr int TEAMS = kBwdThreads / Sh::l;
    auto kern = ln_bwd_kernel<TX, TY, Sh::v, Sh::l, Sh::n>;
    int64_t ctas = (p.rows + TEAMS - 1) / TEAMS;
    const int64_t limit = sms < kLnMaxBwdCtas ? sms : kLnMaxBwdCtas;
    if (ctas > limit) ctas = limit;
    if (ctas < 1) ctas = 1;
    const size_t smem = TEAMS > 1 ? sizeof(float) * TEAMS * 2 * (size_t)p.D : 0;
    constexpr size_t most = TEAMS > 1 ? sizeof(float) * TEAMS * 2 * Sh::l * Sh::n * Sh::v : 0;   // a row's features in registers
    static_assert(most <= 64 * 1024, "teams' sums");
    if constexpr (most > 32 * 1024) {   // (48 KB, what is static among them, go unasked)
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
      if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kBwdThreads), smem, st, p);
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
