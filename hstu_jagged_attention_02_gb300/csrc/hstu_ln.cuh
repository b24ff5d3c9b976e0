// Layer norm with weight and bias: what the forward (hstu_ln_fwd.cu) and the
// backward (hstu_ln_bwd.cu) share.
//
// A row lies in the registers of a team, 8 lanes to a warp or (from 1,024 features on) a
// CTA: thread l of a team of L has the features (i L + l) V + [0, V) for i < N,
// V = 8 where rows are 16-byte aligned (16 or 32 bytes a load, a warp's loads
// cover 256 features), else 1 (a warp's load covers 32 neighbouring features).
#pragma once
#include "hstu_internal.h"

namespace hstu {
namespace ln {

struct LnParams {
  const int64_t* num_rows;
  const void* x;
  const float* weight;
  const float* bias;
  void* y;             // forward
  float* mean;
  float* rstd;
  const void* dy;      // backward
  const void* dres;
  void* dx;
  float* d_weight;
  float* d_bias;
  float* partial;      // [CTAs][2][D] sums of the CTAs
  int* hdr;
  int64_t rows, xs, ys, dxs, drs;
  int D;
  float eps;
};

// Rows that are in use; a count outside [0, rows] is recorded and none taken.
__device__ __forceinline__ int64_t live_rows(const LnParams& p) {
  if (!p.num_rows) return p.rows;
  const int64_t n = *p.num_rows;
  if (n < 0 || n > p.rows) {
    set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return 0;
  }
  return n;
}

// V neighbouring features as they are loaded.
template <typename T, int V> struct Pack;
template <> struct Pack<__nv_bfloat16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
};
template <> struct Pack<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <typename T> struct Pack<T, 1> {
  T a;
  __device__ __forceinline__ void load(const T* p) { a = *p; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f(a); }
};

__device__ __forceinline__ void put(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void put(T* p, const float (&v)[1]) { *p = from_f<T>(v[0]); }

// Sums of two values over a team of L threads.  A CTA's go through red, which is
// free again after the team's next barrier: callers alternate between two.
template <int L>
__device__ __forceinline__ float2 team_sum(float2 v, float2* red) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (L > 32) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < L / 32; ++w) {
      v.x += red[w].x;
      v.y += red[w].y;
    }
  }
  return v;
}
template <int L>
__device__ __forceinline__ float team_sum(float v, float2* red) { return team_sum<L>(make_float2(v, 0.f), red).x; }

// Calls go(V, L, N) as integral constants for D features, wide or not: the
// smallest of a few register counts that holds a row.
template <int V, int L, int N> struct Shape {
  static constexpr int v = V, l = L, n = N;
};
template <typename F>
auto dispatch_shape(int D, bool wide, F&& go) {
  if (wide) {
    if (D <= 64) return go(Shape<8, 8, 1>());
    if (D <= 128) return go(Shape<8, 16, 1>());
    if (D <= 256) return go(Shape<8, 32, 1>());
    if (D <= 512) return go(Shape<8, 32, 2>());
    if (D <= 1024) return go(Shape<8, 32, 4>());
    if (D <= 2048) return go(Shape<8, 256, 1>());
    if (D <= 8192) return go(Shape<8, 256, 4>());
    return go(Shape<8, 512, 4>());
  }
  if (D <= 32) return go(Shape<1, 8, 4>());
  if (D <= 128) return go(Shape<1, 16, 8>());
  if (D <= 320) return go(Shape<1, 32, 10>());
  if (D <= 512) return go(Shape<1, 32, 16>());
  if (D <= 1024) return go(Shape<1, 32, 32>());
  if (D <= 4096) return go(Shape<1, 512, 8>());
  return go(Shape<1, 512, 32>());
}

constexpr int kMaxD = 16384;
constexpr int kTeamsThreads = 256;   // threads of a CTA whose teams are warps or parts of them

}  // namespace ln

// launches (hstu_ln_fwd.cu, hstu_ln_bwd.cu)
cudaError_t launch_ln_fwd(const ln::LnParams& p, int x_dtype, int y_dtype, bool wide, int sms, cudaStream_t st);
cudaError_t launch_ln_bwd(const ln::LnParams& p, int x_dtype, int y_dtype, bool wide, int sms, cudaStream_t st);
constexpr int kLnMaxBwdCtas = 160;   // rows of partial sums in the backward's workspace

}  // namespace hstu
