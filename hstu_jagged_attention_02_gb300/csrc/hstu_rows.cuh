// Rows of d features in the registers of d / 8 lanes, laid out so that the
// rotation of queries and keys pairs features of one lane (hstu_qk.cu,
// hstu_cache.cu).
//
// A lane holds two parts of 4 neighbouring features.  Pairs of halves
// (i, i + rot/2): lane l of a row's lanes has features 4 l .. and rot/2 + 4 l ..
// while 4 l < rot/2, and the lanes behind share the features from rot on, 8
// each.  Pairs of neighbours: lane l has features 8 l .. 8 l + 7.  Either way
// the lane's 4 pairs take 4 neighbouring cosines and sines.
#pragma once

#include "hstu_common.cuh"

namespace hstu {

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  uint2 x;
  x.x = *reinterpret_cast<const uint32_t*>(&a);
  x.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = x;
}

// The packed form of 4 features as it is loaded (16 bytes FP32, 8 bytes BF16).
template <typename T> struct Raw4;
template <> struct Raw4<float> { float4 x; };
template <> struct Raw4<__nv_bfloat16> { uint2 x; };
template <typename T> __device__ __forceinline__ Raw4<T> fetch4(const T* p) {
  Raw4<T> r;
  r.x = *reinterpret_cast<const decltype(r.x)*>(p);
  return r;
}

__device__ __forceinline__ void unpack4(const Raw4<__nv_bfloat16>& r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x.x << 16); v[1] = __uint_as_float(r.x.x & 0xFFFF0000u);
  v[2] = __uint_as_float(r.x.y << 16); v[3] = __uint_as_float(r.x.y & 0xFFFF0000u);
}

// A lane's 8 features of a row as FP32 pairs: v[0], v[1] part 0, v[2], v[3] part 1.
struct Row8 {
  float2 v[4];
  __device__ __forceinline__ Row8() {}
  __device__ __forceinline__ Row8(const Raw4<float>& a, const Raw4<float>& b) {
    v[0] = make_float2(a.x.x, a.x.y); v[1] = make_float2(a.x.z, a.x.w);
    v[2] = make_float2(b.x.x, b.x.y); v[3] = make_float2(b.x.z, b.x.w);
  }
  __device__ __forceinline__ Row8(const Raw4<__nv_bfloat16>& a, const Raw4<__nv_bfloat16>& b) {
    const uint32_t w[4] = {a.x.x, a.x.y, b.x.x, b.x.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void times(float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __fmul2_rn(v[e], make_float2(f, f));
  }
  __device__ __forceinline__ void times(const Row8& o) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __fmul2_rn(v[e], o.v[e]);
  }
  // sum of v o over the lane's features
  __device__ __forceinline__ float dot(const Row8& o) const {
    float2 s = __fmul2_rn(v[0], o.v[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) s = __ffma2_rn(v[e], o.v[e], s);
    return s.x + s.y;
  }
};
__device__ __forceinline__ void store_part(float* p, float2 a, float2 b) {
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_part(__nv_bfloat16* p, float2 a, float2 b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a.x, a.y), y = __floats2bfloat162_rn(b.x, b.y);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&x);
  w.y = *reinterpret_cast<const uint32_t*>(&y);
  *reinterpret_cast<uint2*>(p) = w;
}

// Where lane l of a row's lanes has its two parts, and whether they turn.
struct Parts {
  int f0, f1;
  bool turns;
  __device__ __forceinline__ Parts(int l, int rot, bool interleaved) {
    if (interleaved || 8 * l >= rot) {
      f0 = 8 * l;
      f1 = f0 + 4;
    } else {
      f0 = 4 * l;
      f1 = (rot >> 1) + 4 * l;
    }
    turns = 8 * l < rot;
  }
};

// The cosines and sines of the lane's 4 pairs, and the turn (a, b) -> (a c - b s, b c + a s).
struct Angles {
  float2 c[2], s[2];
  __device__ __forceinline__ void load(const float* cos, const float* sin, float dir) {
    const float4 a = *reinterpret_cast<const float4*>(cos), b = *reinterpret_cast<const float4*>(sin);
    c[0] = make_float2(a.x, a.y); c[1] = make_float2(a.z, a.w);
    s[0] = make_float2(b.x * dir, b.y * dir); s[1] = make_float2(b.z * dir, b.w * dir);
  }
  // the largest magnitude among them
  __device__ __forceinline__ float largest() const {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      m = fmaxf(m, fmaxf(fmaxf(fabsf(c[e].x), fabsf(c[e].y)), fmaxf(fabsf(s[e].x), fabsf(s[e].y))));
    return m;
  }
  __device__ __forceinline__ void turn(Row8& r, bool interleaved) const {
    if (interleaved) {
      const float cc[4] = {c[0].x, c[0].y, c[1].x, c[1].y}, ss[4] = {s[0].x, s[0].y, s[1].x, s[1].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = r.v[e];
        r.v[e] = make_float2(x.x * cc[e] - x.y * ss[e], x.y * cc[e] + x.x * ss[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 x = r.v[e], y = r.v[e + 2], ns = make_float2(-s[e].x, -s[e].y);
        r.v[e] = __ffma2_rn(y, ns, __fmul2_rn(x, c[e]));
        r.v[e + 2] = __ffma2_rn(x, s[e], __fmul2_rn(y, c[e]));
      }
    }
  }
};

// Sum over a row's LANES lanes.
template <int LANES, typename F>
__device__ __forceinline__ F row_sum(F v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace hstu
