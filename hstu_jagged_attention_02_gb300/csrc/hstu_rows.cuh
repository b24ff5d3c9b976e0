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

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xFFFF0000u);
  v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
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
__device__ __forceinline__ void unpack4(const Raw4<float>& r, float (&v)[4]) {
  v[0] = r.x.x; v[1] = r.x.y; v[2] = r.x.z; v[3] = r.x.w;
}
__device__ __forceinline__ void unpack4(const Raw4<__nv_bfloat16>& r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x.x << 16); v[1] = __uint_as_float(r.x.x & 0xFFFF0000u);
  v[2] = __uint_as_float(r.x.y << 16); v[3] = __uint_as_float(r.x.y & 0xFFFF0000u);
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

// The lane's 4 pairs (a, b) -> (a c - b s, b c + a s).
template <typename F>
__device__ __forceinline__ void turn_pairs(F (&x)[4], F (&y)[4], const float (&c)[4], const float (&s)[4], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      F& a = e < 2 ? x[2 * e] : y[2 * e - 4];
      F& b = e < 2 ? x[2 * e + 1] : y[2 * e - 3];
      const F u = a * c[e] - b * s[e], v = b * c[e] + a * s[e];
      a = u;
      b = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const F u = x[e] * c[e] - y[e] * s[e], v = y[e] * c[e] + x[e] * s[e];
      x[e] = u;
      y[e] = v;
    }
  }
}

// Sum over a row's LANES lanes.
template <int LANES, typename F>
__device__ __forceinline__ F row_sum(F v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace hstu
