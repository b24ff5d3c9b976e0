// AdamW over many tensors in one launch, moments in 32 or in 8 bits
// (hstu_adamw_*); the formulas and the 8-bit format are in hstu_attn.h.
//
// HBM-bound: 28 bytes a parameter in 32 bits, 16 with 8-bit moments (and 2 for a BF16 copy).  The tensors are
// cut into chunks of 256 to 2,048 elements once, by init, into a list of records that hold all of a
// chunk's pointers: a warp needs one load before its data, and takes one chunk after the other.
// 16 layers (21 million parameters): 104 us in 32 bits, 6.1 TB/s (89% of a copy's rate); 8 bits 70.0 us, 5.4 TB/s, with
// the arithmetic of the codes (10 rounds of the generator for 4 elements) beside the loads.  Prefetches into L2 and 3
// CTAs an SM were slower.
//
// A lane holds 4 neighbouring elements twice (elements 4 l and 128 + 4 l of the warp's 256).  In 8 bits
// the warp's 256 elements are a block: its largest magnitudes take one reduction over
// the warp.  Decoding and encoding work on the bits of FP32 numbers: a code shifted
// by 20 is the bit pattern of its value times a power of two (the small codes those of
// subnormal numbers), so rounding up or down at random is one integer addition below the cut.
#include <cuda_fp16.h>
#include <stdlib.h>
#include <string.h>

#include <type_traits>

#include "hstu_internal.h"

namespace hstu {

namespace {

constexpr int kBlock = 256;     // elements that share an exponent byte
constexpr int kMaxChunk = 2048; // of a chunk, a power of two from kBlock on
constexpr int kAdamThreads = 256;
constexpr int kMOff = 134, kVOff = 142, kLeastExp = 16;

// What the header of the workspace holds behind the error words.
struct AdamState {
  double pow1, pow2;    // beta^t of the next step
  int64_t steps;        // steps counted
  int64_t chunks;       // of the list
  int32_t kind;         // state_bits, grad_dtype: what the list was made for
  float c1, c2;         // 1 / (1 - beta1^t), 1 / (1 - beta2^t) of the next step
};
constexpr size_t kStateOff = 128;   // another line than the counter of CTAs

struct __align__(16) AdamChunk {
  float* p;
  const void* g;
  __nv_bfloat16* copy;
  void* m;
  void* v;
  uint8_t* me;
  uint8_t* ve;
  int64_t quad0;        // groups of 4 elements before this chunk, all tensors
  int32_t n;            // elements, <= kMaxChunk
  float wd, lr_scale;
  int32_t pad;
};

struct __align__(16) ReadChunk {
  const void* m;
  const void* v;
  const uint8_t* me;
  const uint8_t* ve;
  void* om;
  void* ov;
  int64_t n;
  int64_t pad;
};

struct AdamParams {
  int* hdr;
  const AdamChunk* list;
  const float* lr_at;
  const float* scale;
  const int32_t* skip;
  int64_t chunks;
  int kind;
  float lr, b1, b2, a1, a2, eps;   // a = 1 - b
  double beta1, beta2;
  uint64_t seed;
};

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011)
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// 4 elements from at on, `live` of them there (the others 0)
__device__ __forceinline__ void get4(const float* at, int live, float (&v)[4]) {
  if (live >= 4) {
    const float4 x = *reinterpret_cast<const float4*>(at);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < live ? at[i] : 0.f;
  }
}
__device__ __forceinline__ void get4(const __nv_bfloat16* at, int live, float (&v)[4]) {
  if (live >= 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xFFFF0000u);
    v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < live ? to_f(at[i]) : 0.f;
  }
}
__device__ __forceinline__ uint32_t get4(const uint8_t* at, int live) {
  if (live >= 4) return *reinterpret_cast<const uint32_t*>(at);
  uint32_t x = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < live) x |= (uint32_t)at[i] << (8 * i);
  return x;
}
__device__ __forceinline__ void put4(float* at, int live, const float (&v)[4]) {
  if (live >= 4) {
    *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < live) at[i] = v[i];
  }
}
__device__ __forceinline__ void put4(__nv_bfloat16* at, int live, const float (&v)[4]) {
  if (live >= 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 x;
    x.x = *reinterpret_cast<const uint32_t*>(&a);
    x.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(at) = x;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < live) at[i] = from_f<__nv_bfloat16>(v[i]);
  }
}
__device__ __forceinline__ void put4(uint8_t* at, int live, uint32_t x) {
  if (live >= 4) {
    *reinterpret_cast<uint32_t*>(at) = x;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < live) at[i] = (uint8_t)(x >> (8 * i));
  }
}

// A sum of pairs behind products, which must not become a fused product and sum (as the paired sum does,
// whatever its rounding mode says).
__device__ __forceinline__ float2 sum2(float2 x, float2 y) { return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y)); }

// Values of 4 codes of a block, unit its power of two.  m: e4m3 by the conversion to FP16 (127 a NaN);
// v: a code 20 bits up is the bit pattern of its value times 2^-112.
__device__ __forceinline__ void decode_m(uint32_t codes, float unit, float2 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t x;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(x) : "r"(codes >> (16 * h)));
    v[h] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&x)), make_float2(unit, unit));
  }
}
__device__ __forceinline__ void decode_v(uint32_t codes, float unit, float2 (&v)[2]) {
  constexpr uint32_t mask = 255u << 20;
  const float2 up = make_float2(0x1p112f, 0x1p112f), u = make_float2(unit, unit);
  v[0] = make_float2(__uint_as_float(codes << 20 & mask), __uint_as_float(codes << 12 & mask));
  v[1] = make_float2(__uint_as_float(codes << 4 & mask), __uint_as_float(codes >> 4 & mask));
#pragma unroll
  for (int h = 0; h < 2; ++h) v[h] = __fmul2_rn(__fmul2_rn(v[h], up), u);
}

// Noise for the 20 bits that fall away: 16 r + 8, r a word's low half (m) or high half (v).
__device__ __forceinline__ uint32_t noise_m(uint32_t w) { return (w & 0xffffu) * 16u + 8u; }
__device__ __forceinline__ uint32_t noise_v(uint32_t w) { return (w >> 16) * 16u + 8u; }

// Code of one value rounded up or down by the noise, whatever the value; up: 2^(off - e).
__device__ __forceinline__ uint32_t code_m(float x, float up, uint32_t noise) {
  const float a = fabsf(x) * up * 0x1p-120f;
  const uint32_t c = min((__float_as_uint(a) + noise) >> 20, 126u);
  return (fabsf(x) < __int_as_float(0x7f800000) ? c : 127u) | (__float_as_uint(x) >> 31 << 7);
}
__device__ __forceinline__ uint32_t code_v(float x, float up, uint32_t noise) {
  const float a = x * up * 0x1p-112f;
  const uint32_t c = min((__float_as_uint(a) + noise) >> 20, 255u);
  return x < __int_as_float(0x7f800000) ? c : 255u;
}
// The top bytes of 4 words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
// The same for 4 values of a block that holds finite numbers only: what is largest lies below 2^8 (m)
// or 2^16 (v) times the unit, so no code reaches the end of the range, and the sign stays where it is.
// (bits + 16 r + 8) << 4, as two multiply-adds: the code in the top byte.
__device__ __forceinline__ uint32_t rounded(float a, uint32_t r, uint32_t& sum) {
  sum = __float_as_uint(a);
  asm("" : "+r"(sum));   // nvcc 13.0 loses a shift of the first half of a paired product without this
  sum = r * 16u + sum;
  return sum * 16u + 128u;
}
__device__ __forceinline__ uint32_t codes_m(const float2 (&x)[2], float up, const uint4& w) {
  const float2 u = make_float2(up, up), d = make_float2(0x1p-120f, 0x1p-120f);
  const float2 a = __fmul2_rn(__fmul2_rn(x[0], u), d), b = __fmul2_rn(__fmul2_rn(x[1], u), d);
  const float f[4] = {a.x, a.y, b.x, b.y};
  const uint32_t r[4] = {w.x & 0xffffu, w.y & 0xffffu, w.z & 0xffffu, w.w & 0xffffu};
  uint32_t z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t sum;
    z[i] = rounded(f[i], r[i], sum);
    z[i] = (z[i] & 0x7fffffffu) | (sum & 0x80000000u);
  }
  return top_bytes(z[0], z[1], z[2], z[3]);
}
__device__ __forceinline__ uint32_t codes_v(const float2 (&x)[2], float up, const uint4& w) {
  const float2 u = make_float2(up, up), d = make_float2(0x1p-112f, 0x1p-112f);
  const float2 a = __fmul2_rn(__fmul2_rn(x[0], u), d), b = __fmul2_rn(__fmul2_rn(x[1], u), d);
  const float f[4] = {a.x, a.y, b.x, b.y};
  const uint32_t r[4] = {w.x >> 16, w.y >> 16, w.z >> 16, w.w >> 16};
  uint32_t z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t sum;
    z[i] = rounded(f[i], r[i], sum);
  }
  return top_bytes(z[0], z[1], z[2], z[3]);
}

constexpr uint32_t kInfBits = 0x7f800000u;
// the largest magnitude of a lane's 8 values, a NaN where there is one, as bits
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t top_bits(const float2 (&x)[2][2]) {
  const float a = max3(fabsf(x[0][0].x), fabsf(x[0][0].y), fabsf(x[0][1].x));
  const float b = max3(fabsf(x[0][1].y), fabsf(x[1][0].x), fabsf(x[1][0].y));
  return __float_as_uint(max3(a, b, max3(fabsf(x[1][1].x), fabsf(x[1][1].y), 0.f))) & 0x7fffffffu;
}
// the same of the finite ones
__device__ __forceinline__ uint32_t top_finite_bits(const float2 (&x)[2][2]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = x[j >> 1][j & 1];
    const uint32_t a = __float_as_uint(v.x) & 0x7fffffffu, b = __float_as_uint(v.y) & 0x7fffffffu;
    if (a < kInfBits) top = max(top, a);
    if (b < kInfBits) top = max(top, b);
  }
  return top;
}
__device__ __forceinline__ int exp_byte(uint32_t top) { return max((int)(top >> 23), kLeastExp); }

// The hardware's root and reciprocal, off by a step of FP32 (2^-23) at most each, beside the half steps of the update's other
// products and sums: the moments do not go through them.  They take subnormal numbers for zero; the denominator lies
// between eps and 2^126.
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void pairs(const float (&a)[4], float2 (&b)[2]) {
  b[0] = make_float2(a[0], a[1]);
  b[1] = make_float2(a[2], a[3]);
}
__device__ __forceinline__ void singles(const float2 (&b)[2], float (&a)[4]) {
  a[0] = b[0].x; a[1] = b[0].y; a[2] = b[1].x; a[3] = b[1].y;
}

// A record by its 16-byte parts, the same for all lanes.
template <typename R>
__device__ __forceinline__ R get_record(const R* at) {
  R r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(R) / 16); ++i) reinterpret_cast<uint4*>(&r)[i] = __ldg(reinterpret_cast<const uint4*>(at) + i);
  return r;
}

// A block's bytes, m's and v's; one below the least (memory that was zeroed, say) counts as that.
__device__ __forceinline__ int exps_of(const uint8_t* me, const uint8_t* ve, int block) {
  return max((int)me[block], kLeastExp) | max((int)ve[block], kLeastExp) << 8;
}

template <int BITS, typename TG>
__global__ void __launch_bounds__(kAdamThreads, 4) adamw_kernel(const __grid_constant__ AdamParams p) {
  pdl_wait();
  AdamState* st = reinterpret_cast<AdamState*>(reinterpret_cast<char*>(p.hdr) + kStateOff);
  if (st->chunks != p.chunks || st->kind != p.kind) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return;
  }
  if (p.skip && *p.skip != 0) return;
  const int lane = threadIdx.x & 31;
  const float lr0 = p.lr_at ? *p.lr_at : p.lr, scale = p.scale ? *p.scale : 1.f;
  const float c1s = st->c1, c2s = st->c2;
  const uint64_t t = (uint64_t)st->steps + 1;
  const float2 b1 = make_float2(p.b1, p.b1), a1 = make_float2(p.a1, p.a1), b2 = make_float2(p.b2, p.b2),
               a2 = make_float2(p.a2, p.a2), eps = make_float2(p.eps, p.eps), c2 = make_float2(c2s, c2s);
  constexpr int kWarps = kAdamThreads / 32;
  for (int i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < p.chunks; i += gridDim.x * kWarps) {
    const AdamChunk c = get_record(p.list + i);
    int exps = 0;   // lane b: the bytes of block b, m's and v's
    if (BITS == 8 && lane * kBlock < c.n) exps = exps_of(c.me, c.ve, lane);
    int new_exps = 0;
    const float lr = lr0 * c.lr_scale, keep1 = 1.f - lr * c.wd, c1 = -lr * c1s;
    const float2 keep = make_float2(keep1, keep1), step = make_float2(c1, c1);
#pragma unroll 1
    for (int blk = 0; blk * kBlock < c.n; ++blk) {
      const int at0 = blk * kBlock + 4 * lane;
      float2 w[2][2], g[2][2], m[2][2], v[2][2];
      uint32_t mc[2], vc[2];
      auto load = [&](auto FULL) {
        constexpr bool full = decltype(FULL)::value;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = at0 + 128 * j, live = full ? 4 : c.n - at;
          float a[4];
          get4(c.p + at, live, a); pairs(a, w[j]);
          get4(static_cast<const TG*>(c.g) + at, live, a); pairs(a, g[j]);
          if constexpr (BITS == 32) {
            get4(static_cast<const float*>(c.m) + at, live, a); pairs(a, m[j]);
            get4(static_cast<const float*>(c.v) + at, live, a); pairs(a, v[j]);
          } else {
            mc[j] = get4(static_cast<const uint8_t*>(c.m) + at, live);
            vc[j] = get4(static_cast<const uint8_t*>(c.v) + at, live);
          }
        }
      };
      const bool whole = c.n >= (blk + 1) * kBlock;
      if (whole) load(std::true_type());
      else load(std::false_type());
      float um = 0.f, uv = 0.f;
      if constexpr (BITS == 8) {
        const int e = __shfl_sync(0xffffffffu, exps, blk);
        um = pow2f((e & 255) - kMOff);
        uv = pow2f((e >> 8) - kVOff);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (BITS == 8) {
          decode_m(mc[j], um, m[j]);
          decode_v(vc[j], uv, v[j]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // products and sums one by one: the codes go by their last bits
          const float2 gs = __fmul2_rn(g[j][h], make_float2(scale, scale));
          m[j][h] = sum2(__fmul2_rn(m[j][h], b1), __fmul2_rn(gs, a1));
          v[j][h] = sum2(__fmul2_rn(v[j][h], b2), __fmul2_rn(__fmul2_rn(gs, gs), a2));
          // v / (1 - beta2^t) before the root, which takes a subnormal number for zero: its root, below 2^-63, counts for
          // nothing beside eps, while that of a subnormal v may
          const float2 vh = __fmul2_rn(v[j][h], c2), d = __fadd2_rn(make_float2(sqrt_approx(vh.x), sqrt_approx(vh.y)), eps);
          const float2 u = __fmul2_rn(m[j][h], make_float2(rcp_approx(d.x), rcp_approx(d.y)));
          w[j][h] = __ffma2_rn(u, step, __fmul2_rn(w[j][h], keep));
        }
      }
      uint32_t nm[2] = {}, nv[2] = {};
      if constexpr (BITS == 8) {
        uint32_t tm = __reduce_max_sync(0xffffffffu, top_bits(m)), tv = __reduce_max_sync(0xffffffffu, top_bits(v));
        const bool wild = max(tm, tv) >= kInfBits;   // the same for the whole warp
        if (wild) {
          tm = __reduce_max_sync(0xffffffffu, top_finite_bits(m));
          tv = __reduce_max_sync(0xffffffffu, top_finite_bits(v));
        }
        const int me = exp_byte(tm), ve = exp_byte(tv);
        const float up_m = pow2f(kMOff - me), up_v = pow2f(kVOff - ve);
        if (lane == blk) new_exps = me | ve << 8;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint64_t quad = (uint64_t)c.quad0 + (uint32_t)((at0 + 128 * j) >> 2);
          const uint4 r = philox((uint32_t)quad, (uint32_t)(quad >> 32), (uint32_t)t, (uint32_t)(t >> 32), (uint32_t)p.seed,
                                 (uint32_t)(p.seed >> 32));
          if (!wild) {
            nm[j] = codes_m(m[j], up_m, r);
            nv[j] = codes_v(v[j], up_v, r);
          } else {
            float x[4], y[4];
            singles(m[j], x);
            singles(v[j], y);
            const uint32_t word[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              nm[j] |= code_m(x[e], up_m, noise_m(word[e])) << (8 * e);
              nv[j] |= code_v(y[e], up_v, noise_v(word[e])) << (8 * e);
            }
          }
        }
      }
      auto store = [&](auto FULL) {
        constexpr bool full = decltype(FULL)::value;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = at0 + 128 * j, live = full ? 4 : c.n - at;
          if (!full && live <= 0) continue;
          float a[4];
          singles(w[j], a);
          put4(c.p + at, live, a);
          if (c.copy) put4(c.copy + at, live, a);
          if constexpr (BITS == 32) {
            singles(m[j], a);
            put4(static_cast<float*>(c.m) + at, live, a);
            singles(v[j], a);
            put4(static_cast<float*>(c.v) + at, live, a);
          } else {
            put4(static_cast<uint8_t*>(c.m) + at, live, nm[j]);
            put4(static_cast<uint8_t*>(c.v) + at, live, nv[j]);
          }
        }
      };
      if (whole) store(std::true_type());
      else store(std::false_type());
    }
    if (BITS == 8 && lane * kBlock < c.n) {
      c.me[lane] = (uint8_t)new_exps;
      c.ve[lane] = (uint8_t)(new_exps >> 8);
    }
  }
  // the CTA that ends last counts the step, when all have read what belongs to it
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(p.hdr + WS_NEXT, 1) == (int)gridDim.x - 1) {
      p.hdr[WS_NEXT] = 0;
      st->pow1 *= p.beta1;
      st->pow2 *= p.beta2;
      st->c1 = (float)(1.0 / (1.0 - st->pow1));
      st->c2 = (float)(1.0 / (1.0 - st->pow2));
      st->steps += 1;
    }
  }
}

// A warp takes a chunk, four blocks at a time where it has them: a lane 16 neighbouring elements twice.
template <int BITS, typename TO>
__global__ void __launch_bounds__(kAdamThreads)
adamw_read_kernel(int* hdr, const ReadChunk* __restrict__ list, int chunks, int kind) {
  pdl_wait();
  const AdamState* st = reinterpret_cast<const AdamState*>(reinterpret_cast<const char*>(hdr) + kStateOff);
  if (st->chunks != chunks || st->kind != kind) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return;
  }
  const int lane = threadIdx.x & 31;
  constexpr int kWarps = kAdamThreads / 32;
  for (int i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < chunks; i += gridDim.x * kWarps) {
    const ReadChunk c = get_record(list + i);
    const int n = (int)c.n;
    int exps = 0;
    if (BITS == 8 && lane * kBlock < n) exps = exps_of(c.me, c.ve, lane);
#pragma unroll 1
    for (int blk = 0; blk * kBlock < n; blk += 2) {
      uint32_t mc[4], vc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = blk * kBlock + 128 * j + 4 * lane, live = n - at;
        if constexpr (BITS == 8) {
          if (c.om) mc[j] = get4(static_cast<const uint8_t*>(c.m) + at, live);
          if (c.ov) vc[j] = get4(static_cast<const uint8_t*>(c.v) + at, live);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = blk * kBlock + 128 * j + 4 * lane, live = n - at;
        float um = 0.f, uv = 0.f;
        if constexpr (BITS == 8) {
          const int e = __shfl_sync(0xffffffffu, exps, (blk + (j >> 1)) & 31);
          um = pow2f((e & 255) - kMOff);
          uv = pow2f((e >> 8) - kVOff);
        }
        if (live <= 0) continue;
        float x[4];
        float2 y[2];
        if (c.om) {
          if constexpr (BITS == 8) {
            decode_m(mc[j], um, y);
            singles(y, x);
          } else {
            get4(static_cast<const float*>(c.m) + at, live, x);
          }
          put4(static_cast<TO*>(c.om) + at, live, x);
        }
        if (c.ov) {
          if constexpr (BITS == 8) {
            decode_v(vc[j], uv, y);
            singles(y, x);
          } else {
            get4(static_cast<const float*>(c.v) + at, live, x);
          }
          put4(static_cast<TO*>(c.ov) + at, live, x);
        }
      }
    }
  }
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

hstu_status_t check_desc(const hstu_adamw_desc* d) {
  if (!d || d->struct_size != sizeof(hstu_adamw_desc)) return HSTU_ERR_INVALID_ARG;
  if (d->state_bits != 32 && d->state_bits != 8) return HSTU_ERR_INVALID_ARG;
  if (d->grad_dtype != HSTU_BF16 && d->grad_dtype != HSTU_FP32) return HSTU_ERR_INVALID_ARG;
  if (d->num_tensors < 0 || d->steps_done < -1) return HSTU_ERR_INVALID_ARG;
  const double b[2] = {d->beta1, d->beta2};
  for (double x : b)
    if (!(x >= 0.0 && x < 1.0)) return HSTU_ERR_INVALID_ARG;
  // from 1e-12 on the square root of a subnormal number counts for nothing beside it
  if (!(d->eps >= 1e-12 && d->eps < 1e30) || !(d->lr >= 0.0 && d->lr < 1e30)) return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

// Elements of a chunk: a warp takes one at a time, and every warp of the GPU (4,864) should have a few, as
// the last round is short for some: three with 8-bit moments, whose chunks begin with a round trip for the exponents
// (16 layers: 119.8 us with chunks of 256, 96.4 of 512, 95.1 of 1,024, 99.9 of 2,048), twelve in 32 bits (103.9, 104.8,
// 106.4, 111.3; one layer 7.5, 8.0, 9.3, 12.5).  Longer chunks are a shorter list.
int chunk_of(const hstu_adamw_desc* d, const hstu_adamw_tensor* t) {
  int64_t blocks = 0;
  for (int i = 0; i < d->num_tensors; ++i) blocks += (t[i].n + kBlock - 1) / kBlock;
  const int64_t least = (d->state_bits == 8 ? 3 : 12) * 4864;
  int chunk = kBlock;
  while (chunk < kMaxChunk && blocks / (2 * chunk / kBlock) >= least) chunk *= 2;
  return chunk;
}

// The tensors' checks, and the chunks of their list.
hstu_status_t check_tensors(const hstu_adamw_desc* d, const hstu_adamw_tensor* t, bool stepped, int64_t* chunks) {
  if (d->num_tensors > 0 && !t) return HSTU_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int i = 0; i < d->num_tensors; ++i) {
    const hstu_adamw_tensor& x = t[i];
    if (x.n < 0) return HSTU_ERR_INVALID_ARG;
    if (x.n > ((int64_t)1 << 44)) return HSTU_ERR_UNSUPPORTED;
    if (x.n == 0) continue;
    if (!x.m || !x.v || !aligned(x.m, 16) || !aligned(x.v, 16)) return HSTU_ERR_INVALID_ARG;
    if (d->state_bits == 8 && (!x.m_exp || !x.v_exp)) return HSTU_ERR_INVALID_ARG;
    if (stepped) {
      if (!x.param || !aligned(x.param, 16) || !aligned(x.copy, 8)) return HSTU_ERR_INVALID_ARG;
      if (!aligned(x.grad, 16)) return HSTU_ERR_INVALID_ARG;
      if (!(x.weight_decay >= 0.f && x.weight_decay < 1e30f) || !(x.lr_scale >= 0.f && x.lr_scale < 1e30f))
        return HSTU_ERR_INVALID_ARG;
    }
  }
  const int chunk = chunk_of(d, t);
  for (int i = 0; i < d->num_tensors; ++i)
    if (!stepped || t[i].grad) total += (t[i].n + chunk - 1) / chunk;
  if (total > 0x7ff00000) return HSTU_ERR_UNSUPPORTED;
  *chunks = total;
  return HSTU_OK;
}

size_t list_bytes(int64_t chunks) {
  static_assert(sizeof(AdamChunk) == 80 && sizeof(ReadChunk) == 64, "records of the lists");
  return kWsHeaderBytes + (size_t)chunks * sizeof(AdamChunk);
}

hstu_status_t check_ws(const void* ws, size_t bytes, size_t need) {
  return !ws || !aligned(ws, kWsAlign) || bytes < need ? HSTU_ERR_WORKSPACE : HSTU_OK;
}

hstu_status_t cuda_failed(cudaError_t e, const char* what) {
  (void)cudaGetLastError();
  set_error_detail(e, what);
  return HSTU_ERR_CUDA;
}

// CTAs for a warp a chunk, at most `most`
unsigned ctas_for(int64_t chunks, int most) {
  const int64_t n = (chunks + kAdamThreads / 32 - 1) / (kAdamThreads / 32);
  return (unsigned)(n < 1 ? 1 : (n < most ? n : most));
}

hstu_status_t device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? HSTU_OK : cuda_failed(e, "reading the number of SMs");
}

int kind_of(const hstu_adamw_desc* d, bool read, int out_dtype) {
  return d->state_bits << 8 | (read ? 16 + out_dtype : d->grad_dtype);
}

// Header and list to the workspace; waits until they are there.  The header keeps its counters where keep.
hstu_status_t send(void* ws, const AdamState& state, bool keep, const void* list, size_t bytes, cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  cudaError_t e = cudaSuccess;
  if (!keep) {
    char header[kWsHeaderBytes] = {};
    memcpy(header + kStateOff, &state, sizeof(state));
    e = cudaMemcpyAsync(base, header, sizeof(header), cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  } else {
    const size_t at = kStateOff + offsetof(AdamState, chunks), n = offsetof(AdamState, c1) - offsetof(AdamState, chunks);
    e = cudaMemcpyAsync(base + at, &state.chunks, n, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e == cudaSuccess && bytes > 0) e = cudaMemcpyAsync(base + kWsHeaderBytes, list, bytes, cudaMemcpyHostToDevice, st);
  const cudaError_t f = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? HSTU_OK : cuda_failed(e, "writing the list of chunks");
}

hstu_status_t not_captured(cudaStream_t st) {
  cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(st, &c);
  if (e != cudaSuccess) return cuda_failed(e, "cudaStreamIsCapturing");
  if (c == cudaStreamCaptureStatusNone) return HSTU_OK;
  set_detail_message("a list of chunks cannot be laid out on a stream that is being captured");
  return HSTU_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_adamw_workspace_size(const hstu_adamw_desc* desc, const hstu_adamw_tensor* tensors, size_t* bytes) {
  hstu_status_t s = check_desc(desc);
  int64_t chunks = 0;
  if (s == HSTU_OK) s = check_tensors(desc, tensors, false, &chunks);
  if (s != HSTU_OK) return s;
  if (bytes) *bytes = list_bytes(chunks);
  return HSTU_OK;
}

hstu_status_t hstu_adamw_init(hstu_adamw_desc* d, const hstu_adamw_tensor* tensors, void* workspace, size_t workspace_bytes,
                              hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  int64_t chunks = 0;
  if (s == HSTU_OK) s = check_tensors(d, tensors, true, &chunks);
  if (s == HSTU_OK) s = check_ws(workspace, workspace_bytes, list_bytes(chunks));
  if (s != HSTU_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if ((s = not_captured(st)) != HSTU_OK) return s;
  AdamChunk* list = static_cast<AdamChunk*>(calloc(chunks > 0 ? (size_t)chunks : 1, sizeof(AdamChunk)));
  if (!list) {
    set_detail_message("no host memory for the list of chunks");
    return HSTU_ERR_WORKSPACE;
  }
  int64_t at = 0, block = 0;
  const int chunk = chunk_of(d, tensors);
  const size_t msize = d->state_bits == 8 ? 1 : 4, gsize = d->grad_dtype == HSTU_FP32 ? 4 : 2;
  for (int i = 0; i < d->num_tensors; ++i) {
    const hstu_adamw_tensor& x = tensors[i];
    for (int64_t e = 0; x.grad && e < x.n; e += chunk) {
      AdamChunk& c = list[at++];
      c.p = x.param + e;
      c.g = static_cast<const char*>(x.grad) + e * gsize;
      c.copy = x.copy ? static_cast<__nv_bfloat16*>(x.copy) + e : nullptr;
      c.m = static_cast<char*>(x.m) + e * msize;
      c.v = static_cast<char*>(x.v) + e * msize;
      c.me = x.m_exp ? x.m_exp + e / kBlock : nullptr;
      c.ve = x.v_exp ? x.v_exp + e / kBlock : nullptr;
      c.quad0 = block * (kBlock / 4) + e / 4;
      c.n = (int32_t)(x.n - e < chunk ? x.n - e : chunk);
      c.wd = x.weight_decay;
      c.lr_scale = x.lr_scale;
    }
    block += (x.n + kBlock - 1) / kBlock;
  }
  AdamState state{};
  const bool keep = d->steps_done < 0;
  state.steps = keep ? 0 : d->steps_done;
  state.pow1 = pow(d->beta1, (double)(state.steps + 1));
  state.pow2 = pow(d->beta2, (double)(state.steps + 1));
  state.c1 = (float)(1.0 / (1.0 - state.pow1));
  state.c2 = (float)(1.0 / (1.0 - state.pow2));
  state.chunks = chunks;
  state.kind = kind_of(d, false, 0);
  s = send(workspace, state, keep, list, (size_t)chunks * sizeof(AdamChunk), st);
  free(list);
  if (s == HSTU_OK) d->chunks = chunks;
  return s;
}

hstu_status_t hstu_adamw_step(const hstu_adamw_desc* d, const hstu_adamw_step_args* a, void* workspace,
                              size_t workspace_bytes, hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  if (s != HSTU_OK) return s;
  if (!a || d->chunks < 0 || d->chunks > 0x7ff00000) return HSTU_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)a->lr, (const void*)a->grad_scale, (const void*)a->skip})
    if (!aligned(ptr, 4)) return HSTU_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, list_bytes(d->chunks))) != HSTU_OK) return s;
  AdamParams p{};
  p.hdr = static_cast<int*>(workspace);
  p.list = reinterpret_cast<const AdamChunk*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  p.lr_at = a->lr; p.scale = a->grad_scale; p.skip = a->skip;
  p.chunks = d->chunks; p.kind = kind_of(d, false, 0);
  p.lr = (float)d->lr; p.b1 = (float)d->beta1; p.b2 = (float)d->beta2;
  p.a1 = (float)(1.0 - d->beta1); p.a2 = (float)(1.0 - d->beta2); p.eps = (float)d->eps;
  p.beta1 = d->beta1; p.beta2 = d->beta2; p.seed = d->seed;
  reset_launches();
  int sms = 0;
  if ((s = device_sms(&sms)) != HSTU_OK) return s;
  const dim3 grid(ctas_for(d->chunks, 4 * sms)), block(kAdamThreads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = d->grad_dtype == HSTU_FP32;
  const cudaError_t e = d->state_bits == 32
                            ? (f32 ? launch_pdl(adamw_kernel<32, float>, grid, block, 0, st, p)
                                   : launch_pdl(adamw_kernel<32, __nv_bfloat16>, grid, block, 0, st, p))
                            : (f32 ? launch_pdl(adamw_kernel<8, float>, grid, block, 0, st, p)
                                   : launch_pdl(adamw_kernel<8, __nv_bfloat16>, grid, block, 0, st, p));
  if (e != cudaSuccess) return cuda_failed(e, "launching adamw_kernel");
  note_launches(1);
  return HSTU_OK;
}

hstu_status_t hstu_adamw_read_init(hstu_adamw_desc* d, const hstu_adamw_tensor* tensors, const hstu_adamw_moments* outs,
                                   int32_t out_dtype, void* workspace, size_t workspace_bytes, hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  int64_t chunks = 0;
  if (s == HSTU_OK) s = check_tensors(d, tensors, false, &chunks);
  if (s != HSTU_OK) return s;
  if ((out_dtype != HSTU_BF16 && out_dtype != HSTU_FP32) || (d->num_tensors > 0 && !outs)) return HSTU_ERR_INVALID_ARG;
  for (int i = 0; i < d->num_tensors; ++i)
    if (!aligned(outs[i].m, 16) || !aligned(outs[i].v, 16)) return HSTU_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, list_bytes(chunks))) != HSTU_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if ((s = not_captured(st)) != HSTU_OK) return s;
  ReadChunk* list = static_cast<ReadChunk*>(calloc(chunks > 0 ? (size_t)chunks : 1, sizeof(ReadChunk)));
  if (!list) {
    set_detail_message("no host memory for the list of chunks");
    return HSTU_ERR_WORKSPACE;
  }
  int64_t at = 0;
  const int chunk = chunk_of(d, tensors);
  const size_t msize = d->state_bits == 8 ? 1 : 4, osize = out_dtype == HSTU_FP32 ? 4 : 2;
  for (int i = 0; i < d->num_tensors; ++i) {
    const hstu_adamw_tensor& x = tensors[i];
    for (int64_t e = 0; e < x.n; e += chunk) {
      ReadChunk& c = list[at++];
      c.m = static_cast<const char*>(x.m) + e * msize;
      c.v = static_cast<const char*>(x.v) + e * msize;
      c.me = x.m_exp ? x.m_exp + e / kBlock : nullptr;
      c.ve = x.v_exp ? x.v_exp + e / kBlock : nullptr;
      c.om = outs[i].m ? static_cast<char*>(outs[i].m) + e * osize : nullptr;
      c.ov = outs[i].v ? static_cast<char*>(outs[i].v) + e * osize : nullptr;
      c.n = x.n - e < chunk ? x.n - e : chunk;
    }
  }
  AdamState state{};
  state.chunks = chunks;
  state.kind = kind_of(d, true, out_dtype);
  s = send(workspace, state, false, list, (size_t)chunks * sizeof(ReadChunk), st);
  free(list);
  if (s == HSTU_OK) {
    d->chunks = chunks;
    d->grad_dtype = out_dtype;   // what read goes by
  }
  return s;
}

hstu_status_t hstu_adamw_read(const hstu_adamw_desc* d, void* workspace, size_t workspace_bytes, hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  if (s != HSTU_OK) return s;
  if (d->chunks < 0 || d->chunks > 0x7ff00000) return HSTU_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, list_bytes(d->chunks))) != HSTU_OK) return s;
  reset_launches();
  if (d->chunks == 0) return HSTU_OK;
  int* hdr = static_cast<int*>(workspace);
  const ReadChunk* list = reinterpret_cast<const ReadChunk*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  int sms = 0;
  if ((s = device_sms(&sms)) != HSTU_OK) return s;
  const dim3 grid(ctas_for(d->chunks, 8 * sms)), block(kAdamThreads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int kind = kind_of(d, true, d->grad_dtype);
  const bool f32 = d->grad_dtype == HSTU_FP32;
  const cudaError_t e = d->state_bits == 32
                            ? (f32 ? launch_pdl(adamw_read_kernel<32, float>, grid, block, 0, st, hdr, list, (int)d->chunks, kind)
                                   : launch_pdl(adamw_read_kernel<32, __nv_bfloat16>, grid, block, 0, st, hdr, list, (int)d->chunks, kind))
                            : (f32 ? launch_pdl(adamw_read_kernel<8, float>, grid, block, 0, st, hdr, list, (int)d->chunks, kind)
                                   : launch_pdl(adamw_read_kernel<8, __nv_bfloat16>, grid, block, 0, st, hdr, list, (int)d->chunks, kind));
  if (e != cudaSuccess) return cuda_failed(e, "launching adamw_read_kernel");
  note_launches(1);
  return HSTU_OK;
}

hstu_status_t hstu_adamw_steps(const void* workspace, hstu_stream_t stream, int64_t* steps) {
  if (!workspace || !steps) return HSTU_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  hstu_status_t s = not_captured(st);
  if (s != HSTU_OK) return s;
  const char* at = static_cast<const char*>(workspace) + kStateOff + offsetof(AdamState, steps);
  cudaError_t e = cudaMemcpyAsync(steps, at, sizeof(int64_t), cudaMemcpyDeviceToHost, st);
  const cudaError_t f = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? HSTU_OK : cuda_failed(e, "reading the count of steps");
}

}  // extern "C"
