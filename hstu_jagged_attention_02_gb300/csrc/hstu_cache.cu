// Appending to and reading from the paged 4-bit cache (hstu_cache_append,
// hstu_cache_read).
//
// Append: the BF16 rows it reads and the packed ones it writes (2 d bytes in,
// 9 d / 16 out) would bound it, but coding a feature takes more instructions than
// that leaves room for: 161,000 tokens of four heads of 128, normed and rotated,
// take 220 us (2.0 TB/s; 63 us at the rate of a copy), 1,084 warp instructions a
// token at 2.6 a cycle: issue slots are busy 63% of the time, with the 20 warps an
// SM that 96 registers leave.  Keys that go in as they are take 134 us; more loads
// in flight (through shared memory) or more warps (80 registers) took longer.  The
// read is bound by what it writes: 74 us, 5.8 TB/s.
//
// d / 8 lanes hold a row (hstu_rows.cuh: both features
// of a pair in one lane), a warp takes a token at a time, its keys' and values'
// passes of 256 features side by side, all loads first.  A warp walks
// tokens_per_warp neighbouring tokens, so that the sequence and the page are
// looked up once for them (in a small batch each warp has one token: there the
// chain of lookups is the time; both sides at tokens_per_warp).  A group's
// maximum goes over the 2 or 4 lanes that share it.
//
// Roundings are decided as on real numbers.  A value x that is exact in FP32
// (a BF16 input) meets a border only exactly: its quotient by the scale (4
// significant bits) lies on a border or more than 2^-8 of it away, since x is at
// most 255 units and a border times a scale fewer than 128, of the same or a
// coarser unit.  So the quotient by the reciprocal, rounded to 16 significant
// bits, decides rightly.
// A normed or rotated key is known to 2^-20 of its terms only; where the
// codes (or the scale) of x - d and x + d differ, the warp computes its rows
// again as sums of two FP32 numbers, good to 2^-44, and compares with the
// borders themselves.  That happens to about one row in a thousand.
#include "hstu_fp4.cuh"
#include "hstu_internal.h"
#include "hstu_rows.cuh"
#include "hstu_seq_search.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kManyTokens = 4;
constexpr float kBand = 1.05e-06f;   // 2^-20 of a feature's terms, its quotient by the scale included, and a little
// The terms of a turned feature are |a c| + |b s| <= m (|a| + |b|), m the
// largest cosine or sine of the lane's pairs; kBand is for m <= 1 and grows with
// m (tables may carry a factor).

struct AppendParams {
  const int64_t* off;
  const int32_t* lens;
  const int32_t* table;
  const int64_t* times;
  const float* cos;
  const float* sin;
  const float* gain;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t ks[2], vs[2];
  uint8_t* pages;
  int64_t* page_times;
  int* hdr;
  int64_t T, max_pos;
  int B, H, page_log, num_pages, max_pages;
  int rot, interleaved, norm, tokens_per_warp;
  float eps;
  float k_scale, v_scale;   // 2^-k_exp, 2^-v_exp
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 4 features of a group: their codes and the group's scale.
struct Coded {
  uint32_t codes;   // 4 codes, 16 bits
  uint32_t scale;   // e4m3 byte
};

// y = x / s for a scale s, rounded to 16 significant bits: right on a border
// exactly where the quotient of an exact x is.
__device__ __forceinline__ float snap(float y) { return __uint_as_float((__float_as_uint(y) + 0x80u) & 0xffffff00u); }

__device__ __forceinline__ float inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return s > 0.f ? r : 0.f;
}

// 8 features that are exact in FP32, top the largest magnitude of their group:
// codes (32 bits) and the scale's byte.
__device__ __forceinline__ uint2 encode_exact(const Row8& x, float top) {
  const float want = snap(top * 0.16666667f);                 // a border is met, or more than 2^-8 of it away
  const uint32_t scale = e4m3_of(top == top ? want : top);    // a NaN stays one
  const float inv = inverse(e4m3_float(scale));
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) codes |= e2m1x2_of(snap(x.v[e].x * inv), snap(x.v[e].y * inv)) << (8 * e);
  return make_uint2(codes, scale);
}

// 4 features known to +-d, and their group's largest magnitude to [lo, hi]:
// false where that does not decide the result (a NaN may be two infinities of
// this path's own, each a number beyond FP32 times the cache's power of two).
__device__ __forceinline__ bool encode_banded(const float2 (&x)[2], const float2 (&d)[2], float lo, float hi, Coded& c) {
  c.scale = e4m3_of(hi * (0.16666667f * 1.0000005f));
  const bool sure = c.scale == e4m3_of(lo * (0.16666667f * 0.9999995f)) && c.scale != 0x7fu;
  const float inv = inverse(e4m3_float(c.scale));
  const float2 i2 = make_float2(inv, inv), n2 = make_float2(-inv, -inv);
  uint32_t lower = 0, upper = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float2 y = __fmul2_rn(x[e], i2);
    const float2 a = __ffma2_rn(d[e], n2, y), b = __ffma2_rn(d[e], i2, y);
    lower |= e2m1x2_of(a.x, a.y) << (8 * e);
    upper |= e2m1x2_of(b.x, b.y) << (8 * e);
  }
  c.codes = lower;
  if (lower == upper) return sure;
  // codes that differ, but for the sign of a zero
  const uint32_t diff = lower ^ upper, mags = (lower | upper) & 0x7777u;
  const uint32_t nonzero = (mags | (mags >> 1) | (mags >> 2)) & 0x1111u;
  return sure && (diff & (nonzero * 15u)) == 0;
}

// A number as the sum of two FP32 ones, h the nearest to it: 2^-48 of it in
// precision, on the FP32 units (an FP64 path of the same steps took 7 us to the
// 1 us of this one; the exactness of sums and products in two parts is Dekker's
// and Knuth's).  A result that is not finite has no second part, where the
// steps for it would make an infinity a NaN.
struct Two {
  float h, l;
};
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.4028234663852886e38f; }
__device__ __forceinline__ Two sum_of(float a, float b) {          // exact
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two join(float h, float l) {            // exact for |l| <= |h|
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two s = sum_of(a.h, b.h);
  return finite(s.h) ? join(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))) : Two{s.h, 0.f};
}
__device__ __forceinline__ Two operator*(Two a, float f) {
  const float p = __fmul_rn(a.h, f);
  return finite(p) ? join(p, __fmaf_rn(a.l, f, __fmaf_rn(a.h, f, -p))) : Two{p, 0.f};
}
__device__ __forceinline__ Two operator-(Two a) { return {-a.h, -a.l}; }
// whether |a| lies above a border, or on it too
__device__ __forceinline__ float over(Two a, float border) { return __fadd_rn(__fsub_rn(a.h, border), a.l); }

// 1 / sqrt(a): one Newton step with its quadratic term from the FP32 value.
__device__ __forceinline__ Two rsqrt_two(Two a) {
  const float r = rsqrtf(a.h), p = __fmul_rn(r, r), e = __fmaf_rn(r, r, -p);
  const float t = __fsub_rn(__fmaf_rn(-a.h, p, 1.f), __fmaf_rn(a.h, e, __fmul_rn(a.l, p)));   // 1 - a r^2
  return join(r, __fmul_rn(r, __fmul_rn(t, __fmaf_rn(0.375f, t, 0.5f))));
}

// The same from two parts each (every border compared with itself); bad: a NaN in the group.
__device__ __forceinline__ Coded encode_two(const Two (&x)[4], Two top, bool bad) {
  Coded c;
  // the nearest scale by its FP32 neighbour, then its two borders (halves between scales) times 6
  c.scale = e4m3_of(top.h * 0.16666667f);
  if (c.scale < 0x7eu) {
    const float d = over(top, 3.f * (e4m3_float(c.scale) + e4m3_float(c.scale + 1)));
    if (d > 0.f || (d == 0.f && (c.scale & 1))) c.scale += 1;
  }
  if (c.scale > 0 && c.scale < 0x7fu) {
    const float d = over(top, 3.f * (e4m3_float(c.scale) + e4m3_float(c.scale - 1)));
    if (d < 0.f || (d == 0.f && (c.scale & 1))) c.scale -= 1;
  }
  const float s = e4m3_float(c.scale);
  if (bad) c.scale = 0x7fu;
  c.codes = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const Two a = x[e].h < 0.f ? -x[e] : x[e];
    uint32_t m = 0;
    if (s > 0.f)
      m = (over(a, 0.25f * s) > 0.f) + (over(a, 0.75f * s) >= 0.f) + (over(a, 1.25f * s) > 0.f) + (over(a, 1.75f * s) >= 0.f) +
          (over(a, 2.5f * s) > 0.f) + (over(a, 3.5f * s) >= 0.f) + (over(a, 5.f * s) > 0.f);
    c.codes |= (m | (x[e].h < 0.f ? 8u : 0u)) << (4 * e);
  }
  return c;
}

// A group is 4 lanes' parts of one kind (quad: the turning lanes of pairs of
// halves, rot / 2 a multiple of 16) or both parts of 2 lanes.
template <typename F, typename M>
__device__ __forceinline__ void group_tops(F& x, F& y, bool quad, bool any_quad, M mx) {
  x = mx(x, __shfl_xor_sync(0xffffffffu, x, 1));
  y = mx(y, __shfl_xor_sync(0xffffffffu, y, 1));
  F a = x, b = y;
  if (any_quad) {
    a = mx(x, __shfl_xor_sync(0xffffffffu, x, 2));
    b = mx(y, __shfl_xor_sync(0xffffffffu, y, 2));
  }
  const F both = mx(x, y);
  x = quad ? a : both;
  y = quad ? b : both;
}

// Pairs of halves whose rot / 2 is no multiple of 16: the parts moved to
// neighbouring features, 8 l .. 8 l + 7 in lane l.
template <int LANES, typename F>
__device__ __forceinline__ void to_neighbours(F (&x)[4], F (&y)[4], int lane, int rot) {
  const int l = lane % LANES, half = rot >> 1;
  F out[2][4];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int f = 8 * l + 4 * q;
    const int src = f < half ? f >> 2 : (f < rot ? (f - half) >> 2 : f >> 3);
    const bool second = f < half ? false : (f < rot ? true : (f >> 2) & 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const F a = __shfl_sync(0xffffffffu, x[e], lane - l + src), b = __shfl_sync(0xffffffffu, y[e], lane - l + src);
      out[q][e] = second ? b : a;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) { x[e] = out[0][e]; y[e] = out[1][e]; }
}

// What a lane knows about turning keys.
struct KeyTurn {
  Parts pt;        // as loaded and turned
  bool moved;      // then moved to neighbouring features
  bool quad, any_quad;
};

// A lane's 8 features of a key, normed and turned, coded from FP32; false where that does not decide them.
// turn_band: kBand, of the terms of turned features.
template <int LANES>
__device__ __forceinline__ bool key_f32(const AppendParams& p, const KeyTurn& kt, const Angles& an, float turn_band,
                                        const Row8& gain, int lane, Row8 x, Coded& cx, Coded& cy) {
  float rs = p.k_scale;
  if (p.norm) rs *= rsqrtf(fmaf(row_sum<LANES>(x.dot(x)), 1.f / (8 * LANES), p.eps));
  x.times(rs);
  if (p.gain) x.times(gain);
  Row8 d;
  const float2 band = make_float2(kBand, kBand), tband = make_float2(turn_band, turn_band);
  auto mag = [](float2 a) { return make_float2(fabsf(a.x), fabsf(a.y)); };
  if (kt.pt.turns) {
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = turn_band * (fabsf(x.v[e].x) + fabsf(x.v[e].y));
        d.v[e] = make_float2(m, m);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) d.v[e] = d.v[e + 2] = __fmul2_rn(__fadd2_rn(mag(x.v[e]), mag(x.v[e + 2])), tband);
    }
    an.turn(x, p.interleaved);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) d.v[e] = __fmul2_rn(mag(x.v[e]), band);
  }
  if (kt.moved) {
    float a[4] = {x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y}, b[4] = {x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y};
    float u[4] = {d.v[0].x, d.v[0].y, d.v[1].x, d.v[1].y}, v[4] = {d.v[2].x, d.v[2].y, d.v[3].x, d.v[3].y};
    to_neighbours<LANES>(a, b, lane, p.rot);
    to_neighbours<LANES>(u, v, lane, p.rot);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x.v[e] = make_float2(a[2 * e], a[2 * e + 1]); x.v[e + 2] = make_float2(b[2 * e], b[2 * e + 1]);
      d.v[e] = make_float2(u[2 * e], u[2 * e + 1]); d.v[e + 2] = make_float2(v[2 * e], v[2 * e + 1]);
    }
  }
  float h[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 m = mag(x.v[e]);
    const float2 a = __fadd2_rn(m, d.v[e]), b = __fadd2_rn(m, make_float2(-d.v[e].x, -d.v[e].y));
    h[e >> 1] = max_nan(h[e >> 1], max_nan(a.x, a.y));
    w[e >> 1] = max_nan(w[e >> 1], max_nan(b.x, b.y));
  }
  auto mx = [](float a, float b) { return max_nan(a, b); };
  group_tops(h[0], h[1], kt.quad, kt.any_quad, mx);
  group_tops(w[0], w[1], kt.quad, kt.any_quad, mx);
  const float2 x0[2] = {x.v[0], x.v[1]}, x1[2] = {x.v[2], x.v[3]}, d0[2] = {d.v[0], d.v[1]}, d1[2] = {d.v[2], d.v[3]};
  const bool a = encode_banded(x0, d0, w[0], h[0], cx), b = encode_banded(x1, d1, w[1], h[1], cy);
  return a && b;
}

// The same in two parts each, from the loaded features: the parts' codes in x
// (low and high half), their scales in y.  how: bit 0 turns, 1 moved, 2 quad,
// 3 any_quad.
template <int LANES>
__device__ __noinline__ uint2 key_two(const AppendParams& p, int how, int f0, int f1, int lane, Row8 v, Angles an) {
  const float x0[8] = {v.v[0].x, v.v[0].y, v.v[1].x, v.v[1].y, v.v[2].x, v.v[2].y, v.v[3].x, v.v[3].y};
  const float c[4] = {an.c[0].x, an.c[0].y, an.c[1].x, an.c[1].y}, s[4] = {an.s[0].x, an.s[0].y, an.s[1].x, an.s[1].y};
  const bool quad = how & 4, any_quad = how & 8;
  Two rs = {1.f, 0.f};
  if (p.norm) {
    Two ss = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {     // a BF16 number's square is an FP32 number
      const Two a = sum_of(ss.h, __fmul_rn(x0[e], x0[e]));
      ss = {a.h, __fadd_rn(ss.l, a.l)};
    }
    ss = join(ss.h, ss.l);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
      ss = ss + Two{__shfl_xor_sync(0xffffffffu, ss.h, o), __shfl_xor_sync(0xffffffffu, ss.l, o)};
    rs = rsqrt_two(ss * (1.f / (8 * LANES)) + Two{p.eps, 0.f});
  }
  Two x[4], y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = rs * x0[e] * (p.gain ? p.gain[f0 + e] : 1.f);
    y[e] = rs * x0[4 + e] * (p.gain ? p.gain[f1 + e] : 1.f);
  }
  if (how & 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      Two& a = p.interleaved ? (e < 2 ? x[2 * e] : y[2 * e - 4]) : x[e];
      Two& b = p.interleaved ? (e < 2 ? x[2 * e + 1] : y[2 * e - 3]) : y[e];
      const Two u = a * c[e] + -(b * s[e]), w = b * c[e] + a * s[e];
      a = u;
      b = w;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {     // the power of two last: what passes FP32 here lies above every border
    x[e] = x[e] * p.k_scale;
    y[e] = y[e] * p.k_scale;
  }
  if (how & 2) {
    float xh[4], xl[4], yh[4], yl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) { xh[e] = x[e].h; xl[e] = x[e].l; yh[e] = y[e].h; yl[e] = y[e].l; }
    to_neighbours<LANES>(xh, yh, lane, p.rot);
    to_neighbours<LANES>(xl, yl, lane, p.rot);
#pragma unroll
    for (int e = 0; e < 4; ++e) { x[e] = {xh[e], xl[e]}; y[e] = {yh[e], yl[e]}; }
  }
  // a group's largest magnitude: in the order of (h, l), as one 64-bit number
  unsigned long long tx = 0, ty = 0;
  float bx = 0.f, by = 0.f;           // 1: a NaN
  auto largest = [](Two& a, unsigned long long& top, float& bad) {
    if (a.h != a.h) {
      bad = 1.f;
    } else {
      const Two m = a.h < 0.f ? -a : a;
      const uint32_t low = __float_as_uint(m.l);
      const unsigned long long key = ((unsigned long long)__float_as_uint(fabsf(m.h)) << 32) |
                                     (low ^ ((int)low < 0 ? 0xffffffffu : 0x80000000u));
      top = key > top ? key : top;
    }
  };
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    largest(x[e], tx, bx);
    largest(y[e], ty, by);
  }
  group_tops(tx, ty, quad, any_quad, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; });
  group_tops(bx, by, quad, any_quad, [](float a, float b) { return fmaxf(a, b); });
  auto value = [](unsigned long long key) -> Two {
    const uint32_t low = (uint32_t)key;
    return {__uint_as_float((uint32_t)(key >> 32)), key ? __uint_as_float(low ^ ((int)low < 0 ? 0x80000000u : 0xffffffffu)) : 0.f};
  };
  const Coded cx = encode_two(x, value(tx), bx != 0.f), cy = encode_two(y, value(ty), by != 0.f);
  return make_uint2((cx.codes & 0xffffu) | (cy.codes << 16), cx.scale | (cy.scale << 8));
}

// A position's page and place.
struct Slot {
  int64_t page;
  int place, pos;
};

// false (recorded) where the tables do not give one
__device__ __forceinline__ bool find_slot(const int32_t* table, int max_pages, int page_log, int num_pages, int b, int64_t pos,
                                          int* hdr, Slot& s) {
  bool ok = pos >= 0 && pos < ((int64_t)max_pages << page_log);
  if (ok) {
    s.pos = (int)pos;
    s.page = table[(int64_t)b * max_pages + (s.pos >> page_log)];
    s.place = s.pos & ((1 << page_log) - 1);
    ok = s.page >= 0 && s.page < num_pages;
  }
  if (!ok) set_error(hdr, HSTU_ERR_DEVICE_CHECK, b);
  return ok;
}

// A walk over neighbouring tokens: the token's sequence and place, looked up
// again where a sequence or a page ends.  lens: cache lengths after an append
// (the tokens are the last ones), or starts of a read (NULL: 0).
template <bool APPEND>
struct Places {
  FoundSeq seq;
  Slot slot;
  bool found = false;

  // false: no place (recorded), or a padded batch's row (done)
  template <typename P>
  __device__ __forceinline__ bool at(const P& p, const int32_t* lens, int64_t t, int64_t total) {
    if (!found || t >= seq.end) {
      seq = warp_find_sequence(p.off, lens, p.B, t);
      found = t < total;
      if (!found) return false;
    } else if ((++slot.place & ((1 << p.page_log) - 1)) != 0) {
      ++slot.pos;                         // the next place of the same page
      return true;
    }
    const int64_t pos = APPEND ? seq.aux - (seq.end - t) : seq.aux + (t - seq.begin);
    // the first test fails only for offsets that decrease somewhere
    const bool in = seq.begin <= t && t < seq.end && seq.aux >= (APPEND ? seq.end - seq.begin : 0);
    if (find_slot(p.table, p.max_pages, p.page_log, p.num_pages, seq.b, in ? pos : -1, p.hdr, slot)) return true;
    found = false;
    return false;
  }
};

// Offsets that do not fit the rows are recorded; nothing is done then.
__device__ __forceinline__ bool fits(int64_t first, int64_t total, int64_t T, int* hdr) {
  if (first == 0 && total >= 0 && total <= T) return true;
  if ((threadIdx.x & 31) == 0) set_error(hdr, HSTU_ERR_DEVICE_CHECK, -1);
  return false;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 5) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
  int64_t t = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.tokens_per_warp;
  const int64_t t_end = t + p.tokens_per_warp < p.T ? t + p.tokens_per_warp : p.T;
  if (t >= p.T) return;
  const bool work = p.rot || p.norm;            // keys change on their way
  const int ph = (p.H + PER - 1) / PER;
  KeyTurn kt = {Parts(l, p.rot, p.interleaved), false, false, false};
  const int v0 = 8 * l;                         // values lie side by side
  int f0 = kt.pt.f0, f1 = kt.pt.f1;             // of a key's coded parts
  if (!p.interleaved && p.rot > 8) {
    kt.moved = p.rot % 32 != 0;
    kt.any_quad = !kt.moved;
    kt.quad = kt.any_quad && kt.pt.turns;
    if (kt.moved) { f0 = v0; f1 = v0 + 4; }
  }
  Raw4<__nv_bfloat16> k0, k1, u0, u1;
  auto load = [&](int64_t tok, int i) {
    const int head = i * PER + sub;
    if (head < p.H) {
      const __nv_bfloat16 *k = p.k + tok * p.ks[0] + head * p.ks[1], *v = p.v + tok * p.vs[0] + head * p.vs[1];
      k0 = fetch4(k + kt.pt.f0);
      k1 = fetch4(k + kt.pt.f1);
      u0 = fetch4(v + v0);
      u1 = fetch4(v + v0 + 4);
    }
  };
  load(t, 0);
  const int64_t off0 = p.off[0], total = p.off[p.B];
  Places<true> pl;
  Row8 gain;
  if (p.gain) gain = Row8(fetch4(p.gain + kt.pt.f0), fetch4(p.gain + kt.pt.f1));
  const PageLayout lay(1 << p.page_log, D);
  for (; t < t_end; ++t) {
    bool placed = pl.at(p, p.lens, t, total);
    if (!fits(off0, total, p.T, p.hdr) || t >= total) return;
    const Slot sl = pl.slot;
    if (placed && p.rot && sl.pos >= p.max_pos) {   // behind the tables
      if (lane == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, pl.seq.b);
      placed = false;
    }
    if (!placed) {    // this token is left out; the next ones may belong to other sequences
      if (t + 1 < t_end) load(t + 1, 0);
      continue;
    }
    Angles an;
    float turn_band = kBand;
    if (p.rot && kt.pt.turns) {
      const int64_t at = (int64_t)sl.pos * (p.rot >> 1) + 4 * l;
      an.load(p.cos + at, p.sin + at, 1.f);
      turn_band *= fmaxf(1.f, an.largest());
    }
    uint8_t* block = p.pages + sl.page * p.H * (int64_t)lay.bytes();
    const int place_c = sl.place * lay.code_row, place_s = lay.scales() + sl.place * lay.scale_row;
    for (int i = 0; i < ph; ++i) {
      const int head = i * PER + sub;
      uint8_t* part = block + head * lay.bytes();
      const Row8 kx(k0, k1);
      Row8 vx(u0, u1);
      // the next pass's rows
      if (i + 1 < ph) load(t, i + 1);
      else if (t + 1 < t_end) load(t + 1, 0);
      if (work) {
        Coded cx, cy;
        const bool sure = key_f32<LANES>(p, kt, an, turn_band, gain, lane, kx, cx, cy);
        if (__any_sync(0xffffffffu, !sure && head < p.H)) {
          const uint2 r = key_two<LANES>(
              p, (kt.pt.turns ? 1 : 0) | (kt.moved ? 2 : 0) | (kt.quad ? 4 : 0) | (kt.any_quad ? 8 : 0), kt.pt.f0, kt.pt.f1,
              lane, kx, an);
          cx.codes = r.x & 0xffffu; cy.codes = r.x >> 16;
          cx.scale = r.y & 0xffu; cy.scale = r.y >> 8;
        }
        if (head < p.H) {
          uint8_t *codes = part + place_c, *scales = part + place_s;
          if (kt.quad) {
            *reinterpret_cast<uint16_t*>(codes + (f0 >> 1)) = (uint16_t)cx.codes;
            *reinterpret_cast<uint16_t*>(codes + (f1 >> 1)) = (uint16_t)cy.codes;
            if ((l & 3) == 0) {
              scales[f0 >> 4] = (uint8_t)cx.scale;
              scales[f1 >> 4] = (uint8_t)cy.scale;
            }
          } else {
            *reinterpret_cast<uint32_t*>(codes + (f0 >> 1)) = cx.codes | (cy.codes << 16);
            if ((l & 1) == 0) scales[f0 >> 4] = (uint8_t)cx.scale;
          }
        }
      }
      // values, and keys that go in as they are
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (w == 0 && work) continue;
        Row8 x = w ? vx : kx;
        x.times(w ? p.v_scale : p.k_scale);
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max_nan(top, max_nan(fabsf(x.v[e].x), fabsf(x.v[e].y)));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const uint2 r = encode_exact(x, top);
        if (head < p.H) {
          uint8_t* half = part + (w ? lay.half() : 0);
          *reinterpret_cast<uint32_t*>(half + place_c + 4 * l) = r.x;
          if ((l & 1) == 0) half[place_s + (l >> 1)] = (uint8_t)r.y;
        }
      }
    }
    if (p.page_times && lane == 0) p.page_times[(sl.page << p.page_log) + sl.place] = p.times[t];
  }
}

struct ReadParams {
  const int64_t* off;
  const int32_t* starts;
  const int32_t* table;
  const uint8_t* pages;
  const int64_t* page_times;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int64_t* times;
  int* hdr;
  int64_t T;
  int B, H, page_log, num_pages, max_pages, tokens_per_warp;
  float k_scale, v_scale;   // 2^k_exp, 2^v_exp
};

// A lane takes 8 features (4 bytes of codes, 16 bytes out: a warp's store is
// whole lines), a warp kManyTokens neighbouring tokens' keys and values, 256
// features of each a pass, all loads of a pass first.
template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES;
  const int64_t t = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.tokens_per_warp;
  const int64_t t_end = t + p.tokens_per_warp < p.T ? t + p.tokens_per_warp : p.T;
  if (t >= p.T) return;
  const int64_t off0 = p.off[0], total = p.off[p.B];
  Places<false> pl;
  const PageLayout lay(1 << p.page_log, D);
  const int ph = (p.H + PER - 1) / PER;
  auto two = [&](__half2 v, float s) -> uint32_t {
    const float2 x = __fmul2_rn(__half22float2(v), make_float2(s, s));
    const __nv_bfloat162 y = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&y);
  };
  int64_t from[kManyTokens];    // where a token's codes of head 0 lie; -1: nowhere
  int rel[kManyTokens];         // of its scales, from there
#pragma unroll
  for (int n = 0; n < kManyTokens; ++n) {
    from[n] = -1;
    if (t + n >= t_end) continue;
    const bool placed = pl.at(p, p.starts, t + n, total);
    if (!fits(off0, total, p.T, p.hdr)) return;
    if (!placed) continue;      // a padded batch's row, or recorded
    from[n] = pl.slot.page * p.H * (int64_t)lay.bytes() + pl.slot.place * lay.code_row;
    rel[n] = lay.scales() + pl.slot.place * (lay.scale_row - lay.code_row);
    if (p.times && lane == 0) p.times[t + n] = p.page_times[(pl.slot.page << p.page_log) + pl.slot.place];
  }
  for (int i = 0; i < ph; ++i) {
    const int head = i * PER + sub;
    if (head >= p.H) break;
    uint32_t w[kManyTokens][2];
    uint32_t sc[kManyTokens][2];
#pragma unroll
    for (int n = 0; n < kManyTokens; ++n) {
      if (from[n] < 0) continue;
      const uint8_t* codes = p.pages + from[n] + head * lay.bytes();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        w[n][x] = *reinterpret_cast<const uint32_t*>(codes + x * lay.half() + g * 4);
        sc[n][x] = codes[x * lay.half() + rel[n] + (g >> 1)];
      }
    }
#pragma unroll
    for (int n = 0; n < kManyTokens; ++n) {
      if (from[n] < 0) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        __nv_bfloat16* dst = x ? p.v : p.k;
        if (!dst) continue;
        const float s = e4m3_float(sc[n][x]) * (x ? p.v_scale : p.k_scale);
        const uint32_t c = w[n][x];
        *reinterpret_cast<uint4*>(dst + ((t + n) * p.H + head) * D + g * 8) =
            make_uint4(two(e2m1x2_half2<0>(c), s), two(e2m1x2_half2<1>(c), s), two(e2m1x2_half2<2>(c), s),
                       two(e2m1x2_half2<3>(c), s));
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// One token a warp in a small batch, else four.  Eight sequences, four heads of
// 128, one call after the other, by tokens, one and four a warp: append 1,000 6.8
// and 13.7 us, 4,000 11.1 and 14.6, 7,300 15.4 and 18.4, 12,000 21.4 and 22.3,
// 24,000 38.6 and 36.3, 48,000 76 and 68; read 1,000 3.2 and 3.7, 4,000 3.8 and
// 4.0, 7,300 5.5 and 4.6, 12,000 7.9 and 5.9, 48,000 37 and 25.  The switch lies
// between the read's (5,000) and the append's (some 20,000).
int tokens_per_warp(int64_t T) { return T > 152 * 48 ? kManyTokens : 1; }

int page_log(int page_size) { return page_size == 32 ? 5 : (page_size == 64 ? 6 : 7); }

hstu_status_t launch_error(cudaError_t e, const char* what) {
  (void)cudaGetLastError();
  set_error_detail(e, what);
  return HSTU_ERR_CUDA;
}

}  // namespace

hstu_status_t check_cache_desc(const hstu_cache_desc* c, bool buffers) {
  if (!c || c->struct_size != sizeof(hstu_cache_desc)) return HSTU_ERR_INVALID_ARG;
  if (c->H < 1 || c->num_pages < 1 || c->max_pages < 1) return HSTU_ERR_INVALID_ARG;
  if (c->k_exp < -32 || c->k_exp > 32 || c->v_exp < -32 || c->v_exp > 32) return HSTU_ERR_INVALID_ARG;
  if ((c->d != 64 && c->d != 128) || (c->page_size != 32 && c->page_size != 64 && c->page_size != 128))
    return HSTU_ERR_UNSUPPORTED;
  if (c->H * (int64_t)c->d > 2048) return HSTU_ERR_UNSUPPORTED;
  if (c->max_pages > (1 << 24)) return HSTU_ERR_UNSUPPORTED;   // positions stay below 2^31
  if (buffers && (!c->pages || !aligned16(c->pages) || (c->timestamps && !aligned16(c->timestamps))))
    return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_cache_bytes(const hstu_cache_desc* c, size_t* page_bytes, size_t* total_bytes) {
  const hstu_status_t s = check_cache_desc(c, false);
  if (s != HSTU_OK) return s;
  const size_t page = (size_t)PageLayout(c->page_size, c->d).bytes() * (size_t)c->H;
  if (page_bytes) *page_bytes = page;
  if (total_bytes) *total_bytes = page * (size_t)c->num_pages;
  return HSTU_OK;
}

hstu_status_t hstu_cache_append(const hstu_cache_desc* c, const hstu_cache_append_args* a, void* workspace,
                                size_t workspace_bytes, hstu_stream_t stream) {
  const hstu_status_t s = check_cache_desc(c, true);
  if (s != HSTU_OK) return s;
  if (!a || a->B < 0 || a->total_tokens < 0 || a->reserved != 0 || (a->interleaved & ~1) || (a->norm & ~1))
    return HSTU_ERR_INVALID_ARG;
  if (a->norm && !(a->eps >= 0.f && a->eps < 1e30f)) return HSTU_ERR_INVALID_ARG;
  if (!a->norm && a->k_gain) return HSTU_ERR_INVALID_ARG;
  if (a->rot_dim < 0 || a->rot_dim > c->d || (a->rot_dim > 0 && a->max_position < 1)) return HSTU_ERR_INVALID_ARG;
  if (a->rot_dim % 8 != 0 || a->total_tokens > ((int64_t)1 << 30)) return HSTU_ERR_UNSUPPORTED;
  if (!a->seq_offsets) return HSTU_ERR_INVALID_ARG;
  if (a->total_tokens > 0 && a->B > 0) {
    if (!a->cache_lens || !a->block_table || !a->k || !a->v || (a->rot_dim > 0 && (!a->cos || !a->sin)))
      return HSTU_ERR_INVALID_ARG;
    if ((a->token_times == nullptr) != (c->timestamps == nullptr)) return HSTU_ERR_INVALID_ARG;
  }
  for (const void* ptr : {a->k, a->v, (const void*)a->cos, (const void*)a->sin, (const void*)a->k_gain})
    if (ptr && !aligned16(ptr)) return HSTU_ERR_INVALID_ARG;
  if (a->k_strides[0] % 8 || a->k_strides[1] % 8 || a->v_strides[0] % 8 || a->v_strides[1] % 8)
    return HSTU_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) || workspace_bytes < kWsHeaderBytes)
    return HSTU_ERR_WORKSPACE;
  reset_launches();
  if (a->total_tokens == 0 || a->B == 0) return HSTU_OK;
  AppendParams p{};
  p.off = a->seq_offsets; p.lens = a->cache_lens; p.table = a->block_table; p.times = a->token_times;
  p.cos = a->cos; p.sin = a->sin; p.gain = a->k_gain;
  p.k = static_cast<const __nv_bfloat16*>(a->k); p.v = static_cast<const __nv_bfloat16*>(a->v);
  for (int i = 0; i < 2; ++i) { p.ks[i] = a->k_strides[i]; p.vs[i] = a->v_strides[i]; }
  p.pages = static_cast<uint8_t*>(c->pages); p.page_times = c->timestamps; p.hdr = static_cast<int*>(workspace);
  p.T = a->total_tokens; p.max_pos = a->max_position;
  p.B = a->B; p.H = c->H; p.page_log = page_log(c->page_size); p.num_pages = c->num_pages; p.max_pages = c->max_pages;
  p.rot = a->rot_dim; p.interleaved = a->interleaved; p.norm = a->norm; p.eps = a->eps;
  p.k_scale = ldexpf(1.f, -c->k_exp); p.v_scale = ldexpf(1.f, -c->v_exp);
  p.tokens_per_warp = tokens_per_warp(p.T);
  const unsigned ctas = (unsigned)((p.T + kWarps * p.tokens_per_warp - 1) / (kWarps * p.tokens_per_warp));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c->d == 128 ? launch_pdl(append_kernel<128>, dim3(ctas), dim3(kThreads), 0, st, p)
                                    : launch_pdl(append_kernel<64>, dim3(ctas), dim3(kThreads), 0, st, p);
  if (e != cudaSuccess) return launch_error(e, "launching append_kernel");
  note_launches(1);
  return HSTU_OK;
}

hstu_status_t hstu_cache_read(const hstu_cache_desc* c, const hstu_cache_read_args* a, void* workspace,
                              size_t workspace_bytes, hstu_stream_t stream) {
  const hstu_status_t s = check_cache_desc(c, true);
  if (s != HSTU_OK) return s;
  if (!a || a->B < 0 || a->total_tokens < 0 || a->reserved != 0 || !a->seq_offsets) return HSTU_ERR_INVALID_ARG;
  if (a->total_tokens > ((int64_t)1 << 30)) return HSTU_ERR_UNSUPPORTED;
  if (a->total_tokens > 0 && a->B > 0 && !a->block_table) return HSTU_ERR_INVALID_ARG;
  if (a->token_times && !c->timestamps) return HSTU_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)a->k, (const void*)a->v})
    if (ptr && !aligned16(ptr)) return HSTU_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) || workspace_bytes < kWsHeaderBytes)
    return HSTU_ERR_WORKSPACE;
  reset_launches();
  if (a->total_tokens == 0 || a->B == 0) return HSTU_OK;
  ReadParams p{};
  p.off = a->seq_offsets; p.starts = a->starts; p.table = a->block_table;
  p.pages = static_cast<const uint8_t*>(c->pages); p.page_times = c->timestamps;
  p.k = static_cast<__nv_bfloat16*>(a->k); p.v = static_cast<__nv_bfloat16*>(a->v); p.times = a->token_times;
  p.hdr = static_cast<int*>(workspace);
  p.T = a->total_tokens;
  p.B = a->B; p.H = c->H; p.page_log = page_log(c->page_size); p.num_pages = c->num_pages; p.max_pages = c->max_pages;
  p.k_scale = ldexpf(1.f, c->k_exp); p.v_scale = ldexpf(1.f, c->v_exp);
  p.tokens_per_warp = tokens_per_warp(p.T);
  const unsigned ctas = (unsigned)((p.T + kWarps * p.tokens_per_warp - 1) / (kWarps * p.tokens_per_warp));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c->d == 128 ? launch_pdl(read_kernel<128>, dim3(ctas), dim3(kThreads), 0, st, p)
                                    : launch_pdl(read_kernel<64>, dim3(ctas), dim3(kThreads), 0, st, p);
  if (e != cudaSuccess) return launch_error(e, "launching read_kernel");
  note_launches(1);
  return HSTU_OK;
}

}  // extern "C"
