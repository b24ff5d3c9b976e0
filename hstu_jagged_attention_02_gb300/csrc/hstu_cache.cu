// Appending to and reading from the paged 4-bit cache (hstu_cache_append,
// hstu_cache_read).
//
// Append: bound by the BF16 rows it reads (2 d bytes in, 9 d / 16 out), if the
// instructions are few.  d / 8 lanes hold a row (hstu_rows.cuh: both features
// of a pair in one lane), a warp takes one token, kPasses passes of 256
// features at a time, all loads first; its place in the cache is looked up
// once.  A group's maximum goes over the 2 or 4 lanes that share it.
//
// Roundings are decided as on real numbers.  A value x that is exact in FP32
// (a BF16 input) meets a border only exactly: its quotient by the scale (4
// significant bits) lies at least 2^-13 from a border or on it, so the
// quotient by the reciprocal, rounded to 16 significant bits, decides rightly.
// A normed or rotated key is known to 2^-20 of its terms only; where the
// codes (or the scale) of x - d and x + d differ, the warp computes its rows
// again in FP64 and compares with the borders themselves.  That happens to
// about one row in a thousand.
#include "hstu_fp4.cuh"
#include "hstu_internal.h"
#include "hstu_rows.cuh"
#include "hstu_seq_search.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPasses = 4;
constexpr float kBand = 1.9073486328125e-06f;   // 2^-19: 2^-20 of the terms, and as much for the quotient

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
  int rot, interleaved, norm;
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

__device__ __forceinline__ float max4(const float (&x)[4]) {
  return max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3])));
}

// y = x / s for a scale s, rounded to 16 significant bits: right on a border
// exactly where the quotient of an exact x is.
__device__ __forceinline__ float quotient(float x, float inv) {
  return __uint_as_float((__float_as_uint(x * inv) + 0x80u) & 0xffffff00u);
}

// 4 features that are exact in FP32, top the largest magnitude of their group.
__device__ __forceinline__ Coded encode_exact(const float (&x)[4], float top) {
  Coded c;
  c.scale = e4m3_of(__fdiv_rn(top, 6.f));
  const float s = e4m3_float(c.scale), inv = s > 0.f ? __frcp_rn(s) : 0.f;
  c.codes = e2m1x2_of(quotient(x[0], inv), quotient(x[1], inv)) | (e2m1x2_of(quotient(x[2], inv), quotient(x[3], inv)) << 8);
  return c;
}

// 4 features known to +-d[e], and their group's largest magnitude to [lo, hi]:
// false where that does not decide the result.
__device__ __forceinline__ bool encode_banded(const float (&x)[4], const float (&d)[4], float lo, float hi, Coded& c) {
  c.scale = e4m3_of(hi * (0.16666667f * 1.0000005f));
  bool sure = c.scale == e4m3_of(lo * (0.16666667f * 0.9999995f));
  const float s = e4m3_float(c.scale), inv = s > 0.f ? __frcp_rn(s) : 0.f;
  float a[4], b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = x[e] * inv, w = d[e] * inv;
    a[e] = y - w;
    b[e] = y + w;
  }
  c.codes = e2m1x2_of(a[0], a[1]) | (e2m1x2_of(a[2], a[3]) << 8);
  const uint32_t other = e2m1x2_of(b[0], b[1]) | (e2m1x2_of(b[2], b[3]) << 8);
  // codes that differ, but for the sign of a zero
  const uint32_t diff = (c.codes ^ other) & 0xffffu, mags = (c.codes | other) & 0x7777u;
  const uint32_t nonzero = (mags | (mags >> 1) | (mags >> 2)) & 0x1111u;
  return sure && (diff & (nonzero * 15u)) == 0;
}

// The same from FP64 (every border compared with itself); bad: a NaN in the group.
__device__ __noinline__ Coded encode_f64(double x0, double x1, double x2, double x3, double top, bool bad) {
  const double x[4] = {x0, x1, x2, x3};
  Coded c;
  // the nearest scale by its FP32 neighbour, then its two borders (halves between scales) times 6
  c.scale = e4m3_of((float)(top / 6.0));
  if (c.scale < 0x7eu) {
    const double here = e4m3_float(c.scale), up = e4m3_float(c.scale + 1);
    const double border = 3.0 * (here + up);
    if (top > border || (top == border && (c.scale & 1))) c.scale += 1;
  }
  if (c.scale > 0 && c.scale < 0x7fu) {
    const double here = e4m3_float(c.scale), down = e4m3_float(c.scale - 1);
    const double border = 3.0 * (here + down);
    if (top < border || (top == border && (c.scale & 1))) c.scale -= 1;
  }
  const double s = e4m3_float(c.scale);
  if (bad) c.scale = 0x7fu;
  c.codes = 0;
  for (int e = 0; e < 4; ++e) {
    const double a = fabs(x[e]);
    uint32_t m = 0;
    if (s > 0.0)
      m = (a > 0.25 * s) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) + (a > 2.5 * s) + (a >= 3.5 * s) +
          (a > 5.0 * s);
    c.codes |= (m | (x[e] < 0.0 ? 8u : 0u)) << (4 * e);
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

// What a lane knows about turning the token's keys.
struct KeyTurn {
  Parts pt;        // as loaded and turned
  bool moved;      // then moved to neighbouring features
  bool quad, any_quad;
  float c[4], s[4];
};

// Two parts of a key row, normed and turned, coded from FP32; false where FP64 has to decide.
template <int LANES>
__device__ __forceinline__ bool key_f32(const AppendParams& p, const KeyTurn& kt, int lane, float (&x)[4], float (&y)[4],
                                        Coded& cx, Coded& cy) {
  float rs = p.k_scale;
  if (p.norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
    rs *= __frsqrt_rn(fmaf(row_sum<LANES>(ss), 1.f / (8 * LANES), p.eps));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) { x[e] *= rs; y[e] *= rs; }
  if (p.gain) {
    float a[4], b[4];
    load4(p.gain + kt.pt.f0, a);
    load4(p.gain + kt.pt.f1, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) { x[e] *= a[e]; y[e] *= b[e]; }
  }
  float dx[4], dy[4];
  if (kt.pt.turns) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // the pair's size bounds both of its terms
      if (p.interleaved) {
        dx[e] = kBand * (fabsf(x[e]) + fabsf(x[e ^ 1]));
        dy[e] = kBand * (fabsf(y[e]) + fabsf(y[e ^ 1]));
      } else {
        dx[e] = dy[e] = kBand * (fabsf(x[e]) + fabsf(y[e]));
      }
    }
    turn_pairs(x, y, kt.c, kt.s, p.interleaved);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) { dx[e] = kBand * fabsf(x[e]); dy[e] = kBand * fabsf(y[e]); }
  }
  if (kt.moved) {
    to_neighbours<LANES>(x, y, lane, p.rot);
    to_neighbours<LANES>(dx, dy, lane, p.rot);
  }
  float hx = 0.f, hy = 0.f, lx = 0.f, ly = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hx = max_nan(hx, fabsf(x[e]) + dx[e]);
    hy = max_nan(hy, fabsf(y[e]) + dy[e]);
    lx = max_nan(lx, fabsf(x[e]) - dx[e]);
    ly = max_nan(ly, fabsf(y[e]) - dy[e]);
  }
  auto mx = [](float a, float b) { return max_nan(a, b); };
  group_tops(hx, hy, kt.quad, kt.any_quad, mx);
  group_tops(lx, ly, kt.quad, kt.any_quad, mx);
  const bool a = encode_banded(x, dx, lx, hx, cx), b = encode_banded(y, dy, ly, hy, cy);
  return a && b;
}

// The same in FP64, from the loaded features x, y (cosines c, sines s): the
// parts' codes in x (low and high half), their scales in y.  how: bit 0
// turns, 1 moved, 2 quad, 3 any_quad.
template <int LANES>
__device__ __noinline__ uint2 key_f64(const AppendParams& p, int how, int f0, int f1, int lane, float4 x4, float4 y4, float4 c4,
                                      float4 s4) {
  const float x0[4] = {x4.x, x4.y, x4.z, x4.w}, y0[4] = {y4.x, y4.y, y4.z, y4.w};
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
  const bool quad = how & 4, any_quad = how & 8;
  double x[4], y[4], rs = 1.0;
  if (p.norm) {
    double ss = 0.0;
    for (int e = 0; e < 4; ++e) ss += (double)x0[e] * x0[e] + (double)y0[e] * y0[e];
    rs = 1.0 / sqrt(row_sum<LANES>(ss) / (8 * LANES) + (double)p.eps);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = x0[e] * rs * (p.gain ? (double)p.gain[f0 + e] : 1.0) * p.k_scale;
    y[e] = y0[e] * rs * (p.gain ? (double)p.gain[f1 + e] : 1.0) * p.k_scale;
  }
  if (how & 1) turn_pairs(x, y, c, s, p.interleaved);
  if (how & 2) to_neighbours<LANES>(x, y, lane, p.rot);
  double tx = 0.0, ty = 0.0;
  double bx = 0.0, by = 0.0;        // 1: a NaN, which the maximum passes over
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    tx = fmax(tx, fabs(x[e]));
    ty = fmax(ty, fabs(y[e]));
    if (x[e] != x[e]) bx = 1.0;
    if (y[e] != y[e]) by = 1.0;
  }
  auto mx = [](double a, double b) { return fmax(a, b); };
  group_tops(tx, ty, quad, any_quad, mx);
  group_tops(bx, by, quad, any_quad, mx);
  const Coded cx = encode_f64(x[0], x[1], x[2], x[3], tx, bx != 0.0);
  const Coded cy = encode_f64(y[0], y[1], y[2], y[3], ty, by != 0.0);
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

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const bool work = p.rot || p.norm;            // keys change on their way
  const int ph = (p.H + PER - 1) / PER;         // passes over the keys, then as many over the values
  const Parts kp(l, work ? p.rot : 0, p.interleaved), vp(l, 0, true);
  Raw4<__nv_bfloat16> r0[kPasses], r1[kPasses];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i0 + i >= 2 * ph) break;
      const bool key = i0 + i < ph;
      const int head = min((i0 + i - (key ? 0 : ph)) * PER + sub, p.H - 1);
      const __nv_bfloat16* src = key ? p.k + t * p.ks[0] + head * p.ks[1] : p.v + t * p.vs[0] + head * p.vs[1];
      r0[i] = fetch4(src + (key ? kp.f0 : vp.f0));
      r1[i] = fetch4(src + (key ? kp.f1 : vp.f1));
    }
  };
  load(0);
  const int64_t total = p.off[p.B];
  if (total > p.T || p.off[0] != 0) {
    if (lane == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return;
  }
  if (t >= total) return;                 // a padded batch's row
  const int b = warp_find_sequence(p.off, p.B, t);
  const int64_t o0 = p.off[b], o1 = p.off[b + 1];
  Slot sl;
  const bool in = o0 <= t && t < o1;      // false only for offsets that decrease somewhere
  if (!find_slot(p.table, p.max_pages, p.page_log, p.num_pages, b, in ? p.lens[b] - (o1 - o0) + (t - o0) : -1, p.hdr, sl))
    return;
  KeyTurn kt = {kp, false, false, false, {1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}};
  int f0 = kp.f0, f1 = kp.f1;             // of a key's coded parts
  if (p.rot) {
    if (sl.pos >= p.max_pos) {
      if (lane == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, b);
      return;
    }
    if (kp.turns) {
      const int64_t at = (int64_t)sl.pos * (p.rot >> 1) + 4 * l;
      load4(p.cos + at, kt.c);
      load4(p.sin + at, kt.s);
    }
    if (!p.interleaved && p.rot > 8) {
      kt.moved = p.rot % 32 != 0;
      kt.any_quad = !kt.moved;
      kt.quad = kt.any_quad && kp.turns;
      if (kt.moved) { f0 = vp.f0; f1 = vp.f1; }
    }
  }
  const PageLayout lay(1 << p.page_log, D);
  uint8_t* block = p.pages + sl.page * p.H * (int64_t)lay.bytes();
  for (int i0 = 0; i0 < 2 * ph; i0 += kPasses) {
    if (i0) load(i0);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i0 + i >= 2 * ph) break;
      const bool key = i0 + i < ph;
      const int head = (i0 + i - (key ? 0 : ph)) * PER + sub;
      float x[4], y[4];
      unpack4(r0[i], x);
      unpack4(r1[i], y);
      Coded cx, cy;
      if (key && work) {
        const bool sure = key_f32<LANES>(p, kt, lane, x, y, cx, cy);
        if (__any_sync(0xffffffffu, !sure)) {
          unpack4(r0[i], x);
          unpack4(r1[i], y);
          const uint2 r = key_f64<LANES>(
              p, (kp.turns ? 1 : 0) | (kt.moved ? 2 : 0) | (kt.quad ? 4 : 0) | (kt.any_quad ? 8 : 0), kp.f0, kp.f1, lane,
              make_float4(x[0], x[1], x[2], x[3]), make_float4(y[0], y[1], y[2], y[3]),
              make_float4(kt.c[0], kt.c[1], kt.c[2], kt.c[3]), make_float4(kt.s[0], kt.s[1], kt.s[2], kt.s[3]));
          cx.codes = r.x & 0xffffu; cy.codes = r.x >> 16;
          cx.scale = r.y & 0xffu; cy.scale = r.y >> 8;
        }
      } else {
        const float sc = key ? p.k_scale : p.v_scale;
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[e] *= sc; y[e] *= sc; }
        float top = max_nan(max4(x), max4(y));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        cx = encode_exact(x, top);
        cy = encode_exact(y, top);
      }
      if (head < p.H) {
        uint8_t* part = block + head * lay.bytes() + (key ? 0 : lay.half());
        uint8_t* codes = part + sl.place * lay.code_row;
        uint8_t* scales = part + lay.scales() + sl.place * lay.scale_row;
        const int a = key ? f0 : vp.f0, bb = key ? f1 : vp.f1;
        if (key && kt.quad) {
          *reinterpret_cast<uint16_t*>(codes + (a >> 1)) = (uint16_t)cx.codes;
          *reinterpret_cast<uint16_t*>(codes + (bb >> 1)) = (uint16_t)cy.codes;
          if ((l & 3) == 0) {
            scales[a >> 4] = (uint8_t)cx.scale;
            scales[bb >> 4] = (uint8_t)cy.scale;
          }
        } else {
          *reinterpret_cast<uint32_t*>(codes + (a >> 1)) = (cx.codes & 0xffffu) | (cy.codes << 16);
          if ((l & 1) == 0) scales[a >> 4] = (uint8_t)cx.scale;
        }
      }
    }
  }
  if (p.page_times && lane == 0) p.page_times[(sl.page << p.page_log) + sl.place] = p.times[t];
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
  int B, H, page_log, num_pages, max_pages;
  float k_scale, v_scale;   // 2^k_exp, 2^v_exp
};

// A lane takes 16 features (8 bytes of codes and their scale), a warp one
// token, 512 features a pass, the loads of kPasses passes first.
template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int LANES = D / 16, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int64_t total = p.off[p.B];
  if (total > p.T || p.off[0] != 0) {
    if (lane == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return;
  }
  if (t >= total) return;
  const int b = warp_find_sequence(p.off, p.B, t);
  const int64_t o0 = p.off[b], o1 = p.off[b + 1];
  const int64_t start = p.starts ? p.starts[b] : 0;
  Slot sl;
  if (!find_slot(p.table, p.max_pages, p.page_log, p.num_pages, b, o0 <= t && t < o1 && start >= 0 ? start + (t - o0) : -1,
                 p.hdr, sl))
    return;
  const PageLayout lay(1 << p.page_log, D);
  const uint8_t* block = p.pages + sl.page * p.H * (int64_t)lay.bytes();
  const uint8_t* codes = block + sl.place * lay.code_row + g * 8;
  const uint8_t* scales = block + lay.scales() + sl.place * lay.scale_row + g;
  const int ph = (p.H + PER - 1) / PER;
  for (int i0 = 0; i0 < 2 * ph; i0 += kPasses) {
    uint2 w[kPasses];
    uint32_t sc[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i0 + i >= 2 * ph) break;
      const bool key = i0 + i < ph;
      const int head = min((i0 + i - (key ? 0 : ph)) * PER + sub, p.H - 1);
      const int at = head * lay.bytes() + (key ? 0 : lay.half());
      w[i] = *reinterpret_cast<const uint2*>(codes + at);
      sc[i] = scales[at];
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i0 + i >= 2 * ph) break;
      const bool key = i0 + i < ph;
      const int head = (i0 + i - (key ? 0 : ph)) * PER + sub;
      __nv_bfloat16* dst = key ? p.k : p.v;
      if (head >= p.H || !dst) continue;
      const float s = e4m3_float(sc[i]) * (key ? p.k_scale : p.v_scale);
      auto two = [&](__half2 v) -> uint32_t {
        const float2 x = __half22float2(v);
        const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * s, x.y * s);
        return *reinterpret_cast<const uint32_t*>(&y);
      };
      uint4* to = reinterpret_cast<uint4*>(dst + (t * p.H + head) * D + g * 16);
      to[0] = make_uint4(two(e2m1x2_half2<0>(w[i].x)), two(e2m1x2_half2<1>(w[i].x)), two(e2m1x2_half2<2>(w[i].x)),
                         two(e2m1x2_half2<3>(w[i].x)));
      to[1] = make_uint4(two(e2m1x2_half2<0>(w[i].y)), two(e2m1x2_half2<1>(w[i].y)), two(e2m1x2_half2<2>(w[i].y)),
                         two(e2m1x2_half2<3>(w[i].y)));
    }
  }
  if (p.times && lane == 0) p.times[t] = p.page_times[(sl.page << p.page_log) + sl.place];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

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
  const unsigned ctas = (unsigned)((p.T + kWarps - 1) / kWarps);
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
  const unsigned ctas = (unsigned)((p.T + kWarps - 1) / kWarps);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c->d == 128 ? launch_pdl(read_kernel<128>, dim3(ctas), dim3(kThreads), 0, st, p)
                                    : launch_pdl(read_kernel<64>, dim3(ctas), dim3(kThreads), 0, st, p);
  if (e != cudaSuccess) return launch_error(e, "launching read_kernel");
  note_launches(1);
  return HSTU_OK;
}

}  // extern "C"
