// Appending to and reading from the paged 4-bit cache (hstu_cache_append,
// hstu_cache_read).
//
// Append: HBM-bound on the BF16 rows (2 d bytes in, 9 d / 16 out).  A lane
// holds 4 features, d / 4 lanes a row, 4 lanes a group of 16; a warp takes
// kRows rows of one token at a time, all its loads issued before anything
// else.  The group's maximum goes over 4 lanes by shuffles.
//
// Roundings are decided as on real numbers.  A value x that is exact in FP32
// (a BF16 input) meets a border only exactly: its quotient by the scale (4
// significant bits) lies at least 2^-13 from a border or on it, so the
// quotient corrected by one residual step in FP32 decides rightly.  A
// normed or rotated key is known to 2^-20 of its terms only; where the codes
// (or the scale) of x - d and x + d differ, the warp computes its rows again
// in FP64 and compares with the borders themselves.  That happens to about
// one row in a thousand.
#include "hstu_fp4.cuh"
#include "hstu_internal.h"
#include "hstu_seq_search.cuh"
#include "hstu_vec.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kBand = 9.5367431640625e-07f;   // 2^-20

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
  int B, H, page_size, num_pages, max_pages;
  int rot, interleaved, norm;
  float eps;
  float k_scale, v_scale;   // 2^-k_exp, 2^-v_exp
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Largest of the 4 lanes of a group; NaN if one is.
__device__ __forceinline__ float group_max(float v) {
  v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// x / s to within half a unit (x exact, s a scale): the quotient by the
// reciprocal and one residual step.  x is cut where e2m1 has long saturated,
// so that infinities stay on their side.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  x = fminf(fmaxf(x, -8192.f), 8192.f);
  const float y = x * inv;
  return fmaf(fmaf(-y, s, x), inv, y);
}

struct Coded {
  uint32_t codes;   // 4 codes, 16 bits
  uint32_t scale;   // e4m3 byte of the group
};

// A row part that is exact in FP32.
__device__ __forceinline__ Coded encode_exact(const float (&x)[4]) {
  const float top = group_max(max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3]))));
  Coded c;
  c.scale = e4m3_of(__fdiv_rn(top, 6.f));
  const float s = e4m3_float(c.scale), inv = s > 0.f ? __frcp_rn(s) : 0.f;
  c.codes = e2m1x2_of(quotient(x[0], s, inv), quotient(x[1], s, inv)) |
            (e2m1x2_of(quotient(x[2], s, inv), quotient(x[3], s, inv)) << 8);
  return c;
}

// A row part known to +-d[e]: false where that does not decide the result.
__device__ __forceinline__ bool encode_banded(const float (&x)[4], const float (&d)[4], Coded& c) {
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi = max_nan(hi, fabsf(x[e]) + d[e]);
    lo = max_nan(lo, fabsf(x[e]) - d[e]);
  }
  hi = group_max(hi);
  lo = group_max(lo);
  c.scale = e4m3_of(hi * 0.16666667f * 1.0000005f);
  bool sure = c.scale == e4m3_of(lo * 0.16666667f * 0.9999995f);
  const float s = e4m3_float(c.scale), inv = s > 0.f ? __frcp_rn(s) : 0.f;
  float a[4], b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float xc = fminf(fmaxf(x[e], -8192.f), 8192.f);
    const float y = xc * inv, w = fmaf(fabsf(y), kBand, d[e] * inv);
    a[e] = y - w;
    b[e] = y + w;
  }
  c.codes = e2m1x2_of(a[0], a[1]) | (e2m1x2_of(a[2], a[3]) << 8);
  const uint32_t other = e2m1x2_of(b[0], b[1]) | (e2m1x2_of(b[2], b[3]) << 8);
  // a zero's sign is no difference of value
  const uint32_t diff = c.codes ^ other;
  if (diff) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t m = 0xfu << (4 * e);
      if ((diff & m) && !(((c.codes | other) & (0x7u << (4 * e))) == 0)) sure = false;
    }
  }
  return sure;
}

__device__ __forceinline__ double group_max(double v) {
  v = fmax(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmax(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// The same from FP64: every border compared with itself.
__device__ __noinline__ Coded encode_f64(double x0, double x1, double x2, double x3) {
  const double x[4] = {x0, x1, x2, x3};
  const double top = group_max(fmax(fmax(fabs(x0), fabs(x1)), fmax(fabs(x2), fabs(x3))));
  int bad = x0 != x0 || x1 != x1 || x2 != x2 || x3 != x3;   // a NaN, which the maximum passes over
  bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
  bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
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

template <int LANES, typename F>
__device__ __forceinline__ F lanes_sum(F v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A key row part, normed and turned, in FP32, with what it may be off by.
template <int LANES>
__device__ __forceinline__ void key_f32(const AppendParams& p, const float (&x)[4], int f, int partner,
                                        const float (&gain)[4], const float (&c)[4], const float (&s)[4],
                                        float (&w)[4], float (&d)[4]) {
  float rs = 1.f;
  if (p.norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(x[e], x[e], ss);
    rs = __frsqrt_rn(fmaf(lanes_sum<LANES>(ss), 1.f / (4 * LANES), p.eps));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = x[e] * rs * gain[e] * p.k_scale;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.rot) {
    if (p.interleaved) {
      o[0] = w[1]; o[1] = w[0]; o[2] = w[3]; o[3] = w[2];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(0xffffffffu, w[e], partner);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    d[e] = kBand * (fabsf(w[e]) + (s[e] != 0.f ? fabsf(o[e]) : 0.f));
    w[e] = fmaf(w[e], c[e], o[e] * s[e]);
  }
}

template <int LANES>
__device__ __noinline__ Coded key_f64(const AppendParams& p, float x0, float x1, float x2, float x3, int f, int partner,
                                      float4 c4, float4 s4) {
  const float x[4] = {x0, x1, x2, x3}, c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
  double w[4], o[4] = {0.0, 0.0, 0.0, 0.0}, rs = 1.0;
  if (p.norm) {
    double ss = 0.0;
    for (int e = 0; e < 4; ++e) ss += (double)x[e] * x[e];
    rs = 1.0 / sqrt(lanes_sum<LANES>(ss) / (4 * LANES) + (double)p.eps);
  }
  for (int e = 0; e < 4; ++e) w[e] = x[e] * rs * (p.gain ? (double)p.gain[f + e] : 1.0) * p.k_scale;
  if (p.rot) {
    if (p.interleaved) {
      o[0] = w[1]; o[1] = w[0]; o[2] = w[3]; o[3] = w[2];
    } else {
      for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(0xffffffffu, w[e], partner);
    }
  }
  for (int e = 0; e < 4; ++e) w[e] = w[e] * c[e] + o[e] * s[e];
  return encode_f64(w[0], w[1], w[2], w[3]);
}

// The page block offset of a token's head, or -1 (recorded) where the tables do not give one.
struct Slot {
  int64_t page;
  int place;
  int64_t pos;
};

__device__ __forceinline__ bool find_slot(const int32_t* table, int max_pages, int page_size, int num_pages, int b,
                                          int64_t pos, int* hdr, Slot& s) {
  s.pos = pos;
  bool ok = pos >= 0 && pos < (int64_t)max_pages * page_size;
  if (ok) {
    s.page = table[(int64_t)b * max_pages + pos / page_size];
    s.place = (int)(pos % page_size);
    ok = s.page >= 0 && s.page < num_pages;
  }
  if (!ok) set_error(hdr, HSTU_ERR_DEVICE_CHECK, b);
  return ok;
}

// kRows x (128 / D) of the token's 2 H rows (keys first) a warp.
template <int D, int kRows>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p, int chunks) {
  constexpr int LANES = D / 4, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / chunks;
  const int first = (int)(unit - t * chunks) * kRows * PER;
  if (t >= p.T) return;
  const int f = (lane % LANES) * 4, mine = first + lane / LANES;
  float x[kRows][4];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int hh = mine + r * PER;
    if (hh < p.H) {
      load4(p.k + t * p.ks[0] + (int64_t)hh * p.ks[1] + f, x[r]);
    } else if (hh < 2 * p.H) {
      load4(p.v + t * p.vs[0] + (int64_t)(hh - p.H) * p.vs[1] + f, x[r]);
    } else {
      x[r][0] = x[r][1] = x[r][2] = x[r][3] = 0.f;
    }
  }
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
  if (!find_slot(p.table, p.max_pages, p.page_size, p.num_pages, b, in ? p.lens[b] - (o1 - o0) + (t - o0) : -1, p.hdr, sl))
    return;
  const bool keys = first < p.H;
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f}, gain[4] = {1.f, 1.f, 1.f, 1.f};
  int partner = lane;
  const bool moved = p.rot || p.norm;
  if (keys && moved) {
    if (p.rot && sl.pos >= p.max_pos) {
      if (lane == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, b);
      return;
    }
    if (p.gain) load4(p.gain + f, gain);
    if (f < p.rot) {
      const int half = p.rot >> 1;
      const float* cr = p.cos + sl.pos * half;
      const float* sr = p.sin + sl.pos * half;
      if (p.interleaved) {
        const float2 cc = *reinterpret_cast<const float2*>(cr + (f >> 1));
        const float2 sn = *reinterpret_cast<const float2*>(sr + (f >> 1));
        c[0] = c[1] = cc.x; c[2] = c[3] = cc.y;
        s[0] = -sn.x; s[1] = sn.x; s[2] = -sn.y; s[3] = sn.y;
      } else {
        const bool second = f >= half;
        load4(cr + (second ? f - half : f), c);
        load4(sr + (second ? f - half : f), s);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = second ? s[e] : -s[e];
      }
    }
    const int l = lane % LANES, h = p.rot >> 3;
    partner = lane - l + (l < h ? l + h : (l < 2 * h ? l - h : l));
  }
  const PageLayout lay(p.page_size, D);
  uint8_t* block = p.pages + sl.page * p.H * (int64_t)lay.bytes();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int hh = mine + r * PER;
    const bool is_k = hh < p.H;
    const bool any_k = first + r * PER < p.H;   // the warp's row group holds a key row
    Coded out;
    if (any_k && moved) {
      float w[4], d[4];
      key_f32<LANES>(p, x[r], f, partner, gain, c, s, w, d);
      bool sure = encode_banded(w, d, out);
      if (__any_sync(0xffffffffu, is_k && !sure))
        out = key_f64<LANES>(p, x[r][0], x[r][1], x[r][2], x[r][3], f, partner, make_float4(c[0], c[1], c[2], c[3]),
                             make_float4(s[0], s[1], s[2], s[3]));
    }
    if (!(any_k && moved) || first + r * PER + PER > p.H) {   // values, or keys as they are
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = x[r][e] * (is_k ? p.k_scale : p.v_scale);
      const Coded plain = encode_exact(y);
      if (!(is_k && moved)) out = plain;
    }
    if (hh < 2 * p.H) {
      const int h = is_k ? hh : hh - p.H;
      uint8_t* part = block + (int64_t)h * lay.bytes() + (is_k ? 0 : lay.half());
      *reinterpret_cast<uint16_t*>(part + sl.place * lay.code_row + (f >> 1)) = (uint16_t)out.codes;
      if ((lane & 3) == 0) part[lay.scales() + sl.place * lay.scale_row + (f >> 4)] = (uint8_t)out.scale;
    }
  }
  if (p.page_times && first == 0 && lane == 0) p.page_times[sl.page * p.page_size + sl.place] = p.times[t];
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
  int B, H, page_size, num_pages, max_pages;
  float k_scale, v_scale;   // 2^k_exp, 2^v_exp
};

// A lane takes 16 features (8 bytes of codes and their scale), a warp
// 512 / D rows of one token at a time.
template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int LANES = D / 16, PER = 32 / LANES;
  pdl_wait();
  const int lane = threadIdx.x & 31;
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
  if (!find_slot(p.table, p.max_pages, p.page_size, p.num_pages, b, o0 <= t && t < o1 && start >= 0 ? start + (t - o0) : -1,
                 p.hdr, sl))
    return;
  const PageLayout lay(p.page_size, D);
  const uint8_t* block = p.pages + sl.page * p.H * (int64_t)lay.bytes();
  const int g = lane % LANES;
  for (int hh = lane / LANES; hh < 2 * p.H; hh += PER) {
    const bool is_k = hh < p.H;
    const int h = is_k ? hh : hh - p.H;
    __nv_bfloat16* dst = is_k ? p.k : p.v;
    if (!dst) continue;
    const uint8_t* part = block + (int64_t)h * lay.bytes() + (is_k ? 0 : lay.half());
    const uint2 w = *reinterpret_cast<const uint2*>(part + sl.place * lay.code_row + g * 8);
    const float s = e4m3_float(part[lay.scales() + sl.place * lay.scale_row + g]) * (is_k ? p.k_scale : p.v_scale);
    uint32_t out[8];
    auto two = [&](__half2 v) -> uint32_t {
      const float2 x = __half22float2(v);
      const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * s, x.y * s);
      return *reinterpret_cast<const uint32_t*>(&y);
    };
    out[0] = two(e2m1x2_half2<0>(w.x)); out[1] = two(e2m1x2_half2<1>(w.x));
    out[2] = two(e2m1x2_half2<2>(w.x)); out[3] = two(e2m1x2_half2<3>(w.x));
    out[4] = two(e2m1x2_half2<0>(w.y)); out[5] = two(e2m1x2_half2<1>(w.y));
    out[6] = two(e2m1x2_half2<2>(w.y)); out[7] = two(e2m1x2_half2<3>(w.y));
    uint4* to = reinterpret_cast<uint4*>(dst + (t * p.H + h) * D + g * 16);
    to[0] = make_uint4(out[0], out[1], out[2], out[3]);
    to[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
  if (p.times && lane == 0) p.times[t] = p.page_times[sl.page * p.page_size + sl.place];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

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
  p.B = a->B; p.H = c->H; p.page_size = c->page_size; p.num_pages = c->num_pages; p.max_pages = c->max_pages;
  p.rot = a->rot_dim; p.interleaved = a->interleaved; p.norm = a->norm; p.eps = a->eps;
  p.k_scale = ldexpf(1.f, -c->k_exp); p.v_scale = ldexpf(1.f, -c->v_exp);
  constexpr int R = 4;
  const int per = 128 / c->d, chunks = (2 * c->H + R * per - 1) / (R * per);
  const unsigned ctas = (unsigned)((p.T * chunks + kWarps - 1) / kWarps);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c->d == 128 ? launch_pdl(append_kernel<128, R>, dim3(ctas), dim3(kThreads), 0, st, p, chunks)
                                    : launch_pdl(append_kernel<64, R>, dim3(ctas), dim3(kThreads), 0, st, p, chunks);
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
  p.B = a->B; p.H = c->H; p.page_size = c->page_size; p.num_pages = c->num_pages; p.max_pages = c->max_pages;
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
