// AdamW over many tensors in one launch, moments in 32 or in 8 bits
// (hstu_adamw_*); the formulas and the 8-bit format are in hstu_attn.h.
//
// HBM-bound: 28 bytes a parameter in 32 bits, 16 with 8-bit moments (and 2 for a BF16 copy).  The tensors are
// cut into chunks of 2,048 elements once, by init, into a list of records that hold all of a
// chunk's pointers: a CTA needs one load before its data.
//
// A lane holds 4 neighbouring elements twice (elements 4 l and 128 + 4 l of the warp's 256).  In 8 bits
// the warp's 256 elements are a block: its largest magnitudes take one reduction over
// the warp.  Decoding and encoding work on the bits of FP32 numbers: a code shifted
// by 20 is the bit pattern of its value times a power of two (the small codes those of
// subnormal numbers), so rounding up or down at random is one integer addition below the cut.
#include <stdlib.h>
#include <string.h>

#include "hstu_internal.h"

namespace hstu {

namespace {

constexpr int kBlock = 256;     // elements that share an exponent byte
constexpr int kChunk = 2048;
constexpr int kAdamThreads = kChunk / 8;
constexpr int kMOff = 134, kVOff = 142, kLeastExp = 16;

// What the header of the workspace holds behind the error words (64 bytes on).
struct AdamState {
  double pow1, pow2;    // beta^t of the next step
  int64_t steps;        // steps counted
  int64_t chunks;       // of the list
  int32_t kind;         // state_bits, grad_dtype: what the list was made for
  float c1, c2;         // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t) of the next step
};
constexpr size_t kStateOff = 64;

struct __align__(16) AdamChunk {
  float* p;
  const void* g;
  __nv_bfloat16* copy;
  void* m;
  void* v;
  uint8_t* me;
  uint8_t* ve;
  int64_t quad0;        // groups of 4 elements before this chunk, all tensors
  int32_t n;            // elements, <= kChunk
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

// Values of 4 codes of a block with exponent byte e.  m: sign, 4 and 3 bits, 127 a NaN; v: 5 and 3 bits.
__device__ __forceinline__ void decode_m(uint32_t codes, int e, float (&v)[4]) {
  const float unit = pow2f(e - kMOff);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = codes >> (8 * i);
    const float x = __uint_as_float((c & 127u) << 20) * 0x1p120f * unit;
    const float y = (c & 127u) == 127u ? __int_as_float(0x7fffffff) : x;
    v[i] = __uint_as_float(__float_as_uint(y) | (c & 128u) << 24);
  }
}
__device__ __forceinline__ void decode_v(uint32_t codes, int e, float (&v)[4]) {
  const float unit = pow2f(e - kVOff);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float((codes >> (8 * i) & 255u) << 20) * 0x1p112f * unit;
}

// |x| rounded up or down by the 20-bit noise; up: 2^(off - e)
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
// the exponent byte of a block from this lane's 8 values
__device__ __forceinline__ int block_exp(const float (&x)[2][4]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = __float_as_uint(x[j][i]) & 0x7fffffffu;
      if (b < 0x7f800000u) top = max(top, b);
    }
  return max((int)(__reduce_max_sync(0xffffffffu, top) >> 23), kLeastExp);
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int BITS, typename TG>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamParams p) {
  pdl_wait();
  AdamState* st = reinterpret_cast<AdamState*>(reinterpret_cast<char*>(p.hdr) + kStateOff);
  if (st->chunks != p.chunks || st->kind != p.kind) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return;
  }
  if (p.skip && *p.skip != 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x < p.chunks) {
    const AdamChunk c = p.list[blockIdx.x];
    const int at0 = warp * kBlock + 4 * lane;
    if (warp * kBlock < c.n) {
      const TG* gp = static_cast<const TG*>(c.g);
      float w[2][4], g[2][4], m[2][4], v[2][4];
      uint32_t mc[2], vc[2];
      int me = 0, ve = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = at0 + 128 * j, live = c.n - at;
        get4(c.p + at, live, w[j]);
        get4(gp + at, live, g[j]);
        if constexpr (BITS == 32) {
          get4(static_cast<const float*>(c.m) + at, live, m[j]);
          get4(static_cast<const float*>(c.v) + at, live, v[j]);
        } else {
          mc[j] = get4(static_cast<const uint8_t*>(c.m) + at, live);
          vc[j] = get4(static_cast<const uint8_t*>(c.v) + at, live);
        }
      }
      if constexpr (BITS == 8) {
        me = c.me[warp];
        ve = c.ve[warp];
      }
      const float lr = (p.lr_at ? *p.lr_at : p.lr) * c.lr_scale, keep = 1.f - lr * c.wd;
      const float c1 = -lr * st->c1, c2 = st->c2, scale = p.scale ? *p.scale : 1.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (BITS == 8) {
          decode_m(mc[j], me, m[j]);
          decode_v(vc[j], ve, v[j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // products and sums one by one: the codes go by their last bits
          const float gs = __fmul_rn(g[j][i], scale);
          m[j][i] = __fadd_rn(__fmul_rn(m[j][i], p.b1), __fmul_rn(gs, p.a1));
          v[j][i] = __fadd_rn(__fmul_rn(v[j][i], p.b2), __fmul_rn(__fmul_rn(gs, gs), p.a2));
          const float d = fmaf(sqrt_approx(v[j][i]), c2, p.eps);
          w[j][i] = fmaf(__fdividef(m[j][i], d), c1, w[j][i] * keep);
        }
      }
      if constexpr (BITS == 8) {
        me = block_exp(m);
        ve = block_exp(v);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = at0 + 128 * j, live = c.n - at;
        if (live <= 0) continue;
        put4(c.p + at, live, w[j]);
        if (c.copy) put4(c.copy + at, live, w[j]);
        if constexpr (BITS == 32) {
          put4(static_cast<float*>(c.m) + at, live, m[j]);
          put4(static_cast<float*>(c.v) + at, live, v[j]);
        } else {
          const uint64_t quad = (uint64_t)c.quad0 + (uint64_t)(at >> 2), t = (uint64_t)st->steps + 1;
          const uint4 r = philox((uint32_t)quad, (uint32_t)(quad >> 32), (uint32_t)t, (uint32_t)(t >> 32),
                                 (uint32_t)p.seed, (uint32_t)(p.seed >> 32));
          const uint32_t word[4] = {r.x, r.y, r.z, r.w};
          const float up_m = pow2f(kMOff - me), up_v = pow2f(kVOff - ve);
          uint32_t a = 0, b = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a |= code_m(m[j][i], up_m, ((word[i] & 0xffffu) << 4) + 8) << (8 * i);
            b |= code_v(v[j][i], up_v, (word[i] >> 16 << 4) + 8) << (8 * i);
          }
          put4(static_cast<uint8_t*>(c.m) + at, live, a);
          put4(static_cast<uint8_t*>(c.v) + at, live, b);
        }
      }
      if (BITS == 8 && lane == 0) {
        c.me[warp] = (uint8_t)me;
        c.ve[warp] = (uint8_t)ve;
      }
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
      st->c2 = (float)(1.0 / sqrt(1.0 - st->pow2));
      st->steps += 1;
    }
  }
}

template <int BITS, typename TO>
__global__ void __launch_bounds__(kAdamThreads)
adamw_read_kernel(int* hdr, const ReadChunk* __restrict__ list, int64_t chunks, int kind) {
  pdl_wait();
  const AdamState* st = reinterpret_cast<const AdamState*>(reinterpret_cast<const char*>(hdr) + kStateOff);
  if (st->chunks != chunks || st->kind != kind) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return;
  }
  const ReadChunk c = list[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = warp * kBlock + 128 * j + 4 * lane, live = (int)c.n - at;
    if (live <= 0) continue;
    float m[4], v[4];
    if constexpr (BITS == 32) {
      get4(static_cast<const float*>(c.m) + at, live, m);
      get4(static_cast<const float*>(c.v) + at, live, v);
    } else {
      decode_m(get4(static_cast<const uint8_t*>(c.m) + at, live), c.me[warp], m);
      decode_v(get4(static_cast<const uint8_t*>(c.v) + at, live), c.ve[warp], v);
    }
    if (c.om) put4(static_cast<TO*>(c.om) + at, live, m);
    if (c.ov) put4(static_cast<TO*>(c.ov) + at, live, v);
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
  // eps keeps the quotient's divisor a normal FP32 number
  if (!(d->eps >= 1e-30 && d->eps < 1e30) || !(d->lr >= 0.0 && d->lr < 1e30)) return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

// The tensors' checks, and the chunks of their list.
hstu_status_t check_tensors(const hstu_adamw_desc* d, const hstu_adamw_tensor* t, bool stepped, int64_t* chunks) {
  if (d->num_tensors > 0 && !t) return HSTU_ERR_INVALID_ARG;
  int64_t total = 0;
  const size_t code = d->state_bits == 8 ? 4 : 16;
  for (int i = 0; i < d->num_tensors; ++i) {
    const hstu_adamw_tensor& x = t[i];
    if (x.n < 0) return HSTU_ERR_INVALID_ARG;
    if (x.n > ((int64_t)1 << 44)) return HSTU_ERR_UNSUPPORTED;
    if (x.n == 0) continue;
    if (!x.m || !x.v || !aligned(x.m, code) || !aligned(x.v, code)) return HSTU_ERR_INVALID_ARG;
    if (d->state_bits == 8 && (!x.m_exp || !x.v_exp)) return HSTU_ERR_INVALID_ARG;
    if (stepped) {
      if (!x.param || !aligned(x.param, 16) || !aligned(x.copy, 8)) return HSTU_ERR_INVALID_ARG;
      if (!aligned(x.grad, d->grad_dtype == HSTU_FP32 ? 16 : 8)) return HSTU_ERR_INVALID_ARG;
      if (!(x.weight_decay >= 0.f && x.weight_decay < 1e30f) || !(x.lr_scale >= 0.f && x.lr_scale < 1e30f))
        return HSTU_ERR_INVALID_ARG;
      if (!x.grad) continue;   // left as it is
    }
    total += (x.n + kChunk - 1) / kChunk;
  }
  if (total > 0x7fffffff) return HSTU_ERR_UNSUPPORTED;
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
  const size_t msize = d->state_bits == 8 ? 1 : 4, gsize = d->grad_dtype == HSTU_FP32 ? 4 : 2;
  for (int i = 0; i < d->num_tensors; ++i) {
    const hstu_adamw_tensor& x = tensors[i];
    for (int64_t e = 0; x.grad && e < x.n; e += kChunk) {
      AdamChunk& c = list[at++];
      c.p = x.param + e;
      c.g = static_cast<const char*>(x.grad) + e * gsize;
      c.copy = x.copy ? static_cast<__nv_bfloat16*>(x.copy) + e : nullptr;
      c.m = static_cast<char*>(x.m) + e * msize;
      c.v = static_cast<char*>(x.v) + e * msize;
      c.me = x.m_exp ? x.m_exp + e / kBlock : nullptr;
      c.ve = x.v_exp ? x.v_exp + e / kBlock : nullptr;
      c.quad0 = block * (kBlock / 4) + e / 4;
      c.n = (int32_t)(x.n - e < kChunk ? x.n - e : kChunk);
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
  state.c2 = (float)(1.0 / sqrt(1.0 - state.pow2));
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
  if (!a || d->chunks < 0 || d->chunks > 0x7fffffff) return HSTU_ERR_INVALID_ARG;
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
  const dim3 grid((unsigned)(d->chunks > 0 ? d->chunks : 1)), block(kAdamThreads);
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
  const size_t msize = d->state_bits == 8 ? 1 : 4, osize = out_dtype == HSTU_FP32 ? 4 : 2;
  for (int i = 0; i < d->num_tensors; ++i) {
    const hstu_adamw_tensor& x = tensors[i];
    for (int64_t e = 0; e < x.n; e += kChunk) {
      ReadChunk& c = list[at++];
      c.m = static_cast<const char*>(x.m) + e * msize;
      c.v = static_cast<const char*>(x.v) + e * msize;
      c.me = x.m_exp ? x.m_exp + e / kBlock : nullptr;
      c.ve = x.v_exp ? x.v_exp + e / kBlock : nullptr;
      c.om = outs[i].m ? static_cast<char*>(outs[i].m) + e * osize : nullptr;
      c.ov = outs[i].v ? static_cast<char*>(outs[i].v) + e * osize : nullptr;
      c.n = x.n - e < kChunk ? x.n - e : kChunk;
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
  if (d->chunks < 0 || d->chunks > 0x7fffffff) return HSTU_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, list_bytes(d->chunks))) != HSTU_OK) return s;
  reset_launches();
  if (d->chunks == 0) return HSTU_OK;
  int* hdr = static_cast<int*>(workspace);
  const ReadChunk* list = reinterpret_cast<const ReadChunk*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  const dim3 grid((unsigned)d->chunks), block(kAdamThreads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int kind = kind_of(d, true, d->grad_dtype);
  const bool f32 = d->grad_dtype == HSTU_FP32;
  const cudaError_t e = d->state_bits == 32
                            ? (f32 ? launch_pdl(adamw_read_kernel<32, float>, grid, block, 0, st, hdr, list, d->chunks, kind)
                                   : launch_pdl(adamw_read_kernel<32, __nv_bfloat16>, grid, block, 0, st, hdr, list, d->chunks, kind))
                            : (f32 ? launch_pdl(adamw_read_kernel<8, float>, grid, block, 0, st, hdr, list, d->chunks, kind)
                                   : launch_pdl(adamw_read_kernel<8, __nv_bfloat16>, grid, block, 0, st, hdr, list, d->chunks, kind));
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
