// HSTU attention of new rows over the paged 4-bit cache (hstu_attn_fwd_cached).
//
// Plain kernels: one CTA a (row, head) walks the cached positions that the
// row sees, a warp a position at a time, and leaves the FP32 sum in the
// workspace; one CTA a row adds a candidate's own term and does norm and gate.
#include "hstu_fp4.cuh"
#include "hstu_internal.h"
#include "hstu_seq_search.cuh"
#include "hstu_vec.cuh"

namespace hstu {

hstu_status_t check_cache_desc(const hstu_cache_desc* c, bool buffers);

namespace {

struct CachedParams {
  const int64_t* off;
  const int32_t* lens;
  const int32_t* nt;
  const int32_t* table;
  const int64_t* times;
  const float* rab_pos;
  const float* rab_time;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* u;
  __nv_bfloat16* o;
  __nv_bfloat16* y;
  const uint8_t* pages;
  const int64_t* page_times;
  float* acc;
  int* hdr;
  int64_t T;
  int B, H, page_size, num_pages, max_pages, max_rows, max_n, P, Tb, norm;
  float alpha, inv_n, eps, k_scale, v_scale;
};

struct RowInfo {
  int b, L;
  int64_t pos;       // the row's position
  bool candidate;
};

// false (with the error recorded) where the batch's numbers do not fit together
__device__ __forceinline__ bool find_row(const CachedParams& p, int64_t t, RowInfo& r) {
  const int64_t total = p.off[p.B];
  if (total > p.T || p.off[0] != 0) {
    set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, -1);
    return false;
  }
  if (t >= total) return false;
  r.b = warp_find_sequence(p.off, p.B, t);
  const int64_t o0 = p.off[r.b], n = p.off[r.b + 1] - o0;
  const int64_t m = p.nt ? p.nt[r.b] : 0;
  r.L = p.lens[r.b];
  if (t < o0 || t >= o0 + n || n > p.max_rows || m < 0 || m > n || n - m > r.L || r.L + m > p.max_n ||
      r.L > (int64_t)p.max_pages * p.page_size) {
    set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, r.b);
    return false;
  }
  r.candidate = t - o0 >= n - m;
  r.pos = r.candidate ? r.L : r.L - (n - m) + (t - o0);
  return true;
}

// zero far below zero, minus infinity included
__device__ __forceinline__ float silu(float z) { return z < -1e4f ? 0.f : z / (1.f + expf(-z)); }

template <int D>
__global__ void __launch_bounds__(256) plain_cached_kernel(const __grid_constant__ CachedParams p) {
  constexpr int PER = D / 32;
  __shared__ float part[8][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y;
  RowInfo r;
  if (!find_row(p, t, r)) return;
  const int64_t seen = r.candidate ? r.L : r.pos + 1;
  float q[PER], acc[PER] = {};
  for (int e = 0; e < PER; ++e) q[e] = __bfloat162float(p.q[(t * p.H + h) * D + lane * PER + e]);
  const PageLayout lay(p.page_size, D);
  for (int64_t j = warp; j < seen; j += 8) {
    const int64_t page = p.table[(int64_t)r.b * p.max_pages + j / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      set_error(p.hdr, HSTU_ERR_DEVICE_CHECK, r.b);
      break;
    }
    const int at = (int)(j % p.page_size);
    const uint8_t* kp = p.pages + (page * p.H + h) * lay.bytes();
    const uint8_t* vp = kp + lay.half();
    float dot = 0.f, v[PER];
    for (int e = 0; e < PER; e += 2) {
      const int f = lane * PER + e;
      const float2 a = __half22float2(e2m1x2_half2<0>(kp[at * lay.code_row + f / 2]));
      const float2 b = __half22float2(e2m1x2_half2<0>(vp[at * lay.code_row + f / 2]));
      const float ks = e4m3_float(kp[lay.scales() + at * lay.scale_row + f / 16]) * p.k_scale;
      const float vs = e4m3_float(vp[lay.scales() + at * lay.scale_row + f / 16]) * p.v_scale;
      dot += q[e] * a.x * ks + q[e + 1] * a.y * ks;
      v[e] = b.x * vs;
      v[e + 1] = b.y * vs;
    }
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    float z = p.alpha * dot;
    if (p.rab_pos) z += p.rab_pos[h * p.P + min(r.pos - j, (int64_t)p.P - 1)];
    if (p.rab_time && p.times) z += p.rab_time[h * p.Tb + time_bucket(p.times[t], p.page_times[page * p.page_size + at], p.Tb)];
    const float w = silu(z);
    for (int e = 0; e < PER; ++e) acc[e] += w * v[e];
  }
  for (int e = 0; e < PER; ++e) part[warp][lane * PER + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int w = 0; w < 8; ++w) s += part[w][threadIdx.x];
    p.acc[(t * p.H + h) * D + threadIdx.x] = s;
  }
}

constexpr int kFinThreads = 128;

// One CTA a row, 4 features a thread and step.
template <int D>
__global__ void __launch_bounds__(kFinThreads) finish_kernel(const __grid_constant__ CachedParams p) {
  constexpr int LANES = D / 4;
  __shared__ float red[2][kFinThreads / 32];
  const int64_t t = blockIdx.x;
  const int F = p.H * D, tid = threadIdx.x;
  RowInfo r;
  if (!find_row(p, t, r)) return;
  float o[4][4];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = (i * kFinThreads + tid) * 4;
    const bool on = f < F;
    const int64_t at = t * F + f;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) load4(p.acc + at, a);
    if (r.candidate) {
      float q[4] = {}, k[4] = {}, v[4] = {};
      if (on) {
        load4(p.q + at, q);
        load4(p.k + at, k);
        load4(p.v + at, v);
      }
      float dot = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
      for (int s = LANES / 2; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
      if (on) {
        const int h = f / D;
        float z = p.alpha * dot;
        if (p.rab_pos) z += p.rab_pos[h * p.P];
        if (p.rab_time && p.times) z += p.rab_time[h * p.Tb];
        const float w = silu(z);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] += w * v[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[i][e] = a[e] * p.inv_n;
      sum += on ? o[i][e] : 0.f;
    }
    if (on && p.o) store4(p.o + at, o[i]);
  }
  if (!p.y) return;
  auto total = [&](float v, int slot) -> float {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    if ((tid & 31) == 0) red[slot][tid >> 5] = v;
    __syncthreads();
    float x = 0.f;
    for (int w = 0; w < kFinThreads / 32; ++w) x += red[slot][w];
    return x;
  };
  float mean = 0.f, rstd = 1.f;
  if (p.norm == HSTU_NORM_LAYERNORM) {
    mean = total(sum, 0) / F;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = o[i][e] - mean;
        ss += (i * kFinThreads + tid) * 4 < F ? c * c : 0.f;
      }
    rstd = __frsqrt_rn(total(ss, 1) / F + p.eps);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = (i * kFinThreads + tid) * 4;
    if (f >= F) continue;
    float u[4] = {1.f, 1.f, 1.f, 1.f};
    if (p.u) load4(p.u + t * F + f, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] *= (o[i][e] - mean) * rstd;
    store4(p.y + t * F + f, u);
  }
}

hstu_status_t check_cached(const hstu_attn_desc* d, const hstu_cache_desc* c, int32_t max_rows, bool buffers) {
  hstu_status_t s = hstu_attn_workspace_size(d, nullptr, nullptr);
  if (s != HSTU_OK) return s;
  if ((s = check_cache_desc(c, buffers)) != HSTU_OK) return s;
  if (max_rows < 1) return HSTU_ERR_INVALID_ARG;
  if (d->H != c->H || d->d_qk != c->d) return HSTU_ERR_INVALID_ARG;
  if (d->flags != 0) return HSTU_ERR_INVALID_ARG;
  if (d->dtype != HSTU_BF16 || d->out_dtype != HSTU_BF16 || d->dropout_p > 0.f) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

size_t cached_bytes(const hstu_attn_desc* d) {
  return kWsHeaderBytes + sizeof(float) * (size_t)d->total_tokens * d->H * d->d_v;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_attn_cached_workspace_size(const hstu_attn_desc* d, const hstu_cache_desc* c, int32_t max_rows,
                                              size_t* bytes) {
  const hstu_status_t s = check_cached(d, c, max_rows, false);
  if (s != HSTU_OK) return s;
  if (bytes) *bytes = cached_bytes(d);
  return HSTU_OK;
}

hstu_status_t hstu_attn_fwd_cached(const hstu_attn_desc* d, const hstu_cache_desc* c, const hstu_attn_cached_args* a,
                                   void* workspace, size_t workspace_bytes, hstu_stream_t stream) {
  if (!a) return HSTU_ERR_INVALID_ARG;
  const hstu_status_t s = check_cached(d, c, a->max_rows, true);
  if (s != HSTU_OK) return s;
  if (a->reserved != 0 || !a->seq_offsets) return HSTU_ERR_INVALID_ARG;
  if (d->total_tokens > 0 && d->B > 0 && (!a->cache_lens || !a->block_table || !a->q)) return HSTU_ERR_INVALID_ARG;
  if (d->total_tokens > 0 && d->B > 0 && a->num_targets && (!a->k || !a->v)) return HSTU_ERR_INVALID_ARG;
  if (a->row_times && !c->timestamps) return HSTU_ERR_INVALID_ARG;
  for (const void* ptr : {a->q, a->k, a->v, a->u, (const void*)a->o, (const void*)a->y})
    if (ptr && !aligned16(ptr)) return HSTU_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) || workspace_bytes < cached_bytes(d))
    return HSTU_ERR_WORKSPACE;
  reset_launches();
  if (d->total_tokens == 0 || d->B == 0 || (!a->o && !a->y)) return HSTU_OK;
  CachedParams p{};
  p.off = a->seq_offsets; p.lens = a->cache_lens; p.nt = a->num_targets; p.table = a->block_table; p.times = a->row_times;
  p.rab_pos = a->rab_pos; p.rab_time = a->rab_time;
  p.q = static_cast<const __nv_bfloat16*>(a->q); p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v); p.u = static_cast<const __nv_bfloat16*>(a->u);
  p.o = static_cast<__nv_bfloat16*>(a->o); p.y = static_cast<__nv_bfloat16*>(a->y);
  p.pages = static_cast<const uint8_t*>(c->pages); p.page_times = c->timestamps;
  p.hdr = static_cast<int*>(workspace);
  p.acc = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  p.T = d->total_tokens; p.B = d->B; p.H = d->H;
  p.page_size = c->page_size; p.num_pages = c->num_pages; p.max_pages = c->max_pages;
  p.max_rows = a->max_rows; p.max_n = d->max_seq_len; p.P = d->num_pos_buckets; p.Tb = d->num_time_buckets;
  p.norm = d->norm; p.alpha = d->alpha; p.inv_n = 1.f / (float)d->max_seq_len; p.eps = d->ln_eps;
  p.k_scale = ldexpf(1.f, c->k_exp); p.v_scale = ldexpf(1.f, c->v_exp);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)d->total_tokens, (unsigned)d->H);
  if (c->d == 128) {
    plain_cached_kernel<128><<<grid, 256, 0, st>>>(p);
    finish_kernel<128><<<(unsigned)d->total_tokens, kFinThreads, 0, st>>>(p);
  } else {
    plain_cached_kernel<64><<<grid, 256, 0, st>>>(p);
    finish_kernel<64><<<(unsigned)d->total_tokens, kFinThreads, 0, st>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error_detail(e, "launching the cached attention");
    return HSTU_ERR_CUDA;
  }
  note_launches(2);
  return HSTU_OK;
}

}  // extern "C"
