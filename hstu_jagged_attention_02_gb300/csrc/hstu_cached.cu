// HSTU attention of new rows over the paged 4-bit cache (hstu_attn_fwd_cached):
// the entry point, and the kernel that finishes what the tensor-core kernel
// (hstu_tc_cached.cu) leaves.
//
// Finishing: one CTA a row adds up the pieces' FP32 sums of each head in
// piece order, adds a candidate's own term, SiLU(z_ii) v_i, and does 1/N, norm
// and gate on the row's H d features in registers, 4 a thread and step.  It
// is launched programmatically behind the tensor-core kernel.  HBM traffic is
// the rows' q, k, v, u, o, y; the sums come from L2.  Few rows over a long
// cache have many pieces each (one for every CTA that held a part), so there
// kGroups groups of threads share them and add their sums in shared memory.
#include "hstu_cached.cuh"
#include "hstu_rows.cuh"

namespace hstu {

hstu_status_t check_cache_desc(const hstu_cache_desc* c, bool buffers);

namespace {

// zero far below zero, minus infinity included
__device__ __forceinline__ float silu(float z) { return z < -1e4f ? 0.f : z / (1.f + expf(-z)); }

constexpr int kFin = 128;    // threads that hold a row's features

template <int D, int kGroups>
__global__ void __launch_bounds__(kFin* kGroups) finish_kernel(const __grid_constant__ CachedParams p, int N) {
  constexpr int LANES = D / 4;
  __shared__ float red[2][kFin / 32];
  __shared__ __align__(16) float sums[kGroups > 1 ? kGroups - 1 : 1][4 * kFin];
  const int64_t t = blockIdx.x;
  const int F = p.H * D, tid = threadIdx.x % kFin, group = threadIdx.x / kFin, lane = threadIdx.x & 31;
  pdl_wait();
  const int quota = p.hdr[WS_CA_QUOTA];
  if (quota < 0 || t >= p.off[p.B]) return;    // a refused batch, a padded batch's row
  const int b = warp_find_sequence(p.off, nullptr, p.B, t).b;
  CachedSeq s;
  if (!load_seq(p, b, s)) return;
  const int r = (int)(t - s.row0), qb = r / N;
  const bool candidate = r >= s.n - s.m;
  // where the block's first item begins among all tiles
  int before = 0;
  for (int x = lane; x < qb; x += 32) before += block_tiles(s, x, N);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const int tiles = block_tiles(s, qb, N);
  const int tile0 = p.seq_tiles[b] + before * p.H, item0 = p.seq_items[b] + qb * p.H;
  const float* rows = p.part + (int64_t)(r - qb * N) * D;
  float o[4][4];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = (i * kFin + tid) * 4;
    const bool on = f < F;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (i * kFin * 4 >= F) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      continue;
    }
    const int h = f / D;
    if (on && tiles > 0) {
      const int at = tile0 + h * tiles, c1 = (at + tiles - 1) / quota;
      const float* src = rows + (int64_t)(item0 + h) * N * D + f % D;
#pragma unroll 8
      for (int c = at / quota + group; c <= c1; c += kGroups) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)c * N * D));
        a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
      }
    }
    if (kGroups > 1) {
      __syncthreads();
      if (group > 0) *reinterpret_cast<float4*>(&sums[group - 1][tid * 4]) = make_float4(a[0], a[1], a[2], a[3]);
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int g = 0; g < kGroups - 1; ++g) {
          const float4 x = *reinterpret_cast<const float4*>(&sums[g][tid * 4]);
          a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] *= p.o_scale;
    if (candidate && group == 0) {
      const int64_t at = t * F + f;
      float q[4] = {}, k[4] = {}, v[4] = {};
      if (on) {
        load4(p.q + at, q);
        load4(p.k + at, k);
        load4(p.v + at, v);
      }
      float dot = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
      for (int x = LANES / 2; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
      if (on) {
        float z = p.alpha * dot;
        if (p.rab_pos) z += p.rab_pos[h * p.P];
        if (p.rab_time) z += p.rab_time[h * p.Tb];
        const float w = silu(z) * p.inv_n;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = fmaf(w, v[e], a[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[i][e] = a[e];
      sum += on ? a[e] : 0.f;
    }
    if (on && p.o && group == 0) store4(p.o + t * F + f, o[i]);
  }
  if (!p.y) return;
  auto total = [&](float v, int slot) -> float {
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    if (lane == 0 && group == 0) red[slot][tid >> 5] = v;
    __syncthreads();
    float x = 0.f;
    for (int w = 0; w < kFin / 32; ++w) x += red[slot][w];
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
        ss += (i * kFin + tid) * 4 < F ? c * c : 0.f;
      }
    rstd = __frsqrt_rn(total(ss, 1) / F + p.eps);
  }
  if (group > 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = (i * kFin + tid) * 4;
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
  if (d->total_tokens > ((int64_t)1 << 30)) return HSTU_ERR_UNSUPPORTED;   // one CTA a row finishes
  // tiles of all items are counted in 32 bits
  const int N = cached_block_rows(max_rows);
  const double items = ((double)d->total_tokens / N + d->B) * d->H;
  if (items * (d->max_seq_len / (double)kCachedTile + 1) > 2e9) return HSTU_ERR_UNSUPPORTED;
  if (d->dtype != HSTU_BF16 || d->out_dtype != HSTU_BF16 || d->dropout_p > 0.f) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

constexpr int kMaxCtas = 256;

struct CachedWs {
  size_t tiles, items, part, total;
};

CachedWs cached_ws(const hstu_attn_desc* d, int N) {
  CachedWs w{};
  size_t off = kWsHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + kWsAlign - 1) / kWsAlign * kWsAlign;
    return at;
  };
  w.tiles = take(sizeof(int) * (size_t)d->B);
  w.items = take(sizeof(int) * (size_t)d->B);
  // a sum for every item, and one more for every CTA that ends inside one
  const size_t slots = ((size_t)(d->total_tokens / N) + d->B) * d->H + kMaxCtas;
  w.part = take(sizeof(float) * slots * N * d->d_v);
  w.total = off;
  return w;
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
  if (bytes) *bytes = cached_ws(d, cached_block_rows(max_rows)).total;
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
  const int N = cached_block_rows(a->max_rows);
  const CachedWs w = cached_ws(d, N);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) || workspace_bytes < w.total)
    return HSTU_ERR_WORKSPACE;
  reset_launches();
  if (d->total_tokens == 0 || d->B == 0 || (!a->o && !a->y)) return HSTU_OK;
  CachedParams p{};
  p.off = a->seq_offsets; p.lens = a->cache_lens; p.nt = a->num_targets; p.table = a->block_table; p.times = a->row_times;
  p.rab_pos = a->rab_pos; p.rab_time = a->row_times ? a->rab_time : nullptr;
  p.q = static_cast<const __nv_bfloat16*>(a->q); p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v); p.u = static_cast<const __nv_bfloat16*>(a->u);
  p.o = static_cast<__nv_bfloat16*>(a->o); p.y = static_cast<__nv_bfloat16*>(a->y);
  p.pages = static_cast<const uint8_t*>(c->pages); p.page_times = c->timestamps;
  p.hdr = static_cast<int*>(workspace);
  char* ws = static_cast<char*>(workspace);
  p.seq_tiles = reinterpret_cast<int*>(ws + w.tiles);
  p.seq_items = reinterpret_cast<int*>(ws + w.items);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.T = d->total_tokens; p.B = d->B; p.H = d->H;
  p.page_size = c->page_size; p.page_log = c->page_size == 32 ? 5 : (c->page_size == 64 ? 6 : 7); p.num_pages = c->num_pages; p.max_pages = c->max_pages;
  p.max_rows = a->max_rows; p.max_n = d->max_seq_len; p.P = d->num_pos_buckets; p.Tb = d->num_time_buckets;
  p.norm = d->norm; p.alpha = d->alpha; p.inv_n = 1.f / (float)d->max_seq_len; p.eps = d->ln_eps;
  p.k_scale = ldexpf(1.f, c->k_exp);
  p.o_scale = ldexpf(p.inv_n, c->v_exp - 4);   // the scores carry a factor of 16
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  if (e == cudaSuccess)
    e = N == 8 ? launch_stream_cached(p, c->d, ctas, st) : launch_tc_cached(p, c->d, N, ctas, st);
  if (e == cudaSuccess) {
    const dim3 grid((unsigned)d->total_tokens);
    const bool few = d->total_tokens <= sms;
    if (c->d == 128)
      e = few ? launch_pdl(finish_kernel<128, 4>, grid, dim3(4 * kFin), 0, st, p, N)
              : launch_pdl(finish_kernel<128, 1>, grid, dim3(kFin), 0, st, p, N);
    else
      e = few ? launch_pdl(finish_kernel<64, 4>, grid, dim3(4 * kFin), 0, st, p, N)
              : launch_pdl(finish_kernel<64, 1>, grid, dim3(kFin), 0, st, p, N);
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    if (!*hstu_last_error_detail()) set_error_detail(e, "launching the cached attention");
    return HSTU_ERR_CUDA;
  }
  note_launches(2);
  return HSTU_OK;
}

}  // extern "C"
