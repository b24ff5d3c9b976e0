// HSTU attention of new rows over the paged 4-bit cache (hstu_attn_fwd_cached):
// the entry point, and the kernel that finishes what the tensor-core kernel
// (hstu_tc_cached.cu) leaves.
//
// Finishing: one warp a row adds up the pieces' FP32 sums of each head in
// piece order, adds a candidate's own term, SiLU(z_ii) v_i, and does 1/N, norm
// and gate on the row's H d features in registers.  It is launched
// programmatically behind the tensor-core kernel, which has written where each
// row's sums lie, so that the rows' own loads wait for one record only.  HBM
// traffic is the rows' q, k, v, u, o, y; the sums come from L2.  The heads' sums
// are loaded together: one head after the other took 4 us more for 4,096 rows.
// Few rows over a long cache have many pieces each (one for every CTA that held a
// part), so there 16 warps share a row's and add theirs in shared memory.
//
// Of 81 us for 32 users x 128 candidates (four heads of 128) this kernel takes
// 11: 18 MB of sums from L2 and 24 MB of rows.  One row of 131,000 cached tokens:
// with one warp a row 57.0 us, with 16 32.4 (single calls); 4,096 rows: 86.7 and
// 122.5.
#include "hstu_cached.cuh"
#include "hstu_rows.cuh"

namespace hstu {

hstu_status_t check_cache_desc(const hstu_cache_desc* c, bool buffers);

namespace {

// zero far below zero, minus infinity included
__device__ __forceinline__ float silu(float z) { return z < -1e4f ? 0.f : z / (1.f + expf(-z)); }

constexpr int kFinThreads = 128;   // of a CTA with a warp a row
constexpr int kFewWarps = 16;      // of a CTA with a row

// NV: the row's features in steps of 128 (4 a lane).
template <int D, int NV, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? kFinThreads : 32 * kWarps) finish_kernel(const __grid_constant__ CachedParams p,
                                                                                         int N) {
  constexpr int LANES = D / 4;
  constexpr int SHARE = kWarps / NV > 0 ? kWarps / NV : 1;   // warps that share a step's pieces
  static_assert(kWarps == 1 || kWarps % NV == 0, "as many warps for every step");
  __shared__ __align__(16) float4 sums[kWarps > 1 ? kWarps : 1][kWarps > 1 ? 32 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = kWarps == 1 ? (int64_t)blockIdx.x * (kFinThreads / 32) + warp : blockIdx.x;
  const int F = p.H * D;
  pdl_wait();
  if (t >= p.T) return;
  const int quota = p.hdr[WS_CA_QUOTA];
  const int64_t total = p.off[p.B];
  const int4 rec = p.rows[t];
  if (quota < 0 || t >= total) return;    // a refused batch or a wait that ran out, a padded batch's row
  const bool candidate = p.nt && ((rec.w >> 30) & 1);
  const int64_t row = t * F + lane * 4;
  // the row's own loads, under way while the sums are added up
  Raw4<__nv_bfloat16> q[NV], k[NV], v[NV], u[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool on = i * 128 + lane * 4 < F && (kWarps == 1 || warp == 0);
    q[i].x = k[i].x = v[i].x = make_uint2(0, 0);
    u[i].x = make_uint2(0x3f803f80u, 0x3f803f80u);   // ones
    if (on && candidate) {
      q[i] = fetch4(p.q + row + i * 128);
      k[i] = fetch4(p.k + row + i * 128);
      v[i] = fetch4(p.v + row + i * 128);
    }
    if (on && p.u && p.y) u[i] = fetch4(p.u + row + i * 128);
  }
  // the pieces of features f .. f + 3: their number, and the first one's sum
  const float* rows = p.part + (int64_t)(rec.w & 0xffff) * D;
  auto pieces = [&](int f, const float*& src) -> int {
    if (f >= F) return 0;
    const RowPieces r = row_pieces(rec, f / D, quota, N, p.slots);
    src = rows + r.slot * N * D + f % D;
    return (int)r.n;
  };
  const int64_t next = (int64_t)N * D;    // floats from a piece's sum to the next one's
  float o[NV][4];
  float sum = 0.f;
  if constexpr (kWarps == 1) {
    const float* src[NV];
    int n[NV], most = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      n[i] = pieces(i * 128 + lane * 4, src[i]);
      most = max(most, n[i]);
      o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    for (int c = 0; c < most; ++c) {      // a piece of every step at a time: their loads are under way together
      float4 x[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < n[i]) x[i] = __ldcg(reinterpret_cast<const float4*>(src[i] + c * next));
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) { o[i][0] += x[i].x; o[i][1] += x[i].y; o[i][2] += x[i].z; o[i][3] += x[i].w; }
    }
  } else {
    const float* src = nullptr;
    const int n = pieces((warp / SHARE) * 128 + lane * 4, src);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int c = warp % SHARE; c < n; c += SHARE) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(src + c * next));
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    }
    sums[warp][lane] = a;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      a = sums[i * SHARE][lane];
#pragma unroll
      for (int w = 1; w < SHARE; ++w) {
        const float4 x = sums[i * SHARE + w][lane];
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      }
      o[i][0] = a.x; o[i][1] = a.y; o[i][2] = a.z; o[i][3] = a.w;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int f = i * 128 + lane * 4, h = f / D;
    const bool on = f < F;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] *= p.o_scale;
    if (candidate) {
      float a[4], b[4];
      unpack4(q[i], a);
      unpack4(k[i], b);
      float dot = a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
      unpack4(v[i], b);
#pragma unroll
      for (int x = LANES / 2; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
      if (on) {
        float z = p.alpha * dot;
        if (p.rab_pos) z += p.rab_pos[h * p.P];
        if (p.rab_time) z += p.rab_time[h * p.Tb];
        const float w = silu(z) * p.inv_n;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = fmaf(w, b[e], o[i][e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += on ? o[i][e] : 0.f;
    if (on && p.o) store4(p.o + row + i * 128, o[i]);
  }
  if (!p.y) return;
  float mean = 0.f, rstd = 1.f;
  if (p.norm == HSTU_NORM_LAYERNORM) {
    mean = row_sum<32>(sum) / F;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = o[i][e] - mean;
        ss += i * 128 + lane * 4 < F ? c * c : 0.f;
      }
    rstd = rsqrtf(row_sum<32>(ss) / F + p.eps);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * 128 + lane * 4 >= F) continue;
    float g[4];
    unpack4(u[i], g);
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] *= (o[i][e] - mean) * rstd;
    store4(p.y + row + i * 128, g);
  }
}

template <int D, int NV>
cudaError_t launch_finish(const CachedParams& p, int N, bool few, cudaStream_t st) {
  if (few) return launch_pdl(finish_kernel<D, NV, kFewWarps>, dim3((unsigned)p.T), dim3(32 * kFewWarps), 0, st, p, N);
  const unsigned ctas = (unsigned)((p.T + kFinThreads / 32 - 1) / (kFinThreads / 32));
  return launch_pdl(finish_kernel<D, NV, 1>, dim3(ctas), dim3(kFinThreads), 0, st, p, N);
}

template <int D>
cudaError_t dispatch_finish(const CachedParams& p, int N, bool few, cudaStream_t st) {
  const int F = p.H * D;
  return F <= 128 ? launch_finish<D, 1>(p, N, few, st) : F <= 256 ? launch_finish<D, 2>(p, N, few, st)
       : F <= 512 ? launch_finish<D, 4>(p, N, few, st) : F <= 1024 ? launch_finish<D, 8>(p, N, few, st)
                                                                   : launch_finish<D, 16>(p, N, few, st);
}

hstu_status_t check_cached(const hstu_attn_desc* d, const hstu_cache_desc* c, int32_t max_rows, bool buffers) {
  hstu_status_t s = hstu_attn_workspace_size(d, nullptr, nullptr);
  if (s != HSTU_OK) return s;
  if ((s = check_cache_desc(c, buffers)) != HSTU_OK) return s;
  if (max_rows < 1) return HSTU_ERR_INVALID_ARG;
  if (d->H != c->H || d->d_qk != c->d) return HSTU_ERR_INVALID_ARG;
  if (d->flags & ~HSTU_FLAG_TEST_TIMEOUT) return HSTU_ERR_INVALID_ARG;
  if (d->total_tokens > ((int64_t)1 << 30)) return HSTU_ERR_UNSUPPORTED;   // one CTA a row finishes
  // the tiles' costs of all items are counted in 32 bits
  const int N = cached_block_rows(max_rows);
  const double items = ((double)d->total_tokens / N + d->B) * d->H;
  if (items * (d->max_seq_len / (double)kCachedTile + 1) * kMostTileCost > 2e9) return HSTU_ERR_UNSUPPORTED;
  if (d->dtype != HSTU_BF16 || d->out_dtype != HSTU_BF16 || d->dropout_p > 0.f) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

constexpr int kMaxCtas = 256;

struct CachedWs {
  size_t rows, part, total;
  int64_t slots;   // sums
};

CachedWs cached_ws(const hstu_attn_desc* d, int N) {
  CachedWs w{};
  size_t off = kWsHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + kWsAlign - 1) / kWsAlign * kWsAlign;
    return at;
  };
  w.rows = take(sizeof(int4) * (size_t)d->total_tokens);
  // a sum for every item, and one more for every CTA that ends inside one
  w.slots = (d->total_tokens / N + d->B) * d->H + kMaxCtas;
  w.part = take(sizeof(float) * (size_t)w.slots * N * d->d_v);
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
  p.rows = reinterpret_cast<int4*>(ws + w.rows);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.T = d->total_tokens; p.B = d->B; p.H = d->H; p.slots = w.slots;
  p.withhold = (d->flags & HSTU_FLAG_TEST_TIMEOUT) ? 1 : 0;
  p.wait_ns = p.withhold ? 1000000ull : 2000000000ull;
  p.page_size = c->page_size; p.page_log = c->page_size == 32 ? 5 : (c->page_size == 64 ? 6 : 7);
  p.num_pages = c->num_pages; p.max_pages = c->max_pages;
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
    const bool few = d->total_tokens <= sms;   // fewer rows than SMs: their pieces are many (measured above)
    e = c->d == 128 ? dispatch_finish<128>(p, N, few, st) : dispatch_finish<64>(p, N, few, st);
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
