// Layer norm with weight and bias, forward (hstu_ln_fwd), and the C calls of
// both directions.
//
// HBM-bound: each row is read once, held in registers for its mean, its
// centred squares and its output, and written once (161,293 rows of 512, FP32 to BF16: 79.6 us, 6.2 TB/s, 92% of a
// copy's rate; 64 rows: 3.2 us, a launch).
#include "hstu_ln.cuh"

namespace hstu {

namespace {

using namespace ln;

template <typename TX, typename TY, int V, int L, int N>
__global__ void __launch_bounds__(L <= 32 ? kTeamsThreads : L) ln_fwd_kernel(const __grid_constant__ LnParams p) {
  __shared__ float2 red[2][L <= 32 ? 1 : L / 32];
  constexpr int TEAMS = L <= 32 ? kTeamsThreads / L : 1;
  pdl_wait();
  const int64_t r = (int64_t)blockIdx.x * TEAMS + (L <= 32 ? threadIdx.x / L : 0), rows = live_rows(p);
  // (a warp goes on while one of its teams has a row)
  if (r - (L < 32 ? (threadIdx.x & 31) / L : 0) >= rows) return;
  const int l = threadIdx.x % L, D = L >= 32 || r < rows ? p.D : 0;
  const TX* x = static_cast<const TX*>(p.x) + r * p.xs;
  Pack<TX, V> raw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int f = (i * L + l) * V;
    if (f < D) raw[i].load(x + f);
  }
  float v[N][V];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if ((i * L + l) * V < D) {
      raw[i].get(v[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[i][e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = 0.f;
    }
  }
  const float inv = 1.f / (float)p.D;
  const float mean = team_sum<L>(s, red[0]) * inv;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if ((i * L + l) * V < D) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v[i][e] -= mean;
        q = fmaf(v[i][e], v[i][e], q);
      }
    }
  }
  const float rstd = rsqrtf(fmaf(team_sum<L>(q, red[1]), inv, p.eps));
  if (l == 0 && D > 0) {
    if (p.mean) p.mean[r] = mean;
    if (p.rstd) p.rstd[r] = rstd;
  }
  TY* y = static_cast<TY*>(p.y) + r * p.ys;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int f = (i * L + l) * V;
    if (f < D) {
      Pack<float, V> c;
      float w[V], b[V];
      if (p.weight) { c.load(p.weight + f); c.get(w); }
      if (p.bias) { c.load(p.bias + f); c.get(b); }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float t = v[i][e] * rstd;
        if (p.weight) t *= w[e];
        if (p.bias) t += b[e];
        v[i][e] = t;
      }
      put(y + f, v[i]);
    }
  }
}

template <typename TX, typename TY>
cudaError_t launch_t(const LnParams& p, bool wide, cudaStream_t st) {
  return dispatch_shape(p.D, wide, [&](auto S) {
    using Sh = decltype(S);
    constexpr int TEAMS = Sh::l <= 32 ? kTeamsThreads / Sh::l : 1;
    return launch_pdl(ln_fwd_kernel<TX, TY, Sh::v, Sh::l, Sh::n>, dim3((unsigned)((p.rows + TEAMS - 1) / TEAMS)),
                      dim3(Sh::l <= 32 ? kTeamsThreads : Sh::l), 0, st, p);
  });
}

hstu_status_t check_desc(const hstu_ln_desc* d) {
  if (!d || d->struct_size != sizeof(hstu_ln_desc) || d->reserved != 0) return HSTU_ERR_INVALID_ARG;
  for (int t : {d->x_dtype, d->y_dtype})
    if (t != HSTU_BF16 && t != HSTU_FP32) return HSTU_ERR_INVALID_ARG;
  if (d->D < 1 || d->rows < 0 || !(d->eps >= 0.f && d->eps < 1e30f)) return HSTU_ERR_INVALID_ARG;
  if (d->D > kMaxD || d->rows > 0x7fffffffLL) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

size_t size_of(int dtype) { return dtype == HSTU_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
// whether rows can be read 16 bytes at a time
bool wide_rows(const void* p, int64_t stride, int dtype) {
  return !p || (aligned(p, 16) && stride * (int64_t)size_of(dtype) % 16 == 0);
}
bool wide_vec(const float* p) { return aligned(p, 16); }

size_t bwd_bytes(const hstu_ln_desc* d) { return kWsHeaderBytes + sizeof(float) * kLnMaxBwdCtas * 2 * (size_t)d->D; }

hstu_status_t check_ws(void* ws, size_t bytes, size_t need) {
  return !ws || !aligned(ws, kWsAlign) || bytes < need ? HSTU_ERR_WORKSPACE : HSTU_OK;
}

hstu_status_t device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) return HSTU_OK;
  (void)cudaGetLastError();
  set_error_detail(e, "reading the number of SMs");
  return HSTU_ERR_CUDA;
}

hstu_status_t launched(cudaError_t e, const char* what, int n) {
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    set_error_detail(e, what);
    return HSTU_ERR_CUDA;
  }
  note_launches(n);
  return HSTU_OK;
}

}  // namespace

cudaError_t launch_ln_fwd(const LnParams& p, int x_dtype, int y_dtype, bool wide, int, cudaStream_t st) {
  if (x_dtype == HSTU_BF16)
    return y_dtype == HSTU_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(p, wide, st)
                                : launch_t<__nv_bfloat16, float>(p, wide, st);
  return y_dtype == HSTU_BF16 ? launch_t<float, __nv_bfloat16>(p, wide, st) : launch_t<float, float>(p, wide, st);
}

}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_ln_workspace_size(const hstu_ln_desc* desc, size_t* fwd, size_t* bwd) {
  const hstu_status_t s = check_desc(desc);
  if (s != HSTU_OK) return s;
  if (fwd) *fwd = kWsHeaderBytes;
  if (bwd) *bwd = bwd_bytes(desc);
  return HSTU_OK;
}

hstu_status_t hstu_ln_fwd(const hstu_ln_desc* d, const hstu_ln_fwd_args* a, void* workspace, size_t workspace_bytes,
                          hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  if (s != HSTU_OK) return s;
  if (!a || (d->rows > 0 && (!a->x || !a->y))) return HSTU_ERR_INVALID_ARG;
  if (!aligned(a->x, size_of(d->x_dtype)) || !aligned(a->y, size_of(d->y_dtype)) || !aligned(a->weight, 4) ||
      !aligned(a->bias, 4))
    return HSTU_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, kWsHeaderBytes)) != HSTU_OK) return s;
  reset_launches();
  if (d->rows == 0) return HSTU_OK;
  LnParams p{};
  p.num_rows = a->num_rows;
  p.x = a->x; p.weight = a->weight; p.bias = a->bias; p.y = a->y; p.mean = a->mean; p.rstd = a->rstd;
  p.hdr = static_cast<int*>(workspace);
  p.rows = d->rows; p.xs = d->x_stride; p.ys = d->y_stride; p.D = d->D; p.eps = d->eps;
  const bool wide = d->D % 8 == 0 && wide_rows(a->x, d->x_stride, d->x_dtype) &&
                    wide_rows(a->y, d->y_stride, d->y_dtype) && wide_vec(a->weight) && wide_vec(a->bias);
  return launched(launch_ln_fwd(p, d->x_dtype, d->y_dtype, wide, 0, reinterpret_cast<cudaStream_t>(stream)),
                  "launching ln_fwd_kernel", 1);
}

hstu_status_t hstu_ln_bwd(const hstu_ln_desc* d, const hstu_ln_bwd_args* a, void* workspace, size_t workspace_bytes,
                          hstu_stream_t stream) {
  hstu_status_t s = check_desc(d);
  if (s != HSTU_OK) return s;
  if (!a || (d->rows > 0 && (!a->x || !a->dy || !a->dx || !a->mean || !a->rstd))) return HSTU_ERR_INVALID_ARG;
  for (const void* ptr : {a->x, a->dres, (const void*)a->dx})
    if (!aligned(ptr, size_of(d->x_dtype))) return HSTU_ERR_INVALID_ARG;
  if (!aligned(a->dy, size_of(d->y_dtype)) || !aligned(a->weight, 4) || !aligned(a->d_weight, 4) || !aligned(a->d_bias, 4))
    return HSTU_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, bwd_bytes(d))) != HSTU_OK) return s;
  reset_launches();
  if (d->rows == 0 && !a->d_weight && !a->d_bias) return HSTU_OK;   // no row: the sums are zero
  LnParams p{};
  p.num_rows = a->num_rows;
  p.x = a->x; p.weight = a->weight; p.mean = const_cast<float*>(a->mean); p.rstd = const_cast<float*>(a->rstd);
  p.dy = a->dy; p.dres = a->dres; p.dx = a->dx; p.d_weight = a->d_weight; p.d_bias = a->d_bias;
  p.hdr = static_cast<int*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  p.rows = d->rows; p.xs = d->x_stride; p.ys = d->y_stride; p.dxs = d->dx_stride; p.drs = d->dres_stride;
  p.D = d->D; p.eps = d->eps;
  const bool wide = d->D % 8 == 0 && wide_rows(a->x, d->x_stride, d->x_dtype) &&
                    wide_rows(a->dy, d->y_stride, d->y_dtype) && wide_rows(a->dx, d->dx_stride, d->x_dtype) &&
                    wide_rows(a->dres, d->dres_stride, d->x_dtype) && wide_vec(a->weight);
  int sms = 0;
  if ((s = device_sms(&sms)) != HSTU_OK) return s;
  return launched(launch_ln_bwd(p, d->x_dtype, d->y_dtype, wide, sms, reinterpret_cast<cudaStream_t>(stream)),
                  "launching ln_bwd_kernel", a->d_weight || a->d_bias ? 2 : 1);
}

}  // extern "C"
