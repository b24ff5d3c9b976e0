/*
 * hstu_attn.h -- C ABI of the GB300 (sm_103a) HSTU jagged attention library
 * (libhstu_attn.so).
 *
 * The operation (HSTU "Spatial Aggregation" and "Pointwise Transformation",
 * ai6s.net generative-recommendation survey, section 2.1.2, equations (2)
 * and (3); the equations are images on the page, the prose describes a
 * softmax-free "pointwise aggregated attention" with a position/time bias and
 * a U gate):
 *
 *   for each sequence b and head h, tokens i, j of the sequence:
 *     z_ij = alpha * <q_i, k_j> + rab_pos[h][bp(i,j)] + rab_time[h][bt(i,j)]
 *     o_i  = sum over allowed j of SiLU(z_ij) / N * v_j        (no softmax)
 *   y_t = Norm(concat_h o_t) * u_t
 *
 * Jagged layout (KeyedJaggedTensor convention, same survey, section 3.1.2):
 * tokens of all sequences are packed back to back, row-major, no padding;
 * seq_offsets[b] is the first token of sequence b, seq_offsets[B] == T.
 *   q, k     [T, H, d_qk]     v, o  [T, H, d_v]     u, y, dy, du  [T, H*d_v]
 * Every row is dense and contiguous; every tensor pointer must be 16-byte
 * aligned.  q, k, v, u have the element type `dtype`; o, y, dy and the
 * gradients have `out_dtype` (BF16 inputs with FP32 outputs keep the final
 * rounding out of the result; BF16 outputs halve the output traffic).
 *
 * Mask (the ranking task's candidates, section 2.1.2, and the compound
 * causal + context/target mask of the Ascend HSTU fused operator, wmrh.cn
 * RecSDK page, "HSTU acceleration operator" paragraph).  A sequence of n
 * tokens has c = num_contexts[b] context tokens in front and
 * m = num_targets[b] candidates at the end; h_end = n - m:
 *   j >= h_end : allowed iff i == j
 *   j <  h_end : allowed iff j <= i  or  (i < c and j < c)
 * Buckets: pos(i) = min(i, h_end);  bp = min(|pos(i) - pos(j)|, P - 1);
 *          bt = 0 if t_i == t_j else min(Tb - 1, floor(log2|t_i - t_j|) + 1).
 * Norm:    LAYERNORM normalises each token's H*d_v features (population
 *          variance, eps = ln_eps, no affine); NONE leaves them as they are.
 *
 * Conventions
 *  - Every pointer is a device pointer except the host_* outputs of
 *    hstu_attn_debug_plan and hstu_get_device_error.  The caller owns every
 *    buffer, including the workspace; the library never allocates device
 *    memory and keeps no state between calls.  The one exception is
 *    hstu_attn_fwd_noalloc: it uses a fixed buffer built into the library
 *    in place of a workspace, shared by all its calls on a device (its own
 *    comment gives the size limit and the race between overlapping calls).
 *    What one call leaves in a workspace for a later one is the caller's
 *    to keep: the backward's plan kept with HSTU_FLAG_PLAN_BWD.
 *  - Calls are stream-ordered and return without synchronising, except
 *    hstu_attn_debug_plan and hstu_get_device_error, which synchronise the
 *    given stream.  Concurrent calls must use distinct workspaces.
 *  - Host-side checks return an error code before anything is launched.
 *    Problems seen on the device (inconsistent offsets or counts, a pipeline
 *    wait that ran out) are recorded in the workspace and read back with
 *    hstu_get_device_error; outputs are undefined then.  The library never
 *    traps or aborts.
 */
#ifndef HSTU_ATTN_H_
#define HSTU_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HSTU_ATTN_ABI_VERSION 2

typedef struct CUstream_st* hstu_stream_t; /* same type as cudaStream_t; NULL = legacy default stream */

typedef enum {
  HSTU_OK = 0,
  HSTU_ERR_INVALID_ARG = 1,   /* a NULL required pointer, bad size or misalignment */
  HSTU_ERR_UNSUPPORTED = 2,   /* a valid request this build does not implement */
  HSTU_ERR_WORKSPACE = 3,     /* workspace NULL, misaligned or too small */
  HSTU_ERR_CUDA = 4,          /* a CUDA runtime call failed */
  HSTU_ERR_TIMEOUT = 5,       /* device: a pipeline wait ran out of its limit */
  HSTU_ERR_DEVICE_CHECK = 6   /* device: offsets/counts inconsistent with the descriptor */
} hstu_status_t;

typedef enum { HSTU_BF16 = 0, HSTU_FP32 = 1 } hstu_dtype_t;
typedef enum { HSTU_NORM_NONE = 0, HSTU_NORM_LAYERNORM = 1 } hstu_norm_t;

/* Flags */
#define HSTU_FLAG_FORCE_SIMT (1u << 0)   /* use the CUDA-core kernels even where the tensor-core path applies;
                                            BF16 work the tensor-core kernels do not take (the backward
                                            needs d = 128, the forward d = 64 or 128) runs only with this
                                            flag, else the call returns HSTU_ERR_UNSUPPORTED */
#define HSTU_FLAG_TEST_TIMEOUT (1u << 1) /* test only: the tensor-core forward withholds one load (the
                                            first K/V tile of work item 0) and its waits give up after about
                                            a millisecond, so the timeout path runs without a hang; the
                                            result is HSTU_ERR_TIMEOUT.  In hstu_layer_fwd it applies to the
                                            tensor-core input projection instead (its CTA 0 skips its first
                                            load), and hstu_layer_bwd rejects it.  In hstu_attn_fwd_cached
                                            CTA 0 prepares none of its work */
#define HSTU_FLAG_U_FP32 (1u << 2)       /* u is FP32 whatever dtype is (requires out_dtype FP32).  The
                                            gate multiplies y element by element, so a BF16 rounding of u
                                            is never averaged out; q, k, v stay in dtype */
#define HSTU_FLAG_PLAN_BWD (1u << 3)     /* hstu_attn_fwd only: its planner launch also plans the
                                            backward's tiling (a second CTA of the same launch) and keeps
                                            it in the workspace, which must then have the backward's size */
#define HSTU_FLAG_REUSE_PLAN (1u << 4)   /* hstu_attn_bwd only: launch no planner and use the plan kept by
                                            the last hstu_attn_fwd with HSTU_FLAG_PLAN_BWD on this
                                            workspace.  The backward checks on the device that the plan was
                                            made for the same B, total_tokens, max_seq_len and path, from
                                            the same seq_offsets, num_targets, num_contexts and first
                                            timestamp of every sequence; otherwise it computes nothing and
                                            records HSTU_ERR_DEVICE_CHECK.  A kept plan serves any number of
                                            backward calls until another planner launch on the workspace
                                            (any forward, a backward without this flag, a debug plan)
                                            voids it.  Rejected by the layer, delta and no-alloc calls */

typedef struct {
  uint32_t struct_size;     /* sizeof(hstu_attn_desc) */
  int32_t dtype;            /* hstu_dtype_t of the inputs q, k, v, u */
  int32_t out_dtype;        /* hstu_dtype_t of o, y, dy, dq, dk, dv, du; FP32 when dtype is FP32 */
  int32_t B;                /* number of sequences, >= 0 */
  int32_t H;                /* heads, >= 1 */
  int32_t d_qk, d_v;        /* head dims; this build: d_qk == d_v in {32, 64, 128} */
  int64_t total_tokens;     /* T == seq_offsets[B] */
  int32_t max_seq_len;      /* N of the 1/N scale; every sequence must have n <= N */
  float alpha;              /* scale of <q, k> */
  int32_t num_pos_buckets;  /* P >= 1 (128 in the reference workloads) */
  int32_t num_time_buckets; /* Tb >= 1 (64) */
  int32_t norm;             /* hstu_norm_t */
  float ln_eps;             /* LayerNorm epsilon (1e-5) */
  uint32_t flags;           /* HSTU_FLAG_* */
  float dropout_p;          /* fused dropout on y, 0 <= p < 1 (0: none); see below */
  uint32_t reserved;        /* must be 0 */
} hstu_attn_desc;

/* Fused dropout (ai6s.net survey, section 2.1.3, "memory optimisation":
 * dropout fused with its neighbouring operators).  With dropout_p = p > 0
 * the forward's y becomes dropout(Norm(o) * u) and the backward takes dy as
 * the gradient of that dropped-out y.  The keep decision of element (t, f)
 * of the [T, F] output (F = H * d_v) comes from the counter-based generator
 * Philox4x64-10 (Salmon, Moraes, Dror, Shaw, SC 2011):
 *
 *   e = t F + f;  r = Philox4x64-10(counter (e >> 3, dropout_offset, 0, 0),
 *                                   key (dropout_seed, 0))
 *   w = 32-bit word (e & 7) of r[0..3] (low half of each 64-bit word first)
 *   keep iff w >= floor(p 2^32); kept elements are multiplied by 1 / (1 - p)
 *
 * so the backward regenerates the forward's mask from the same seed and
 * offset (a caller advances the offset, or changes the seed, per step).  The
 * mask does not depend on the batch's split into sequences. */

typedef struct {
  const int64_t* seq_offsets;  /* [B+1], non-decreasing, seq_offsets[0] == 0 */
  const int32_t* num_targets;  /* [B] candidates at the end of each sequence, or NULL (none) */
  const int32_t* num_contexts; /* [B] context tokens at the front, or NULL (none) */
  const int64_t* timestamps;   /* [T] integer seconds, or NULL (no time bias) */
  const float* rab_pos;        /* [H, P] position-bucket bias, or NULL */
  const float* rab_time;       /* [H, Tb] time-bucket bias, or NULL; ignored without timestamps */
  const void* q;               /* [T, H, d_qk] */
  const void* k;               /* [T, H, d_qk] */
  const void* v;               /* [T, H, d_v] */
  const void* u;               /* [T, H*d_v] gate, or NULL (gate of one); FP32 with HSTU_FLAG_U_FP32 */
  void* o;                     /* out [T, H, d_v]: A.V, kept for the backward */
  void* y;                     /* out [T, H*d_v]: Norm(o) * u, or NULL (not produced) */
  float* ln_mean;              /* out [T] or NULL: per-token mean of o (LAYERNORM) */
  float* ln_rstd;              /* out [T] or NULL: per-token 1/sqrt(var + eps) (LAYERNORM) */
  uint64_t dropout_seed;       /* fused dropout (desc->dropout_p > 0): generator key */
  uint64_t dropout_offset;     /* and counter word 1 */
} hstu_attn_fwd_args;

typedef struct {
  /* the forward's inputs, unchanged */
  const int64_t* seq_offsets;
  const int32_t* num_targets;
  const int32_t* num_contexts;
  const int64_t* timestamps;
  const float* rab_pos;
  const float* rab_time;
  const void* q;
  const void* k;
  const void* v;
  const void* u;
  const void* o;               /* the forward's o */
  const void* dy;              /* [T, H*d_v] gradient of the loss w.r.t. y */
  /* outputs, overwritten (not accumulated) */
  void* dq;                    /* [T, H, d_qk] */
  void* dk;                    /* [T, H, d_qk] */
  void* dv;                    /* [T, H, d_v] */
  void* du;                    /* [T, H*d_v]; required iff u != NULL */
  float* d_rab_pos;            /* [H, P] or NULL (not wanted) */
  float* d_rab_time;           /* [H, Tb] or NULL */
  uint64_t dropout_seed;       /* the forward's dropout seed and offset */
  uint64_t dropout_offset;
} hstu_attn_bwd_args;

/* Workspace bytes the forward and the backward need for this descriptor
 * (a bound valid for any seq_offsets consistent with it).  The workspace must
 * be 256-byte aligned.  Either output pointer may be NULL. */
hstu_status_t hstu_attn_workspace_size(const hstu_attn_desc* desc, size_t* fwd_bytes, size_t* bwd_bytes);

/* Forward: o = A.V and, if y != NULL, y = Norm(o) * u (eqs. (2), (3)).
 * One planner launch, the attention kernel and (with y or the statistics) the
 * norm-gate kernel.  With HSTU_FLAG_PLAN_BWD the planner also plans the
 * backward, so a training step (forward, then the backward with
 * HSTU_FLAG_REUSE_PLAN on the same workspace) launches one planner. */
hstu_status_t hstu_attn_fwd(const hstu_attn_desc* desc, const hstu_attn_fwd_args* args,
                            void* workspace, size_t workspace_bytes, hstu_stream_t stream);

/* Backward: dq, dk, dv, du, d_rab_pos, d_rab_time from dy; A is recomputed
 * tile by tile, never stored (HSTU's memory design, section 2.1.3 "memory
 * optimisation": sub-layer activations are not kept). */
hstu_status_t hstu_attn_bwd(const hstu_attn_desc* desc, const hstu_attn_bwd_args* args,
                            void* workspace, size_t workspace_bytes, hstu_stream_t stream);

/* The tile plan of one pass, as the kernels walk it (compound-mask tile
 * skipping, wmrh.cn RecSDK page, "HSTU acceleration operator" paragraph).
 * pass 0 = forward (query-block work items), 1 = backward (key-block items).
 * Writes up to host_capacity records of 6 int32 (b, q_block, k_block, class,
 * q_rows, k_rows) to host_tiles for every tile that is not skipped; class 1 =
 * partial, 2 = full; q_rows x k_rows = the tile shape of the path this
 * descriptor selects (tensor-core or CUDA-core).  *n_tiles receives the total
 * count.  The workspace must hold the forward workspace plus
 * 24 * host_capacity bytes (rounded up to 256).  Synchronises the stream. */
hstu_status_t hstu_attn_debug_plan(const hstu_attn_desc* desc, const int64_t* seq_offsets,
                                   const int32_t* num_targets, const int32_t* num_contexts, int32_t pass,
                                   void* workspace, size_t workspace_bytes, int32_t* host_tiles,
                                   int64_t host_capacity, int64_t* n_tiles, hstu_stream_t stream);

/* Forward without a caller workspace, for callers that are not allowed to
 * allocate device memory (a framework that owns all device memory through its
 * own pool, a latency-bound server that cannot afford an allocation, an
 * integration with no allocator at hand).  The pages describe no counterpart;
 * this is a library convenience.
 *
 * Same operation, arguments and outputs as hstu_attn_fwd; the caller still
 * passes every input and output buffer.  The scratch comes from a 1 MiB
 * buffer built into the library (every GPU that loads the library holds it
 * until the process exits).  The plan of T tokens in B sequences needs
 * 256 + 4 (B + 1) + 80 (ceil(T / 32) + B) bytes (each part rounded up to
 * 256), roughly 2.5 T + 84 B + 1 KiB, which must fit in 1 MiB: e.g. 250,000
 * tokens in 4,000 sequences.  Larger problems return HSTU_ERR_WORKSPACE
 * (hstu_last_error_detail says how much was needed) without launching.
 *
 * Each call looks up the buffer's device address (cudaGetSymbolAddress) with
 * the current device, which must be the stream's device (else
 * HSTU_ERR_INVALID_ARG).  The address is not cached, so a device reset
 * between calls does not leave a stale pointer behind.  The first call on a
 * device may load the library's device code, so make that first call before
 * any stream capture.  Every call shares the one buffer: calls that may
 * overlap on the GPU (other streams, other host threads) race and must be
 * serialised by the caller.  The buffer keeps the last call's contents; the
 * planner rewrites everything it reads on every call.
 *
 * host_device_error: NULL, or a host int32 that receives the call's device
 * error code (as hstu_get_device_error reports it); non-NULL makes the call
 * synchronise the stream. */
hstu_status_t hstu_attn_fwd_noalloc(const hstu_attn_desc* desc, const hstu_attn_fwd_args* args,
                                    hstu_stream_t stream, int32_t* host_device_error);

/* ------------------------------------------------------------------------
 * The full HSTU layer around the attention (ai6s.net survey, section 2.1.2,
 * equations (1)-(3), with the residual connection between layers; section
 * 2.1.3: two linear layers per block).  With D = H * d_v (= H * d_qk):
 *
 *   Z1 = X W1                                   [T, 4D]  (FP32 accumulation)
 *   U | V | Q | K = SiLU(Z1), column blocks of width D in that order
 *   o, y = attention(Q, K, V, U) as in hstu_attn_fwd (y = Norm(o) * U)
 *   out  = X + y W2                             [T, D]
 *
 * Precision: X, W1, W2 BF16; V, Q, K = SiLU(Z1) are rounded to BF16 (the
 * attention's MMA operands) while the gate U stays FP32 (it scales y element
 * by element, where a rounding is never averaged out).  The computed GEMM
 * operands y (y W2, y^T dout) and dZ1 (X^T dZ1, dZ1 W1^T) enter as BF16
 * pairs hi + lo (about 16 bits, two accumulating GEMMs each); dout is
 * rounded to BF16 for dout W2^T and y^T dout.  Every accumulation, o, y,
 * out, dx and all gradients are FP32.  The descriptor is the
 * attention's and must have dtype BF16, out_dtype FP32, d_qk == d_v.
 *
 * When D is a multiple of 128 the forward's two projections are this
 * library's tensor-core GEMMs: Z1 = X W1 with the SiLU split in its epilogue
 * (z1, U, V, Q, K written once), and out = X + y_hi W2 + y_lo W2 with the
 * residual in its epilogue.  Otherwise, and for the backward's GEMMs, they
 * are plain cuBLAS GEMMs (BF16 x BF16 -> FP32) around this library's
 * element-wise kernels.  cuBLAS's scratch comes from the caller's
 * workspace, but the first call on each (host thread, device) that uses
 * cuBLAS creates a cuBLAS handle, which allocates cuBLAS's own small state:
 * make that first call outside any stream capture.
 * ------------------------------------------------------------------------ */
typedef struct {
  const int64_t* seq_offsets;  /* as hstu_attn_fwd_args */
  const int32_t* num_targets;
  const int32_t* num_contexts;
  const int64_t* timestamps;
  const float* rab_pos;
  const float* rab_time;
  const void* x;               /* [T, D] BF16 layer input */
  const void* w1;              /* [D, 4D] BF16, row-major (x W1) */
  const void* w2;              /* [D, D] BF16, row-major (y W2) */
  float* out;                  /* out [T, D] FP32: x + y W2 */
  float* z1;                   /* out [T, 4D] FP32: x W1, kept for the backward */
  float* u;                    /* out [T, D] FP32: the gate U */
  void* vqk;                   /* out [3, T, D] BF16: V, Q, K, each [T, H, d] */
  void* o;                     /* out [T, D] FP32: A.V, kept for the backward */
  void* y;                     /* out [T, D] FP32: Norm(o) * U (dropped out when desc->dropout_p > 0) */
  uint64_t dropout_seed;       /* fused dropout on y, as hstu_attn_fwd_args */
  uint64_t dropout_offset;
} hstu_layer_fwd_args;

typedef struct {
  const int64_t* seq_offsets;  /* the forward's inputs, unchanged */
  const int32_t* num_targets;
  const int32_t* num_contexts;
  const int64_t* timestamps;
  const float* rab_pos;
  const float* rab_time;
  const void* x;
  const void* w1;
  const void* w2;
  const float* z1;             /* the forward's z1, u, vqk, o, y */
  const float* u;
  const void* vqk;
  const void* o;
  const void* y;
  const float* dout;           /* [T, D] FP32 gradient of the loss w.r.t. out */
  float* dx;                   /* out [T, D]: dout + dZ1 W1^T */
  float* dw1;                  /* out [D, 4D]: X^T dZ1 */
  float* dw2;                  /* out [D, D]: y^T dout */
  float* d_rab_pos;            /* out [H, P] or NULL */
  float* d_rab_time;           /* out [H, Tb] or NULL */
  uint64_t dropout_seed;       /* the forward's dropout seed and offset */
  uint64_t dropout_offset;
} hstu_layer_bwd_args;

/* Workspace bytes of hstu_layer_fwd / hstu_layer_bwd (256-byte aligned
 * workspace; either output may be NULL).  HSTU_ERR_UNSUPPORTED unless dtype
 * is BF16, out_dtype FP32 and D a multiple of 8. */
hstu_status_t hstu_layer_workspace_size(const hstu_attn_desc* desc, size_t* fwd_bytes, size_t* bwd_bytes);

/* Layer forward (above).  All pointers device, 16-byte aligned; outputs are
 * overwritten.  Device-side problems (the attention's, or a tensor-core
 * projection's wait that ran out: HSTU_ERR_TIMEOUT) land in the error word
 * at the start of the workspace (hstu_get_device_error). */
hstu_status_t hstu_layer_fwd(const hstu_attn_desc* desc, const hstu_layer_fwd_args* args,
                             void* workspace, size_t workspace_bytes, hstu_stream_t stream);

/* Layer backward: dx, dw1, dw2 and the bias-table gradients, recomputing the
 * attention tile by tile from the saved u, vqk and o.  All pointers device,
 * 16-byte aligned; outputs are overwritten.  With D % 128 == 0 the four
 * GEMMs run on the library's tensor-core kernels: dw1 and dw2 are then sums
 * over ranges of tokens added in no fixed order (FP32 rounding may differ
 * from call to call); otherwise on cuBLAS.  A tensor-core GEMM's wait that
 * runs out is reported as HSTU_ERR_TIMEOUT in the workspace's error word. */
hstu_status_t hstu_layer_bwd(const hstu_attn_desc* desc, const hstu_layer_bwd_args* args,
                             void* workspace, size_t workspace_bytes, hstu_stream_t stream);

/* ------------------------------------------------------------------------
 * Delta forward: KV-cached, candidate-only inference (P2 "HSTU acceleration
 * operator" paragraph: variable-length sequences with a KV cache; P1 section
 * 2.1.2: the ranking task scores all candidates of a request in one pass).
 *
 * Sequence b has L_b cached tokens (its context and history, already
 * processed: their K and V are kept) and m_b new candidates.  The call
 * computes, for the candidates only, exactly the candidate rows of
 * hstu_attn_fwd on the whole sequence (n = L_b + m_b, num_targets = m_b):
 * candidate r attends every cached token j < L_b (position bucket
 * min(L_b - j, P - 1)) and itself (position bucket 0), never another
 * candidate; o and y as in hstu_attn_fwd.  num_contexts play no part (a
 * candidate sees all cached tokens either way).
 *
 * The descriptor is hstu_attn_fwd's with total_tokens = T_cand (candidates
 * in the batch); max_seq_len = N must bound every L_b + m_b.  Workspace: the
 * forward size from hstu_attn_workspace_size.  Tensor-core path only: BF16,
 * d_qk = d_v in {64, 128}, T_cand >= 128 and T_cache == 0 or >= 128, and no
 * dropout (inference), else HSTU_ERR_UNSUPPORTED.  Offsets inconsistent with the counts are reported
 * through the workspace error word (HSTU_ERR_DEVICE_CHECK).
 * ------------------------------------------------------------------------ */
typedef struct {
  const int64_t* cand_offsets;      /* [B+1] candidates of each sequence, packed; [B] == T_cand */
  const int64_t* cache_offsets;     /* [B+1] cached tokens of each sequence, packed; [B] == cache_tokens */
  int64_t cache_tokens;             /* T_cache */
  const int64_t* cand_timestamps;   /* [T_cand] or NULL (no time bias) */
  const int64_t* cache_timestamps;  /* [T_cache]; NULL iff cand_timestamps is NULL (when T_cache > 0) */
  const float* rab_pos;             /* [H, P] or NULL */
  const float* rab_time;            /* [H, Tb] or NULL */
  const void* q;                    /* [T_cand, H, d] candidates */
  const void* k;                    /* [T_cand, H, d] candidates' own keys */
  const void* v;                    /* [T_cand, H, d] */
  const void* u;                    /* [T_cand, H*d] gate or NULL */
  const void* k_cache;              /* [T_cache, H, d] */
  const void* v_cache;              /* [T_cache, H, d] */
  void* o;                          /* out [T_cand, H, d] */
  void* y;                          /* out [T_cand, H*d] or NULL */
  float* ln_mean;                   /* out [T_cand] or NULL */
  float* ln_rstd;                   /* out [T_cand] or NULL */
} hstu_attn_delta_args;

hstu_status_t hstu_attn_fwd_delta(const hstu_attn_desc* desc, const hstu_attn_delta_args* args,
                                  void* workspace, size_t workspace_bytes, hstu_stream_t stream);

/* ------------------------------------------------------------------------
 * Queries and keys on their way into the attention: an RMS norm per head and
 * a rotation by the token's position, in one pass over both tensors, with its
 * backward.  For one head's d features x of a token at position p:
 *
 *   r = 1 / sqrt(mean(x^2) + eps);  w_i = x_i r gain_i      (norm = 1; else w = x)
 *   pair i of the first rot_dim features, i < rot_dim / 2:
 *     (a, b) = (w_i, w_{i + rot_dim/2}), or (w_{2i}, w_{2i+1}) with interleaved
 *     a' = a cos[p][i] - b sin[p][i];   b' = b cos[p][i] + a sin[p][i]
 *   the features from rot_dim on stay w.
 *
 * The tables are the caller's ([max_position, rot_dim / 2] FP32 each), and
 * so are the positions: a candidate of the ranking task has the position
 * h_end of its sequence, like in the attention's position buckets.  Sums and
 * products are FP32 (mean(x^2) + eps has to be a normal FP32 number), each output
 * is rounded once.  Backward, with e = the
 * incoming gradient turned back by the rotation:
 *   dgain_i = sum over tokens and heads of e_i x_i r
 *   dx = r (e gain - x r mean(e gain x r))                  (norm = 0: dx = e)
 *
 * Either of q, k may be absent (its head count 0).  Tensors are strided: the
 * d features of a head are contiguous, heads and tokens lie any multiple of
 * 16 bytes apart (q and k may be parts of one projection's output).  An
 * output may be its input (same pointer and strides); other overlaps of an
 * output with anything are the caller's error.  d is 32, 64 or 128, rot_dim a
 * multiple of 8 (0: no rotation) of at most d.
 *
 * The workspace (256-byte aligned) starts with a 256-byte header that must
 * be zero before its first use.  An error that the device finds (a position
 * outside the tables: HSTU_ERR_DEVICE_CHECK, that row's output is undefined)
 * stays in the header, read by hstu_get_device_error, until the caller zeroes
 * it.  Calls that overlap in time need workspaces of their own.
 * ------------------------------------------------------------------------ */
typedef struct {
  uint32_t struct_size;      /* sizeof(hstu_qk_desc) */
  int32_t dtype;             /* of q, k and everything shaped like them */
  int32_t Hq, Hk;            /* heads of q and of k; 0: absent */
  int32_t d;
  int32_t rot_dim;
  int32_t interleaved;       /* pairs of neighbours instead of halves */
  int32_t norm;              /* 1: RMS norm with gain, 0: none */
  float eps;
  uint32_t reserved;         /* must be 0 */
  int64_t total_tokens;      /* T */
  int64_t max_position;      /* rows of cos and sin */
  int64_t q_strides[2];      /* of q: elements from token to token, from head to head */
  int64_t k_strides[2];
  int64_t q_out_strides[2];  /* of q_out (forward) and dq_out (backward) */
  int64_t k_out_strides[2];
  int64_t dq_strides[2];     /* of dq (backward only) */
  int64_t dk_strides[2];
} hstu_qk_desc;

typedef struct {
  const int64_t* num_tokens; /* device: tokens to work on, <= T (e.g. &seq_offsets[B]); rows behind them are left
                                as they are.  NULL: all T */
  const int32_t* positions;  /* [T]; may be NULL when rot_dim is 0 */
  const float* cos;          /* [max_position, rot_dim / 2] */
  const float* sin;
  const float* q_gain;       /* [d], shared by all heads, or NULL (ones); only with norm */
  const float* k_gain;
  const void* q;             /* [T, Hq, d] strided */
  const void* k;             /* [T, Hk, d] strided */
  void* q_out;
  void* k_out;
} hstu_qk_fwd_args;

typedef struct {
  const int64_t* num_tokens;
  const int32_t* positions;
  const float* cos;
  const float* sin;
  const float* q_gain;
  const float* k_gain;
  const void* q;             /* the forward's inputs */
  const void* k;
  const void* dq_out;        /* gradients of the forward's outputs */
  const void* dk_out;
  void* dq;                  /* out */
  void* dk;
  float* d_q_gain;           /* out [d] FP32 or NULL (not wanted); summed in a fixed order */
  float* d_k_gain;
} hstu_qk_bwd_args;

hstu_status_t hstu_qk_workspace_size(const hstu_qk_desc* desc, size_t* fwd_bytes, size_t* bwd_bytes);
hstu_status_t hstu_qk_norm_rope_fwd(const hstu_qk_desc* desc, const hstu_qk_fwd_args* args, void* workspace,
                                    size_t workspace_bytes, hstu_stream_t stream);
hstu_status_t hstu_qk_norm_rope_bwd(const hstu_qk_desc* desc, const hstu_qk_bwd_args* args, void* workspace,
                                    size_t workspace_bytes, hstu_stream_t stream);

/* ------------------------------------------------------------------------
 * A paged cache of keys and values in 4 bits, for serving.
 *
 * The 16 features [16 g, 16 g + 16) of one head of one token share a scale s
 * in e4m3 (4 exponent and 3 mantissa bits); each is held as a code in e2m1,
 * whose magnitudes are 0, .5, 1, 1.5, 2, 3, 4, 6.  With E = k_exp for keys and
 * v_exp for values, one power of two for the whole cache:
 *
 *   s = e4m3(max |x| 2^-E / 6), at most 448;  code = e2m1(x 2^-E / s), at most 6
 *   value = code s 2^E        (s = 0: all values 0; a NaN in the group: all NaN;
 *                              an infinity: the largest code of s = 448)
 *
 * both rounded to nearest, ties to the even mantissa, as real numbers would be
 * (the borders are decided exactly).  A value has 6 significant bits: it is a
 * BF16 number, and before the 2^E a FP16 number too.  A group's smallest
 * scale is 2^-9, so E should bring the data's usual magnitude near 1.
 *
 * pages is [num_pages][H] blocks of 2 page_size (d/2 + d/16) bytes, each
 *   K codes [page_size][d/2] | K scales [page_size][d/16] | V codes | V scales,
 * feature 2i in the low half of byte i.  A sequence of L tokens lies in the
 * pages block_table[b][0 .. ceil(L / page_size)), position j at place
 * j % page_size of entry j / page_size.  Sequences may share pages that are
 * only read; a position that is being written belongs to one sequence.
 * timestamps, when the time bias is wanted, are [num_pages][page_size].
 *
 * The calls below take workspaces as hstu_qk_norm_rope_fwd does (zero header,
 * errors stay until the header is zeroed), and tokens or rows behind
 * seq_offsets[B] (a batch padded to a fixed total_tokens) are left as they
 * are.  Inconsistent offsets or lengths and page numbers outside the cache
 * are found on the device (HSTU_ERR_DEVICE_CHECK); nothing outside the given
 * buffers is touched then.  An append or a read leaves out the tokens that
 * have no place (or no row of the tables) and does all others, unless the
 * offsets do not fit the rows: then it does nothing.
 * ------------------------------------------------------------------------ */
typedef struct {
  uint32_t struct_size;      /* sizeof(hstu_cache_desc) */
  int32_t H, d;              /* d = 64 or 128 */
  int32_t page_size;         /* 32, 64 or 128 */
  int32_t num_pages;
  int32_t k_exp, v_exp;      /* -32 .. 32 */
  int32_t max_pages;         /* entries of a row of the block tables */
  void* pages;               /* 16-byte aligned */
  int64_t* timestamps;       /* 16-byte aligned, or NULL */
} hstu_cache_desc;

/* Append: token i of the n_b = seq_offsets[b+1] - seq_offsets[b] new ones of
 * sequence b is written at position cache_lens[b] - n_b + i, where cache_lens
 * counts the new tokens too.  On its way a key goes through the norm and the
 * rotation of hstu_qk_norm_rope_fwd (p = its position in the cache), without
 * being rounded in between.  k and v are BF16, strided as there. */
typedef struct {
  int32_t B;
  int32_t rot_dim, interleaved, norm;
  float eps;
  uint32_t reserved;           /* must be 0 */
  int64_t total_tokens;        /* rows of k, v, timestamps */
  int64_t max_position;        /* rows of cos, sin; every written position lies below it (with rot_dim > 0) */
  int64_t k_strides[2], v_strides[2];
  const int64_t* seq_offsets;  /* [B+1], non-decreasing, seq_offsets[0] == 0, seq_offsets[B] <= total_tokens */
  const int32_t* cache_lens;   /* [B] */
  const int32_t* block_table;  /* [B][max_pages] */
  const int64_t* token_times;  /* [total_tokens], written to the cache's timestamps; NULL iff those are NULL */
  const float* cos;
  const float* sin;
  const float* k_gain;         /* [d] or NULL */
  const void* k;
  const void* v;
} hstu_cache_append_args;

/* Read: positions [starts[b], starts[b] + n_b) of sequence b into rows
 * seq_offsets[b].. of dense BF16 k, v [total_tokens, H, d] (and times). */
typedef struct {
  int32_t B;
  uint32_t reserved;           /* must be 0 */
  int64_t total_tokens;
  const int64_t* seq_offsets;  /* [B+1] */
  const int32_t* starts;       /* [B] first position, or NULL (0) */
  const int32_t* block_table;
  void* k;                     /* out, or NULL */
  void* v;                     /* out, or NULL */
  int64_t* token_times;        /* out, or NULL */
} hstu_cache_read_args;

/* Bytes of pages for this descriptor's H, d, page_size and num_pages. */
hstu_status_t hstu_cache_bytes(const hstu_cache_desc* cache, size_t* page_bytes, size_t* total_bytes);
/* Workspace: 256 bytes for both. */
hstu_status_t hstu_cache_append(const hstu_cache_desc* cache, const hstu_cache_append_args* args, void* workspace,
                                size_t workspace_bytes, hstu_stream_t stream);
hstu_status_t hstu_cache_read(const hstu_cache_desc* cache, const hstu_cache_read_args* args, void* workspace,
                              size_t workspace_bytes, hstu_stream_t stream);

/* ------------------------------------------------------------------------
 * HSTU attention of new rows over the paged cache (the delta forward's
 * serving form).  Sequence b has L = cache_lens[b] cached tokens and
 * n = seq_offsets[b+1] - seq_offsets[b] rows, of which the last m =
 * num_targets[b] are candidates and the first n - m are its newest history
 * tokens, already appended: row r < n - m is the token at position
 * L - (n - m) + r and sees the cached positions up to its own; a candidate
 * has position L, sees the whole cache and itself (its own BF16 key and
 * value, which are not in the cache), never another candidate.  Buckets, 1/N,
 * norm and gate as in hstu_attn_fwd without contexts.  k, v are read for
 * candidates only.
 *
 * The descriptor is the attention's: dtype and out_dtype BF16, d_qk == d_v ==
 * the cache's d, H <= its H * d limit, total_tokens = rows, max_seq_len = N
 * bounding every L + m, no flags but HSTU_FLAG_TEST_TIMEOUT, no dropout.
 * max_rows bounds every n (it picks the tile's width for all sequences of the
 * call: 8, 32, 64 or 128 rows).  Outputs are left as they are where the batch
 * is refused on the device; where a wait ran out (HSTU_ERR_TIMEOUT) they are
 * undefined.
 *
 * Precision: K, V and q enter the tensor cores exactly; 16 SiLU(z) is rounded
 * once to FP16 (so scores of 4094 and more overflow to infinity; a bias of
 * minus infinity leaves the pair out, and a NaN value in a token that a history
 * row does not see yet still reaches it where both lie in one block of rows);
 * sums, norm and gate are FP32 and o and y are rounded once.  The cache's tiles
 * are dealt to the CTAs by their cost, whatever sequence they belong to, and
 * partial sums added in a fixed order: equal inputs give equal bits.
 * ------------------------------------------------------------------------ */
typedef struct {
  int32_t max_rows;
  uint32_t reserved;             /* must be 0 */
  const int64_t* seq_offsets;    /* [B+1], seq_offsets[B] <= total_tokens */
  const int32_t* cache_lens;     /* [B] */
  const int32_t* num_targets;    /* [B] or NULL (no candidates) */
  const int32_t* block_table;    /* [B][max_pages] */
  const int64_t* row_times;      /* [T] or NULL (no time bias); needs the cache's timestamps */
  const float* rab_pos;          /* [H, P] or NULL */
  const float* rab_time;         /* [H, Tb] or NULL; ignored without row_times */
  const void* q;                 /* [T, H, d] dense, like k, v */
  const void* k;                 /* may be NULL without num_targets */
  const void* v;
  const void* u;                 /* [T, H*d] BF16 gate or NULL (one) */
  void* o;                       /* out [T, H, d] or NULL */
  void* y;                       /* out [T, H*d] or NULL */
} hstu_attn_cached_args;

hstu_status_t hstu_attn_cached_workspace_size(const hstu_attn_desc* desc, const hstu_cache_desc* cache,
                                              int32_t max_rows, size_t* bytes);
hstu_status_t hstu_attn_fwd_cached(const hstu_attn_desc* desc, const hstu_cache_desc* cache,
                                   const hstu_attn_cached_args* args, void* workspace, size_t workspace_bytes,
                                   hstu_stream_t stream);

/* ------------------------------------------------------------------------
 * Layer norm over the D features of a row, with weight and bias, and its
 * backward (what the input of a projection goes through; the attention's own
 * norm-gate has neither weight nor bias):
 *
 *   mean = mean(x);  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 *   y = (x - mean) rstd weight + bias
 * Backward, with h = (x - mean) rstd and e = dy weight:
 *   dx = rstd (e - mean(e) - h mean(e h)) [+ dres]
 *   d_weight = sum over rows of dy h;   d_bias = sum over rows of dy
 *
 * x (and dx, dres) and y (or dy) are BF16 or FP32 each on its own; weight,
 * bias, the statistics and their gradients are FP32.  Sums and products are
 * FP32, each output is rounded once.  Rows are strided: features contiguous,
 * rows any number of elements apart (rows that are 16-byte aligned with D a
 * multiple of 8 take wide loads).  1 <= D <= 16384.  An output may be an input
 * of the same type (same pointer and stride); other overlaps are the
 * caller's error.  d_weight and d_bias are summed in an order that depends on
 * the sizes only: equal inputs give equal bits.
 *
 * The workspace (256-byte aligned) starts with a 256-byte header that must be
 * zero before its first use; an error found on the device (num_rows outside
 * [0, rows]: HSTU_ERR_DEVICE_CHECK, no row is taken) stays in it until the
 * caller zeroes it.  Calls that overlap in time need workspaces of their own.
 * ------------------------------------------------------------------------ */
typedef struct {
  uint32_t struct_size;      /* sizeof(hstu_ln_desc) */
  int32_t x_dtype;           /* of x, dx, dres */
  int32_t y_dtype;           /* of y (forward), dy (backward) */
  int32_t D;
  float eps;
  uint32_t reserved;         /* must be 0 */
  int64_t rows;
  int64_t x_stride;          /* elements from row to row */
  int64_t y_stride;          /* of y, or of dy */
  int64_t dx_stride;         /* backward only */
  int64_t dres_stride;       /* backward with dres only */
} hstu_ln_desc;

typedef struct {
  const int64_t* num_rows;   /* device: rows to work on, <= rows; rows behind them are left as they are and
                                do not count.  NULL: all */
  const void* x;             /* [rows, D] strided */
  const float* weight;       /* [D] or NULL (ones) */
  const float* bias;         /* [D] or NULL (zeros) */
  void* y;                   /* out [rows, D] strided */
  float* mean;               /* out [rows] or NULL */
  float* rstd;               /* out [rows] or NULL */
} hstu_ln_fwd_args;

typedef struct {
  const int64_t* num_rows;
  const void* x;
  const float* weight;
  const float* mean;         /* the forward's */
  const float* rstd;
  const void* dy;            /* [rows, D] strided */
  const void* dres;          /* [rows, D] strided, added to dx, or NULL */
  void* dx;                  /* out [rows, D] strided */
  float* d_weight;           /* out [D] or NULL (not wanted) */
  float* d_bias;             /* out [D] or NULL */
} hstu_ln_bwd_args;

hstu_status_t hstu_ln_workspace_size(const hstu_ln_desc* desc, size_t* fwd_bytes, size_t* bwd_bytes);
hstu_status_t hstu_ln_fwd(const hstu_ln_desc* desc, const hstu_ln_fwd_args* args, void* workspace,
                          size_t workspace_bytes, hstu_stream_t stream);
hstu_status_t hstu_ln_bwd(const hstu_ln_desc* desc, const hstu_ln_bwd_args* args, void* workspace,
                          size_t workspace_bytes, hstu_stream_t stream);

/* ------------------------------------------------------------------------
 * Products of ragged groups of rows, each with a weight matrix of its own (a
 * projection per kind of token, scenario or expert), and their gradients:
 *
 *   y[r]  = x[r] W[g]                       for the rows r of group g
 *   dx[r] = dy[r] W[g]^T
 *   dW[g] = sum over its rows of x[r]^T dy[r]   (zero for a group without rows)
 *
 * Rows lie in the order of their groups: group g has rows
 * [group_offsets[g], group_offsets[g + 1]), offsets on the device, from 0 on,
 * not decreasing, the last one at most `rows`.  Rows behind the last group
 * are left as they are and not read into any result.  x, W, dy are BF16, sums FP32 on the tensor cores; y and dx
 * are rounded once to their type, dW is FP32.  K and N are multiples of 8, rows
 * a multiple of 16 bytes apart (any row stride that is a multiple of 8
 * elements); W and dW are dense [groups][K][N].  Up to 4096 groups.  Outputs
 * must not overlap inputs.  Equal inputs give equal bits.
 *
 * The workspace is 256-byte aligned; its first 256 bytes, the header, must be zero
 * before its first use.  Offsets that break the rules above (HSTU_ERR_DEVICE_CHECK:
 * nothing is computed) and a pipeline wait that ran out (HSTU_ERR_TIMEOUT) stay in the
 * header until the caller zeroes it.  zero_bytes are the header and the counters behind
 * it, the same for every shape; the backward clears its counters itself, so a workspace may serve
 * calls of other shapes and operators in turn.  Calls that overlap in time need
 * workspaces of their own.
 * ------------------------------------------------------------------------ */
typedef struct {
  uint32_t struct_size;      /* sizeof(hstu_group_desc) */
  int32_t groups;            /* 1 .. 4096 */
  int32_t K, N;
  int32_t y_dtype;           /* of y: HSTU_BF16 or HSTU_FP32 */
  int32_t dx_dtype;          /* of dx */
  uint32_t flags;            /* 0, or HSTU_FLAG_TEST_TIMEOUT: the first load is withheld and waits give up
                                after about a millisecond */
  uint32_t reserved;         /* must be 0 */
  int64_t rows;              /* T */
  int64_t x_stride;          /* elements from row to row, multiples of 8 */
  int64_t y_stride;          /* of y (forward) and dy (backward) */
  int64_t dx_stride;         /* backward only */
} hstu_group_desc;

typedef struct {
  const int64_t* group_offsets; /* [groups + 1] */
  const void* x;             /* [T, K] strided, BF16 */
  const void* w;             /* [groups, K, N] BF16 */
  void* y;                   /* out [T, N] strided */
} hstu_group_fwd_args;

typedef struct {
  const int64_t* group_offsets;
  const void* x;             /* for dw */
  const void* w;             /* for dx */
  const void* dy;            /* [T, N] strided, BF16 */
  void* dx;                  /* out [T, K] strided, or NULL (not wanted) */
  float* dw;                 /* out [groups, K, N], or NULL (not wanted) */
} hstu_group_bwd_args;

hstu_status_t hstu_group_workspace_size(const hstu_group_desc* desc, size_t* fwd_bytes, size_t* bwd_bytes,
                                        size_t* zero_bytes);
hstu_status_t hstu_group_fwd(const hstu_group_desc* desc, const hstu_group_fwd_args* args, void* workspace,
                             size_t workspace_bytes, hstu_stream_t stream);
hstu_status_t hstu_group_bwd(const hstu_group_desc* desc, const hstu_group_bwd_args* args, void* workspace,
                             size_t workspace_bytes, hstu_stream_t stream);

/* ------------------------------------------------------------------------
 * An AdamW step over many tensors in one launch:
 *
 *   g = grad grad_scale
 *   m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr' wd) - lr' / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * with t the step (counted on the device, from steps_done + 1 on; one count for
 * all tensors, those that had no gradient in earlier steps among them) and
 * lr' = lr times the tensor's lr_scale.  Parameters are FP32; a tensor may
 * have a BF16 copy (the projections' operands), which is written with the
 * rounded new value.  Gradients are FP32 or BF16.  FP32 arithmetic; m and v
 * are computed product by product without contraction.
 *
 * state_bits 32: m and v are FP32.  state_bits 8: 256 neighbouring elements of
 * a tensor form a block with one byte E a moment, the FP32 exponent field of
 * its largest finite magnitude, at least 16 (a byte below 16 counts as 16).  m is a sign, 4 exponent bits (bias 7) and 3
 * of mantissa, times 2^(E - 134); v is 5 exponent bits (bias 15) and 3 of
 * mantissa, times 2^(E - 142).  The parameters take the new moments before
 * they are rounded.  Rounding is up or down at random, so that means are kept
 * (rounding to the nearest would leave v as it is for ever: a step's decay of a
 * thousandth is far below half a step of 3 bits): the magnitude's 20 bits
 * that fall away get 16 r + 8 added, r 16 random bits.  Element e of the
 * blocks (all blocks counted through the tensors in their order) takes word e mod 4 of Philox4x32-10
 * (Salmon, Moraes, Dror, Shaw, SC 2011) at counter (e div 4, t), key seed;
 * its low half serves m, the high half v.  A new m that is not finite is kept as
 * NaN (code 127), such a v as the largest value.
 *
 * hstu_adamw_init checks the tensors (host array), lays out the workspace (256-byte aligned)
 * and synchronises the stream; a stream that is being captured is refused
 * (HSTU_ERR_INVALID_ARG).  hstu_adamw_step launches one kernel and may be captured: each
 * replay is a step.  A descriptor that is not the one the workspace was laid out
 * for is found on the device (HSTU_ERR_DEVICE_CHECK, nothing is written).  lr and grad_scale on the device, where given, are read at
 * every step in place of the descriptor's lr (and of one).  skip, where given, is
 * read at every step: not zero, nothing changes and the step does not count (a
 * batch whose gradients overflowed).
 * hstu_adamw_read writes the tensors' moments as FP32 or BF16 values (8-bit
 * moments are exact in either, but for what BF16 and FP32 call subnormal):
 * hstu_adamw_read_init lays out a workspace of its own for it.
 *
 * Tensors must not overlap.  Pointers are 16-byte aligned (copies
 * 8 bytes; exponent bytes any).  One call at a time on a workspace.
 * ------------------------------------------------------------------------ */
typedef struct {
  uint32_t struct_size;      /* sizeof(hstu_adamw_desc) */
  int32_t state_bits;        /* 32 or 8 */
  int32_t grad_dtype;        /* HSTU_BF16 or HSTU_FP32 */
  int32_t num_tensors;       /* >= 0 */
  double lr, beta1, beta2, eps;  /* 0 <= beta < 1, eps >= 1e-12 */
  uint64_t seed;             /* of the 8-bit moments' rounding */
  int64_t steps_done;        /* init: steps taken before; -1: what the workspace has counted is kept */
  int64_t chunks;            /* set by init (read_init): the length of the workspace's list */
} hstu_adamw_desc;

typedef struct {
  float* param;              /* [n] */
  const void* grad;          /* [n], or NULL: this tensor is left as it is */
  void* copy;                /* [n] BF16, or NULL */
  void* m;                   /* [n] FP32, or uint8 codes */
  void* v;
  uint8_t* m_exp;            /* [ceil(n / 256)], 8 bits only */
  uint8_t* v_exp;
  int64_t n;                 /* elements, >= 0 */
  float weight_decay;
  float lr_scale;
} hstu_adamw_tensor;

typedef struct {
  const float* lr;           /* device, or NULL: desc->lr */
  const float* grad_scale;   /* device, or NULL: 1 */
  const int32_t* skip;       /* device, or NULL: 0 */
} hstu_adamw_step_args;

typedef struct {
  void* m;                   /* out [n], or NULL (not wanted); 16-byte aligned */
  void* v;
} hstu_adamw_moments;

hstu_status_t hstu_adamw_workspace_size(const hstu_adamw_desc* desc, const hstu_adamw_tensor* tensors, size_t* bytes);
hstu_status_t hstu_adamw_init(hstu_adamw_desc* desc, const hstu_adamw_tensor* tensors, void* workspace,
                              size_t workspace_bytes, hstu_stream_t stream);
hstu_status_t hstu_adamw_step(const hstu_adamw_desc* desc, const hstu_adamw_step_args* args, void* workspace,
                              size_t workspace_bytes, hstu_stream_t stream);
hstu_status_t hstu_adamw_read_init(hstu_adamw_desc* desc, const hstu_adamw_tensor* tensors,
                                   const hstu_adamw_moments* outs, int32_t out_dtype, void* workspace,
                                   size_t workspace_bytes, hstu_stream_t stream);
hstu_status_t hstu_adamw_read(const hstu_adamw_desc* desc, void* workspace, size_t workspace_bytes, hstu_stream_t stream);
/* Steps counted on this workspace (steps_done included).  Synchronises the stream. */
hstu_status_t hstu_adamw_steps(const void* workspace, hstu_stream_t stream, int64_t* steps);

/* Reads the device error word of the last call that used this workspace
 * (HSTU_OK when none).  Synchronises the stream. */
hstu_status_t hstu_get_device_error(const void* workspace, hstu_stream_t stream, int32_t* code);

/* Static string for a status code. */
const char* hstu_status_string(hstu_status_t status);

/* After HSTU_ERR_CUDA: the failing CUDA call of the last call on this thread,
 * by name, or the kernel launch with its resource attributes (registers,
 * threads per block, shared memory).  Empty when the last call did not fail
 * in CUDA.  The string belongs to the library and lives until the next call
 * on this thread. */
const char* hstu_last_error_detail(void);

/* Number of this library's kernels that the last successful hstu_attn_fwd,
 * hstu_attn_bwd, hstu_attn_fwd_delta, hstu_layer_*, hstu_qk_*, hstu_cache_*,
 * hstu_attn_fwd_cached, hstu_ln_*, hstu_group_* or hstu_adamw_* call on this thread launched (for launch accounting; cuBLAS's kernels inside
 * the layer calls are not counted). */
int32_t hstu_last_launch_count(void);

/* Measurement hook.  start_event and stop_event are cudaEvent_t handles (or
 * both NULL to clear).  The next hstu_attn_fwd or hstu_attn_bwd call on this
 * thread records start_event on its stream right before launching its
 * attention kernel and stop_event right after, then forgets them.  Under
 * stream capture they are recorded as external event nodes, so each replay
 * of the graph timestamps them. */
hstu_status_t hstu_time_next_attention_kernel(void* start_event, void* stop_event);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_ATTN_H_ */
