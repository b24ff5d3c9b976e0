// What the cached attention's two kernels share: the call's parameters, the
// checks of a sequence's numbers, and how its work is cut into tiles.
//
// A sequence's n rows form blocks of N; a block's keys are the 128-token
// tiles [0, tiles) of its cache, up to the last position that one of its rows
// sees.  An item is a (block, head).  All items' tiles in a row, ordered by
// sequence, block, head and tile, are cut into equal parts, one a CTA; a CTA's
// part of an item is a piece, and leaves one FP32 sum [N][d] in the workspace
// at slot item + CTA (no two pieces share one: every further piece crosses
// the border of an item, of a CTA, or both).
#pragma once

#include "hstu_fp4.cuh"
#include "hstu_internal.h"
#include "hstu_seq_search.cuh"

namespace hstu {

constexpr int kCachedTile = 128;

struct CachedParams {
  const int64_t* off;
  const int32_t* lens;
  const int32_t* nt;
  const int32_t* table;
  const int64_t* times;       // NULL: no time bias
  const float* rab_pos;
  const float* rab_time;      // NULL without times
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* u;
  __nv_bfloat16* o;
  __nv_bfloat16* y;
  const uint8_t* pages;
  const int64_t* page_times;
  float* part;                // [slots][N][d]
  int* seq_tiles;             // [B] tiles of all items before the sequence
  int* seq_items;             // [B] items before it
  int* hdr;
  int64_t T;
  int B, H, page_size, num_pages, max_pages, max_rows, max_n, P, Tb, norm;
  float alpha, inv_n, eps;
  float k_scale;              // 2^k_exp
  float o_scale;              // 2^v_exp / 16 / N of a tensor-core sum
};

// header words of the cached attention's workspace (beside WS_ERR)
enum : int { WS_CA_QUOTA = 16 };   // tiles a CTA, -1 where the batch was refused

struct CachedSeq {
  int64_t row0;   // first row
  int n, m, L;    // rows, candidates among them, cached tokens
};

// Loads sequence b; false where its numbers do not fit together.
__device__ __forceinline__ bool load_seq(const CachedParams& p, int b, CachedSeq& s) {
  const int64_t o0 = p.off[b], n = p.off[b + 1] - o0;
  s.row0 = o0;
  s.m = p.nt ? p.nt[b] : 0;
  s.L = p.lens[b];
  s.n = (int)n;
  return o0 >= 0 && n >= 0 && o0 + n <= p.T && n <= p.max_rows && s.m >= 0 && s.m <= n && s.L >= n - s.m &&
         (int64_t)s.L + s.m <= p.max_n && s.L <= (int64_t)p.max_pages * p.page_size;
}

// Tiles of block qb of N rows.
__device__ __forceinline__ int block_tiles(const CachedSeq& s, int qb, int N) {
  const int last = min(s.n, (qb + 1) * N) - 1, hist = s.n - s.m;
  const int seen = last >= hist ? s.L : s.L - hist + last + 1;
  return (seen + kCachedTile - 1) / kCachedTile;
}

int cached_block_rows(int max_rows);                 // N of a call
cudaError_t launch_tc_cached(const CachedParams& p, int d, int N, int ctas, cudaStream_t st);

}  // namespace hstu
