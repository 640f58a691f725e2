// How the attention of drafted tokens over a paged cache is divided among its CTAs.
//
// A tile is (sequence b, key head m, row group): up to `rows` of the T * g query rows that
// share key head m (row r = token r / g, query head m g + r % g).  Its keys are blocks of
// 64: the pages of the context that some row can see, then the draft's own tokens.  All
// tiles' blocks, laid end to end, are one list of W items; CTA c of G takes the items
// [c W / G, (c + 1) W / G), whatever sequences they belong to, so a batch of one long and
// many short sequences divides as evenly as a single sequence.  The lengths are read on
// the device: a captured graph follows them.
//
// A tile that lies in one CTA's items is finished there.  Of the others each CTA writes a
// partial result (row maximum, row sum, unnormalised output): the tile that it begins in
// to slot 2c, the one that it ends in to slot 2c + 1; the joining kernel finds a tile's
// partials by the same arithmetic.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gca {

struct SeqBlocks {
  int len;    // context tokens
  int p0;     // first page that some row can see
  int np;     // pages from there
  int nb;     // blocks: pages, then the draft's
};

__device__ __forceinline__ SeqBlocks seq_blocks(const TreeArgs& a, int b, bool flag) {
  SeqBlocks s;
  const int n = a.lengths[b], most = (int)min((int64_t)a.width * kChunk, (int64_t)INT32_MAX);
  s.len = min(max(n, 0), most);
  if (flag && s.len != n) flag_bad_index(a.err, n);
  // Every position is at least len, so no row sees tokens before len - window + 1.
  const int low = a.window > 0 ? max(0, s.len - a.window + 1) : 0;
  s.p0 = low / kChunk;
  s.np = (int)(((int64_t)s.len + kChunk - 1) / kChunk) - s.p0;
  if (s.np < 0) s.np = 0;
  s.nb = s.np + a.nd;
  return s;
}

struct Share {
  int b;          // sequence that item `lo` lies in
  int64_t off;    // its offset among that sequence's items
  int64_t lo, hi; // this CTA's items
  int64_t W;      // all items
  int64_t G;      // CTAs that have work
};

// Called by all `NT` threads of a CTA; `buf` holds NT / 32 + 1 values.  With `find` >= 0 the
// item of a given sequence's start is returned in `lo` instead of this CTA's share.
template <int NT>
__device__ __forceinline__ Share share_of(const TreeArgs& a, int cta, int find, int64_t* buf, Share* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + NT - 1) / NT, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  const int64_t tiles = (int64_t)a.Hkv * a.nrt;
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += seq_blocks(a, b, cta == 0).nb * tiles;
  int64_t incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) buf[warp] = incl;
  __syncthreads();
  int64_t before = 0, W = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) before = W;
    W += buf[w];
  }
  const int64_t excl = before + incl - sum;
  const int64_t G = min((int64_t)a.grid, max((int64_t)1, (W + a.min_blocks - 1) / a.min_blocks));
  const int64_t lo = find >= 0 ? 0 : (cta < G ? W * cta / G : W);
  const int64_t hi = find >= 0 ? 0 : (cta < G ? W * (cta + 1) / G : W);
  if (find >= 0 ? (find >= b0 && find < b1) : (lo >= excl && lo < excl + sum)) {
    int64_t at = excl;
    int b = b0;
    for (;; ++b) {
      const int64_t n = seq_blocks(a, b, false).nb * tiles;
      if (find >= 0 ? b == find : lo < at + n) break;
      at += n;
    }
    *out = find >= 0 ? Share{b, 0, at, 0, W, G} : Share{b, lo - at, lo, hi, W, G};
  } else if (find < 0 && lo >= W && tid == 0) {
    *out = Share{0, 0, lo, hi, W, G};
  }
  __syncthreads();
  return *out;
}

// Whether key u of the draft is seen by row t (mask words, or the causal chain), before the window.
__device__ __forceinline__ bool sees_draft(const TreeArgs& a, int b, int t, int u) {
  if (!a.mask) return u <= t;
  return (a.mask[((int64_t)b * a.T + t) * a.words + (u >> 6)] >> (u & 63)) & 1;
}

// Position of token t (never below the context's length), or -1 for padding.
__device__ __forceinline__ int64_t token_position(const TreeArgs& a, int b, int t, int len) {
  if (!a.positions) return (int64_t)len + t;
  const int p = a.positions[(int64_t)b * a.T + t];
  return p < 0 ? -1 : max(p, len);
}

}  // namespace gca
