// How the attention of drafted tokens over a paged cache is divided among its CTAs.
//
// The work is a list of W items: for each sequence b, for each set of `hl * hw` key heads side by
// side, its blocks of 64 keys (the pages of the context that some row can see, then the
// draft's own tokens).  The list is cut into G shares of W / G items in a row (one more or
// less), whatever sequences they belong to, so a batch of one long and many short sequences
// divides as evenly as a single sequence.  The lengths are read on the device: a captured
// graph follows them.
//
// A share has hl * nrt CTAs, which walk its items together: one for each `hw` of the set's key
// heads, and of each key head m one for each `rows` of the T * g query rows that share it (row
// r = token r / g, query head m g + r % g).  The heads of a token lie side by side in memory:
// read at the same time they make long runs for DRAM, read at different times pieces of
// 128 bytes (measured: 12 heads of 64 over 4 x 64K tokens, 32 rows a head: 142 us together, 203
// us apart); and the row groups after the first find their pages in L2.
//
// A tile (sequence, hw heads, row group) whose blocks lie in one share is finished there.  Of
// the others each CTA writes a partial result (row maximum, row sum, unnormalised output): the
// one that its share begins in to the first of its two slots, the one that it ends in to the
// second; the joining kernel finds a tile's partials by the same arithmetic.
//
// Where the tiles are short and all of them find a CTA at once, a share is a sequence, its CTAs
// finish a tile each, and there is nothing to join.
//
// Going on to another tile costs a CTA the queries' load, a pipeline that fills again and a
// second result.  So each tile has `lead` items without work before its first block, about
// what that costs in blocks: a share that holds them has fewer blocks.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gca {

struct SeqBlocks {
  int len;    // context tokens
  int p0;     // first page that some row can see
  int np;     // pages from there
  int nb;     // blocks: pages, then the draft's
  int items;  // the blocks and the lead
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
  s.items = a.lead + s.nb;
  return s;
}

struct Share {
  int W, G;      // all items, shares
  int q, rem;    // W = q G + rem: the first rem shares have q + 1 items, the others q
  int lo, hi;    // items of this share
  int b, off;    // the sequence that item lo lies in, and its offset among that sequence's items
};
__device__ __forceinline__ int first_item(const Share& s, int share) { return s.q * share + min(share, s.rem); }
__device__ __forceinline__ int owner_of(const Share& s, int item) {
  const int t = s.rem * (s.q + 1);
  return item < t ? item / (s.q + 1) : s.rem + (item - t) / s.q;
}

// Items of all sequences, and of those before b, summed by one warp.  (The host sees to it that
// all items together stay below 2^31.)
__device__ __forceinline__ int all_items(const TreeArgs& a, int b, int& before, bool flag) {
  int sum = 0, part = 0;
  for (int i = threadIdx.x & 31; i < a.B; i += 32) {
    const int n = seq_blocks(a, i, flag).items;
    sum += n;
    if (i < b) part += n;
  }
  const int sets = a.Hkv / (a.hw * a.hl);
  before = __reduce_add_sync(0xffffffffu, part) * sets;
  return __reduce_add_sync(0xffffffffu, sum) * sets;
}
__device__ __forceinline__ Share shares(const TreeArgs& a, int W) {
  Share s;
  s.W = W;
  s.G = max(1, min(a.grid, W >> (W > a.far ? a.least + 1 : a.least)));
  s.q = W / s.G;
  s.rem = W - s.q * s.G;
  return s;
}

// This CTA's share; called by whole warps, each for itself.
__device__ __forceinline__ Share my_share(const TreeArgs& a) {
  const int lane = threadIdx.x & 31, tiles = a.Hkv / (a.hw * a.hl), share = blockIdx.x / (a.hl * a.nrt);
  if (a.whole) {
    Share s{};
    s.b = share;
    s.hi = seq_blocks(a, share, blockIdx.x % (a.hl * a.nrt) == 0 && threadIdx.x == 0).items;
    return s;
  }
  int before;
  Share s = shares(a, all_items(a, 0, before, blockIdx.x == 0 && threadIdx.x < 32));
  s.lo = share < s.G ? first_item(s, share) : s.W;
  s.hi = share < s.G ? first_item(s, share + 1) : s.W;
  s.b = s.off = 0;
  if (s.lo >= s.hi) return s;
  for (int b0 = 0, at = 0;; b0 += 32) {
    const int n = b0 + lane < a.B ? seq_blocks(a, b0 + lane, false).items * tiles : 0;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const uint32_t in = __ballot_sync(0xffffffffu, n > 0 && s.lo < at + incl);
    if (in) {
      const int l = __ffs(in) - 1;
      s.b = b0 + l;
      s.off = s.lo - at - __shfl_sync(0xffffffffu, incl - n, l);
      return s;
    }
    at += __shfl_sync(0xffffffffu, incl, 31);
    if (b0 + 32 >= a.B) return s;
  }
}

// The segments of a share, one after the other: blocks blk0 .. blk1 - 1 of tile `tile` of
// sequence b.
struct Walk {
  int b, off, item, hi;
  SeqBlocks sb;
  int tile, blk0, blk1;
  __device__ __forceinline__ Walk(const TreeArgs& a, const Share& s) : b(s.b), off(s.off), item(s.lo), hi(s.hi), tile(0), blk0(0), blk1(0) {
    if (item < hi) sb = seq_blocks(a, b, false);
  }
  __device__ __forceinline__ bool next(const TreeArgs& a) {
    const int tiles = a.Hkv / (a.hw * a.hl);
    while (item < hi) {
      while ((tile = off / sb.items) >= tiles) {
        sb = seq_blocks(a, ++b, false);
        off = 0;
      }
      const int from = off - tile * sb.items - a.lead;  // below 0: in the lead
      blk0 = max(from, 0);
      blk1 = min(sb.nb, from + hi - item);
      off += blk1 - from;
      item += blk1 - from;
      if (blk0 < blk1) return true;
    }
    return false;
  }
};

// This CTA's row group, and the first key head of tile t of its sequence.
__device__ __forceinline__ int my_rows(const TreeArgs& a) { return blockIdx.x % a.nrt; }
__device__ __forceinline__ int my_heads(const TreeArgs& a, int t) {
  return (t * a.hl + (int)(blockIdx.x / a.nrt) % a.hl) * a.hw;
}

constexpr float kTreeLog2e = 1.4426950408889634f;
constexpr float kTreeLn2 = 0.6931471805599453f;

// Partial results.
// A slot: n = hw rows maxima (of log2 e times the scaled logits), as many sums, and the outputs:
// [n][dh], or, where a thread holds a row (`a.pieces`), [dh / 4][n][4], so that a warp writes runs.
struct Part {
  float* m; float* l; float* o;
  int row, piece;  // from a row to the next, from four columns to the next
  __device__ __forceinline__ float* at(int r, int col) const { return o + r * row + (col >> 2) * piece + (col & 3); }
};
__device__ __forceinline__ Part part_of(const TreeArgs& a, int64_t cta, int which) {
  const int n = a.hw * a.rows;
  float* p = reinterpret_cast<float*>(a.part) + (cta * 2 + which) * n * (a.dh + 2);
  return a.pieces ? Part{p, p + n, p + 2 * n, 4, 4 * n} : Part{p, p + n, p + 2 * n, a.dh, 4};
}

// Where row r of a tile goes: token t, query head h.
__device__ __forceinline__ void row_of(const TreeArgs& a, int r, int m, int& t, int& h) {
  t = r / a.g;
  h = m * a.g + (r - t * a.g);
}

// Position of token t (never below the context's length), or -1 for padding.
__device__ __forceinline__ int64_t token_position(const TreeArgs& a, int b, int t, int len) {
  if (!a.positions) return (int64_t)len + t;
  const int p = a.positions[(int64_t)b * a.T + t];
  return p < 0 ? -1 : max(p, len);
}

// Of the draft's tokens 64 w .. 64 w + 63, those in token t's mask (bit k: token 64 w + k).
__device__ __forceinline__ uint64_t draft_word(const TreeArgs& a, int b, int t, int w) {
  if (a.mask) return a.mask[((int64_t)b * a.T + t) * a.words + w];
  const int past = t - 64 * w;
  return past >= 63 ? ~0ull : (past < 0 ? 0ull : (2ull << past) - 1);
}
// Of the tokens `first` + k with bit k in `word` (all of them there), those at a position above `low`.
// `at`: the sequence's positions, or null.
__device__ __forceinline__ uint64_t draft_above(const int32_t* at, int len, int first, uint64_t word, int low) {
  uint64_t left = 0;
  for (; word; word &= word - 1) {
    const int k = __ffsll((long long)word) - 1, u = first + k;
    if ((at ? max(at[u], len) : len + u) > low) left |= 1ull << k;
  }
  return left;
}

}  // namespace gca
