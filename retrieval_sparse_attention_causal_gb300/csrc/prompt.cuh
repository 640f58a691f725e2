// Packed sequences and their tiles: what the kernels of the attention over prompts share.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace gca {

// A tile of a packed sequence: rows first .. first + T - 1 of the sequence that starts at row `off` and
// has `len` rows.
struct PromptTile {
  int b, tile, off, len;
};

// Rows of sequence b; one whose offsets are out of order or out of the tensor counts as empty (flagged).
__device__ __forceinline__ int prompt_length(const PromptArgs& a, int b) {
  const int s = a.offsets[b], e = a.offsets[b + 1];
  if (s < 0 || e < s || e > a.N) {
    if (blockIdx.x == 0) flag_bad_index(a.err, s < 0 || s > a.N ? s : e);
    return 0;
  }
  return e - s;
}

// Tiles of T rows of the sequences, for many lookups by a warp: lane l has those of sequences l, l + 32 and so on in
// registers.  (Read anew from the offsets for each work item, beyond the first 256 sequences, they took time that grew with
// the square of the sequences: 1024 prompts of 64 tokens, 12 heads, forward 864 us and gradients 2020, now 192 and 672; 256 67
// and 197, now 56 and 185.)  It is made before the CTA's first barrier, beside what the other warps prepare: a
// prompt's gradients take 2 us longer otherwise.
template <int T>
struct PromptTiles {
  static constexpr int kEach = GCA_MAX_SEQUENCES / 32;
  int n[kEach];
  __device__ __forceinline__ PromptTiles() {}  // (of the warps that find no items)
  __device__ __forceinline__ explicit PromptTiles(const PromptArgs& a) {
#pragma unroll
    for (int j = 0; j < kEach; ++j) n[j] = 0;
    any(a, [&](int j) {
      const int b = 32 * j + (threadIdx.x & 31);
      if (b < a.B) n[j] = (prompt_length(a, b) + T - 1) / T;
      return false;
    });
  }
  // Whether f(j) holds for one of the n's that hold sequences, asked in order up to the first; few sequences ask few.
  template <typename F>
  static __device__ __forceinline__ bool any(const PromptArgs& a, const F& f) {
    if (f(0)) return true;
    if (a.B <= 32) return false;
#pragma unroll
    for (int j = 1; j < 4; ++j)
      if (f(j)) return true;
    if (a.B <= 128) return false;
#pragma unroll
    for (int j = 4; j < kEach; ++j)
      if (f(j)) return true;
    return false;
  }
};

// Tile number `rank` of the call: tiles of T rows in the order of their work, the most first, so that
// those that start last are short.  Under the causal mask that is the order of their number in their
// sequence, from the highest down (`back`: counted from the sequence's end, for the side of the keys),
// sequences of equal tiles in order.  With S(i) the tiles numbered i or higher, tile `rank` has the number
// i with S(i + 1) <= rank < S(i).  `of` says how many of a sequence's tiles count.  Called by a whole warp; false
// behind the last tile.
template <int T, typename Of>
__device__ __forceinline__ bool prompt_tile(const PromptArgs& a, const PromptTiles<T>& tiles, const Of& of, int rank, bool back, PromptTile& x) {
  const int lane = threadIdx.x & 31;
  auto from = [&](int i) {
    int n = 0;
    tiles.any(a, [&](int j) {
      n += max(of(tiles.n[j]) - i, 0);
      return false;
    });
    return (int)__reduce_add_sync(0xffffffffu, n);
  };
  int most = 0;
  tiles.any(a, [&](int j) {
    most = max(most, of(tiles.n[j]));
    return false;
  });
  int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, most), below = 0;  // from(lo) > rank >= from(hi) = below
  if (from(0) <= rank) return false;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, n = from(mid);
    if (n > rank) {
      lo = mid;
    } else {
      hi = mid;
      below = n;
    }
  }
  int left = rank - below;  // of the sequences with more than `lo` tiles, in order
  int first = 0, count = 0;
  uint32_t those = 0;
  const bool found = tiles.any(a, [&](int j) {
    first = 32 * j;
    count = of(tiles.n[j]);
    those = __ballot_sync(0xffffffffu, count > lo);
    if (left < __popc(those)) return true;
    left -= __popc(those);
    return false;
  });
  // The lane of the bit that `left` others lie below.
  const bool it = found && count > lo && __popc(those & ((1u << lane) - 1)) == left;
  const int at = __ffs(__ballot_sync(0xffffffffu, it)) - 1;
  if (at < 0) return false;  // (offsets out of order can make more tiles than an int counts)
  x.b = first + at;
  x.tile = back ? __shfl_sync(0xffffffffu, count, at) - 1 - lo : lo;
  x.off = a.offsets[x.b];
  x.len = a.offsets[x.b + 1] - x.off;
  return true;
}
__device__ __forceinline__ int all_tiles(int n) { return n; }

// The work item of a persistent CTA's turn n: every other turn the CTAs take theirs in the opposite order, so that
// the same ones do not always get the larger (in order, 1024 items over 152 CTAs left a CTA 13 % over the mean).
__device__ __forceinline__ int prompt_turn(int n) {
  return n * gridDim.x + (n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Work items on their way from the warp that finds them to those that work on them.  Each warp finding its own took
// two to three thousand cycles an item, most of it the way of code that is rarely run to the warp.
template <typename I>
struct PromptItems {
  static constexpr int kSlots = 4;
  uint64_t full[kSlots], empty[kSlots];
  I item[kSlots];
};
template <typename I>
__device__ __forceinline__ void init_items(PromptItems<I>& r, int readers) {  // one thread
  for (int i = 0; i < r.kSlots; ++i) {
    tc::mbar_init(&r.full[i], 1);
    tc::mbar_init(&r.empty[i], readers);
  }
}
// Item n, by a whole warp; `waited` as in the kernels.  False where a wait gave up.
template <typename I, typename W>
__device__ __forceinline__ bool put_item(PromptItems<I>& r, int n, const I& it, const W& waited, int site) {
  const int s = n % r.kSlots;
  if (!waited(&r.empty[s], ((n / r.kSlots) & 1) ^ 1, site, n)) return false;
  if ((threadIdx.x & 31) == 0) {
    r.item[s] = it;
    tc::mbar_arrive(&r.full[s]);
  }
  __syncwarp();
  return true;
}
template <typename I, typename W>
__device__ __forceinline__ bool take_item(PromptItems<I>& r, int n, I& it, const W& waited, int site) {
  const int s = n % r.kSlots;
  if (!waited(&r.full[s], (n / r.kSlots) & 1, site, n)) return false;
  it = r.item[s];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&r.empty[s]);
  return true;
}

// The backward pass's scratch rows, two sums of each row of a head: row off + t of a sequence that starts at `off` is
// number prompt_sums(a, off, h) + t.  There is a set for sequences that start at even rows and one for odd rows, in
// which a row has its own number, less one in the odd set.  So rows that differ never share a number, in whatever order
// the offsets are, and a sequence starts at an even one: what is read two rows at a time is aligned, and a copy of 16-byte
// units (kSumsOfTile rows for a tile) starts off & 2 rows before it.
__device__ __forceinline__ int64_t prompt_sums(const PromptArgs& a, int off, int h) {
  return ((off & 1) * (int64_t)a.H + h) * a.np + (off & ~1);
}
constexpr int kSumsOfTile = 128 + 4;

}  // namespace gca
