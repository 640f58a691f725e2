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

// What every search needs of the counts of tiles (PromptTiles, or what is made of them): made once, by each warp that
// searches.
template <typename Tiles>
__device__ __forceinline__ void prompt_totals(const PromptArgs& a, Tiles& tiles) {
  const int lane = threadIdx.x & 31;
  int n = tiles(a, lane), most = n, total = n;
  tiles.mine = n;
  for (int b = lane + 32; b < a.B; b += 32) {
    n = tiles(a, b);
    most = max(most, n);
    total += n;
  }
  tiles.most = (int)__reduce_max_sync(0xffffffffu, most);
  tiles.total = (int)__reduce_add_sync(0xffffffffu, total);
  tiles.lo = tiles.below = tiles.above = 0;
}

// Tiles of T rows of the sequences, for many lookups: in shared memory, a byte each (kMore: as many or more, to be
// looked up), and a lane's own of the first 32 in a register.  All threads of the CTA make it, with a barrier between `fill`
// and the first use.
// With 256 of them kept, and sums over all sequences made for each work item, the time of many short prompts grew with the
// square of their number: 1024 of 64 tokens, 12 heads of 64, forward 847 us and gradients 2016, now 230 and 753; 256 67 and
// 191, now 50 to 53 and 170; 48 of up to 300 27.8 and 72.9, now 26.7 and 70.  (All counts in the lanes' registers, searched
// in unrolled code: 190 and 668 for the 1024, but one prompt's gradients 14.8 us for 13.8 and windows 2 % slower.)
template <int T>
struct PromptTiles {
  static constexpr int kKeep = GCA_MAX_SEQUENCES, kMore = 255;
  const uint8_t* kept;
  int mine, most, total;  // the lane's of the first 32 sequences; the most of a sequence, of all together
  int lo, below, above;   // of the last search: the tile's number i, S(i + 1) and S(i)
  static __device__ __forceinline__ int of(const PromptArgs& a, int b) { return b < a.B ? (prompt_length(a, b) + T - 1) / T : 0; }
  static __device__ __forceinline__ void fill(const PromptArgs& a, uint8_t* keep) {
    for (int b = threadIdx.x; b < max(a.B, 32); b += blockDim.x) keep[b] = (uint8_t)min(of(a, b), kMore);
  }
  __device__ __forceinline__ PromptTiles(const PromptArgs& a, const uint8_t* keep) : kept(keep) { prompt_totals(a, *this); }
  __device__ __forceinline__ int operator()(const PromptArgs& a, int b) const {
    const int n = kept[b];
    return n < kMore ? n : of(a, b);
  }
};

// Tile number `rank` of the call: tiles of T rows in the order of their work, the most first, so that
// those that start last are short.  Under the causal mask that is the order of their number in their
// sequence, from the highest down (`back`: counted from the sequence's end, for the side of the keys),
// sequences of equal tiles in order.  With S(i) the tiles numbered i or higher, tile `rank` has the number
// i with S(i + 1) <= rank < S(i).  Called by a whole warp, with ranks that do not fall, so that most have the number of
// the last; false behind the last tile.
template <typename Tiles>
__device__ __forceinline__ bool prompt_tile(const PromptArgs& a, Tiles& tiles, int rank, bool back, PromptTile& x) {
  const int lane = threadIdx.x & 31;
  const int mine = tiles.mine;  // the first 32 sequences stay in registers
  auto from = [&](int i) {
    int n = max(mine - i, 0);
    for (int b = lane + 32; b < a.B; b += 32) n += max(tiles(a, b) - i, 0);
    return (int)__reduce_add_sync(0xffffffffu, n);
  };
  if (tiles.total <= rank) return false;
  if (rank >= tiles.above) {
    int lo = 0, hi = tiles.most, below = 0, above = tiles.total;  // above = from(lo) > rank >= from(hi) = below
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, n = from(mid);
      if (n > rank) {
        lo = mid;
        above = n;
      } else {
        hi = mid;
        below = n;
      }
    }
    tiles.lo = lo;
    tiles.below = below;
    tiles.above = above;
  }
  const int lo = tiles.lo;
  int left = rank - tiles.below;  // of the sequences with more than `lo` tiles, in order
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int n = b0 ? (b0 + lane < a.B ? tiles(a, b0 + lane) : 0) : mine;
    const uint32_t those = __ballot_sync(0xffffffffu, n > lo);
    if (left < __popc(those)) {
      // The lane of the bit that `left` others lie below.
      const bool it = n > lo && __popc(those & ((1u << lane) - 1)) == left;
      const int at = __ffs(__ballot_sync(0xffffffffu, it)) - 1;
      if (at < 0) return false;  // (offsets out of order can make more tiles than an int counts)
      x.b = b0 + at;
      x.tile = back ? __shfl_sync(0xffffffffu, n, at) - 1 - lo : lo;
      x.off = a.offsets[x.b];
      x.len = a.offsets[x.b + 1] - x.off;
      return true;
    }
    left -= __popc(those);
  }
  return false;
}

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
