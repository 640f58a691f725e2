// Causal attention over packed sequences, bf16, on the 5th-generation tensor cores.
//
// With 128 rows and 128 keys a tile asks 4 * 128 * 128 * dh operations and 128 * 128 exponentials: at dh
// 64 the tensor pipe and the exponentials' pipe take about 512 cycles each, at dh 128 the tensor pipe
// takes twice as long.  Both have to work at once, so a CTA (one on an SM, persistent) holds two tiles of
// rows that take turns: while one tile's softmax runs, the other's products do.  The two tiles are two
// heads that share a key head where their number is even, else two neighbouring tiles of one head; either
// way they read the same keys.  (A last tile without a neighbour: see item_of.)
//   * one warp loads: the rows' tiles, and blocks of 128 keys of K and V in turn through a ring, from the
//     diagonal down (so a tile's first block is the one with the causal mask, which has to be weighed by
//     its maximum anyway);
//   * one warp issues the logits' products S = Q K^T, one the outputs' O += P V with P in the TMEM columns
//     that S lay in.  S goes into the next of three buffers (two at dh 128) as soon as the product of the P that
//     was there is done: with three, a softmax finds its next logits when it has stored its weights.  (One
//     warp for both, and a buffer a tile: 1.4 thousand cycles a unit of 128 x 128 at dh 64, 1.75 at dh 128; now
//     0.9 and 1.15.)
//   * four warps a tile do the softmax, a thread a row, as in tree_tc.cu: the weights are exp(s - r) by a
//     reference r that need not stay the maximum; when the sum of a row's 128 weights passes 2^14 the
//     block is weighed again by the new maximum, and the output and the sum so far are scaled to it.
//     P is rounded to bf16, the type of the product's other operand, so each weight is off by half a
//     step (2^-8 of it) at most, like the output itself; the sum is of the float32 weights.
// Blocks that a sequence's end cuts may hold anything behind it: those rows of V become zeros in shared
// memory, for a weight of 0 times what lies in them must stay 0.  dh 32 is read as 64 with zeros behind
// it (the tensor map fills them in).
// Measured, bf16, in a graph: one prompt of 32768 tokens, 16 heads of 128 and 4 key heads, 2.5 ms (1.75 PFLOP/s, the
// tensor pipe), with dh 64 1.61 ms (1.37; exponentials and products each busy for 0.57 of it, the rest waits); four documents
// of 46 thousand tokens in all, 12 heads of 64, 0.70 ms (1.27), of 32, which take as long, 0.70; 54 thousand tokens, 16 and 4
// heads, in a window of 512 176 us; 48 prompts of up to 300 tokens 26.7 us, three or four work items a CTA of some 5 thousand
// cycles each: load, masked block, store; 1024 prompts of 64 tokens, 12 heads, 230 us.
#include <algorithm>
#include <type_traits>

#include "prompt.cuh"
#include "tc.cuh"
#include "tc_rows.cuh"
#include "waits.cuh"

namespace gca {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kT = 128;           // rows of a tile, keys of a block
constexpr int kThreads = 352;     // warps 0-3: softmax of tile 0, 4-7: of tile 1, 8: logits, 9: outputs, 10: loads
constexpr int kTile = kT * 128;   // bytes of 128 rows x 64 elements
constexpr uint32_t kCols = 512;   // of TMEM: two tiles' logits, then their outputs
constexpr float kMost = 16384.f;  // the largest sum of a row's weights over a block by an outgrown reference
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
enum { kSiteFull = 1, kSiteEmpty, kSiteQ, kSiteQFree, kSiteS, kSiteP, kSiteDone, kSiteO, kSiteOFree, kSiteV, kSiteItem };

__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* abort_flag, ErrWord* err, int site, int tile, int at) {
  return __all_sync(kAll, park_or_abort(bar, parity, abort_flag, err, site, tile, at)) != 0;
}

template <int DH>
struct Tc {
  static constexpr int SUB = DH / 64;              // 64-element parts of a head
  static constexpr int BLOCK = kTile * SUB;        // a tile of Q, a block of K or of V
  static constexpr int NS = DH == 64 ? 11 : 5;     // ring slots: what shared memory holds beside two tiles of Q
  static constexpr int NBUF = DH == 64 ? 3 : 2;    // buffers of logits: what TMEM holds beside two outputs
  static constexpr int SMEM = 1024 + 2 * BLOCK + NS * BLOCK;
};

// A work item: up to two tiles of rows and the blocks of keys that they see, from hi down to lo.  Its units
// of work are (block, tile), block after block from the highest down, tile 0 before tile 1.
struct Item {
  PromptTile x;
  int head[2], tile[2];        // of each tile of rows
  int hi[2], lo[2];            // its blocks; hi < lo: there is no such tile
  int m[2];                    // their key heads
  int own;                     // 1: each tile has blocks of its own, of its key head (they see the same ones)
  int more;                    // 0: there is none any more
  __device__ __forceinline__ int top() const { return max(hi[0], hi[1]); }
  __device__ __forceinline__ int low() const { return hi[1] < lo[1] ? lo[0] : min(lo[0], lo[1]); }
  __device__ __forceinline__ bool has(int t, int n) const { return t ? n <= hi[1] && n >= lo[1] : n <= hi[0] && n >= lo[0]; }
  __device__ __forceinline__ int units() const { return max(0, hi[0] - lo[0] + 1) + max(0, hi[1] - lo[1] + 1); }
};

// Of the sequences' tiles of 128 rows those in pairs (COUNT 2), or the last one where it is alone (COUNT 1).
template <int COUNT>
struct Counts {
  const PromptTiles<kT>& tiles;
  int mine, most, total, lo, below, above;
  static __device__ __forceinline__ int of(int n) { return COUNT == 2 ? n >> 1 : n & 1; }
  __device__ __forceinline__ Counts(const PromptArgs& a, const PromptTiles<kT>& all) : tiles(all) { prompt_totals(a, *this); }
  __device__ __forceinline__ int operator()(const PromptArgs& a, int b) const { return of(tiles(a, b)); }
};
// Work item w.  Two heads that share a key head have the same tile, where their number is even.  Else an item is two
// neighbouring tiles of a head, and the last tile of a sequence that has none beside it goes with the next head's, each
// with its own keys: 48 prompts of up to 300 tokens 32 us alone, 29 together, 64 of 100 tokens 29 and 21.  (These
// come first: there may be long ones among them.)  Where there are CTAs for all of them they stay alone, for a tile by
// itself is done sooner.
__device__ __forceinline__ bool item_of(const PromptArgs& a, PromptTiles<kT>& tiles, Counts<1>& alone, Counts<2>& pairs, int w, Item& it) {
  it.own = 0;
  bool second = true;
  if (a.g % 2 == 0) {
    const int h = 2 * (w % (a.H / 2));
    if (!prompt_tile(a, tiles, w / (a.H / 2), false, it.x)) return false;
    it.head[0] = h;
    it.head[1] = h + 1;
    it.tile[0] = it.tile[1] = it.x.tile;
  } else {
    it.own = (int64_t)alone.total * a.H > gridDim.x;
    const int per = it.own ? (a.H + 1) / 2 : a.H, h = w % per;
    if (w < alone.total * per) {
      if (!prompt_tile(a, alone, w / per, false, it.x)) return false;
      it.head[0] = it.own ? 2 * h : h;
      it.head[1] = it.head[0] + 1;
      it.tile[0] = it.tile[1] = (it.x.len - 1) / kT;
      second = it.own && it.head[1] < a.H;
    } else {
      it.own = 0;
      w -= alone.total * per;
      if (!prompt_tile(a, pairs, w / a.H, false, it.x)) return false;
      it.head[0] = it.head[1] = w % a.H;
      it.tile[0] = 2 * it.x.tile;
      it.tile[1] = 2 * it.x.tile + 1;
    }
  }
  it.own = it.own && second;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.m[t] = it.head[t] / a.g;
    it.hi[t] = t == 0 || second ? it.tile[t] : -1;
    it.lo[t] = a.window ? max(0, it.tile[t] * kT - a.window + 1) / kT : 0;
  }
  return true;
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
prompt_tc_kernel(PromptArgs a, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV) {
  using C = Tc<DH>;
  constexpr int SUB = C::SUB, NS = C::NS, NBUF = C::NBUF;
  constexpr uint32_t kIdS = tc::idesc_bf16(kT, kT, false), kIdPV = tc::idesc_bf16(kT, 64, true);
  extern __shared__ unsigned char dsm[];
  unsigned char* Qs = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = Qs + 2 * C::BLOCK;
  __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_q[2], bar_qfree[2], bar_s[2][NBUF], bar_p[NBUF], bar_done[NBUF],
      bar_o[2], bar_ofree[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ uint8_t keep[PromptTiles<kT>::kKeep];
  __shared__ __align__(8) PromptItems<Item> items;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 320) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&bar_full[i], 1);
      tc::mbar_init(&bar_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&bar_q[t], 1);
      tc::mbar_init(&bar_qfree[t], 1);
      tc::mbar_init(&bar_o[t], 1);
      tc::mbar_init(&bar_ofree[t], 4);
    }
    for (int i = 0; i < NBUF; ++i) {
      tc::mbar_init(&bar_s[0][i], 1);
      tc::mbar_init(&bar_s[1][i], 1);
      tc::mbar_init(&bar_p[i], 4);
      tc::mbar_init(&bar_done[i], 1);
    }
    init_items(items, kThreads / 32 - 1);
    abort_s = 0;
    tc::fence_mbar_init();
  }
  PromptTiles<kT>::fill(a, keep);
  if (warp == 8) tc::tmem_alloc(&tmem_slot, kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  auto waited = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    if (__builtin_expect(__all_sync(kAll, tc::mbar_try(bar, parity)), 1)) return true;
    return wait_on(bar, parity, &abort_s, a.err, site, blockIdx.x, at);
  };
  // A waiting warp has to see every phase of a barrier, or its parity says nothing: so the logits' barriers are each
  // tile's own (a tile that an item lacks skips units), in turn for as many units as there are buffers.
  bool ok = true;
  Item it;
  auto take = [&](int n) { return (ok = ok && take_item(items, n, it, waited, kSiteItem)) && it.more; };

  if (warp == 10) {
    // ---------------------------------------------------------------- loads
    int id = 0, st = 0;      // slots so far, the next
    uint32_t parity = 0;     // of its filling
    int nq[2] = {0, 0};      // tiles of rows so far
    PromptTiles<kT> counts(a, keep);
    Counts<1> alone(a, counts);
    Counts<2> pairs(a, counts);
    for (int turn = 0; ok; ++turn) {
      it.more = item_of(a, counts, alone, pairs, prompt_turn(turn), it);
      ok = put_item(items, turn, it, waited, kSiteItem);
      if (!ok || !it.more) break;
      auto rows = [&](auto tile) {
        constexpr int t = decltype(tile)::value;
        if (it.hi[t] < it.lo[t]) return;
        ok = ok && waited(&bar_qfree[t], (nq[t] & 1) ^ 1, kSiteQFree, turn);
        if (!ok) return;
        tc::mbar_expect_tx_warp(&bar_q[t], C::BLOCK);
#pragma unroll
        for (int s = 0; s < SUB; ++s)
          tc::tma_load_4d_warp(Qs + t * C::BLOCK + s * kTile, &tmQ, 64 * s, a.q_hs ? it.head[t] : 0, it.x.off + it.tile[t] * kT, 0, &bar_q[t]);
        ++nq[t];
      };
      const int top = it.top(), low = it.low();
      for (int n = top; n >= low && ok; --n)
#pragma unroll 1
        for (int u = 0; u < 2 + 2 * it.own && ok; ++u) {  // K, then V; of both tiles' key heads where they have their own
          const int v = u & 1, m = u < 2 ? it.m[0] : it.m[1];
          if (n == top && u == 0) rows(std::integral_constant<int, 0>{});
          if (n == top && u == 1) rows(std::integral_constant<int, 1>{});
          ok = ok && waited(&bar_empty[st], parity ^ 1, kSiteEmpty, n);
          if (!ok) break;
          tc::mbar_expect_tx_warp(&bar_full[st], C::BLOCK);
#pragma unroll
          for (int s = 0; s < SUB; ++s)
            tc::tma_load_4d_warp(ring + st * C::BLOCK + s * kTile, v ? &tmV : &tmK, 64 * s, (v ? a.v_hs : a.k_hs) ? m : 0,
                                 it.x.off + n * kT, 0, &bar_full[st]);
          ++id;
          if (++st == NS) {
            st = 0;
            parity ^= 1;
          }
        }
    }
    if (!ok) {  // let the copies in flight land before the CTA ends
      for (int i = max(0, id - NS); i < id; ++i) tc::mbar_wait(&bar_full[i % NS], (i / NS) & 1, 1u << 16);
      for (int t = 0; t < 2; ++t)
        if (nq[t]) tc::mbar_wait(&bar_q[t], (nq[t] - 1) & 1, 1u << 16);
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- logits: S = Q K^T into the buffer of the unit
    int ks = 0, buf = 0, nq[2] = {0, 0}, own_units[2] = {0, 0};  // K's slot, the buffer; tiles and units of each tile's warps so far
    uint32_t kp = 0, bp = 1;              // the parities of K's filling, and of the buffer's last use
    const uint64_t dQ = tc::desc_km(tc::su32(Qs));
    auto blocks = [&](auto own) {
      const int low = it.low();
      for (int n = it.top(); n >= low && ok; --n) {
        auto fetched = [&]() { return ok = waited(&bar_full[ks], kp, kSiteFull, n); };
        auto read = [&]() {
          tc::commit_warp(&bar_empty[ks]);
          ks += 2;
          if (ks >= NS) {
            ks -= NS;
            kp ^= 1;
          }
        };
        if (!fetched()) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!it.has(t, n)) continue;
          if (decltype(own)::value && t == 1 && !fetched()) break;
          if (n == it.hi[t]) {
            ok = waited(&bar_q[t], nq[t] & 1, kSiteQ, n);
            ++nq[t];
          }
          ok = ok && waited(&bar_done[buf], bp, kSiteDone, n);
          if (!ok) break;
          tc::fence_after();
          const uint32_t k = tc::su32(ring + ks * C::BLOCK);
#pragma unroll
          for (int s = 0; s < SUB; ++s)
            tc::mma4_ss<tc::kKStepKm, tc::kKStepKm>(tmem + kT * buf, dQ + ((t * C::BLOCK + s * kTile) >> 4), tc::desc_km(k + s * kTile), kIdS, s ? 1u : 0u);
          tc::commit_warp(&bar_s[t][own_units[t]]);
          if (++own_units[t] == NBUF) own_units[t] = 0;
          if (n == it.lo[t]) tc::commit_warp(&bar_qfree[t]);
          if (++buf == NBUF) {
            buf = 0;
            bp ^= 1;
          }
          if (decltype(own)::value && t == 0) read();
        }
        if (!ok) break;
        read();
      }
    };
    for (int turn = 0; take(turn); ++turn) {
      if (it.own) blocks(std::true_type{});
      else blocks(std::false_type{});
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- outputs: O += P V
    int vs = 1, buf = 0, no[2] = {0, 0};
    uint32_t vp = 0, bp = 0;
    auto blocks = [&](auto own) {
      const int low = it.low();
      for (int n = it.top(); n >= low && ok; --n) {
        auto fetched = [&]() { return ok = waited(&bar_full[vs], vp, kSiteFull, n); };
        auto read = [&]() {
          tc::commit_warp(&bar_empty[vs]);
          vs += 2;
          if (vs >= NS) {
            vs -= NS;
            vp ^= 1;
          }
        };
        if (!fetched()) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!it.has(t, n)) continue;
          if (decltype(own)::value && t == 1 && !fetched()) break;
          if (n == it.hi[t]) {
            ok = waited(&bar_ofree[t], (no[t] & 1) ^ 1, kSiteOFree, n);  // read by the tile before
            ++no[t];
          }
          ok = ok && waited(&bar_p[buf], bp, kSiteP, n);
          if (!ok) break;
          tc::fence_after();
          const uint32_t v = tc::su32(ring + vs * C::BLOCK);
          const uint32_t tO = tmem + NBUF * kT + DH * t, tP = tmem + kT * buf;
#pragma unroll
          for (int s = 0; s < SUB; ++s) {
            tc::mma4_ts<8, 16, 24, tc::kKStepMn>(tO + 64 * s, tP, tc::desc_mn(v + s * kTile), kIdPV, n < it.hi[t] ? 1u : 0u);
            tc::mma4_ts<8, 16, 24, tc::kKStepMn>(tO + 64 * s, tP + 32, tc::desc_mn(v + s * kTile + kTile / 2), kIdPV, 1u);
          }
          tc::commit_warp(&bar_done[buf]);
          if (n == it.lo[t]) tc::commit_warp(&bar_o[t]);
          if (++buf == NBUF) {
            buf = 0;
            bp ^= 1;
          }
          if (decltype(own)::value && t == 0) read();
        }
        if (!ok) break;
        read();
      }
    };
    for (int turn = 0; take(turn); ++turn) {
      if (it.own) blocks(std::true_type{});
      else blocks(std::false_type{});
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 2, r = tid & 127;  // the tile, the row of it
    const float sl2 = a.scale * kLog2e;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + NBUF * kT + DH * t + lanes;
    int unit0 = 0, slot = 0, no = 0, own = 0;  // units of work and ring slots before the item, own tiles and own units so far
    for (int turn = 0; take(turn); ++turn) {
      // (Chosen, not indexed by t: the item stays in registers.)
      const int hi = t ? it.hi[1] : it.hi[0], lo = t ? it.lo[1] : it.lo[0], top = it.top();
      const int tile = t ? it.tile[1] : it.tile[0], head = t ? it.head[1] : it.head[0];
      const int pos = tile * kT + r;
      const bool on = pos < it.x.len;
      const int first = a.window ? max(0, pos - a.window + 1) : 0;  // the first key that the row sees
      const int whole = a.window ? (max(0, tile * kT + kT - a.window) + kT - 1) / kT : 0;  // blocks from here to hi - 1 are seen whole
      float mx = -CUDART_INF_F, l = 0.f;
      const uint64_t k2 = tc::f2(sl2, sl2);
      uint64_t sums[4], b2 = 0;
      auto weigh = [&](const float (&s)[32], uint32_t* p) {  // by the row's reference
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x, y;
          tc::uf2(tc::fma2(tc::f2(s[2 * i], s[2 * i + 1]), k2, b2), x, y);
          x = tc::ex2(x);
          y = tc::ex2(y);
          sums[i & 3] = tc::add2(sums[i & 3], tc::f2(x, y));
          p[i] = pack_bf16(x, y);
        }
      };
      auto total = [&]() {
        float x, y;
        tc::uf2(tc::add2(tc::add2(sums[0], sums[1]), tc::add2(sums[2], sums[3])), x, y);
        return x + y;
      };
      // A row that does not exist weighs nothing.
      auto set_base = [&]() {
        const float base = !on ? -CUDART_INF_F : mx == -CUDART_INF_F ? 0.f : -mx * sl2;
        b2 = tc::f2(base, base);
      };
      // The tile's first unit: those of the other tile's blocks before it.
      int unit = unit0 + (t ? max(0, it.hi[0] - max(hi, it.lo[0]) + 1) : max(0, it.hi[1] - max(hi + 1, it.lo[1]) + 1)), last = unit;
      for (int n = hi; n >= lo && ok; --n) {
        const int buf = unit % NBUF;
        const uint32_t tS = tmem + kT * buf + lanes;
        ok = waited(&bar_s[t][own % NBUF], (own / NBUF) & 1, kSiteS, n);
        ++own;
        if (!ok) break;
        tc::fence_after();
        // Of quarter q of the block, a bit a key that the row sees.
        auto seen = [&](int q) {
          const int lo = min(max(first - n * kT - 32 * q, 0), 32), n1 = on ? min(max(pos - n * kT + 1 - 32 * q, 0), 32) : 0;
          return lo >= n1 ? 0u : (n1 == 32 ? ~0u : (1u << n1) - 1) & ~((1u << lo) - 1);
        };
        // The block's weights by references that hold, in one straight run; false where one is outgrown.
        auto run = [&](auto edge) {
          float s0[32], s1[32];
          uint32_t p[64];
          auto hide = [&](int q, float (&s)[32]) {
            if constexpr (decltype(edge)::value) {
              const uint32_t see = seen(q);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see >> i) & 1)) s[i] = -CUDART_INF_F;
            }
          };
          sums[0] = sums[1] = sums[2] = sums[3] = 0;
          tc::ld32x32b_x32(tS, s0);
          tc::ld_wait_row(s0);
          tc::ld32x32b_x32(tS + 32, s1);  // on its way while the first quarter is weighed
          hide(0, s0);
          weigh(s0, p);
          tc::ld_wait_row(s1);
          tc::ld32x32b_x32(tS + 64, s0);
          hide(1, s1);
          weigh(s1, p + 16);
          tc::ld_wait_row(s0);
          tc::ld32x32b_x32(tS + 96, s1);
          hide(2, s0);
          weigh(s0, p + 32);
          tc::ld_wait_row(s1);
          hide(3, s1);
          weigh(s1, p + 48);
          const float sum = total();
          if (__builtin_expect(__any_sync(kAll, sum > kMost), 0)) return false;
          l += sum;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t q[8] = {p[8 * i], p[8 * i + 1], p[8 * i + 2], p[8 * i + 3], p[8 * i + 4], p[8 * i + 5], p[8 * i + 6], p[8 * i + 7]};
            tc::st32x32b_x8(tS + 8 * i, q);
          }
          return true;
        };
        bool done = false;
        if (__builtin_expect(n < hi && n >= whole, 1)) done = run(std::false_type{});
        else if (n < hi) done = run(std::true_type{});  // the window's edge
        if (__builtin_expect(!done, 0)) {
          // Some row of the warp sees keys of quarters q0 .. q1 - 1.  The maximum with this block, and the weights by it.
          const int c0 = max(first - n * kT, 0), c1 = on ? min(pos - n * kT + 1, kT) : 0;  // keys c0 .. c1 - 1 are seen
          const int q0 = min(__shfl_sync(kAll, c0, 0) / 32, 4), q1 = ((int)__reduce_max_sync(kAll, c1) + 31) / 32;
          if (n == hi && (n + 1) * kT > it.x.len) {
            // Rows of V behind the sequence become zeros (by this tile's softmax where it is the tile that
            // reaches them, or by both with the same zeros).
            const int i = slot + (2 + 2 * it.own) * (top - n) + 1 + 2 * t * it.own;
            ok = waited(&bar_full[i % NS], (i / NS) & 1, kSiteV, n);
            if (!ok) break;
            if (n * kT + r >= it.x.len)
#pragma unroll
              for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int u = 0; u < 8; ++u)
                  *reinterpret_cast<uint4*>(ring + (i % NS) * C::BLOCK + s * kTile + r * 128 + u * 16) = make_uint4(0, 0, 0, 0);
            tc::fence_async_smem();
          }
          // A quarter's logits; what the row does not see becomes -inf.
          auto logits = [&](int q, float (&s)[32]) {
            tc::ld32x32b_x32(tS + 32 * q, s);
            tc::ld_wait_row(s);
            const uint32_t see = seen(q);
            if (__all_sync(kAll, see == ~0u)) return;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((see >> i) & 1)) s[i] = -CUDART_INF_F;
          };
          float now = mx;
#pragma unroll 1
          for (int q = q0; q < q1; ++q) {
            float s[32];
            logits(q, s);
#pragma unroll
            for (int i = 0; i < 32; i += 2) now = tc::max3(now, s[i], s[i + 1]);
          }
          const float f = now == -CUDART_INF_F ? 1.f : tc::ex2((mx - now) * sl2);
          mx = now;
          l *= f;
          if (n < hi && __any_sync(kAll, f != 1.f)) {
            ok = waited(&bar_done[last % NBUF], (last / NBUF) & 1, kSiteDone, n);  // (the products are issued in order: none behind this unit's)
            if (!ok) break;
            tc::fence_after();
#pragma unroll 1
            for (int q = 0; q < DH / 32; ++q) {
              float o[32];
              tc::ld32x32b_x32(tO + 32 * q, o);
              tc::ld_wait_row(o);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(o[8 * i + e] * f);
                tc::st32x32b_x8(tO + 32 * q + 8 * i, x);
              }
            }
          }
          set_base();
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t p[16];
            if (q < q0 || q >= q1) {
#pragma unroll
              for (int i = 0; i < 16; ++i) p[i] = 0;
            } else {
              float s[32];
              logits(q, s);
              sums[0] = sums[1] = sums[2] = sums[3] = 0;
              weigh(s, p);
              l += total();
            }
            const uint32_t p0[8] = {p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]}, p1[8] = {p[8], p[9], p[10], p[11], p[12], p[13], p[14], p[15]};
            tc::st32x32b_x8(tS + 16 * q, p0);  // over logits that have been read
            tc::st32x32b_x8(tS + 16 * q + 8, p1);
          }
        }
        tc::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar_p[buf]);
        last = unit;
        unit += 1 + it.has(1 - t, t ? n - 1 : n);
      }
      unit0 += it.units();
      slot += (2 + 2 * it.own) * (top - it.low() + 1);
      const int64_t to = (int64_t)(it.x.off + pos) * a.H + head;
      if (!ok || hi < lo) continue;
      ok = waited(&bar_o[t], no & 1, kSiteO, -1);  // (of its own: a buffer's could be two units further by now)
      ++no;
      if (!ok) break;
      tc::fence_after();
      const float inv = 1.f / l;
      uint4* rows = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.o) + ((int64_t)it.x.off * a.H + head) * a.dh);
#pragma unroll
      for (int half = 0; half < DH / 64; ++half) {
        uint4 x[8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float o[32];
          tc::ld32x32b_x32(tO + 64 * half + 32 * q, o);
          tc::ld_wait_row(o);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[4 * q + i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                      pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        }
        tc::store_rows(x, rows + 8 * half, (int64_t)a.H * (a.dh / 8), pos, it.x.len, a.dh / 8);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar_ofree[t]);
      if (on) a.lse[to] = mx * a.scale + logf(l);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::tmem_dealloc(tmem_slot, kCols);
  }
}

template <int DH>
cudaError_t run_tc(const PromptArgs& a, cudaStream_t s) {
  using C = Tc<DH>;
  CUtensorMap q, k, v;
  cudaError_t e = make_packed_tmap(&q, a.q, a.dh, a.H, a.N, a.q_hs, a.q_ts);
  if (e == cudaSuccess) e = make_packed_tmap(&k, a.k, a.dh, a.Hkv, a.N, a.k_hs, a.k_ts);
  if (e == cudaSuccess) e = make_packed_tmap(&v, a.v, a.dh, a.Hkv, a.N, a.v_hs, a.v_ts);
  if (e == cudaSuccess) e = allow_smem((const void*)prompt_tc_kernel<DH>, C::SMEM);
  if (e != cudaSuccess) return e;
  // Items: whole tiles of rows, and at most one that is not whole a sequence.
  const int rows = a.g % 2 == 0 ? kT : 2 * kT;
  const int64_t items = (a.N / rows + std::min<int64_t>(a.B, a.N)) * (a.g % 2 == 0 ? a.H / 2 : a.H);
  launch_begin("prompt_tc", s);
  prompt_tc_kernel<DH><<<(unsigned)std::min<int64_t>(items, kSMs), kThreads, C::SMEM, s>>>(a, q, k, v);
  return launch_end("prompt_tc", s);
}

}  // namespace

cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t s) { return a.dh <= 64 ? run_tc<64>(a, s) : run_tc<128>(a, s); }

}  // namespace gca
