// Attention of drafted tokens over a paged cache where there is much to read, bf16, dh 64 or
// 128, on the 5th-generation tensor cores.
//
// With 128 rows a byte of K or V asks 128 operations: still below the balance of memory and
// tensor pipes (about 290), so the aim is a stream of pages that never waits.  One CTA walks
// its share of the blocks for 128 rows (padded) of one key head; two CTAs share an SM.
//   * one warp loads: page numbers of 32 blocks at a time (and the next 32 on their way), and TMA
//     tiles of 64 x 64 into a ring of 16 KB slots, K and V in turn (two tiles a barrier: waiting
//     for one and announcing a load take about 200 cycles, which at 8 KB a slot held a CTA to 14
//     bytes a cycle, less than its share of DRAM).  Ring and Q take all of an SM's shared memory:
//     a slot more was 3 % at dh 64, 7 % at dh 128.
//   * one warp issues the products: S(n) = Q K(n)^T into one of two TMEM buffers; O += P(n) V(n)
//     with P in the buffer that S(n) lay in; behind that S(n + 2), which takes the buffer over, so
//     that the softmax always has a block to go on with.
//     Barriers of blocks (S ready, P ready, O done) come in pairs, one for even and one for odd
//     blocks: S(n) is issued before P V (n - 1), so a thread that has seen S(n) knows that
//     P V (n - 2) is done, not that P V (n - 1) is, and one barrier's parity would not tell.
//   * four warps do the softmax: a thread owns a row.  The weights are exp(s - r) with a reference r
//     that is the row's maximum when it is taken.  It need not stay that: a larger logit only
//     makes larger weights, and bf16 and float32 round relative to the value.  So a block's
//     maximum is not computed; when the sum of a row's 64 weights passes 2^14, the block is
//     weighed again by the new maximum, and the output and the sum so far are scaled to it.
//     P is rounded to bf16, the type of the product's other operand, so each weight is off by half a
//     step (2^-8 of it) at most, like the output itself; the sum is of the float32 weights.
// The last page, the window's edge and the draft's own block are masked by a 64-bit word a
// row; there the rows of V that nobody sees are set to zeros in shared memory, for a weight
// of 0 times what lies in them must stay 0.
//
// What costs beside the memory is the way of the code to the warps: six warps of three kinds
// share the instruction caches, and a CTA walks a few blocks to a few hundred.  So blocks that
// are seen whole run through one straight loop, everything else is rolled up and there once,
// and a wait whose first probe fails goes on in a function of its own.  Against code that was
// inlined and unrolled throughout: 2 x 256K tokens, 64 drafted, 16 query and 4 key heads of 64,
// 200 -> 131 us (1074 MB from L2, half of that from DRAM; issue slots 53 %, tensor pipe 44 %, the
// exponentials' pipe 44 %, DRAM 52 %: none alone bounds it); 64 of 12 heads over 2 x 128K, 137
// -> 129 us (6.2 TB/s); 16 sequences of trees in a window of 512, 22.5 -> 18.9 us, and 13.0 with
// whole tiles and no join (a launch, the chain of a first block: lengths, page numbers, tiles,
// products, about 6 us, and 0.5 a block).
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"
#include "tc_rows.cuh"
#include "tree_sched.cuh"
#include "waits.cuh"

namespace gca {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 192;
constexpr int kCtas = 2;         // on an SM
constexpr int kCols = 256;       // of TMEM: two buffers of logits, the output behind them
constexpr int kRows = 128;       // the lanes of TMEM
constexpr int kTile = 8192;      // 64 tokens x 64 elements
constexpr int kSlot = 2 * kTile;
constexpr float kMost = 16384.f;  // the largest sum of a row's weights over a block by an outgrown reference
constexpr uint32_t kAll = 0xffffffffu;
enum { kSiteFull = 1, kSiteEmpty, kSiteQ, kSiteS, kSiteP, kSiteO, kSiteV, kSiteRing };

// The rest of a wait that its first probe did not end: off the straight path, and one copy of it.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* abort_flag, ErrWord* err, int site, int tile, int at) {
  return __all_sync(kAll, wait_or_abort(bar, parity, abort_flag, err, site, tile, at)) != 0;
}

// Masks of a draft whose windows end inside it: of the tokens `first` + k with bit k in `there`, those that
// tokens x0, x0 + step, .. below x1 see.  Off the straight path too.
__device__ __noinline__ uint64_t seen_in_windows(const uint64_t* mask, int words, const int32_t* where, int len, int window, int first,
                                                 uint64_t there, int x0, int x1, int step) {
  uint64_t seen = 0;
  for (int x = x0; x < x1; x += step) {
    const int p = where ? (where[x] < 0 ? -1 : max(where[x], len)) : len + x;
    if (p < 0) continue;
    const uint64_t d = there & (mask ? mask[x * words + first / kChunk] : (x - first >= 63 ? ~0ull : (x < first ? 0ull : (2ull << (x - first)) - 1)));
    seen |= draft_above(where, len, first, d, p - window);
  }
  return seen;
}

template <int DH>
struct Tc {
  static constexpr int SUB = DH / 64;               // 64-element parts of a head
  static constexpr int PB = 2 / SUB;                // blocks of 64 keys of a ring slot: 16 KB of K or of V
  static constexpr int QB = 2 * kTile * SUB;        // a row tile of Q
  static constexpr int NS = DH == 64 ? 6 : 5;       // ring slots: with 1 KB of barriers and 1 KB of the system's, half of an SM's 228 KB
  static constexpr int SMEM = QB + NS * kSlot;
};

template <int DH>
__global__ void __launch_bounds__(kThreads, kCtas)
tree_tc_kernel(TreeArgs a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmKn, const __grid_constant__ CUtensorMap tmVn) {
  using C = Tc<DH>;
  constexpr int SUB = C::SUB, NS = C::NS, PB = C::PB;
  constexpr uint32_t kIdS = tc::idesc_bf16(kRows, 64, false), kIdPV = tc::idesc_bf16(kRows, 64, true);
  extern __shared__ __align__(1024) unsigned char dsm[];
  unsigned char* Qs = dsm;
  unsigned char* ring = Qs + C::QB;
  __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_q, bar_s[2], bar_p[2], bar_o[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next();
  if (tc::su32(dsm) & 1023) {  // the tiles' swizzle counts on it
    if (tid == 0) flag_timeout(a.err, kSiteRing, blockIdx.x, 0, 0);
    return;
  }
  if (tid == 160) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmKn);
    prefetch_tmap(&tmVn);
  }
  const Share sh = my_share(a);
  if (sh.lo >= sh.hi) return;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&bar_full[i], 1);
      tc::mbar_init(&bar_empty[i], 1);
    }
    tc::mbar_init(&bar_q, 4);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bar_s[i], 1);
      tc::mbar_init(&bar_p[i], 4);
      tc::mbar_init(&bar_o[i], 1);
    }
    abort_s = 0;
    tc::fence_mbar_init();
  }
  if (warp == 4) tc::tmem_alloc(&tmem_slot, kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  const int rt = my_rows(a);

  // The segments of this CTA, walked by every role.
  Walk at(a, sh);
  const SeqBlocks& sb = at.sb;
  const int &b = at.b, &tile = at.tile, &blk0 = at.blk0, &blk1 = at.blk1;
  // Waits of a warp: it goes on or gives up as a whole.
  auto waited = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    if (__builtin_expect(__all_sync(kAll, tc::mbar_try(bar, parity)), 1)) return true;
    return wait_on(bar, parity, &abort_s, a.err, site, tile, at);
  };
  bool ok = true;

  if (warp == 5) {
    // ---------------------------------------------------------------- loads
    int id = 0, st = 0;     // slots so far, the next
    uint32_t parity = 0;    // of its filling
    while (ok && at.next(a)) {
      const int m = my_heads(a, tile), n = blk1 - blk0;
      // 32 page numbers at a time, one a lane, and the next 32; behind the pool, which reads zeros,
      // where there is no page.
      int pages = 0, next = 0;
      auto pages_at = [&](int blk) {
        int page = -1;
        if (blk + lane < sb.np) page = a.table[(int64_t)b * a.width + sb.p0 + blk + lane];
        if (page >= 0 && page < a.pages) return page;
        if (page != -1) flag_bad_index(a.err, page);
        return (int)a.pages;
      };
      for (int x = 0; x < n && ok; x += PB) {
        if (x % 32 == 0) {
          pages = x == 0 ? pages_at(blk0) : next;
          if (x + 32 < n) next = pages_at(blk0 + x + 32);
        }
        int page[PB];
#pragma unroll
        for (int i = 0; i < PB; ++i) page[i] = __shfl_sync(kAll, pages, (x + i) % 32);
        const int count = min(PB, n - x);
        const bool full = x + PB <= min(n, sb.np - blk0);  // blocks of the context
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {  // K, then V
          ok = ok && waited(&bar_empty[st], parity ^ 1, kSiteEmpty, x);
          if (!ok) break;
          unsigned char* to = ring + st * kSlot;
          uint64_t* bar = &bar_full[st];
          if (__builtin_expect(full, 1)) {
            tc::mbar_expect_tx_warp(bar, kSlot);
#pragma unroll
            for (int i = 0; i < PB; ++i)
#pragma unroll
              for (int s = 0; s < SUB; ++s)
                tc::tma_load_4d_warp(to + (i * SUB + s) * kTile, v ? &tmV : &tmK, 64 * s, m, 0, page[i], bar);
          } else {
            tc::mbar_expect_tx_warp(bar, count * SUB * kTile);
#pragma unroll
            for (int i = 0; i < PB; ++i) {
              if (i >= count) break;
              const int blk = blk0 + x + i;
#pragma unroll
              for (int s = 0; s < SUB; ++s, to += kTile) {
                if (blk < sb.np) {
                  tc::tma_load_4d_warp(to, v ? &tmV : &tmK, 64 * s, m, 0, page[i], bar);
                } else {  // the draft's (an axis of stride 0 has one entry in the map)
                  const int64_t hs = v ? a.vn_hs : a.kn_hs, ts = v ? a.vn_ts : a.kn_ts, bs = v ? a.vn_bs : a.kn_bs;
                  tc::tma_load_4d_warp(to, v ? &tmVn : &tmKn, 64 * s, hs ? m : 0, ts ? (blk - sb.np) * kChunk : 0, bs ? b : 0, bar);
                }
              }
            }
          }
          ++id;
          if (++st == NS) {
            st = 0;
            parity ^= 1;
          }
        }
      }
    }
    if (!ok)  // let the copies in flight land before the CTA ends
      for (int i = max(0, id - NS); i < id; ++i) tc::mbar_wait(&bar_full[i % NS], (i / NS) & 1, 1u << 16);
  } else if (warp == 4) {
    // ---------------------------------------------------------------- products
    int seg = 0, nth = 0;  // segments and blocks so far
    int ks = 0, vs = 1;    // the slots that K and V come from, and the parities they are filled at
    uint32_t kp = 0, vp = 0;
    auto pass = [](int& slot, uint32_t& parity) {
      slot += 2;
      if (slot >= NS) {
        slot -= NS;
        parity ^= 1;
      }
    };
    const uint64_t dQ = tc::desc_km(tc::su32(Qs));
    while (ok && at.next(a)) {
      const int n = blk1 - blk0;
      ok = waited(&bar_q, seg & 1, kSiteQ, seg);
      ++seg;
      // Step x: P V of block x, and the logits of block x + 2 in the buffer that P lay in.
      for (int x0 = -2; x0 < n && ok; x0 += PB) {
#pragma unroll
        for (int i = 0; i < PB; ++i) {
          const int x = x0 + i, j = nth + x;
          if (x >= n) break;
          if (x >= 0) {
            if (i == 0) ok = waited(&bar_full[vs], vp, kSiteFull, x);
            ok = ok && waited(&bar_p[j & 1], (j >> 1) & 1, kSiteP, x);
            if (!ok) break;
            const uint32_t v = tc::su32(ring + vs * kSlot + i * kTile);
            tc::fence_after();
#pragma unroll
            for (int s = 0; s < SUB; ++s)
              tc::mma4_ts<8, 16, 24, tc::kKStepMn>(tmem + 64 * (2 + s), tmem + 64 * (j & 1), tc::desc_mn(v + s * kTile), kIdPV,
                                                   x > 0 ? 1u : 0u);
            tc::commit_warp(&bar_o[j & 1]);
            if (i == PB - 1 || x == n - 1) {
              tc::commit_warp(&bar_empty[vs]);
              pass(vs, vp);
            }
          }
          if (x + 2 < n) {
            if (i == 0) ok = waited(&bar_full[ks], kp, kSiteFull, x + 2);
            if (!ok) break;
            const uint32_t k = tc::su32(ring + ks * kSlot + i * kTile);
            tc::fence_after();
#pragma unroll
            for (int s = 0; s < SUB; ++s)
              tc::mma4_ss<tc::kKStepKm, tc::kKStepKm>(tmem + 64 * (j & 1), dQ + s * (2 * kTile >> 4), tc::desc_km(k + s * kTile),
                                                      kIdS, s ? 1u : 0u);
            tc::commit_warp(&bar_s[j & 1]);
            if (i == PB - 1 || x + 2 == n - 1) {
              tc::commit_warp(&bar_empty[ks]);
              pass(ks, kp);
            }
          }
        }
      }
      nth += n;
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const float sl2 = a.scale * kTreeLog2e;
    const int R = a.T * a.g;
    const uint32_t tS = tmem + ((uint32_t)(32 * warp) << 16), tO = tS + 128;
    int nth = 0, id = 0;  // blocks and ring slots so far
    int slot = 0;
    while (ok && at.next(a)) {
      const int m = my_heads(a, tile), r = rt * kRows + tid, n = blk1 - blk0;
      const bool on = r < R, idle = rt * kRows + 32 * warp >= R;
      int t = 0, h = 0, pos = -1;
      // What the segment asks of memory, all of it before the first use: Q, the row's position, the
      // page numbers, and of the draft's first block the mask and the positions.
      auto page_at = [&](int blk) { return a.table[(int64_t)b * a.width + sb.p0 + blk]; };
      const int32_t* where = a.positions ? a.positions + (int64_t)b * a.T : nullptr;
      if (on) row_of(a, r, m, t, h);
      uint4 w[DH / 8];
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.q) + b * a.q_bs + t * a.q_ts + h * a.q_hs);
#pragma unroll
      for (int u = 0; u < DH / 8; ++u) w[u] = on ? src[u] : make_uint4(0, 0, 0, 0);
      if (on) pos = (int)token_position(a, b, t, sb.len);
      const int held = min(blk1, sb.np);
      int page = blk0 + lane < held ? page_at(blk0 + lane) : 0;
      const bool draft = blk1 > sb.np;
      const int x0 = rt * kRows / a.g + lane, x1 = min(a.T, ((rt + 1) * kRows - 1) / a.g + 1);  // tokens of the CTA's rows
      // The lowest and the highest position of the CTA's rows.
      int near = where ? INT32_MAX : sb.len + rt * kRows / a.g, most = where ? -1 : sb.len + x1 - 1;
      uint64_t own = 0, any = 0;  // of the first draft block: this row's mask, all rows' masks
      int real0 = 0, real1 = 0;   // positions of its tokens
      if (draft && on) own = draft_word(a, b, t, 0);
      if (draft || (where && a.window > 0))
        for (int x = x0; x < x1; x += 32) {
          const int p = where ? where[x] : 0;
          const uint64_t d = draft ? draft_word(a, b, x, 0) : 0;
          any |= p >= 0 ? d : 0;
          if (where && p >= 0) {
            near = min(near, p);
            most = max(most, p);
          }
        }
      if (draft && where) {
        real0 = where[min(lane, a.T - 1)];
        real1 = where[min(32 + lane, a.T - 1)];
      }
#pragma unroll
      for (int u = 0; u < DH / 8; ++u) *reinterpret_cast<uint4*>(Qs + (u / 8) * 2 * kTile + swz<128>(tid, u % 8)) = w[u];
      tc::fence_async_smem();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar_q);
      float mx = -CUDART_INF_F, l = 0.f;
      int far = __reduce_max_sync(kAll, pos);
      bool passes = false;  // a window ends inside the draft
      if (a.window > 0) {
        near = __reduce_min_sync(kAll, near);
        near = near == INT32_MAX ? sb.len : max(near, sb.len);  // (where all rows are padding, what they see is of no account)
        far = max(far, near);
        passes = (int)__reduce_max_sync(kAll, most) - a.window >= sb.len;
      }
      // Blocks in0 .. in1 - 1 are seen whole by every row of this warp, unless there are holes.
      const int in0 = a.window > 0 && far >= a.window ? (far - a.window) / kChunk + 1 - sb.p0 : 0, in1 = sb.len / kChunk - sb.p0;
      bool hole = page < 0 || page >= a.pages;  // a page that is not held
      for (int blk = blk0 + 32 + lane; blk < held; blk += 32) {
        page = page_at(blk);
        hole = hole || page < 0 || page >= a.pages;
      }
      const bool holes = __any_sync(kAll, hole);
      bool settled = false;  // every row that sees something has a reference
      const int run1 = holes || idle ? blk0 : min(in1, blk1);
      uint64_t sums[4], b2 = 0;
      const uint64_t k2 = tc::f2(sl2, sl2);
      auto weigh = [&](const float (&s)[32], uint32_t (&p)[2][8]) {  // by the row's reference
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x, y;
          tc::uf2(tc::fma2(tc::f2(s[2 * i], s[2 * i + 1]), k2, b2), x, y);
          x = tc::ex2(x);
          y = tc::ex2(y);
          sums[i & 3] = tc::add2(sums[i & 3], tc::f2(x, y));
          p[i / 8][i % 8] = pack_bf16(x, y);
        }
      };
      auto total = [&]() {
        float x, y;
        tc::uf2(tc::add2(tc::add2(sums[0], sums[1]), tc::add2(sums[2], sums[3])), x, y);
        return x + y;
      };
      auto set_base = [&]() {
        const float base = mx == -CUDART_INF_F ? 0.f : -mx * sl2;
        b2 = tc::f2(base, base);
      };
      for (int blk = blk0; blk < blk1 && ok; ++blk, ++nth) {
        // Blocks that are seen whole, by references that hold: one straight run of instructions.  (Each branch
        // that was taken cost a warp 50 to 200 cycles; a block's arithmetic takes 700.)
        if (settled && blk >= in0 && blk < run1) {
          set_base();
          uint32_t there = 0;  // the block's logits were seen to be complete
          for (;;) {
            if (__builtin_expect(!__all_sync(kAll, there), 0)) {
              ok = waited(&bar_s[nth & 1], (nth >> 1) & 1, kSiteS, blk);
              if (!ok) break;
            }
            tc::fence_after();
            const uint32_t tP = tS + 64 * (nth & 1);
            float s0[32], s1[32];
            tc::ld32x32b_x32(tP, s0);
            tc::ld_wait_row(s0);
            tc::ld32x32b_x32(tP + 32, s1);  // on its way while the first half is weighed
            uint32_t p0[2][8], p1[2][8];
            sums[0] = sums[1] = sums[2] = sums[3] = 0;
            weigh(s0, p0);
            tc::ld_wait_row(s1);
            weigh(s1, p1);
            const float sum = total();
            if (__builtin_expect(__any_sync(kAll, sum > kMost), 0)) break;  // weighed again below
            l += sum;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              tc::st32x32b_x8(tP + 8 * i, p0[i]);
              tc::st32x32b_x8(tP + 16 + 8 * i, p1[i]);
            }
            there = tc::mbar_test(&bar_s[(nth + 1) & 1], ((nth + 1) >> 1) & 1);  // used at the next block
            tc::st_wait();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar_p[nth & 1]);
            ++nth;
            if (++blk >= run1) break;
          }
          if (!ok || blk >= blk1) break;
        }
        const bool inner = blk >= in0 && blk < in1 && !holes;
        uint64_t see = ~0ull;  // keys that this row sees
        uint64_t used = 0;     // where `blank`: keys that some row of the CTA sees
        bool blank = false;
        if (__builtin_expect(!inner, 0)) {
          const bool ctx = blk < sb.np;
          const int j0 = ctx ? (sb.p0 + blk) * kChunk : (blk - sb.np) * kChunk;
          // Keys lo .. hi - 1 of the block exist.
          int lo = 0, hi = min(kChunk, (ctx ? sb.len : a.T) - j0);
          if (ctx && a.window > 0) lo = min(max(near - a.window + 1 - j0, 0), kChunk);
          if (ctx && holes) {
            const int page = page_at(blk);
            if (page < 0 || page >= a.pages) hi = 0;
          }
          int c0 = lo;
          if (ctx && a.window > 0) c0 = max(c0, pos - a.window + 1 - j0);
          c0 = min(c0, kChunk);
          see = c0 >= hi ? 0ull : ((hi == 64 ? ~0ull : (1ull << hi) - 1) & ~((c0 == 64 ? 0ull : 1ull << c0) - 1));
          if (c0 == 64) see = 0;
          uint64_t seen = 0;  // by some row of the CTA
          if (!ctx) {
            uint64_t real = ~0ull;  // tokens that are not padding
            if (j0 > 0) {
              own = on ? draft_word(a, b, t, j0 / kChunk) : 0;
              any = 0;
              for (int x = x0; x < x1; x += 32)
                if (!where || where[x] >= 0) any |= draft_word(a, b, x, j0 / kChunk);
              if (where) {
                real0 = where[min(j0 + lane, a.T - 1)];
                real1 = where[min(j0 + 32 + lane, a.T - 1)];
              }
            }
            if (where) real = ((uint64_t)__ballot_sync(kAll, real1 >= 0) << 32) | __ballot_sync(kAll, real0 >= 0);
            real &= see;
            uint64_t word = pos >= 0 ? own & real : 0;
            if (__builtin_expect(passes, 0)) {
              const uint64_t* mask = a.mask ? a.mask + (int64_t)b * a.T * a.words : nullptr;
              any = seen_in_windows(mask, a.words, where, sb.len, a.window, j0, real, x0, x1, 32);
              word = seen_in_windows(mask, a.words, where, sb.len, a.window, j0, word, t, pos >= 0 ? t + 1 : t, 1);
            }
            seen = real & (((uint64_t)__reduce_or_sync(kAll, (uint32_t)(any >> 32)) << 32) | __reduce_or_sync(kAll, (uint32_t)any));
            see = word;
          }
          if (!ctx || lo > 0 || hi < kChunk) {
            blank = true;
            used = hi == 64 ? ~0ull : (1ull << max(hi, 0)) - 1;
            used &= lo >= 64 ? 0ull : ~((1ull << lo) - 1);
            if (!ctx) used &= seen;
          }
        }
        ok = ok && waited(&bar_s[nth & 1], (nth >> 1) & 1, kSiteS, blk);
        if (blank) {
          // V's rows that no row of the CTA sees become zeros.  S(n) has been seen, so the slot's last
          // tile (V(n - 2) at the nearest) has been read, and the parity below is that of this one.
          const int i = id + 2 * ((blk - blk0) / PB) + 1, part = (blk - blk0) % PB;
          ok = ok && waited(&bar_full[i % NS], (i / NS) & 1, kSiteV, blk);
          if (ok && !((used >> (tid >> 1)) & 1)) {
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(ring + (i % NS) * kSlot + (part + s) * kTile + (tid >> 1) * 128 + (tid & 1) * 64 + u * 16) =
                    make_uint4(0, 0, 0, 0);
          }
          tc::fence_async_smem();
        }
        if (!ok) break;
        if (idle) {  // no row of this warp exists: what P holds for them goes nowhere
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar_p[nth & 1]);
          continue;
        }
        tc::fence_after();
        const uint32_t tP = tS + 64 * (nth & 1);
        // Of 32 logits of the row, what it does not see becomes -inf.
        auto hide = [&](float (&s)[32], int q) {
          const uint32_t w = (uint32_t)(see >> (32 * q));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((w >> i) & 1)) s[i] = -CUDART_INF_F;
        };
        // The maximum with this block, and the weights by it.  Loops that are not unrolled: few blocks
        // come here, and code that is short leaves the caches of instructions to the straight run.
        float now = mx;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          float s[32];
          tc::ld32x32b_x32(tP + 32 * q, s);
          tc::ld_wait_row(s);
          hide(s, q);
#pragma unroll
          for (int i = 0; i < 32; i += 2) now = tc::max3(now, s[i], s[i + 1]);
        }
        const float f = now == -CUDART_INF_F ? 1.f : tc::ex2((mx - now) * sl2);
        mx = now;
        l *= f;
        settled = __all_sync(kAll, mx != -CUDART_INF_F || pos < 0);
        if (blk > blk0 && __any_sync(kAll, f != 1.f)) {
          ok = waited(&bar_o[(nth - 1) & 1], ((nth - 1) >> 1) & 1, kSiteO, blk);
          tc::fence_after();
#pragma unroll 1
          for (int q = 0; q < DH / 32; ++q) {
            float o[32];
            tc::ld32x32b_x32(tO + 32 * q, o);
            tc::ld_wait_row(o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[8 * i + e] * f);
              tc::st32x32b_x8(tO + 32 * q + 8 * i, w);
            }
          }
        }
        set_base();
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          float s[32];
          tc::ld32x32b_x32(tP + 32 * q, s);
          tc::ld_wait_row(s);
          hide(s, q);
          uint32_t w[2][8];
          sums[0] = sums[1] = sums[2] = sums[3] = 0;
          weigh(s, w);
          l += total();
          tc::st32x32b_x8(tP + 16 * q, w[0]);  // over logits that have been read
          tc::st32x32b_x8(tP + 16 * q + 8, w[1]);
        }
        tc::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar_p[nth & 1]);
      }
      id += 2 * ((n + PB - 1) / PB);
      if (!ok) break;
      ok = waited(&bar_o[(nth - 1) & 1], ((nth - 1) >> 1) & 1, kSiteO, -1);
      if (!ok) break;
      tc::fence_after();
      if (pos < 0) l = 0.f;
      const bool whole = blk0 == 0 && blk1 == sb.nb;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t to = ((int64_t)b * a.T + t) * a.H + h;
      const Part part = part_of(a, blockIdx.x, slot);
#pragma unroll 1
      for (int q = 0; q < DH / 32; ++q) {
        float o[32];
        tc::ld32x32b_x32(tO + 32 * q, o);
        tc::ld_wait_row(o);
        if (!on) continue;
        if (whole) {
          uint4* row = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.o) + to * DH + 32 * q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = l == 0.f ? 0u : pack_bf16(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv);
            row[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          #pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(part.at(tid, 32 * q + 4 * i)) =
                l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (on) {
        if (whole) {
          a.lse[to] = l == 0.f ? -CUDART_INF_F : mx * a.scale + logf(l);
        } else {
          part.m[tid] = l == 0.f ? -CUDART_INF_F : mx * sl2;
          part.l[tid] = l;
        }
      }
      slot = 1;
      tc::fence_before();
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 4) {
    tc::fence_after();
    tc::tmem_dealloc(tmem_slot, kCols);
  }
}

template <int DH>
cudaError_t run_tc(const TreeArgs& a, cudaStream_t s) {
  using C = Tc<DH>;
  CUtensorMap tk, tv, tkn, tvn;
  cudaError_t e = make_pages_tmap(&tk, a.kp, DH, a.Hkv, a.pages);
  if (e == cudaSuccess) e = make_pages_tmap(&tv, a.vp, DH, a.Hkv, a.pages);
  if (e == cudaSuccess) e = make_draft_tmap(&tkn, a.kn, DH, a.Hkv, a.T, a.B, a.kn_hs, a.kn_ts, a.kn_bs);
  if (e == cudaSuccess) e = make_draft_tmap(&tvn, a.vn, DH, a.Hkv, a.T, a.B, a.vn_hs, a.vn_ts, a.vn_bs);
  if (e == cudaSuccess) e = allow_smem((const void*)tree_tc_kernel<DH>, C::SMEM);
  if (e != cudaSuccess) return e;
  launch_begin("tree_tc", s);
  tree_tc_kernel<DH><<<a.grid * a.hl * a.nrt, kThreads, C::SMEM, s>>>(a, tk, tv, tkn, tvn);
  return launch_end("tree_tc", s);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t s) { return a.dh == 64 ? run_tc<64>(a, s) : run_tc<128>(a, s); }

}  // namespace gca
