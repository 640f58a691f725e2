// Gradients of the attention over packed sequences, bf16, on the 5th-generation tensor cores.
//
// Two passes without atomics, as in window_bwd.cu: first the queries' side (dQ, and a better D) walks the keys
// that a tile of 128 rows sees, then the keys' side (dK, dV) the rows that see a tile of 128 keys, of all heads that
// share it.  Each computes the logits and <dO, V> anew: 3 and 4 products of 128 x 128 x dh a pair of tiles, 7 where
// the gradients themselves need 5.  Both are persistent, a CTA an SM: one warp loads, one or two issue the
// products, eight (queries' side, 64 columns of 32 TMEM lanes each) or sixteen (keys' side, 32) do the arithmetic.
//   * Queries' side: S = Q K^T of the next block is issued as soon as this one's is in registers; dP = dO V^T has two
//     buffers, whose columns dS takes over as the A operand of dQ += dS K, which another warp issues: one for
//     all products took as long as its own instructions (waits, elections and commits, 80 to 140 cycles each),
//     1.77 thousand cycles a block at dh 64.  Now 1.5: 1.0 of arithmetic, where the warps, all in step, have
//     their exponentials (0.5) and sums (0.45) one after the other, the rest waits that are over but take their time.
//   * Keys' side: S^T = K Q^T, dP^T = V dO^T; P^T and dS^T take the columns that they came from as the A
//     operands of dV += P^T dO and dK += dS^T Q.  The products go in the order dV(x), S^T(x + 1), dK(x),
//     dP^T(x + 1), so each follows only the one that read the columns it overwrites (the tensor pipe runs one
//     warp's products in order).  At dh 64 the warps are two groups, each with half of a block's rows and with
//     products, barriers and accumulators of its own (added at the end): one's exponentials run beside the
//     other's sums.  2.14 thousand cycles a block, 2.24 without.  At dh 128 the accumulators fill TMEM.
// P and dS are rounded to bf16, the type of the products' other operands (half a step, 2^-8 of each).
// With that dQ and dK are off by 1.4 times their own rounding.
// Rows behind a sequence's end may hold anything: as operands that are summed over they become zeros in
// shared memory, elsewhere their results are not used.
// Measured, bf16, in a graph, with the rows' sums of prompt_attn.cu: four documents of 46 thousand tokens in all, 12
// heads of 64, 2.59 ms (866 TFLOP/s of five products; queries' side 1.09, keys' side 1.51, rows 0.04); one prompt of
// 32768 tokens, 16 heads of 128 and 4 key heads, 9.7 ms (1.13 PFLOP/s); 54 thousand tokens, 16 and 4 heads of 64, in
// a window of 512 0.62 ms; 1024 prompts of 64 tokens, 12 heads of 64, 0.75; one prompt of 77 tokens 14 us, where each of
// the two starts while what is ahead of it ends (17 without).
#include <algorithm>
#include <type_traits>

#include "prompt.cuh"
#include "tc.cuh"
#include "tc_rows.cuh"
#include "waits.cuh"

namespace gca {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kT = 128;             // rows, and keys, of a tile
// Warps that do the arithmetic: of each 32 rows, two with 64 columns each on the queries' side, four with 32 on the
// keys' side.  The warps of the other roles come behind them: products; on the queries' side the sums', on the
// keys' side the second group's products; loads.
constexpr int kElemQ = 8, kElemKv = 16;
constexpr int threads_of(int elem, int issuing) { return 32 * (elem + issuing + 1); }
constexpr int kTile = kT * 128;     // bytes of 128 rows x 64 elements
constexpr uint32_t kCols = 512;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
enum { kSiteFull = 1, kSiteEmpty, kSiteTile, kSiteTileFree, kSiteS, kSiteDp, kSiteP, kSiteTaken, kSiteDs, kSiteDone, kSiteAcc, kSiteAccFree, kSiteRows, kSiteRest, kSiteItem };

__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* abort_flag, ErrWord* err, int site, int tile, int at) {
  return __all_sync(kAll, park_or_abort(bar, parity, abort_flag, err, site, tile, at)) != 0;
}

template <int DH>
struct Tc {
  static constexpr int SUB = DH / 64;                   // 64-element parts of a head
  static constexpr int BLOCK = kTile * SUB;             // 128 rows of a head
  static constexpr int G = DH == 64 ? 2 : 1;            // keys' side: groups of warps that take turns
  static constexpr int NB = DH == 64 ? 2 : 1;           // buffers of the tile that stays (Q and dO, or K and V)
  static constexpr int NK = DH == 64 ? 8 : 5;           // queries' side: ring slots, a block of K or of V each
  static constexpr int NS = DH == 64 ? 4 : 2;           // keys' side: stages, a tile of Q and of dO and the rows' two sums
  static constexpr int SMEM_Q = 1024 + NB * 2 * BLOCK + NK * BLOCK;
  static constexpr int SMEM_KV = 1024 + NB * 2 * BLOCK + NS * (2 * BLOCK + 2 * kSumsOfTile * 4);
};

// Shared memory and barriers of a CTA, the same for both passes.
template <int DH>
struct Shared {
  uint64_t full[Tc<DH>::NK], empty[Tc<DH>::NK];  // slots, or stages
  uint64_t tile[2], tile_free[2];                // the tile that stays
  // Of each group of warps (on the queries' side dp, ds and done are of each of two buffers):
  uint64_t s[2], dp[2];                          // products that are there: S and dP (or their transposes)
  uint64_t s_taken;                              // queries' side: S is in registers
  uint64_t p[2], ds[2], done[2];                 // P and dS in TMEM; dS's product done
  uint64_t rest;                                 // queries' side: the rows' sums of dS in TMEM
  uint64_t acc, acc_free;                        // the tile's gradients: complete, read
  uint32_t tmem;
  int abort;
  uint8_t keep[PromptTiles<kT>::kKeep];
};

template <int DH, int G, int E, typename I>
__device__ __forceinline__ void set_up(const PromptArgs& a, Shared<DH>& sh, PromptItems<I>& items, int readers) {
  PromptTiles<kT>::fill(a, sh.keep);
  if (threadIdx.x == 0) {
    for (int i = 0; i < Tc<DH>::NK; ++i) {
      tc::mbar_init(&sh.full[i], 1);
      tc::mbar_init(&sh.empty[i], G);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.tile[i], 1);
      tc::mbar_init(&sh.tile_free[i], G);
    }
    for (int i = 0; i < G; ++i) {
      tc::mbar_init(&sh.s[i], 1);
      tc::mbar_init(&sh.p[i], E / G);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.dp[i], 1);
      tc::mbar_init(&sh.ds[i], E / G);
      tc::mbar_init(&sh.done[i], 1);
    }
    tc::mbar_init(&sh.s_taken, E);
    tc::mbar_init(&sh.rest, E);
    tc::mbar_init(&sh.acc, G);
    tc::mbar_init(&sh.acc_free, E);
    init_items(items, readers);
    sh.abort = 0;
    tc::fence_mbar_init();
  }
  if (threadIdx.x / 32 == E) tc::tmem_alloc(&sh.tmem, kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
}

// Of group `grp`'s rows of a block in shared memory those from `have` on become zeros; called by 128 threads.
template <int DH, int G>
__device__ __forceinline__ void blank(unsigned char* block, int grp, int thread, int have) {
  constexpr int U = 8 / G;  // 16-byte units of a row part a thread
  const int r = grp * (kT / G) + thread / G, u0 = thread % G * U;
  if (r < have) return;
#pragma unroll
  for (int s = 0; s < Tc<DH>::SUB; ++s)
#pragma unroll
    for (int u = 0; u < U; ++u) *reinterpret_cast<uint4*>(block + s * kTile + r * 128 + (u0 + u) * 16) = make_uint4(0, 0, 0, 0);
}

// D = A B^T of two K-major blocks: group `grp`'s columns, 128 or 64 of them.
template <int DH, int G>
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b, int grp) {
  constexpr int N = kT / G;
#pragma unroll
  for (int s = 0; s < Tc<DH>::SUB; ++s)
    tc::mma4_ss<tc::kKStepKm, tc::kKStepKm>(d + N * grp, tc::desc_km(a + s * kTile), tc::desc_km(b + s * kTile + grp * N * 128),
                                            tc::idesc_bf16(kT, N, false), s ? 1u : 0u);
}
// D[128 x DH] (+)= A B with group `grp`'s columns of A [128 x 128] in TMEM, each 16 of them in front of 16 others, and rows
// of B [128 x DH] in shared memory.
template <int DH, int G>
__device__ __forceinline__ void accumulate(uint32_t d, uint32_t at, uint32_t b, int grp, bool add) {
  constexpr int H = 2 / G;  // runs of 64 rows
#pragma unroll
  for (int s = 0; s < Tc<DH>::SUB; ++s)
#pragma unroll
    for (int h = 0; h < H; ++h)
      tc::mma4_ts<8, 32, 40, tc::kKStepMn>(d + 64 * s, at + 64 * (H * grp + h),
                                         tc::desc_mn(b + s * kTile + kTile / 2 * (H * grp + h)), tc::idesc_bf16(kT, 64, true), add || h ? 1u : 0u);
}

// W columns of a row of the groups' accumulators, `apart` columns from one to the next, summed and scaled, to
// global memory: `to` is the first of them in row 0, with `have` columns there, `pos` the lane's row of `len`.
template <int W, int G>
__device__ __forceinline__ void write_rows(uint32_t at, int apart, bf16* to, int64_t stride, int pos, int len, float scale, int have) {
  uint4 x[W / 8];
#pragma unroll
  for (int c = 0; c < W; c += 32) {
    float o[32], more[32];
    tc::ld32x32b_x32(at + c, o);
    if constexpr (G == 2) tc::ld32x32b_x32(at + apart + c, more);
    tc::ld_wait_row(o);
    if constexpr (G == 2) {
      tc::ld_wait_row(more);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] += more[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[c / 8 + i] = make_uint4(pack_bf16(o[8 * i] * scale, o[8 * i + 1] * scale), pack_bf16(o[8 * i + 2] * scale, o[8 * i + 3] * scale),
                                pack_bf16(o[8 * i + 4] * scale, o[8 * i + 5] * scale), pack_bf16(o[8 * i + 6] * scale, o[8 * i + 7] * scale));
  }
  tc::store_rows(x, reinterpret_cast<uint4*>(to), stride / 8, pos, len, have / 8);
}

struct Maps {
  CUtensorMap q, k, v, g;
};

// Work of the queries' side: a tile of rows of a head, and its blocks lo .. tile of keys.
struct QItem {
  PromptTile x;
  int h, m, lo, more;  // more: 0 behind the last
};
__device__ __forceinline__ bool q_item(const PromptArgs& a, PromptTiles<kT>& tiles, int w, QItem& it) {
  it.h = w % a.H;
  it.m = it.h / a.g;
  if (!prompt_tile(a, tiles, w / a.H, false, it.x)) return false;
  it.lo = a.window ? max(0, it.x.tile * kT - a.window + 1) / kT : 0;
  return true;
}

// ------------------------------------------------------------------ the queries' side
template <int DH>
__global__ void __launch_bounds__(threads_of(kElemQ, 2), 1) prompt_dq_tc_kernel(PromptArgs a, const __grid_constant__ Maps tm) {
  using C = Tc<DH>;
  constexpr int NK = C::NK, NB = C::NB, SUB = C::SUB;
  extern __shared__ unsigned char dsm[];
  unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = tiles + NB * 2 * C::BLOCK;
  __shared__ __align__(8) Shared<DH> sh;
  __shared__ __align__(8) PromptItems<QItem> items;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  set_up<DH, 1, kElemQ>(a, sh, items, kElemQ + 2);
  let_next();
  const uint32_t tS = sh.tmem, tP = tS + 128, tQ = tS + 384;  // S, two of dP, dQ
  bool ok = true;
  auto waited = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    if (__builtin_expect(__all_sync(kAll, tc::mbar_try(bar, parity)), 1)) return true;
    return wait_on(bar, parity, &sh.abort, a.err, site, blockIdx.x, at);
  };
  QItem it;
  auto take_into = [&](int n, QItem& x) { return (ok = ok && take_item(items, n, x, waited, kSiteItem)) && x.more; };
  auto take = [&](int n) { return take_into(n, it); };

  if (warp == kElemQ + 2) {
    // ---------------------------------------------------------------- loads
    int id = 0, nt = 0;
    PromptTiles<kT> counts(a, sh.keep);
    for (; ok; ++nt) {
      it.more = q_item(a, counts, prompt_turn(nt), it);
      ok = put_item(items, nt, it, waited, kSiteItem);
      if (!ok || !it.more) break;
      const int buf = nt % NB;
      ok = waited(&sh.tile_free[buf], ((nt / NB) & 1) ^ 1, kSiteTileFree, nt);
      if (!ok) break;
      tc::mbar_expect_tx_warp(&sh.tile[buf], 2 * C::BLOCK);
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        unsigned char* to = tiles + buf * 2 * C::BLOCK + s * kTile;
        tc::tma_load_4d_warp(to, &tm.q, 64 * s, a.q_hs ? it.h : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
        tc::tma_load_4d_warp(to + C::BLOCK, &tm.g, 64 * s, a.do_hs ? it.h : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
      }
      for (int n = it.lo; n <= it.x.tile && ok; ++n)
#pragma unroll 1
        for (int v = 0; v < 2; ++v, ++id) {  // K, then V
          const int st = id % NK;
          ok = waited(&sh.empty[st], ((id / NK) & 1) ^ 1, kSiteEmpty, n);
          if (!ok) break;
          tc::mbar_expect_tx_warp(&sh.full[st], C::BLOCK);
#pragma unroll
          for (int s = 0; s < SUB; ++s)
            tc::tma_load_4d_warp(ring + st * C::BLOCK + s * kTile, v ? &tm.v : &tm.k, 64 * s, (v ? a.v_hs : a.k_hs) ? it.m : 0, it.x.off + n * kT, 0,
                                 &sh.full[st]);
        }
    }
    if (!ok) {  // let the copies in flight land before the CTA ends
      for (int i = max(0, id - NK); i < id; ++i) tc::mbar_wait(&sh.full[i % NK], (i / NK) & 1, 1u << 16);
      for (int i = max(0, nt + 1 - NB); i <= nt; ++i) tc::mbar_wait(&sh.tile[i % NB], (i / NB) & 1, 1u << 16);
    }
  } else if (warp == kElemQ) {
    // ---------------------------------------------------------------- S once the last is in registers, dP two blocks ahead
    int id = 0, nt = 0;  // blocks, tiles so far
    for (; take(nt); ++nt) {
      const uint32_t q = tc::su32(tiles + (nt % NB) * 2 * C::BLOCK), g = q + C::BLOCK;
      ok = waited(&sh.tile[nt % NB], (nt / NB) & 1, kSiteTile, nt);
      for (int n = it.lo; n <= it.x.tile && ok; ++n, ++id) {
        const int ks = 2 * id % NK, vs = (2 * id + 1) % NK;
        ok = waited(&sh.full[ks], (2 * id / NK) & 1, kSiteFull, n) && (id == 0 || waited(&sh.s_taken, (id - 1) & 1, kSiteTaken, n));
        if (!ok) break;
        tc::fence_after();
        product<DH, 1>(tS, q, tc::su32(ring + ks * C::BLOCK), 0);
        tc::commit_warp(&sh.s[0]);
        ok = waited(&sh.full[vs], ((2 * id + 1) / NK) & 1, kSiteFull, n) && (id < 2 || waited(&sh.done[id & 1], ((id >> 1) - 1) & 1, kSiteDone, n));
        if (!ok) break;
        tc::fence_after();
        product<DH, 1>(tP + 128 * (id & 1), g, tc::su32(ring + vs * C::BLOCK), 0);
        tc::commit_warp(&sh.dp[id & 1]);
        tc::commit_warp(&sh.empty[vs]);
      }
      if (!ok) break;
      tc::commit_warp(&sh.tile_free[nt % NB]);
    }
  } else if (warp == kElemQ + 1) {
    // ---------------------------------------------------------------- dQ += dS K
    int id = 0, nt = 0;
    for (; take(nt); ++nt) {
      ok = waited(&sh.acc_free, (nt & 1) ^ 1, kSiteAccFree, nt);
      for (int n = it.lo; n <= it.x.tile && ok; ++n, ++id) {
        const int ks = 2 * id % NK;
        ok = waited(&sh.ds[id & 1], (id >> 1) & 1, kSiteDs, n);
        if (!ok) break;
        tc::fence_after();
        accumulate<DH, 1>(tQ, tP + 128 * (id & 1), tc::su32(ring + ks * C::BLOCK), 0, n > it.lo);
        tc::commit_warp(&sh.done[id & 1]);
        tc::commit_warp(&sh.empty[ks]);
      }
      if (!ok) break;
      tc::commit_warp(&sh.acc);
    }
  } else {
    // ---------------------------------------------------------------- arithmetic
    const int r = 32 * (warp & 3) + lane, part = warp >> 2;  // row of the tile; columns 64 part ..
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float sl2 = a.scale * kLog2e;
    const uint64_t k2 = tc::f2(sl2, sl2);
    int id = 0, nt = 0, met = 0;
    // The sum over a row's two warps.  They meet in columns of dQ that each has read (or that hold nothing yet), in
    // another one every other time: until then both have read.
    auto meet = [&](float own) {
      float both[1];
      const uint32_t at = tQ + lanes + (met & 1);
      tc::st32x32b_x1(at + part * (DH / 2), __float_as_uint(own));
      tc::st_wait();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.rest);
      ok = waited(&sh.rest, met & 1, kSiteRest, nt);
      ++met;
      if (!ok) return 0.f;
      tc::fence_after();
      tc::ld32x32b_x1(at + (part ^ 1) * (DH / 2), both[0]);
      tc::ld_wait_row(both);
      return own + both[0];
    };
    // -lse log2(e) and -D of the item's row; a row that does not exist weighs nothing.
    auto row_of = [&](const QItem& x) { return prompt_sums(a, x.x.off, x.h) + x.x.tile * kT + r; };
    float nl = -CUDART_INF_F, nd = 0.f;
    bool more = take(0);
    after_previous();  // the rows' sums
    if (more && it.x.tile * kT + r < it.x.len) {
      nl = a.nlse[row_of(it)];
      nd = a.nD[row_of(it)];
    }
    for (; more; ++nt) {
      const int pos = it.x.tile * kT + r;
      const bool on = pos < it.x.len;
      const uint64_t nl2 = tc::f2(nl, nl);
      uint64_t rest = 0;  // sum of dS
      const int first = a.window ? max(0, pos - a.window + 1) : 0;
      const int whole = a.window ? (max(0, it.x.tile * kT + kT - a.window) + kT - 1) / kT : 0;
      if (it.lo == it.x.tile) {
        // One block alone, so rows that see few keys: what the rounding of o puts into D is largest there.  dS is summed
        // once beforehand, for a D that is right when it is rounded.  (Without that dQ of sequences of two tokens is off
        // by 4.0e-3 of its size, of 17 by 2.9e-3, now by 2.4e-3; of single tokens, whose gradient is 0, it is 0.  It
        // costs short prompts' gradients some 5 us of 73.  Later rows see few keys only in small windows, where D comes
        // right: prompt_few_rows_kernel.)
        ok = waited(&sh.s[0], id & 1, kSiteS, nt) && waited(&sh.dp[id & 1], (id >> 1) & 1, kSiteDp, nt);
        if (!ok) break;
        tc::fence_after();
        float sum = 0.f;
#pragma unroll 1
        for (int c = 64 * part; c < 64 * part + 64; c += 32) {
          float s[32], dp[32];
          tc::ld32x32b_x32(tS + lanes + c, s);
          tc::ld32x32b_x32(tP + 128 * (id & 1) + lanes + c, dp);
          tc::ld_wait_row(s);
          tc::ld_wait_row(dp);
          const int k0 = it.x.tile * kT + c;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (on && k0 + i <= pos && k0 + i >= first) sum += tc::ex2(fmaf(s[i], sl2, nl)) * (dp[i] + nd);
        }
        sum = meet(sum);
        if (!ok) break;
        nd -= sum;
      }
      const uint64_t nd2 = tc::f2(nd, nd);
      for (int n = it.lo; n <= it.x.tile; ++n, ++id) {
        ok = waited(&sh.s[0], id & 1, kSiteS, n);
        if (!ok) break;
        tc::fence_after();
        float s[2][32], dp[32];
        tc::ld32x32b_x32(tS + lanes + 64 * part, s[0]);
        tc::ld32x32b_x32(tS + lanes + 64 * part + 32, s[1]);
        tc::ld_wait_row(s[0]);
        tc::ld_wait_row(s[1]);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.s_taken);
        ok = waited(&sh.dp[id & 1], (id >> 1) & 1, kSiteDp, n);
        if (!ok) break;
        tc::fence_after();
        const uint32_t to = tP + 128 * (id & 1) + lanes + 64 * part;
        tc::ld32x32b_x32(to, dp);  // on its way while the logits are weighed
        uint32_t d[2][16];
        auto probabilities = [&](float (&s)[32]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            tc::uf2(tc::fma2(tc::f2(s[2 * i], s[2 * i + 1]), k2, nl2), x, y);
            s[2 * i] = tc::ex2(x);
            s[2 * i + 1] = tc::ex2(y);
          }
        };
        auto weigh = [&](auto edge, const float (&s)[32], uint32_t (&d)[16], int c0, int c1) {  // at an edge: keys c0 .. c1 - 1 are seen
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            tc::uf2(tc::mul2(tc::f2(s[2 * i], s[2 * i + 1]), tc::add2(tc::f2(dp[2 * i], dp[2 * i + 1]), nd2)), x, y);
            if constexpr (decltype(edge)::value) {
              if (2 * i < c0 || 2 * i >= c1) x = 0.f;
              if (2 * i + 1 < c0 || 2 * i + 1 >= c1) y = 0.f;
            }
            rest = tc::add2(rest, tc::f2(x, y));
            d[i] = pack_bf16(x, y);
          }
        };
        auto both = [&](auto edge) {
          const int c0 = first - n * kT - 64 * part, c1 = on ? pos - n * kT - 64 * part + 1 : 0;
          probabilities(s[0]);
          tc::ld_wait_row(dp);
          weigh(edge, s[0], d[0], c0, c1);
          tc::ld32x32b_x32(to + 32, dp);
          probabilities(s[1]);
          tc::ld_wait_row(dp);
          weigh(edge, s[1], d[1], c0 - 32, c1 - 32);
        };
        if (n == it.x.tile || n < whole) both(std::true_type{});  // keys that the row does not see, and rows that do not exist
        else both(std::false_type{});
        if ((n + 1) * kT > it.x.len) {  // rows of K behind the sequence
          ok = waited(&sh.full[2 * id % NK], (2 * id / NK) & 1, kSiteRows, n);
          if (!ok) break;
          if (part == 0) blank<DH, 1>(ring + (2 * id % NK) * C::BLOCK, 0, r, it.x.len - n * kT);
          tc::fence_async_smem();
        }
        // Over columns that have been read: an A operand's 16 of each 32.
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t d0[8] = {d[c][0], d[c][1], d[c][2], d[c][3], d[c][4], d[c][5], d[c][6], d[c][7]};
          const uint32_t d1[8] = {d[c][8], d[c][9], d[c][10], d[c][11], d[c][12], d[c][13], d[c][14], d[c][15]};
          tc::st32x32b_x8(to + 32 * c, d0);
          tc::st32x32b_x8(to + 32 * c + 8, d1);
        }
        tc::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.ds[id & 1]);  // (a warp is never two blocks ahead of another: dP of the second waits for all)
      }
      if (!ok) break;
      // The next row's sums are on their way while this one's gradients are written.
      QItem next;
      more = take_into(nt + 1, next);
      if (!ok) break;
      float next_nl = -CUDART_INF_F, next_nd = 0.f;
      if (more && next.x.tile * kT + r < next.x.len) {
        next_nl = a.nlse[row_of(next)];
        next_nd = a.nD[row_of(next)];
      }
      ok = waited(&sh.acc, nt & 1, kSiteAcc, nt);
      if (!ok) break;
      tc::fence_after();
      const int col = part * (DH / 2);
      bf16* to = reinterpret_cast<bf16*>(a.dq) + (int64_t)it.x.off * a.dq_ts + it.h * a.dq_hs + col;
      if (col < a.dh) write_rows<DH / 2, 1>(tQ + lanes + col, 0, to, a.dq_ts, pos, it.x.len, a.scale, a.dh - col);
      // A row of dS sums to 0 by its D; what is left is how far D, of the rounded output, is off.  The keys' side takes
      // the D that is right: in rows that see few keys the difference is as large as the roundings of dS.
      float x, y;
      tc::uf2(rest, x, y);
      const float left = meet(x + y);
      if (!ok) break;
      if (part == 0 && on) a.nD[row_of(it)] = nd - left;
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.acc_free);
      it = next;
      nl = next_nl;
      nd = next_nd;
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kElemQ) {
    tc::fence_after();
    tc::tmem_dealloc(sh.tmem, kCols);
  }
}

// Work of the keys' side: a tile of keys of a key head; for each of the g heads that share it, the tiles
// tile .. end - 1 of rows.
struct KvItem {
  PromptTile x;
  int m, end, more;
};
__device__ __forceinline__ bool kv_item(const PromptArgs& a, PromptTiles<kT>& tiles, int w, KvItem& it) {
  it.m = w % a.Hkv;
  if (!prompt_tile(a, tiles, w / a.Hkv, true, it.x)) return false;
  const int k = min(it.x.tile * kT + kT, it.x.len) - 1;  // the tile's last key
  it.end = (a.window ? (int)min((int64_t)it.x.len - 1, (int64_t)k + a.window - 1) : it.x.len - 1) / kT + 1;
  return true;
}

// ------------------------------------------------------------------ the keys' side
template <int DH>
__global__ void __launch_bounds__(threads_of(kElemKv, Tc<DH>::G), 1) prompt_dkv_tc_kernel(PromptArgs a, const __grid_constant__ Maps tm) {
  using C = Tc<DH>;
  constexpr int NS = C::NS, NB = C::NB, SUB = C::SUB, G = C::G;
  extern __shared__ unsigned char dsm[];
  unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = tiles + NB * 2 * C::BLOCK;
  float* rows = reinterpret_cast<float*>(ring + NS * 2 * C::BLOCK);  // of each stage: -lse log2(e), -D
  __shared__ __align__(8) Shared<DH> sh;
  __shared__ __align__(8) PromptItems<KvItem> items;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  set_up<DH, G, kElemKv>(a, sh, items, kElemKv + G);
  if (warp != kElemKv + G) after_previous();  // (before any wait with a limit: the queries' side may take long)
  // P^T and dS^T lie in the columns that S^T and dP^T came in; behind those dV and dK, of each group its own.
  const uint32_t tS = sh.tmem, tP = tS + 128, tV = tS + 256, tK = tV + DH;
  bool ok = true;
  auto waited = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    if (__builtin_expect(__all_sync(kAll, tc::mbar_try(bar, parity)), 1)) return true;
    return wait_on(bar, parity, &sh.abort, a.err, site, blockIdx.x, at);
  };
  KvItem it;
  auto take = [&](int n) { return (ok = ok && take_item(items, n, it, waited, kSiteItem)) && it.more; };

  if (warp == kElemKv + G) {
    // ---------------------------------------------------------------- loads
    int id = 0, nt = 0;
    PromptTiles<kT> counts(a, sh.keep);
    for (; ok; ++nt) {
      it.more = kv_item(a, counts, prompt_turn(nt), it);
      ok = put_item(items, nt, it, waited, kSiteItem);
      if (!ok || !it.more) break;
      const int buf = nt % NB;
      ok = waited(&sh.tile_free[buf], ((nt / NB) & 1) ^ 1, kSiteTileFree, nt);
      if (!ok) break;
      tc::mbar_expect_tx_warp(&sh.tile[buf], 2 * C::BLOCK);
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        unsigned char* to = tiles + buf * 2 * C::BLOCK + s * kTile;
        tc::tma_load_4d_warp(to, &tm.k, 64 * s, a.k_hs ? it.m : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
        tc::tma_load_4d_warp(to + C::BLOCK, &tm.v, 64 * s, a.v_hs ? it.m : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
      }
      if (nt == 0) after_previous();  // the rows' sums, as the queries' side left them
      for (int h = it.m * a.g; h < it.m * a.g + a.g && ok; ++h)
        for (int i = it.x.tile; i < it.end; ++i, ++id) {
          const int st = id % NS;
          ok = waited(&sh.empty[st], ((id / NS) & 1) ^ 1, kSiteEmpty, i);
          if (!ok) break;
          tc::mbar_expect_tx_warp(&sh.full[st], 2 * C::BLOCK + 2 * kSumsOfTile * 4);
#pragma unroll
          for (int s = 0; s < SUB; ++s) {
            unsigned char* to = ring + st * 2 * C::BLOCK + s * kTile;
            tc::tma_load_4d_warp(to, &tm.q, 64 * s, a.q_hs ? h : 0, it.x.off + i * kT, 0, &sh.full[st]);
            tc::tma_load_4d_warp(to + C::BLOCK, &tm.g, 64 * s, a.do_hs ? h : 0, it.x.off + i * kT, 0, &sh.full[st]);
          }
          const int64_t row = prompt_sums(a, it.x.off, h) + i * kT - (it.x.off & 2);
          if (lane == 0) {
            tc::bulk_load(rows + st * 2 * kSumsOfTile, a.nlse + row, kSumsOfTile * 4, &sh.full[st]);
            tc::bulk_load(rows + (st * 2 + 1) * kSumsOfTile, a.nD + row, kSumsOfTile * 4, &sh.full[st]);
          }
          __syncwarp();
        }
    }
    if (!ok) {
      for (int i = max(0, id - NS); i < id; ++i) tc::mbar_wait(&sh.full[i % NS], (i / NS) & 1, 1u << 16);
      for (int i = max(0, nt + 1 - NB); i <= nt; ++i) tc::mbar_wait(&sh.tile[i % NB], (i / NB) & 1, 1u << 16);
    }
  } else if (warp >= kElemKv) {
    // ---------------------------------------------------------------- products of a group
    const int w = G == 1 ? 0 : warp - kElemKv;
    const uint32_t tVw = tV + 2 * DH * w, tKw = tVw + DH;
    int id = 0, nt = 0;  // blocks, tiles so far
    for (; take(nt); ++nt) {
      const uint32_t k = tc::su32(tiles + (nt % NB) * 2 * C::BLOCK), v = k + C::BLOCK;
      const int count = (it.end - it.x.tile) * a.g;
      ok = waited(&sh.tile[nt % NB], (nt / NB) & 1, kSiteTile, nt);
      for (int x = -1; x < count && ok; ++x) {
        const int i = id + x, st = i % NS, next = (i + 1) % NS;
        const uint32_t q = tc::su32(ring + st * 2 * C::BLOCK), qn = tc::su32(ring + next * 2 * C::BLOCK);
        if (x >= 0) {
          ok = (x > 0 || waited(&sh.acc_free, (nt & 1) ^ 1, kSiteAccFree, nt)) && waited(&sh.p[w], i & 1, kSiteP, x);
          if (!ok) break;
          tc::fence_after();
          accumulate<DH, G>(tVw, tS, q + C::BLOCK, w, x > 0);
        }
        if (x + 1 < count) {
          ok = waited(&sh.full[next], ((i + 1) / NS) & 1, kSiteFull, x);
          if (!ok) break;
          tc::fence_after();
          product<DH, G>(tS, k, qn, w);
          tc::commit_warp(&sh.s[w]);
        }
        if (x >= 0) {
          ok = waited(&sh.ds[w], i & 1, kSiteDs, x);
          if (!ok) break;
          tc::fence_after();
          accumulate<DH, G>(tKw, tP, q, w, x > 0);
          tc::commit_warp(&sh.empty[st]);
        }
        if (x + 1 < count) {
          product<DH, G>(tP, v, qn + C::BLOCK, w);
          tc::commit_warp(&sh.dp[w]);
        }
      }
      if (!ok) break;
      tc::commit_warp(&sh.tile_free[nt % NB]);
      tc::commit_warp(&sh.acc);
      id += count;
    }
  } else {
    // ---------------------------------------------------------------- arithmetic
    // A warp's 32 keys (lanes) and 32 rows (columns 32 part ..) in fragments: of each 16 keys and 8 rows a thread has
    // keys lane / 4 and lane / 4 + 8 and rows 2 (lane % 4) and the next.  So it needs eight rows' sums, not all 32:
    // in whole rows a thread their loads from shared memory (four wavefronts a vector, broadcast or not) took longer
    // than the operands of the products.
    const int part = warp >> 2, grp = G == 2 ? part >> 1 : 0, group = lane >> 2, two = 2 * (lane & 3);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float sl2 = a.scale * kLog2e;
    const uint64_t k2 = tc::f2(sl2, sl2);
    int id = 0, nt = 0;
    for (; take(nt); ++nt) {
      const int key0 = it.x.tile * kT + 32 * (warp & 3) + group;  // keys key0 + 0, 8, 16, 24
      for (int h = 0; h < a.g && ok; ++h)
        for (int i = it.x.tile; i < it.end; ++i, ++id) {
          const int st = id % NS, t0 = i * kT + 32 * part + two;  // rows t0 + 8 n, and the next
          ok = waited(&sh.full[st], (id / NS) & 1, kSiteRows, i) && waited(&sh.s[grp], id & 1, kSiteS, i);
          if (!ok) break;
          tc::fence_after();
          // Every row sees every key of blocks inside.
          const bool edge = i == it.x.tile || (i + 1) * kT > it.x.len || (a.window && i * kT + kT - a.window > it.x.tile * kT);
          auto seen = [&](int t, int key) { return t >= key && t < it.x.len && (a.window == 0 || t - key < a.window); };
          float p[2][4][4];
          tc::ld16x256_x4(tS + lanes + 32 * part, p[0]);
          tc::ld16x256_x4(tS + lanes + (16u << 16) + 32 * part, p[1]);
          if ((G == 2 || part < 2) && (i + 1) * kT > it.x.len) {  // rows of Q and dO behind the sequence
            blank<DH, G>(ring + st * 2 * C::BLOCK + part % 2 * C::BLOCK, grp, 32 * (warp & 3) + lane, it.x.len - i * kT);
            tc::fence_async_smem();
          }
          const float* nl = rows + st * 2 * kSumsOfTile + (it.x.off & 2) + 32 * part + two;
          const float* nd = nl + kSumsOfTile;
          tc::ld_wait(p[0]);
          tc::ld_wait(p[1]);
          uint32_t x[2][8];
          auto weigh = [&](auto at_edge) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint64_t l = *reinterpret_cast<const uint64_t*>(nl + 8 * n);
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  float e, f;
                  tc::uf2(tc::fma2(tc::f2(p[k][n][2 * u], p[k][n][2 * u + 1]), k2, l), e, f);
                  e = tc::ex2(e);
                  f = tc::ex2(f);
                  if constexpr (decltype(at_edge)::value) {
                    const int key = key0 + 16 * k + 8 * u;
                    if (!seen(t0 + 8 * n, key)) e = 0.f;
                    if (!seen(t0 + 8 * n + 1, key)) f = 0.f;
                  }
                  p[k][n][2 * u] = e;
                  p[k][n][2 * u + 1] = f;
                  x[k][2 * n + u] = pack_bf16(e, f);
                }
            }
          };
          if (edge) weigh(std::true_type{});
          else weigh(std::false_type{});
          // Over columns that have been read: an A operand's 16 of each 32.
          tc::st16x128_x4(tS + lanes + 32 * part, x[0]);
          tc::st16x128_x4(tS + lanes + (16u << 16) + 32 * part, x[1]);
          tc::st_wait();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.p[grp]);
          ok = waited(&sh.dp[grp], id & 1, kSiteDp, i);
          if (!ok) break;
          tc::fence_after();
          float d[2][4][4];
          tc::ld16x256_x4(tP + lanes + 32 * part, d[0]);
          tc::ld16x256_x4(tP + lanes + (16u << 16) + 32 * part, d[1]);
          tc::ld_wait(d[0]);
          tc::ld_wait(d[1]);
          auto differ = [&](auto at_edge) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint64_t l = *reinterpret_cast<const uint64_t*>(nd + 8 * n);
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  float e, f;
                  tc::uf2(tc::mul2(tc::f2(p[k][n][2 * u], p[k][n][2 * u + 1]), tc::add2(tc::f2(d[k][n][2 * u], d[k][n][2 * u + 1]), l)), e, f);
                  if constexpr (decltype(at_edge)::value) {  // (what is not seen may be anything, an infinity times 0 too)
                    const int key = key0 + 16 * k + 8 * u;
                    if (!seen(t0 + 8 * n, key)) e = 0.f;
                    if (!seen(t0 + 8 * n + 1, key)) f = 0.f;
                  }
                  x[k][2 * n + u] = pack_bf16(e, f);
                }
            }
          };
          if (edge) differ(std::true_type{});
          else differ(std::false_type{});
          tc::st16x128_x4(tP + lanes + 32 * part, x[0]);
          tc::st16x128_x4(tP + lanes + (16u << 16) + 32 * part, x[1]);
          tc::st_wait();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.ds[grp]);
        }
      if (!ok) break;
      ok = waited(&sh.acc, nt & 1, kSiteAcc, nt);
      if (!ok) break;
      tc::fence_after();
      // Half a row of dV, or of dK, a warp.
      const int key = it.x.tile * kT + 32 * (warp & 3) + lane, col = (part & 1) * (DH / 2);
      if (col < a.dh) {
        if (part < 2)
          write_rows<DH / 2, G>(tV + lanes + col, 2 * DH, reinterpret_cast<bf16*>(a.dv) + (int64_t)it.x.off * a.dv_ts + it.m * a.dv_hs + col,
                                a.dv_ts, key, it.x.len, 1.f, a.dh - col);
        else
          write_rows<DH / 2, G>(tK + lanes + col, 2 * DH, reinterpret_cast<bf16*>(a.dk) + (int64_t)it.x.off * a.dk_ts + it.m * a.dk_hs + col,
                                a.dk_ts, key, it.x.len, a.scale, a.dh - col);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.acc_free);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kElemKv) {
    tc::fence_after();
    tc::tmem_dealloc(sh.tmem, kCols);
  }
}

template <int DH>
cudaError_t run_tc(const PromptArgs& a, cudaStream_t s) {
  using C = Tc<DH>;
  Maps tm;
  cudaError_t e = make_packed_tmap(&tm.q, a.q, a.dh, a.H, a.N, a.q_hs, a.q_ts);
  if (e == cudaSuccess) e = make_packed_tmap(&tm.k, a.k, a.dh, a.Hkv, a.N, a.k_hs, a.k_ts);
  if (e == cudaSuccess) e = make_packed_tmap(&tm.v, a.v, a.dh, a.Hkv, a.N, a.v_hs, a.v_ts);
  if (e == cudaSuccess) e = make_packed_tmap(&tm.g, a.dout, a.dh, a.H, a.N, a.do_hs, a.do_ts);
  if (e == cudaSuccess) e = allow_smem((const void*)prompt_dq_tc_kernel<DH>, C::SMEM_Q);
  if (e == cudaSuccess) e = allow_smem((const void*)prompt_dkv_tc_kernel<DH>, C::SMEM_KV);
  if (e != cudaSuccess) return e;
  const int64_t tiles = a.N / kT + std::min<int64_t>(a.B, a.N);
  launch_begin("prompt_dq_tc", s);
  e = launch_after_smem(prompt_dq_tc_kernel<DH>, dim3((unsigned)std::min<int64_t>(tiles * a.H, kSMs)), dim3(threads_of(kElemQ, 2)), C::SMEM_Q, s, a, tm);
  cudaError_t last = launch_end("prompt_dq_tc", s);
  if (e == cudaSuccess) e = last;
  if (e != cudaSuccess) return e;
  launch_begin("prompt_dkv_tc", s);
  e = launch_after_smem(prompt_dkv_tc_kernel<DH>, dim3((unsigned)std::min<int64_t>(tiles * a.Hkv, kSMs)), dim3(threads_of(kElemKv, C::G)), C::SMEM_KV, s, a, tm);
  last = launch_end("prompt_dkv_tc", s);
  return e != cudaSuccess ? e : last;
}

}  // namespace

cudaError_t launch_prompt_bwd_tc(const PromptArgs& a, cudaStream_t s) { return a.dh <= 64 ? run_tc<64>(a, s) : run_tc<128>(a, s); }

}  // namespace gca
