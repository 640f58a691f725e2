// Attention of drafted tokens over a paged cache where many query rows share a key head
// (T g > 16), bf16, dh 64 or 128, on the 5th-generation tensor cores.
//
// With 128 rows a byte of K or V asks 128 operations: still below the balance of memory and
// tensor pipes (about 290), so the aim is a stream of pages that never waits.  One CTA walks
// its share of the blocks for 128 rows (padded) of one key head; two CTAs share an SM.
//   * warp 5 (loads): page numbers of 32 blocks at a time, and one TMA load per 64 x 64 tile
//     of K and V into a ring, in the order the products read them: K(0), K(1), V(0), K(2), ...
//   * warp 4 (products): S(n) = Q K(n)^T into one of two TMEM buffers, one block ahead of the
//     softmax; O += P(n) V(n) with P in the buffer that S(n) lay in.
//     Barriers of blocks (S ready, P ready, O done) come in pairs, one for even and one for odd
//     blocks: S(n) is issued before P V (n - 1), so a thread that has seen S(n) knows that
//     P V (n - 2) is done, not that P V (n - 1) is, and one barrier's parity would not tell.
//   * warps 0-3 (softmax): a thread owns a row.  Running maximum and sum; the output is only
//     rescaled when a row's maximum has grown by more than 2^8 over the one in use, which
//     keeps the weights below 2^8 (their sum stays in 32 bits, and bf16 rounds relative to
//     the weight, so nothing is lost); after a few blocks that no longer happens.
// The last page, the window's edge and the draft's own block are masked by a 64-bit word a
// row; there the rows of V that nobody sees are set to zeros in shared memory, for a weight
// of 0 times what lies in them must stay 0.
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
constexpr int kRows = 128;
constexpr int kTile = 8192;     // 64 tokens x 64 elements
constexpr float kGrow = 8.f;    // log2 of how far a row's maximum may outgrow the one in use
constexpr uint32_t kAll = 0xffffffffu;
enum { kSiteFull = 1, kSiteEmpty, kSiteQ, kSiteS, kSiteP, kSiteO, kSiteV };

template <int DH>
struct Tc {
  static constexpr int SUB = DH / 64;               // 64-element parts of a head
  static constexpr int STAGE = kTile * SUB;         // K or V of a block
  static constexpr int QB = 2 * kTile * SUB;        // 128 rows
  static constexpr int NS = DH == 64 ? 11 : 4;      // ring stages
  static constexpr int SMEM = QB + NS * STAGE + 1024;
};

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++stage == n) {
      stage = 0;
      phase ^= 1;
    }
  }
};

template <int DH>
__global__ void __launch_bounds__(kThreads, 2)
tree_tc_kernel(TreeArgs a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmKn, const __grid_constant__ CUtensorMap tmVn) {
  using C = Tc<DH>;
  constexpr int SUB = C::SUB, NS = C::NS;
  constexpr uint32_t kIdS = tc::idesc_bf16(kRows, 64, false), kIdPV = tc::idesc_bf16(kRows, 64, true);
  extern __shared__ __align__(1024) unsigned char dsm[];
  unsigned char* Qs = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = Qs + C::QB;
  __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_q, bar_s[2], bar_p[2], bar_o[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  if (warp == 4) tc::tmem_alloc(&tmem_slot, 256);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = tmem_slot, tO = tmem_slot + 128;
  const int rt = my_rows(a);

  // The segments of this CTA, walked by every role: blocks blk0 .. blk1 - 1 of tile `tile`.
  int b = sh.b, off = sh.off, item = sh.lo;
  SeqBlocks sb = seq_blocks(a, b, false);
  int tile = 0, blk0 = 0, blk1 = 0;
  auto segment = [&]() -> bool {
    if (item >= sh.hi) return false;
    while ((tile = off / sb.nb) >= a.Hkv / a.hl) {
      sb = seq_blocks(a, ++b, false);
      off = 0;
    }
    blk0 = off - tile * sb.nb;
    blk1 = min(sb.nb, blk0 + sh.hi - item);
    off += blk1 - blk0;
    item += blk1 - blk0;
    return true;
  };
  // Waits of a warp: it goes on or gives up as a whole.
  auto spun = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    return __all_sync(kAll, spin_or_abort(bar, parity, &abort_s, a.err, site, tile, at)) != 0;
  };
  auto waited = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    return __all_sync(kAll, wait_or_abort(bar, parity, &abort_s, a.err, site, tile, at)) != 0;
  };
  bool ok = true;

  if (warp == 5) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      prefetch_tmap(&tmKn);
      prefetch_tmap(&tmVn);
    }
    Ring r;
    int issued = 0;
    while (ok && segment()) {
      const int m = my_heads(a, tile), n = blk1 - blk0;
      int kfirst = -64, kpages = -1, vfirst = -64, vpages = -1;  // 32 page numbers, one a lane, for K and for V
      auto load = [&](int blk, bool value) {
        int& first = value ? vfirst : kfirst;
        int& pages = value ? vpages : kpages;
        int page = -1;
        const bool ctx = blk < sb.np;
        if (ctx) {
          if (blk - first >= 32) {
            first = blk;
            pages = blk + lane < sb.np ? a.table[(int64_t)b * a.width + sb.p0 + blk + lane] : -1;
          }
          page = __shfl_sync(kAll, pages, blk - first);
          if (page < 0 || page >= a.pages) {
            if (page != -1 && !value && lane == 0) flag_bad_index(a.err, page);
            page = (int)a.pages;  // behind the pool: reads zeros
          }
        }
        if (issued >= NS) ok = spun(&bar_empty[r.stage], r.phase ^ 1, kSiteEmpty, blk);
        if (!ok) return;
        if (lane == 0) {
          unsigned char* to = ring + r.stage * C::STAGE;
          tc::mbar_expect_tx(&bar_full[r.stage], C::STAGE);
#pragma unroll
          for (int s = 0; s < SUB; ++s) {
            if (ctx) tc::tma_load_4d(to + s * kTile, value ? &tmV : &tmK, 64 * s, m, 0, page, &bar_full[r.stage]);
            else
              tc::tma_load_4d(to + s * kTile, value ? &tmVn : &tmKn, 64 * s, value ? (a.vn_hs ? m : 0) : (a.kn_hs ? m : 0),
                              (value ? a.vn_ts : a.kn_ts) ? (blk - sb.np) * kChunk : 0,
                              (value ? a.vn_bs : a.kn_bs) ? b : 0, &bar_full[r.stage]);
          }
        }
        __syncwarp();
        ++issued;
        r.next(NS);
      };
      load(blk0, false);
      for (int i = 0; i < n && ok; ++i) {
        if (i + 1 < n) load(blk0 + i + 1, false);
        if (ok) load(blk0 + i, true);
      }
    }
    if (!ok)  // let the copies in flight land before the CTA ends
      for (int i = 0; i < min(issued, NS); ++i) {
        r.stage = (r.stage + NS - 1) % NS;
        if (r.stage == NS - 1) r.phase ^= 1;
        tc::mbar_wait(&bar_full[r.stage], r.phase, 1u << 16);
      }
  } else if (warp == 4) {
    // ---------------------------------------------------------------- products
    Ring r;
    int seg = 0, nth = 0;  // segments, and blocks, so far
    const uint64_t dQ = tc::desc_km(tc::su32(Qs));
    auto wait_full = [&](int blk) {
      ok = ok && spun(&bar_full[r.stage], r.phase, kSiteFull, blk);
      tc::fence_after();
    };
    auto logits = [&](int blk, int i) {
      wait_full(blk);
      if (!ok) return;
      const uint32_t k = tc::su32(ring + r.stage * C::STAGE);
#pragma unroll
      for (int s = 0; s < SUB; ++s)
        tc::mma4_ss<tc::kKStepKm, tc::kKStepKm>(tS + 64 * (i & 1), dQ + s * (2 * kTile >> 4), tc::desc_km(k + s * kTile), kIdS,
                                                s ? 1u : 0u);
      tc::commit_warp(&bar_empty[r.stage]);
      tc::commit_warp(&bar_s[i & 1]);
      r.next(NS);
    };
    while (ok && segment()) {
      ok = spun(&bar_q, seg & 1, kSiteQ, seg);
      tc::fence_after();
      ++seg;
      if (ok) logits(blk0, nth);
      for (int blk = blk0; blk < blk1 && ok; ++blk, ++nth) {
        if (blk + 1 < blk1) logits(blk + 1, nth + 1);
        if (!ok) break;
        ok = spun(&bar_p[nth & 1], (nth >> 1) & 1, kSiteP, blk);
        if (ok) wait_full(blk);
        if (!ok) break;
        const uint32_t v = tc::su32(ring + r.stage * C::STAGE);
#pragma unroll
        for (int s = 0; s < SUB; ++s)
          tc::mma4_ts<8, 16, 24, tc::kKStepMn>(tO + 64 * s, tS + 64 * (nth & 1), tc::desc_mn(v + s * kTile), kIdPV,
                                               blk > blk0 ? 1u : 0u);
        tc::commit_warp(&bar_empty[r.stage]);
        tc::commit_warp(&bar_o[nth & 1]);
        r.next(NS);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const float sl2 = a.scale * kTreeLog2e;
    const int R = a.T * a.g;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    int nth = 0, tiles_read = 0;  // blocks, and ring tiles, so far
    int slot = 0;
    while (ok && segment()) {
      const int m = my_heads(a, tile), r = rt * kRows + tid, n = blk1 - blk0;
      const bool on = r < R, idle = rt * kRows + 32 * warp >= R;
      int t = 0, h = 0, pos = -1;
      {
        uint4 w[DH / 8];
        if (on) {
          row_of(a, r, m, t, h);
          pos = (int)token_position(a, b, t, sb.len);
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.q) + b * a.q_bs + t * a.q_ts + h * a.q_hs);
#pragma unroll
          for (int u = 0; u < DH / 8; ++u) w[u] = src[u];
        } else {
#pragma unroll
          for (int u = 0; u < DH / 8; ++u) w[u] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < DH / 8; ++u)
          *reinterpret_cast<uint4*>(Qs + (u / 8) * 2 * kTile + swz<128>(tid, u % 8)) = w[u];
      }
      tc::fence_async_smem();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar_q);
      const int far = __reduce_max_sync(kAll, pos);  // of this warp's rows
      float mx = -CUDART_INF_F, l = 0.f;
      auto page_at = [&](int blk) { return blk < sb.np ? a.table[(int64_t)b * a.width + sb.p0 + blk] : 0; };
      int page = page_at(blk0);
      for (int blk = blk0; blk < blk1 && ok; ++blk, ++nth) {
        const bool ctx = blk < sb.np;
        const int j0 = ctx ? (sb.p0 + blk) * kChunk : (blk - sb.np) * kChunk;
        // Keys lo .. hi - 1 of the block exist.
        int lo = 0, hi = min(kChunk, (ctx ? sb.len : a.T) - j0);
        if (ctx && a.window > 0) lo = max(0, sb.len - a.window + 1 - j0);
        if (ctx && (page < 0 || page >= a.pages)) hi = 0;
        const int next_page = blk + 1 < blk1 ? page_at(blk + 1) : 0;
        const bool edge = !ctx || lo > 0 || hi < kChunk;
        uint64_t see = ~0ull, real = ~0ull;  // keys that this row sees; draft tokens that are not padding
        auto draft_word = [&](int x) {       // of the draft's tokens in this block, those in row x's mask
          if (a.mask) return a.mask[((int64_t)b * a.T + x) * a.words + blk - sb.np];
          return (uint64_t)(x - j0 >= 63 ? ~0ull : (x < j0 ? 0ull : (2ull << (x - j0)) - 1));
        };
        if (edge || (a.window > 0 && j0 <= far - a.window)) {
          int c0 = lo;
          if (ctx && a.window > 0) c0 = max(c0, pos - a.window + 1 - j0);
          c0 = min(c0, kChunk);
          see = c0 >= hi ? 0ull : ((hi == 64 ? ~0ull : (1ull << hi) - 1) & ~((c0 == 64 ? 0ull : 1ull << c0) - 1));
          if (c0 == 64) see = 0;
          if (!ctx) {
            if (a.positions) {
              const int32_t* p = a.positions + (int64_t)b * a.T;
              const uint32_t p0 = __ballot_sync(kAll, j0 + lane < a.T && p[min(j0 + lane, a.T - 1)] >= 0);
              const uint32_t p1 = __ballot_sync(kAll, j0 + 32 + lane < a.T && p[min(j0 + 32 + lane, a.T - 1)] >= 0);
              real = ((uint64_t)p1 << 32) | p0;
            }
            uint64_t word = 0;
            if (pos >= 0) {
              word = draft_word(t) & see & real;
              if (a.window > 0 && pos - a.window >= sb.len)  // the window ends inside the draft
                for (int u = 0; u < kChunk; ++u)
                  if ((word >> u) & 1 && token_position(a, b, j0 + u, sb.len) <= (int64_t)pos - a.window) word &= ~(1ull << u);
            }
            see = word;
          }
        }
        if (edge) {
          // V's rows that no row of the tile sees become zeros.
          uint64_t used = hi == 64 ? ~0ull : (1ull << max(hi, 0)) - 1;
          used &= lo >= 64 ? 0ull : ~((1ull << lo) - 1);
          if (!ctx) {
            uint64_t any = 0;
            for (int x = rt * kRows / a.g + lane; x < min(a.T, (rt * kRows + kRows - 1) / a.g + 1); x += 32)
              if (token_position(a, b, x, sb.len) >= 0) any |= draft_word(x);
            any &= real;
            used &= ((uint64_t)__reduce_or_sync(kAll, (uint32_t)(any >> 32)) << 32) | __reduce_or_sync(kAll, (uint32_t)any);
          }
          const int at = tiles_read + (blk + 1 < blk1 ? 2 + 2 * (blk - blk0) : 2 * n - 1);
          ok = waited(&bar_full[at % NS], (at / NS) & 1, kSiteV, blk);
          const int row = tid >> 1;
          if (ok && !((used >> row) & 1)) {
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(ring + (at % NS) * C::STAGE + s * kTile + row * 128 + (tid & 1) * 64 + u * 16) =
                    make_uint4(0, 0, 0, 0);
          }
          tc::fence_async_smem();
        }
        ok = ok && waited(&bar_s[nth & 1], (nth >> 1) & 1, kSiteS, blk);
        if (!ok) break;
        page = next_page;
        if (idle) {  // no row of this warp exists: what P holds for them goes nowhere
          if (lane == 0) tc::mbar_arrive(&bar_p[nth & 1]);
          continue;
        }
        tc::fence_after();
        const uint32_t tP = tS + 64 * (nth & 1) + lanes;
        float s[2][32];
        tc::ld32x32b_x32(tP, s[0]);
        tc::ld32x32b_x32(tP + 32, s[1]);
        tc::ld_wait_row(s[0]);
        tc::ld_wait_row(s[1]);
        if (see != ~0ull) {
          const uint32_t w[2] = {(uint32_t)see, (uint32_t)(see >> 32)};
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((w[q] >> i) & 1)) s[q][i] = -CUDART_INF_F;
        }
        float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 32; i += 2) tops[(i >> 1) & 3] = tc::max3(tops[(i >> 1) & 3], s[q][i], s[q][i + 1]);
        const float top = fmaxf(tc::max3(tops[0], tops[1], tops[2]), tops[3]);
        const bool grow = (top - mx) * sl2 > kGrow || (mx == -CUDART_INF_F && top > mx);
        if (__any_sync(kAll, grow)) {
          const float now = grow ? top : mx;
          const float f = now == -CUDART_INF_F ? 1.f : tc::ex2((mx - now) * sl2);
          mx = now;
          l *= f;
          if (blk > blk0) {
            ok = waited(&bar_o[(nth - 1) & 1], ((nth - 1) >> 1) & 1, kSiteO, blk);
            tc::fence_after();
#pragma unroll
            for (int q = 0; q < DH / 32; ++q) {
              float o[32];
              tc::ld32x32b_x32(tO + lanes + 32 * q, o);
              tc::ld_wait_row(o);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[8 * i + e] * f);
                tc::st32x32b_x8(tO + lanes + 32 * q + 8 * i, w);
              }
            }
          }
        }
        const float base = mx == -CUDART_INF_F ? 0.f : -mx * sl2;
        const uint64_t k2 = tc::f2(sl2, sl2), b2 = tc::f2(base, base);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x, y;
              tc::uf2(tc::fma2(tc::f2(s[q][8 * i + 2 * e], s[q][8 * i + 2 * e + 1]), k2, b2), x, y);
              x = tc::ex2(x);
              y = tc::ex2(y);
              sum[e & 1] = tc::add2(sum[e & 1], tc::f2(x, y));
              w[e] = pack_bf16(x, y);
            }
            tc::st32x32b_x4(tP + 16 * q + 4 * i, w);
          }
        float x0, x1, x2, x3;
        tc::uf2(sum[0], x0, x1);
        tc::uf2(sum[1], x2, x3);
        l += (x0 + x1) + (x2 + x3);
        tc::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar_p[nth & 1]);
      }
      tiles_read += 2 * n;
      if (!ok) break;
      ok = waited(&bar_o[(nth - 1) & 1], ((nth - 1) >> 1) & 1, kSiteO, -1);
      if (!ok) break;
      tc::fence_after();
      if (pos < 0) l = 0.f;
      const bool whole = blk0 == 0 && blk1 == sb.nb;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t at = ((int64_t)b * a.T + t) * a.H + h;
      const Part part = part_of(a, blockIdx.x, slot);
#pragma unroll
      for (int q = 0; q < DH / 32; ++q) {
        float o[32];
        tc::ld32x32b_x32(tO + lanes + 32 * q, o);
        tc::ld_wait_row(o);
        if (!on) continue;
        if (whole) {
          uint4* to = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.o) + at * DH + 32 * q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = l == 0.f ? 0u : pack_bf16(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv);
            to[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* to = reinterpret_cast<float4*>(part.o + (int64_t)tid * DH + 32 * q);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[i] = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (on) {
        if (whole) {
          a.lse[at] = l == 0.f ? -CUDART_INF_F : mx * a.scale + logf(l);
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
    tc::tmem_dealloc(tmem_slot, 256);
  }
}

template <int DH>
cudaError_t run_tc(const TreeArgs& a, cudaStream_t s) {
  CUtensorMap tk, tv, tkn, tvn;
  cudaError_t e = make_pages_tmap(&tk, a.kp, DH, a.Hkv, a.pages);
  if (e == cudaSuccess) e = make_pages_tmap(&tv, a.vp, DH, a.Hkv, a.pages);
  if (e == cudaSuccess) e = make_draft_tmap(&tkn, a.kn, DH, a.Hkv, a.T, a.B, a.kn_hs, a.kn_ts, a.kn_bs);
  if (e == cudaSuccess) e = make_draft_tmap(&tvn, a.vn, DH, a.Hkv, a.T, a.B, a.vn_hs, a.vn_ts, a.vn_bs);
  if (e == cudaSuccess) e = allow_smem((const void*)tree_tc_kernel<DH>, Tc<DH>::SMEM);
  if (e != cudaSuccess) return e;
  launch_begin("tree_tc", s);
  tree_tc_kernel<DH><<<a.grid * a.hl * a.nrt, kThreads, Tc<DH>::SMEM, s>>>(a, tk, tv, tkn, tvn);
  return launch_end("tree_tc", s);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t s) { return a.dh == 64 ? run_tc<64>(a, s) : run_tc<128>(a, s); }

}  // namespace gca
