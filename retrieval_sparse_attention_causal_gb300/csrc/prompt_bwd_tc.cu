// Gradients of the attention over packed sequences, bf16, on the 5th-generation tensor cores.
//
// Two passes without atomics, as in window_bwd.cu: the queries' side (dQ) walks the keys that a tile of
// 128 rows sees, the keys' side (dK, dV) the rows that see a tile of 128 keys, of all heads that share it.
// Each computes the logits and <dO, V> anew: 3 and 4 products of 128 x 128 x dh a pair of tiles, 7 where
// the gradients themselves need 5.  Both are persistent, a CTA an SM: one warp loads, one issues the
// products, eight warps do the arithmetic, a row (TMEM lane) and 64 columns a thread.
//   * Queries' side: S = Q K^T and dP = dO V^T of the next block are issued as soon as this one's are in
//     registers; dS goes to one of two buffers as the A operand of dQ += dS K.
//   * Keys' side: S^T = K Q^T, dP^T = V dO^T; P^T and dS^T take the columns that they came from as the A
//     operands of dV += P^T dO and dK += dS^T Q.  The products go in the order dV(x), S^T(x + 1), dK(x),
//     dP^T(x + 1), so each follows only the one that read the columns it overwrites, and the weights of
//     x + 1 are computed while dK(x) and dP^T(x + 1) run.
// P and dS are rounded to bf16, the type of the products' other operands (half a step, 2^-8 of each).
// Rows behind a sequence's end may hold anything: as operands that are summed over they become zeros in
// shared memory, elsewhere their results are not used.
#include <algorithm>

#include "prompt.cuh"
#include "tc.cuh"
#include "tc_rows.cuh"
#include "waits.cuh"

namespace gca {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kT = 128;             // rows, and keys, of a tile
constexpr int kElem = 8;            // warps that do the arithmetic
constexpr int kThreads = 32 * (kElem + 2);
constexpr int kTile = kT * 128;     // bytes of 128 rows x 64 elements
constexpr uint32_t kCols = 512;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
enum { kSiteFull = 1, kSiteEmpty, kSiteTile, kSiteTileFree, kSiteS, kSiteP, kSiteTaken, kSiteDs, kSiteAcc, kSiteAccFree, kSiteRows };

__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* abort_flag, ErrWord* err, int site, int tile, int at) {
  return __all_sync(kAll, park_or_abort(bar, parity, abort_flag, err, site, tile, at)) != 0;
}

template <int DH>
struct Tc {
  static constexpr int SUB = DH / 64;                   // 64-element parts of a head
  static constexpr int BLOCK = kTile * SUB;             // 128 rows of a head
  static constexpr int NB = DH == 64 ? 2 : 1;           // buffers of the tile that stays (Q and dO, or K and V)
  static constexpr int NS = DH == 64 ? 4 : 2;           // stages of what is walked
  static constexpr int SMEM = 1024 + NB * 2 * BLOCK + NS * (2 * BLOCK + 2 * kT * 4);  // a stage: two operands, the rows' two sums
};

// Shared memory and barriers of a CTA, the same for both passes.
template <int DH>
struct Shared {
  uint64_t full[Tc<DH>::NS], empty[Tc<DH>::NS];  // stages
  uint64_t tile[2], tile_free[2];                // the tile that stays
  uint64_t s, dp, p, ds, acc, acc_free;
  uint32_t tmem;
  int abort;
};

template <int DH>
__device__ __forceinline__ void set_up(Shared<DH>& sh) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < Tc<DH>::NS; ++i) {
      tc::mbar_init(&sh.full[i], 1);
      tc::mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.tile[i], 1);
      tc::mbar_init(&sh.tile_free[i], 1);
    }
    tc::mbar_init(&sh.s, 1);
    tc::mbar_init(&sh.dp, 1);
    tc::mbar_init(&sh.p, kElem);
    tc::mbar_init(&sh.ds, kElem);
    tc::mbar_init(&sh.acc, 1);
    tc::mbar_init(&sh.acc_free, kElem);
    sh.abort = 0;
    tc::fence_mbar_init();
  }
  if (threadIdx.x / 32 == kElem) tc::tmem_alloc(&sh.tmem, kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
}

// Rows `have` .. 127 of a block in shared memory become zeros; called by 128 threads, r the thread's row.
template <int DH>
__device__ __forceinline__ void blank(unsigned char* block, int r, int have) {
  if (r < have) return;
#pragma unroll
  for (int s = 0; s < Tc<DH>::SUB; ++s)
#pragma unroll
    for (int u = 0; u < 8; ++u) *reinterpret_cast<uint4*>(block + s * kTile + r * 128 + u * 16) = make_uint4(0, 0, 0, 0);
}

// D[128 x 128] = A B^T of two K-major blocks.
template <int DH>
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int s = 0; s < Tc<DH>::SUB; ++s)
    tc::mma4_ss<tc::kKStepKm, tc::kKStepKm>(d, tc::desc_km(a + s * kTile), tc::desc_km(b + s * kTile), tc::idesc_bf16(kT, kT, false), s ? 1u : 0u);
}
// D[128 x DH] (+)= A B with A [128 x 128] in TMEM (64 columns at a0, 64 at a1) and B [128 x DH] in shared memory.
template <int DH>
__device__ __forceinline__ void accumulate(uint32_t d, uint32_t a0, uint32_t a1, uint32_t b, bool add) {
#pragma unroll
  for (int s = 0; s < Tc<DH>::SUB; ++s) {
    tc::mma4_ts<8, 16, 24, tc::kKStepMn>(d + 64 * s, a0, tc::desc_mn(b + s * kTile), tc::idesc_bf16(kT, 64, true), add ? 1u : 0u);
    tc::mma4_ts<8, 16, 24, tc::kKStepMn>(d + 64 * s, a1, tc::desc_mn(b + s * kTile + kTile / 2), tc::idesc_bf16(kT, 64, true), 1u);
  }
}

// 32 columns of an accumulator's row, scaled, to global memory.
__device__ __forceinline__ void write_row(uint32_t at, bf16* to, float scale, bool on) {
  float o[32];
  tc::ld32x32b_x32(at, o);
  tc::ld_wait_row(o);
  if (!on) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(to + 8 * i) =
        make_uint4(pack_bf16(o[8 * i] * scale, o[8 * i + 1] * scale), pack_bf16(o[8 * i + 2] * scale, o[8 * i + 3] * scale),
                   pack_bf16(o[8 * i + 4] * scale, o[8 * i + 5] * scale), pack_bf16(o[8 * i + 6] * scale, o[8 * i + 7] * scale));
}

struct Maps {
  CUtensorMap q, k, v, g;
};

// Work of the queries' side: a tile of rows of a head, and its blocks lo .. tile of keys.
struct QItem {
  PromptTile x;
  int h, m, lo;
};
__device__ __forceinline__ bool q_item(const PromptArgs& a, int w, QItem& it) {
  it.h = w % a.H;
  it.m = it.h / a.g;
  if (!prompt_tile<kT>(a, w / a.H, false, it.x)) return false;
  it.lo = a.window ? max(0, it.x.tile * kT - a.window + 1) / kT : 0;
  return true;
}

// ------------------------------------------------------------------ the queries' side
template <int DH>
__global__ void __launch_bounds__(kThreads, 1) prompt_dq_tc_kernel(PromptArgs a, const __grid_constant__ Maps tm) {
  using C = Tc<DH>;
  constexpr int NS = C::NS, NB = C::NB, SUB = C::SUB;
  extern __shared__ unsigned char dsm[];
  unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = tiles + NB * 2 * C::BLOCK;
  __shared__ __align__(8) Shared<DH> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  set_up<DH>(sh);
  const uint32_t tS = sh.tmem, tP = tS + 128, tD = tS + 256, tQ = tS + 384;  // S, dP, two buffers of dS, dQ
  bool ok = true;
  auto waited = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    if (__builtin_expect(__all_sync(kAll, tc::mbar_try(bar, parity)), 1)) return true;
    return wait_on(bar, parity, &sh.abort, a.err, site, blockIdx.x, at);
  };
  QItem it;

  if (warp == kElem + 1) {
    // ---------------------------------------------------------------- loads
    int id = 0, nt = 0;
    for (int w = blockIdx.x; ok && q_item(a, w, it); w += gridDim.x, ++nt) {
      const int buf = nt % NB;
      ok = waited(&sh.tile_free[buf], ((nt / NB) & 1) ^ 1, kSiteTileFree, w);
      if (!ok) break;
      tc::mbar_expect_tx_warp(&sh.tile[buf], 2 * C::BLOCK);
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        unsigned char* to = tiles + buf * 2 * C::BLOCK + s * kTile;
        tc::tma_load_4d_warp(to, &tm.q, 64 * s, a.q_hs ? it.h : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
        tc::tma_load_4d_warp(to + C::BLOCK, &tm.g, 64 * s, a.do_hs ? it.h : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
      }
      for (int n = it.lo; n <= it.x.tile; ++n, ++id) {
        const int st = id % NS;
        ok = waited(&sh.empty[st], ((id / NS) & 1) ^ 1, kSiteEmpty, n);
        if (!ok) break;
        tc::mbar_expect_tx_warp(&sh.full[st], 2 * C::BLOCK);
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          unsigned char* to = ring + st * 2 * C::BLOCK + s * kTile;
          tc::tma_load_4d_warp(to, &tm.k, 64 * s, a.k_hs ? it.m : 0, it.x.off + n * kT, 0, &sh.full[st]);
          tc::tma_load_4d_warp(to + C::BLOCK, &tm.v, 64 * s, a.v_hs ? it.m : 0, it.x.off + n * kT, 0, &sh.full[st]);
        }
      }
    }
    if (!ok) {  // let the copies in flight land before the CTA ends
      for (int i = max(0, id - NS); i < id; ++i) tc::mbar_wait(&sh.full[i % NS], (i / NS) & 1, 1u << 16);
      for (int i = max(0, nt + 1 - NB); i <= nt; ++i) tc::mbar_wait(&sh.tile[i % NB], (i / NB) & 1, 1u << 16);
    }
  } else if (warp == kElem) {
    // ---------------------------------------------------------------- products
    int id = 0, nt = 0;
    for (int w = blockIdx.x; ok && q_item(a, w, it); w += gridDim.x, ++nt) {
      const int n = it.x.tile - it.lo + 1;
      const uint32_t q = tc::su32(tiles + (nt % NB) * 2 * C::BLOCK), g = q + C::BLOCK;
      ok = waited(&sh.tile[nt % NB], (nt / NB) & 1, kSiteTile, w);
      // Step x: S and dP of block x, and dQ of the block before.
      for (int x = 0; x <= n && ok; ++x) {
        if (x < n) {
          const int i = id + x, st = i % NS;
          ok = waited(&sh.full[st], (i / NS) & 1, kSiteFull, x);
          if (i > 0) ok = ok && waited(&sh.p, (i - 1) & 1, kSiteTaken, x);  // the block before is in registers
          if (!ok) break;
          tc::fence_after();
          const uint32_t k = tc::su32(ring + st * 2 * C::BLOCK);
          product<DH>(tS, q, k);
          product<DH>(tP, g, k + C::BLOCK);
          tc::commit_warp(&sh.s);
          if (x == n - 1) tc::commit_warp(&sh.tile_free[nt % NB]);
        }
        if (x > 0) {
          const int i = id + x - 1, st = i % NS;
          if (x == 1) ok = waited(&sh.acc_free, (nt & 1) ^ 1, kSiteAccFree, x);
          ok = ok && waited(&sh.ds, i & 1, kSiteDs, x);
          if (!ok) break;
          tc::fence_after();
          accumulate<DH>(tQ, tD + 64 * (i & 1), tD + 64 * (i & 1) + 32, tc::su32(ring + st * 2 * C::BLOCK), x > 1);
          tc::commit_warp(&sh.empty[st]);
        }
      }
      if (!ok) break;
      tc::commit_warp(&sh.acc);
      id += n;
    }
  } else {
    // ---------------------------------------------------------------- arithmetic
    const int r = 32 * (warp & 3) + lane, half = warp >> 2;  // row of the tile; columns 64 half ..
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float sl2 = a.scale * kLog2e;
    const uint64_t k2 = tc::f2(sl2, sl2);
    int id = 0, nt = 0;
    for (int w = blockIdx.x; ok && q_item(a, w, it); w += gridDim.x, ++nt) {
      const int pos = it.x.tile * kT + r;
      const bool on = pos < it.x.len;
      const int64_t row = it.h * a.np + prompt_pad(it.x.off, it.x.b) + pos;
      const float nl = on ? a.nlse[row] : -CUDART_INF_F, nd = on ? a.nD[row] : 0.f;  // a row that does not exist weighs nothing
      const uint64_t nl2 = tc::f2(nl, nl), nd2 = tc::f2(nd, nd);
      const int first = a.window ? max(0, pos - a.window + 1) : 0;
      const int whole = a.window ? (max(0, it.x.tile * kT + kT - a.window) + kT - 1) / kT : 0;
      for (int n = it.lo; n <= it.x.tile; ++n, ++id) {
        ok = waited(&sh.s, id & 1, kSiteS, n);
        if (!ok) break;
        tc::fence_after();
        float s[2][32], dp[2][32];
        tc::ld32x32b_x32(tS + lanes + 64 * half, s[0]);
        tc::ld32x32b_x32(tS + lanes + 64 * half + 32, s[1]);
        tc::ld32x32b_x32(tP + lanes + 64 * half, dp[0]);
        tc::ld32x32b_x32(tP + lanes + 64 * half + 32, dp[1]);
        tc::ld_wait_row(s[0]);
        tc::ld_wait_row(s[1]);
        tc::ld_wait_row(dp[0]);
        tc::ld_wait_row(dp[1]);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.p);
        uint32_t d[32];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            tc::uf2(tc::fma2(tc::f2(s[c][2 * i], s[c][2 * i + 1]), k2, nl2), x, y);
            const uint64_t p = tc::f2(tc::ex2(x), tc::ex2(y));
            tc::uf2(tc::mul2(p, tc::add2(tc::f2(dp[c][2 * i], dp[c][2 * i + 1]), nd2)), x, y);
            s[c][2 * i] = x;
            s[c][2 * i + 1] = y;
          }
        if (n == it.x.tile || n < whole) {  // keys that the row does not see, and rows that do not exist
          const int c0 = first - n * kT - 64 * half, c1 = on ? pos - n * kT - 64 * half + 1 : 0;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i < c0 || 32 * c + i >= c1) s[c][i] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) d[16 * c + i] = pack_bf16(s[c][2 * i], s[c][2 * i + 1]);
        if ((n + 1) * kT > it.x.len) {  // rows of K behind the sequence
          ok = waited(&sh.full[id % NS], (id / NS) & 1, kSiteRows, n);
          if (!ok) break;
          if (half == 0) blank<DH>(ring + (id % NS) * 2 * C::BLOCK, r, it.x.len - n * kT);
          tc::fence_async_smem();
        }
        // The buffer's last reader, dQ of two blocks ago, was issued before S(n) and is done.
        const uint32_t to = tD + lanes + 64 * (id & 1) + 32 * half;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x[8] = {d[8 * i], d[8 * i + 1], d[8 * i + 2], d[8 * i + 3], d[8 * i + 4], d[8 * i + 5], d[8 * i + 6], d[8 * i + 7]};
          tc::st32x32b_x8(to + 8 * i, x);
        }
        tc::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.ds);
      }
      if (!ok) break;
      ok = waited(&sh.acc, nt & 1, kSiteAcc, w);
      if (!ok) break;
      tc::fence_after();
      bf16* to = reinterpret_cast<bf16*>(a.dq) + (int64_t)(it.x.off + pos) * a.dq_ts + it.h * a.dq_hs;
#pragma unroll
      for (int c = 0; c < DH / 64; ++c) {
        const int col = half * (DH / 2) + 32 * c;
        if (col < a.dh) write_row(tQ + lanes + col, to + col, a.scale, on);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.acc_free);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kElem) {
    tc::fence_after();
    tc::tmem_dealloc(sh.tmem, kCols);
  }
}

// Work of the keys' side: a tile of keys of a key head; for each of the g heads that share it, the tiles
// tile .. end - 1 of rows.
struct KvItem {
  PromptTile x;
  int m, end;
};
__device__ __forceinline__ bool kv_item(const PromptArgs& a, int w, KvItem& it) {
  it.m = w % a.Hkv;
  if (!prompt_tile<kT>(a, w / a.Hkv, true, it.x)) return false;
  const int k = min(it.x.tile * kT + kT, it.x.len) - 1;  // the tile's last key
  it.end = (a.window ? (int)min((int64_t)it.x.len - 1, (int64_t)k + a.window - 1) : it.x.len - 1) / kT + 1;
  return true;
}

// ------------------------------------------------------------------ the keys' side
template <int DH>
__global__ void __launch_bounds__(kThreads, 1) prompt_dkv_tc_kernel(PromptArgs a, const __grid_constant__ Maps tm) {
  using C = Tc<DH>;
  constexpr int NS = C::NS, NB = C::NB, SUB = C::SUB;
  extern __shared__ unsigned char dsm[];
  unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = tiles + NB * 2 * C::BLOCK;
  float* rows = reinterpret_cast<float*>(ring + NS * 2 * C::BLOCK);  // of each stage: -lse log2(e), -D
  __shared__ __align__(8) Shared<DH> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  set_up<DH>(sh);
  const uint32_t tS = sh.tmem, tP = tS + 128, tV = tS + 256, tK = tV + DH;
  bool ok = true;
  auto waited = [&](uint64_t* bar, uint32_t parity, int site, int at) {
    if (__builtin_expect(__all_sync(kAll, tc::mbar_try(bar, parity)), 1)) return true;
    return wait_on(bar, parity, &sh.abort, a.err, site, blockIdx.x, at);
  };
  KvItem it;

  if (warp == kElem + 1) {
    // ---------------------------------------------------------------- loads
    int id = 0, nt = 0;
    for (int w = blockIdx.x; ok && kv_item(a, w, it); w += gridDim.x, ++nt) {
      const int buf = nt % NB;
      ok = waited(&sh.tile_free[buf], ((nt / NB) & 1) ^ 1, kSiteTileFree, w);
      if (!ok) break;
      tc::mbar_expect_tx_warp(&sh.tile[buf], 2 * C::BLOCK);
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        unsigned char* to = tiles + buf * 2 * C::BLOCK + s * kTile;
        tc::tma_load_4d_warp(to, &tm.k, 64 * s, a.k_hs ? it.m : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
        tc::tma_load_4d_warp(to + C::BLOCK, &tm.v, 64 * s, a.v_hs ? it.m : 0, it.x.off + it.x.tile * kT, 0, &sh.tile[buf]);
      }
      for (int h = it.m * a.g; h < it.m * a.g + a.g && ok; ++h)
        for (int i = it.x.tile; i < it.end; ++i, ++id) {
          const int st = id % NS;
          ok = waited(&sh.empty[st], ((id / NS) & 1) ^ 1, kSiteEmpty, i);
          if (!ok) break;
          tc::mbar_expect_tx_warp(&sh.full[st], 2 * C::BLOCK + 2 * kT * 4);
#pragma unroll
          for (int s = 0; s < SUB; ++s) {
            unsigned char* to = ring + st * 2 * C::BLOCK + s * kTile;
            tc::tma_load_4d_warp(to, &tm.q, 64 * s, a.q_hs ? h : 0, it.x.off + i * kT, 0, &sh.full[st]);
            tc::tma_load_4d_warp(to + C::BLOCK, &tm.g, 64 * s, a.do_hs ? h : 0, it.x.off + i * kT, 0, &sh.full[st]);
          }
          const int64_t row = h * a.np + prompt_pad(it.x.off, it.x.b) + i * kT;
          if (lane == 0) {
            tc::bulk_load(rows + st * 2 * kT, a.nlse + row, kT * 4, &sh.full[st]);
            tc::bulk_load(rows + st * 2 * kT + kT, a.nD + row, kT * 4, &sh.full[st]);
          }
          __syncwarp();
        }
    }
    if (!ok) {
      for (int i = max(0, id - NS); i < id; ++i) tc::mbar_wait(&sh.full[i % NS], (i / NS) & 1, 1u << 16);
      for (int i = max(0, nt + 1 - NB); i <= nt; ++i) tc::mbar_wait(&sh.tile[i % NB], (i / NB) & 1, 1u << 16);
    }
  } else if (warp == kElem) {
    // ---------------------------------------------------------------- products
    int id = 0, nt = 0;
    for (int w = blockIdx.x; ok && kv_item(a, w, it); w += gridDim.x, ++nt) {
      const int n = (it.end - it.x.tile) * a.g;
      const uint32_t k = tc::su32(tiles + (nt % NB) * 2 * C::BLOCK), v = k + C::BLOCK;
      ok = waited(&sh.tile[nt % NB], (nt / NB) & 1, kSiteTile, w);
      for (int x = -1; x < n && ok; ++x) {
        const int i = id + x, st = i % NS, next = (i + 1) % NS;
        const uint32_t q = tc::su32(ring + st * 2 * C::BLOCK), qn = tc::su32(ring + next * 2 * C::BLOCK);
        if (x >= 0) {
          if (x == 0) ok = waited(&sh.acc_free, (nt & 1) ^ 1, kSiteAccFree, x);
          ok = ok && waited(&sh.p, i & 1, kSiteP, x);
          if (!ok) break;
          tc::fence_after();
          accumulate<DH>(tV, tS, tS + 64, q + C::BLOCK, x > 0);
        }
        if (x + 1 < n) {
          ok = waited(&sh.full[next], ((i + 1) / NS) & 1, kSiteFull, x);
          if (!ok) break;
          tc::fence_after();
          product<DH>(tS, k, qn);
          tc::commit_warp(&sh.s);
        }
        if (x >= 0) {
          ok = waited(&sh.ds, i & 1, kSiteDs, x);
          if (!ok) break;
          tc::fence_after();
          accumulate<DH>(tK, tP, tP + 64, q, x > 0);
          tc::commit_warp(&sh.empty[st]);
        }
        if (x + 1 < n) {
          product<DH>(tP, v, qn + C::BLOCK);
          tc::commit_warp(&sh.dp);
        }
      }
      if (!ok) break;
      tc::commit_warp(&sh.tile_free[nt % NB]);
      tc::commit_warp(&sh.acc);
      id += n;
    }
  } else {
    // ---------------------------------------------------------------- arithmetic
    const int r = 32 * (warp & 3) + lane, half = warp >> 2;  // key of the tile; rows 64 half .. of a block
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float sl2 = a.scale * kLog2e;
    const uint64_t k2 = tc::f2(sl2, sl2);
    int id = 0, nt = 0;
    for (int w = blockIdx.x; ok && kv_item(a, w, it); w += gridDim.x, ++nt) {
      const int key = it.x.tile * kT + r;
      for (int h = 0; h < a.g && ok; ++h)
        for (int i = it.x.tile; i < it.end; ++i, ++id) {
          const int st = id % NS, t0 = i * kT + 64 * half;
          ok = waited(&sh.full[st], (id / NS) & 1, kSiteRows, i) && waited(&sh.s, id & 1, kSiteS, i);
          if (!ok) break;
          tc::fence_after();
          // Rows c0 .. c1 - 1 of this half see the key; every row sees every key of blocks inside.
          const bool edge = i == it.x.tile || (i + 1) * kT > it.x.len || (a.window && i * kT + kT - a.window > it.x.tile * kT);
          int c0 = 0, c1 = 64;
          if (edge) {
            c0 = key - t0;
            c1 = it.x.len - t0;
            if (a.window) c1 = (int)min((int64_t)c1, (int64_t)key + a.window - t0);
          }
          float p[2][32];
          tc::ld32x32b_x32(tS + lanes + 64 * half, p[0]);
          tc::ld32x32b_x32(tS + lanes + 64 * half + 32, p[1]);
          if ((i + 1) * kT > it.x.len) {  // rows of Q and dO behind the sequence
            blank<DH>(ring + st * 2 * C::BLOCK + half * C::BLOCK, r, it.x.len - i * kT);
            tc::fence_async_smem();
          }
          const float4* nl = reinterpret_cast<const float4*>(rows + st * 2 * kT + 64 * half);
          const float4* nd = nl + kT / 4;
          tc::ld_wait_row(p[0]);
          tc::ld_wait_row(p[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 l = nl[8 * c + j];
              float x, y, z, u;
              tc::uf2(tc::fma2(tc::f2(p[c][4 * j], p[c][4 * j + 1]), k2, tc::f2(l.x, l.y)), x, y);
              tc::uf2(tc::fma2(tc::f2(p[c][4 * j + 2], p[c][4 * j + 3]), k2, tc::f2(l.z, l.w)), z, u);
              p[c][4 * j] = tc::ex2(x);
              p[c][4 * j + 1] = tc::ex2(y);
              p[c][4 * j + 2] = tc::ex2(z);
              p[c][4 * j + 3] = tc::ex2(u);
            }
          if (edge) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (32 * c + j < c0 || 32 * c + j >= c1) p[c][j] = 0.f;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = pack_bf16(p[c][16 * j + 2 * e], p[c][16 * j + 2 * e + 1]);
              tc::st32x32b_x8(tS + lanes + 64 * half + 16 * c + 8 * j, x);
            }
          tc::st_wait();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.p);
          ok = waited(&sh.dp, id & 1, kSiteDs, i);
          if (!ok) break;
          tc::fence_after();
          float d[2][32];
          tc::ld32x32b_x32(tP + lanes + 64 * half, d[0]);
          tc::ld_wait_row(d[0]);
          tc::ld32x32b_x32(tP + lanes + 64 * half + 32, d[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c == 1) tc::ld_wait_row(d[1]);
            uint32_t x[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 l = nd[8 * c + j];
              float e0, e1, e2, e3;
              tc::uf2(tc::mul2(tc::f2(p[c][4 * j], p[c][4 * j + 1]), tc::add2(tc::f2(d[c][4 * j], d[c][4 * j + 1]), tc::f2(l.x, l.y))), e0, e1);
              tc::uf2(tc::mul2(tc::f2(p[c][4 * j + 2], p[c][4 * j + 3]), tc::add2(tc::f2(d[c][4 * j + 2], d[c][4 * j + 3]), tc::f2(l.z, l.w))), e2, e3);
              if (edge) {  // (what is not seen may be anything, an infinity times 0 too)
                const int at = 32 * c + 4 * j;
                if (at < c0 || at >= c1) e0 = 0.f;
                if (at + 1 < c0 || at + 1 >= c1) e1 = 0.f;
                if (at + 2 < c0 || at + 2 >= c1) e2 = 0.f;
                if (at + 3 < c0 || at + 3 >= c1) e3 = 0.f;
              }
              x[2 * j] = pack_bf16(e0, e1);
              x[2 * j + 1] = pack_bf16(e2, e3);
            }
            const uint32_t x0[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}, x1[8] = {x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15]};
            tc::st32x32b_x8(tP + lanes + 64 * half + 16 * c, x0);  // over columns that have been read
            tc::st32x32b_x8(tP + lanes + 64 * half + 16 * c + 8, x1);
          }
          tc::st_wait();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.ds);
        }
      if (!ok) break;
      ok = waited(&sh.acc, nt & 1, kSiteAcc, w);
      if (!ok) break;
      tc::fence_after();
      const bool on = key < it.x.len;
      bf16* kt = reinterpret_cast<bf16*>(a.dk) + (int64_t)(it.x.off + key) * a.dk_ts + it.m * a.dk_hs;
      bf16* vt = reinterpret_cast<bf16*>(a.dv) + (int64_t)(it.x.off + key) * a.dv_ts + it.m * a.dv_hs;
#pragma unroll
      for (int c = 0; c < DH / 64; ++c) {
        const int col = half * (DH / 2) + 32 * c;
        if (col >= a.dh) break;
        write_row(tV + lanes + col, vt + col, 1.f, on);
        write_row(tK + lanes + col, kt + col, a.scale, on);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.acc_free);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kElem) {
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
  if (e == cudaSuccess) e = allow_smem((const void*)prompt_dq_tc_kernel<DH>, C::SMEM);
  if (e == cudaSuccess) e = allow_smem((const void*)prompt_dkv_tc_kernel<DH>, C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = a.N / kT + std::min<int64_t>(a.B, a.N);
  launch_begin("prompt_dkv_tc", s);
  prompt_dkv_tc_kernel<DH><<<(unsigned)std::min<int64_t>(tiles * a.Hkv, kSMs), kThreads, C::SMEM, s>>>(a, tm);
  e = launch_end("prompt_dkv_tc", s);
  if (e != cudaSuccess) return e;
  launch_begin("prompt_dq_tc", s);
  prompt_dq_tc_kernel<DH><<<(unsigned)std::min<int64_t>(tiles * a.H, kSMs), kThreads, C::SMEM, s>>>(a, tm);
  return launch_end("prompt_dq_tc", s);
}

}  // namespace

cudaError_t launch_prompt_bwd_tc(const PromptArgs& a, cudaStream_t s) { return a.dh <= 64 ? run_tc<64>(a, s) : run_tc<128>(a, s); }

}  // namespace gca
