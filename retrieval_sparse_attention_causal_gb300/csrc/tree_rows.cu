// Attention of drafted tokens over a paged cache where there is little to read (single tokens,
// short drafts, short contexts and windows; and all drafts of heads of 32), bf16, without shared
// memory on the way.
//
// Bound by memory: 16 rows ask 16 operations of each byte of K and V, a twentieth of what
// the tensor pipes of mma.sync give.  So the keys and values go straight from global memory
// to the registers that the products read, and nothing waits at a barrier:
//   * mma m16n8k16 takes the contraction in any order, as long as both operands agree.  A
//     thread of the B operand of S = Q K^T owns one key and four values of each step of 16;
//     here those are 16 consecutive values of the key's row (one 32-byte load), and Q is laid
//     out to match.  A warp's load covers whole 128-byte rows.
//   * for O = P V a thread owns one column of each block of 8 and four keys of each step of
//     16; the columns may be in any order too, so block i's column n stands for element
//     (dh / 8) n + i, and a thread's columns of all blocks are consecutive values of a row.
//     Pairs of keys are put together by byte permutation.
// Each warp walks its own units of 4 KB of K and 4 KB of V with its own running maximum and
// sum, and asks for the next unit's keys and values as soon as the products have read the
// registers they land in.  The four warps of a CTA take 4, 2 or 1 key heads side by side
// (which lie next to each other in a token's row, so that DRAM sees longer runs) and share
// the units of a head; the warps of one head join their results in shared memory once per
// tile.
//
// Such calls are bound by latency.  One token of 12 heads over 4000 tokens: 10.0 us, of which 1.8 are
// the bytes' at DRAM's rate: about 2 us of launches, 1.1 to the share, 0.8 to the queries, 2.5 for one
// block, 0.7 for the results, 2.6 for the join.  64 single tokens with a window of 512: 27.7 us (3.6
// TB/s).  Tried and slower or equal: one copy of the loop's code (28.8 us there), the partial
// results written by all rows' threads (28.6).
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"
#include "tree_sched.cuh"

namespace gca {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 128, kWarps = 4;
template <int DH> constexpr int kCtas = DH == 32 ? 3 : 2;  // on an SM
constexpr uint32_t kAll = 0xffffffffu;

// Off the loop's path (inlined it cost 64 single tokens over 600 0.8 of 31 us).
__device__ __noinline__ uint64_t in_window(const int32_t* at, int len, int first, uint64_t word, int low) {
  return draft_above(at, len, first, word, low);
}

template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t* r, const void* p, bool wide) {
  if constexpr (WORDS == 8) {
    if (!wide) {
      load_words<4>(r, p, false);
      load_words<4>(r + 4, static_cast<const char*>(p) + 16, false);
      return;
    }
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
  } else if constexpr (WORDS == 4) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
  }
}

template <int DH>
struct Geo {
  static constexpr int KB = 2048 / DH;     // keys of a unit
  static constexpr int NB = KB / 8;        // blocks of 8 keys
  static constexpr int KS = DH / 16;       // steps of the contraction of S
  static constexpr int ST = KB / 16;       // steps of the contraction of P V
  static constexpr int VW = DH / 16;       // 32-bit words of a thread's part of a V row
  static constexpr int UPB = kChunk / KB;  // units of a block of 64 keys
};

// A unit's addresses and the keys of it that exist.
struct UnitAt {
  const bf16 *k, *v;
  int64_t kts, vts;
  int lim;     // largest row that may be read
  int lo, hi;  // keys lo .. hi - 1 exist
  int j0;      // index of its first key, in the context or in the draft
  bool ctx;
  bool wide;   // rows on 32-byte boundaries
};

template <int DH>
struct UnitData {
  uint32_t k[Geo<DH>::NB][DH / 8];
  uint32_t v[Geo<DH>::ST][4][Geo<DH>::VW];
};

// K row of thread (n, c) of block j: words of the elements 16 c .. 16 c + 15 of each 64.
template <int DH>
__device__ __forceinline__ void load_key_row(uint32_t (&r)[DH / 8], const bf16* row, int c, bool wide) {
  if constexpr (DH == 32) {
    load_words<4>(r, row + 8 * c, false);
  } else {
#pragma unroll
    for (int i = 0; i < DH / 64; ++i) load_words<8>(r + 8 * i, row + 64 * i + 16 * c, wide);
  }
}

template <int DH>
__device__ __forceinline__ void load_keys(UnitData<DH>& d, const UnitAt& u, int lane) {
#pragma unroll
  for (int j = 0; j < Geo<DH>::NB; ++j)
    load_key_row<DH>(d.k[j], u.k + min(8 * j + (lane >> 2), u.lim) * u.kts, lane & 3, u.wide);
}
template <int DH>
__device__ __forceinline__ void load_values(UnitData<DH>& d, const UnitAt& u, int lane) {
  using G = Geo<DH>;
#pragma unroll
  for (int t = 0; t < G::ST; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 16 * t + 2 * (lane & 3) + (e & 1) + 8 * (e >> 1);
      load_words<G::VW>(d.v[t][e], u.v + min(r, u.lim) * u.vts + (DH / 8) * (lane >> 2), u.wide);
    }
}

template <int DH>
__global__ void __launch_bounds__(kThreads, kCtas<DH>) tree_rows_kernel(TreeArgs a) {
  using G = Geo<DH>;
  constexpr int NV = DH / 8;  // output blocks of 8 columns
  __shared__ float join_m[kWarps][16], join_l[kWarps][16];
  // Q fragments of the CTA's heads while the keys are walked, the warps' outputs after that.
  __shared__ __align__(16) unsigned char both[sizeof(float) * kWarps * 16 * (DH + 4)];
  float (*join_o)[16][DH + 4] = reinterpret_cast<float (*)[16][DH + 4]>(both);
  uint4 (*q_s)[G::KS][32] = reinterpret_cast<uint4 (*)[G::KS][32]>(both);
  static_assert(kWarps * G::KS * 32 * sizeof(uint4) <= sizeof both, "");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, c = lane & 3;
  let_next();
  const Share sh = my_share(a);
  if (sh.lo >= sh.hi) return;
  const float sl2 = a.scale * kTreeLog2e;
  const int rt = my_rows(a), R = a.T * a.g - 16 * rt;  // rows from this CTA's first on
  Walk walk(a, sh);
  const SeqBlocks& sb = walk.sb;
  const int &b = walk.b, &tile = walk.tile, &blk0 = walk.blk0, &blk1 = walk.blk1;
  int slot = 0;
  while (walk.next(a)) {
    const int m = my_heads(a, tile) + warp % a.hw;  // this warp's key head
    // Q fragments, and the two rows' positions and masks.
    uint32_t qf[G::KS][4];
    int pos[2], tok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = n + 8 * i;
      uint32_t w[DH / 8] = {};
      pos[i] = -1;
      tok[i] = 0;
      if (r < R) {
        int t, h;
        row_of(a, 16 * rt + r, m, t, h);
        load_key_row<DH>(w, reinterpret_cast<const bf16*>(a.q) + b * a.q_bs + t * a.q_ts + h * a.q_hs, c, false);
        pos[i] = (int)token_position(a, b, t, sb.len);
        tok[i] = t;
      }
#pragma unroll
      for (int ks = 0; ks < G::KS; ++ks) {
        qf[ks][i] = w[2 * ks];
        qf[ks][2 + i] = w[2 * ks + 1];
      }
    }
    if (warp < a.hw)
#pragma unroll
      for (int ks = 0; ks < G::KS; ++ks) q_s[warp][ks][lane] = make_uint4(qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3]);
    __syncthreads();
    int far = max(pos[0], pos[1]);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) far = max(far, __shfl_xor_sync(kAll, far, d));

    float mx[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f}, o[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    // The page numbers of 32 blocks at a time, one a lane, and the next 32.
    int tb = 0, tcur = -1, tnext = -1;
    auto table_at = [&](int first) {
      const int x = first + lane;
      return x < sb.np ? a.table[(int64_t)b * a.width + sb.p0 + x] : -1;
    };
    auto locate = [&](int x) {
      UnitAt u;
      const int blk = x / G::UPB, k0 = (x % G::UPB) * G::KB;
      u.ctx = blk < sb.np;
      if (u.ctx) {
        if (blk - tb >= 32) {
          tb += 32;
          tcur = tnext;
          tnext = table_at(tb + 32);
        }
        int page = __shfl_sync(kAll, tcur, blk - tb);
        u.j0 = (sb.p0 + blk) * kChunk + k0;
        u.lo = a.window > 0 ? max(0, sb.len - a.window + 1 - u.j0) : 0;
        u.hi = min(G::KB, sb.len - u.j0);
        if (page < 0 || page >= a.pages) {
          if (page != -1 && lane == 0) flag_bad_index(a.err, page);
          page = 0;
          u.hi = 0;
        }
        const int64_t at = (((int64_t)page * kChunk + k0) * a.Hkv + m) * DH;
        u.k = reinterpret_cast<const bf16*>(a.kp) + at;
        u.v = reinterpret_cast<const bf16*>(a.vp) + at;
        u.kts = u.vts = (int64_t)a.Hkv * DH;
        u.lim = G::KB - 1;
        u.wide = a.wide;
      } else {
        u.j0 = (blk - sb.np) * kChunk + k0;
        u.lo = 0;
        u.hi = min(G::KB, a.T - u.j0);
        const int first = min(u.j0, a.T - 1);
        u.lim = min(G::KB - 1, a.T - 1 - first);
        u.k = reinterpret_cast<const bf16*>(a.kn) + b * a.kn_bs + first * a.kn_ts + m * a.kn_hs;
        u.v = reinterpret_cast<const bf16*>(a.vn) + b * a.vn_bs + first * a.vn_ts + m * a.vn_hs;
        u.kts = a.kn_ts;
        u.vts = a.vn_ts;
        u.wide = false;
      }
      return u;
    };
    auto logits = [&](const UnitData<DH>& d, float (&s)[G::NB][4]) {
#pragma unroll
      for (int j = 0; j < G::NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < G::KS; ++ks) {
        const uint4 w = q_s[warp % a.hw][ks][lane];
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < G::NB; ++j) mma_bf16(s[j], q, d.k[j][2 * ks], d.k[j][2 * ks + 1]);
      }
    };
    auto weigh = [&](UnitData<DH>& d, float (&s)[G::NB][4], const UnitAt& u) {
      if (!u.ctx || u.lo > 0 || u.hi < G::KB || (a.window > 0 && u.j0 <= far - a.window)) {
        // Bit k of see[i]: row i of this thread sees key k; of used: some row of the CTA may.
        uint64_t see[2], used;
        const uint64_t there = (u.hi >= 64 ? ~0ull : (1ull << max(u.hi, 0)) - 1) & ~((u.lo >= 64 ? 0ull : 1ull << u.lo) - 1);
        if (u.ctx) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int gone = a.window > 0 ? pos[i] - a.window + 1 - u.j0 : 0;  // keys that the window has passed
            see[i] = pos[i] < 0 || u.lo >= 64 || gone >= 64 ? 0ull : there & ~((1ull << max(gone, 0)) - 1);
          }
        } else {
          uint64_t real = ~0ull;  // tokens that are not padding
          if (a.positions) {
            const int32_t* p = a.positions + (int64_t)b * a.T;
            const uint32_t p0 = __ballot_sync(kAll, p[min(u.j0 + lane, a.T - 1)] >= 0);
            const uint32_t p1 = G::KB > 32 ? __ballot_sync(kAll, p[min(u.j0 + 32 + lane, a.T - 1)] >= 0) : 0;
            real = ((uint64_t)p1 << 32) | p0;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            see[i] = 0;
            if (pos[i] < 0) continue;
            see[i] = draft_word(a, b, tok[i], u.j0 >> 6) >> (u.j0 & 63) & there & real;
            if (a.window > 0 && pos[i] - a.window >= sb.len)  // the window ends inside the draft
              see[i] = in_window(a.positions ? a.positions + (int64_t)b * a.T : nullptr, sb.len, u.j0, see[i], pos[i] - a.window);
          }
        }
        used = see[0] | see[1];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) used |= __shfl_xor_sync(kAll, used, d);
#pragma unroll
        for (int j = 0; j < G::NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((see[e >> 1] >> (8 * j + 2 * c + (e & 1))) & 1)) s[j][e] = -CUDART_INF_F;
        // What nobody sees is zeros: a weight of 0 times what lies there must stay 0.
#pragma unroll
        for (int t = 0; t < G::ST; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((used >> (16 * t + 2 * c + (e & 1) + 8 * (e >> 1))) & 1))
#pragma unroll
              for (int w = 0; w < G::VW; ++w) d.v[t][e][w] = 0;
      }
      float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int j = 0; j < G::NB; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) top[i] = fmaxf(top[i], fmaxf(s[j][2 * i], s[j][2 * i + 1]));
      float base[2], f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 2));
        const float now = fmaxf(mx[i], top[i]);
        f[i] = now == -CUDART_INF_F ? 1.f : tc::ex2((mx[i] - now) * sl2);
        base[i] = now == -CUDART_INF_F ? 0.f : -now * sl2;
        mx[i] = now;
      }
      if (__any_sync(kAll, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          o[i][0] *= f[0];
          o[i][1] *= f[0];
          o[i][2] *= f[1];
          o[i][3] *= f[1];
        }
        l[0] *= f[0];
        l[1] *= f[1];
      }
#pragma unroll
      for (int t = 0; t < G::ST; ++t) {
        uint32_t p[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float (&x)[4] = s[2 * t + q];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = tc::ex2(fmaf(x[e], sl2, base[e >> 1]));
          l[0] += x[0] + x[1];
          l[1] += x[2] + x[3];
          p[2 * q] = pack_bf16(x[0], x[1]);
          p[2 * q + 1] = pack_bf16(x[2], x[3]);
        }
#pragma unroll
        for (int w = 0; w < G::VW; ++w) {
          mma_bf16(o[2 * w], p, __byte_perm(d.v[t][0][w], d.v[t][1][w], 0x5410), __byte_perm(d.v[t][2][w], d.v[t][3][w], 0x5410));
          mma_bf16(o[2 * w + 1], p, __byte_perm(d.v[t][0][w], d.v[t][1][w], 0x7632),
                   __byte_perm(d.v[t][2][w], d.v[t][3][w], 0x7632));
        }
      }
    };

    const int x1 = blk1 * G::UPB;
    const int step = kWarps / a.hw;
    int x = blk0 * G::UPB + warp / a.hw;
    tb = x / G::UPB;
    tcur = table_at(tb);
    tnext = table_at(tb + 32);
    if (x < x1) {
      UnitData<DH> d;
      UnitAt u = locate(x);
      load_keys<DH>(d, u, lane);
      load_values<DH>(d, u, lane);
      for (;;) {
        float s[G::NB][4];
        logits(d, s);
        x += step;
        UnitAt next = u;
        if (x < x1) {  // K's registers are free: the next unit's keys
          next = locate(x);
          load_keys<DH>(d, next, lane);
        }
        weigh(d, s, u);
        if (x >= x1) break;
        load_values<DH>(d, next, lane);
        u = next;
      }
    }

    __syncthreads();  // Q is read
    // The four warps' results.  Block i's column q stands for element (dh / 8) q + i.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(kAll, l[i], 1);
      l[i] += __shfl_xor_sync(kAll, l[i], 2);
      const int r = n + 8 * i;
      if (r >= R) continue;
      if (c == 0) {
        join_m[warp][r] = pos[i] < 0 ? -CUDART_INF_F : mx[i] * sl2;
        join_l[warp][r] = pos[i] < 0 ? 0.f : l[i];
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < NV; e += 4)
          *reinterpret_cast<float4*>(&join_o[warp][r][NV * (2 * c + q) + e]) =
              make_float4(o[e][2 * i + q], o[e + 1][2 * i + q], o[e + 2][2 * i + q], o[e + 3][2 * i + q]);
    }
    __syncthreads();
    const int there = min(R, 16);  // rows
    for (int task = tid; task < a.hw * there * 8; task += kThreads) {
      const int row = task >> 3, i = row / there, r = row - i * there, d0 = (task & 7) * NV, m = my_heads(a, tile) + i;
      float top = -CUDART_INF_F;
      for (int w = i; w < kWarps; w += a.hw) top = fmaxf(top, join_m[w][r]);
      float sum = 0.f, out[NV];
#pragma unroll
      for (int e = 0; e < NV; ++e) out[e] = 0.f;
      for (int w = i; w < kWarps; w += a.hw) {
        if (join_l[w][r] == 0.f) continue;  // saw nothing (or padding)
        const float f = tc::ex2(join_m[w][r] - top);
        sum = fmaf(join_l[w][r], f, sum);
#pragma unroll
        for (int e = 0; e < NV; ++e) out[e] = fmaf(join_o[w][r][d0 + e], f, out[e]);
      }
      if (blk0 == 0 && blk1 == sb.nb) {
        int t, h;
        row_of(a, 16 * rt + r, m, t, h);
        const int64_t at = ((int64_t)b * a.T + t) * a.H + h;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (d0 == 0) a.lse[at] = sum == 0.f ? -CUDART_INF_F : top * kTreeLn2 + logf(sum);
        uint32_t w[NV / 2];
#pragma unroll
        for (int e = 0; e < NV / 2; ++e) w[e] = pack_bf16(out[2 * e] * inv, out[2 * e + 1] * inv);
        uint32_t* to = reinterpret_cast<uint32_t*>(reinterpret_cast<bf16*>(a.o) + at * DH + d0);
#pragma unroll
        for (int e = 0; e < NV / 2; e += 2) *reinterpret_cast<uint2*>(to + e) = make_uint2(w[e], w[e + 1]);
      } else {
        const Part part = part_of(a, blockIdx.x, slot);
        const int at = i * a.rows + r;
        if (d0 == 0) {
          part.m[at] = top;
          part.l[at] = sum;
        }
#pragma unroll
        for (int e = 0; e < NV; e += 4)
          *reinterpret_cast<float4*>(part.at(at, d0 + e)) = make_float4(out[e], out[e + 1], out[e + 2], out[e + 3]);
      }
    }
    __syncthreads();  // join_* are free again
    slot = 1;
  }
}

}  // namespace

cudaError_t launch_tree_rows(const TreeArgs& a, cudaStream_t s) {
  launch_begin("tree_rows", s);
  if (a.dh == 32) tree_rows_kernel<32><<<a.grid * a.hl * a.nrt, kThreads, 0, s>>>(a);
  else if (a.dh == 64) tree_rows_kernel<64><<<a.grid * a.hl * a.nrt, kThreads, 0, s>>>(a);
  else tree_rows_kernel<128><<<a.grid * a.hl * a.nrt, kThreads, 0, s>>>(a);
  return launch_end("tree_rows", s);
}

}  // namespace gca
