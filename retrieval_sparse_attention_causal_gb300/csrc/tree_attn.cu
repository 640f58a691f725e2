// Attention of newly drafted tokens over a paged cache, and the plan of a draft's tree.
//
// Row (t, h) of sequence b attends with one softmax to the cache's tokens j < len (page
// table[b][j / 64], row j % 64) and to the draft's tokens u that mask row t names:
//     s = scale <q, k>,  o = sum exp(s - lse) v,  lse = log sum exp(s).
// A window keeps j > pos_t - window and pos_u > pos_t - window.
//
// The keys are walked once with the running maximum and sum of a softmax; the walk is
// divided among the CTAs as tree_sched.cuh says and the partial results are joined by
// tree_join_kernel.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tree_sched.cuh"

namespace gca {
namespace {

using bf16 = __nv_bfloat16;
// ------------------------------------------------------------------ CUDA-core kernel (float32)
// 128 threads; thread (ty, tx) owns rows ty RT .. ty RT + RT - 1, of a block's logits the
// keys tx + 16 j, and of the output DH / 16 columns.  K and V pass through shared memory.
// The path of exact results: products, sums and weights in float32 (a tensor core would round
// its operands).  Bound by the reads of shared memory: five of 16 bytes for 16 products a thread
// where a thread has one row, eight for 64 where it has four; nothing hides a block's load but
// the other CTAs of the SM (four; with two, 12 heads over 64K tokens took 320 us where four took 207).
// Measured: one token of 12 heads over 64K, 192 us (2.1 TB/s); 8 drafts of 16 over 4K, 124 us (10
// TFLOP/s); 64 drafted tokens of 16 and 4 heads over 16K, 143 us (30 TFLOP/s).
constexpr int kSimtThreads = 128;
template <int DH, int RT>
constexpr int simt_smem() { return (8 * RT * (DH + 4) + 2 * 64 * (DH + 4) + 8 * RT * 68) * 4; }

template <int DH, int RT>
__global__ void __launch_bounds__(kSimtThreads) tree_simt_kernel(TreeArgs a) {
  using T = float;
  constexpr int MT = 8 * RT, QS = DH + 4, CV = DH >= 64 ? 4 : 2, NC = DH / 16 / CV;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + MT * QS;
  float* Vs = Ks + 64 * QS;
  float* Ps = Vs + 64 * QS;
  __shared__ int row_pos[MT];
  __shared__ unsigned long long used_s, row_see[MT];
  __shared__ uint32_t real_s[2];
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  let_next();
  const Share sh = my_share(a);
  const float sl2 = a.scale * kTreeLog2e;
  const int R = a.T * a.g, rt = my_rows(a);
  Walk walk(a, sh);
  const SeqBlocks& sb = walk.sb;
  const int &b = walk.b, &tile = walk.tile, &blk0 = walk.blk0, &blk1 = walk.blk1;
  int slot = 0;
  while (walk.next(a)) {
    const int m = my_heads(a, tile);
    const int rows = min(MT, R - rt * MT);
    __syncthreads();
    for (int i = tid; i < MT * DH / 4; i += kSimtThreads) {
      const int r = i / (DH / 4), d = i % (DH / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        int t, h;
        row_of(a, rt * MT + r, m, t, h);
        v = *reinterpret_cast<const float4*>(reinterpret_cast<const T*>(a.q) + b * a.q_bs + t * a.q_ts + h * a.q_hs + d);
      }
      *reinterpret_cast<float4*>(Qs + r * QS + d) = v;
    }
    if (tid < MT) row_pos[tid] = tid < rows ? (int)token_position(a, b, (rt * MT + tid) / a.g, sb.len) : -1;
    float mx[RT], l[RT], o[RT][NC * CV];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      mx[i] = -CUDART_INF_F;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC * CV; ++c) o[i][c] = 0.f;
    }
    int near = INT32_MAX;  // the lowest position of a row
    for (int blk = blk0; blk < blk1; ++blk) {
      const bool ctx = blk < sb.np;
      int lo = 0, hi = 0, j0 = 0;       // keys lo .. hi - 1 of the block, of which j0 is the first's index
      const T *kb = nullptr, *vb = nullptr;
      int64_t kts = (int64_t)a.Hkv * DH, vts = kts;
      if (ctx) {
        j0 = (sb.p0 + blk) * kChunk;
        const int page = a.table[(int64_t)b * a.width + sb.p0 + blk];
        if (page >= 0 && page < a.pages) {
          hi = min(kChunk, sb.len - j0);
          const int64_t at = ((int64_t)page * kChunk * a.Hkv + m) * DH;
          kb = reinterpret_cast<const T*>(a.kp) + at;
          vb = reinterpret_cast<const T*>(a.vp) + at;
        } else if (page != -1 && tid == 0) {
          flag_bad_index(a.err, page);
        }
      } else {
        j0 = (blk - sb.np) * kChunk;
        hi = min(kChunk, a.T - j0);
        kb = reinterpret_cast<const T*>(a.kn) + b * a.kn_bs + j0 * a.kn_ts + m * a.kn_hs;
        vb = reinterpret_cast<const T*>(a.vn) + b * a.vn_bs + j0 * a.vn_ts + m * a.vn_hs;
        kts = a.kn_ts;
        vts = a.vn_ts;
      }
      __syncthreads();  // the last block's readers are done; row_pos is written
      if (a.window > 0 && ctx) {
        if (blk == blk0)
          for (int r = 0; r < MT; ++r)
            if (row_pos[r] >= 0) near = min(near, row_pos[r]);
        lo = min(max(near - a.window + 1 - j0, 0), kChunk);
      }
      // Which keys each row sees, one bit a key; of the draft's, those that any row sees.
      if (!ctx) {
        if (tid < 64) {
          const bool real = j0 + tid < a.T && token_position(a, b, j0 + tid, sb.len) >= 0;
          const uint32_t w = __ballot_sync(0xffffffffu, real);
          if ((tid & 31) == 0) real_s[tid >> 5] = w;
        }
        if (tid == 0) used_s = 0;
        __syncthreads();
      }
      if (tid < MT) {
        const int pos = row_pos[tid];
        unsigned long long see = 0;
        if (pos >= 0) {
          int c0 = lo;
          if (ctx && a.window > 0) c0 = min(max(c0, pos - a.window + 1 - j0), kChunk);
          see = c0 >= hi ? 0ull : (hi == 64 ? ~0ull : (1ull << hi) - 1) & ~((1ull << c0) - 1);
          if (!ctx) {
            const int t = (rt * MT + tid) / a.g;
            see &= ((unsigned long long)real_s[1] << 32) | real_s[0];
            see &= draft_word(a, b, t, j0 >> 6);
            if (a.window > 0 && pos - a.window >= sb.len)  // the window ends inside the draft
              see = draft_above(a.positions ? a.positions + (int64_t)b * a.T : nullptr, sb.len, j0, see, pos - a.window);
            atomicOr(&used_s, see);
          }
        }
        row_see[tid] = see;
      }
      __syncthreads();
      const unsigned long long used = ctx ? ~0ull : used_s;
      // Rows that nobody sees are zeros: a weight of 0 times what lies there must stay 0.
#pragma unroll 4
      for (int i = tid; i < kChunk * DH / 4; i += kSimtThreads) {
        const int r = i / (DH / 4), d = i % (DH / 4) * 4;
        float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
        if (r >= lo && r < hi && ((used >> r) & 1)) {
          kv = *reinterpret_cast<const float4*>(kb + r * kts + d);
          vv = *reinterpret_cast<const float4*>(vb + r * vts + d);
        }
        *reinterpret_cast<float4*>(Ks + r * QS + d) = kv;
        *reinterpret_cast<float4*>(Vs + r * QS + d) = vv;
      }
      __syncthreads();
      float s[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < DH; d += 4) {
        float4 kv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * QS + d);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(Qs + (ty * RT + i) * QS + d);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(qv.x, kv[j].x, fmaf(qv.y, kv[j].y, fmaf(qv.z, kv[j].z, fmaf(qv.w, kv[j].w, s[i][j]))));
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int r = ty * RT + i;
        const unsigned long long see = row_see[r];
        float top = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool on = (see >> (tx + 16 * j)) & 1;
          s[i][j] = on ? s[i][j] * sl2 : -CUDART_INF_F;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float n = fmaxf(mx[i], top), base = n == -CUDART_INF_F ? 0.f : n;
        const float f = exp2f(mx[i] - base);  // 0 while the row has seen nothing
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - base);
          Ps[r * 68 + tx + 16 * j] = p;
          sum += p;
        }
        mx[i] = n;
        l[i] = l[i] * f + sum;  // this thread's keys; summed over tx at the end
#pragma unroll
        for (int c = 0; c < NC * CV; ++c) o[i][c] *= f;
      }
      __syncwarp();  // a row's weights are written and read by one half of one warp
#pragma unroll 4
      for (int k = 0; k < kChunk; ++k) {
        float v[NC * CV];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < CV; ++e) v[c * CV + e] = Vs[k * QS + c * 16 * CV + tx * CV + e];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float p = Ps[(ty * RT + i) * 68 + k];
#pragma unroll
          for (int c = 0; c < NC * CV; ++c) o[i][c] = fmaf(p, v[c], o[i][c]);
        }
      }
    }
    const bool whole = blk0 == 0 && blk1 == sb.nb;
    const Part part = part_of(a, blockIdx.x, slot);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty * RT + i;
      float sum = l[i];
#pragma unroll
      for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (r >= rows) continue;
      if (sum == 0.f)  // the row saw nothing: what was weighed by 0 goes nowhere
#pragma unroll
        for (int c = 0; c < NC * CV; ++c) o[i][c] = 0.f;
      if (whole) {
        int t, h;
        row_of(a, rt * MT + r, m, t, h);
        const int64_t at = ((int64_t)b * a.T + t) * a.H + h;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (tx == 0) a.lse[at] = sum == 0.f ? -CUDART_INF_F : mx[i] * kTreeLn2 + logf(sum);
#pragma unroll
        for (int c = 0; c < NC * CV; ++c)
          Elem<T>::st(reinterpret_cast<T*>(a.o) + at * DH + (c / CV) * 16 * CV + tx * CV + c % CV, o[i][c] * inv);
      } else {
        if (tx == 0) {
          part.m[r] = mx[i];
          part.l[r] = sum;
        }
#pragma unroll
        for (int c = 0; c < NC * CV; ++c) *part.at(r, (c / CV) * 16 * CV + tx * CV + c % CV) = o[i][c];
      }
    }
    slot = 1;
  }
}

// ------------------------------------------------------------------ joining the partials
// CTA (tile, sequence, row group): rg rows, each by 16 threads over the columns and 16 / rg
// sets of threads over the partials.  A thread walks its partials once, with a running
// maximum; the sets are joined in shared memory.  It finds its partials while the kernel before it
// still runs, and waits for that one's end.  Bound by latency and by how fast lines that other SMs
// have just written come back: 1024 rows of 38 partials (10 MB), 6 us from the last partial to the
// end; 12 rows of 64, 2.6 us.  More CTAs than run at once were slower (9 us there with 1024), a
// column's rows read a line at a time no faster.
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 4 * kSMs;
constexpr int kJoinFly = 4;  // partials that a thread has on their way

template <typename T, int DH>
__global__ void __launch_bounds__(kJoinThreads, DH == 128 ? 3 : 4) tree_join_kernel(TreeArgs a, int rg) {
  constexpr int NC = DH / 16, CV = NC < 4 ? NC : 4, NQ = NC / CV;  // a thread's columns: NQ runs of CV
  __shared__ float red_m[16], red_l[16];
  __shared__ __align__(16) float red_o[16][DH + 4];
  const int b = blockIdx.y, tile = blockIdx.x, hg = tile / a.nrt, rt = tile % a.nrt;
  int before;
  const Share sh = shares(a, all_items(a, b, before, false));
  const SeqBlocks sb = seq_blocks(a, b, false);
  const int s0 = before + hg / a.hl * sb.items;
  const int c0 = owner_of(sh, s0 + a.lead), c1 = owner_of(sh, s0 + sb.items - 1);  // shares of its first and last block
  after_previous();      // (by every CTA: the grid must not end before the one ahead of it)
  if (c0 == c1) return;  // finished there
  // Threads of a row, or of a column's rows, side by side: as the partials lie.
  const int ps = 16 / rg, ri = a.pieces ? threadIdx.x % rg : threadIdx.x / 16 % rg,
            x = a.pieces ? threadIdx.x / rg % 16 : threadIdx.x % 16, pi = threadIdx.x / (16 * rg), y = pi * rg + ri;
  const int most = min(a.rows, a.T * a.g - rt * a.rows), v = blockIdx.z * rg + ri;
  const int hi = v / most, r = v - hi * most, at = hi * a.rows + r;  // key head of the tile, row, place in the slot
  const bool on = hi < a.hw;
  float mx = -CUDART_INF_F, l = 0.f, o[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) o[i] = 0.f;
  const bool late = first_item(sh, c0) < s0;  // the first of them began in another tile
  if (on) {
    constexpr int U = kJoinFly;
    for (int c = c0 + pi; c <= c1; c += U * ps) {
      float m[U], w[U], y4[U][NC];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int cc = c + k * ps;
        m[k] = -CUDART_INF_F;
        w[k] = 0.f;
        if (cc <= c1) {
          const Part p = part_of(a, ((int64_t)cc * a.hl + hg % a.hl) * a.nrt + rt, cc == c0 && late ? 1 : 0);
          m[k] = p.m[at];
          w[k] = p.l[at];
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if constexpr (CV == 4) {
              const float4 f = *reinterpret_cast<const float4*>(p.at(at, 64 * q + 4 * x));
              y4[k][4 * q] = f.x, y4[k][4 * q + 1] = f.y, y4[k][4 * q + 2] = f.z, y4[k][4 * q + 3] = f.w;
            } else {
              const float2 f = *reinterpret_cast<const float2*>(p.at(at, 2 * x));
              y4[k][0] = f.x, y4[k][1] = f.y;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < NC; ++i) y4[k][i] = 0.f;
        }
      }
      float now = mx;
#pragma unroll
      for (int k = 0; k < U; ++k) now = fmaxf(now, m[k]);
      const float base = now == -CUDART_INF_F ? 0.f : now, f0 = exp2f(mx - base);
      mx = now;
      l *= f0;
#pragma unroll
      for (int i = 0; i < NC; ++i) o[i] *= f0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float f = exp2f(m[k] - base);
        l = fmaf(w[k], f, l);
#pragma unroll
        for (int i = 0; i < NC; ++i) o[i] = fmaf(y4[k][i], f, o[i]);
      }
    }
  }
  // Each set by the maximum of all; then their sum.
  if (x == 0) red_m[y] = mx;
  __syncthreads();
  float top = -CUDART_INF_F;
#pragma unroll 4
  for (int p = 0; p < ps; ++p) top = fmaxf(top, red_m[p * rg + ri]);
  const float f0 = exp2f(mx - (top == -CUDART_INF_F ? 0.f : top));
  l *= f0;
#pragma unroll
  for (int i = 0; i < NC; ++i) o[i] *= f0;
  if (pi > 0) {
    if (x == 0) red_l[y] = l;
#pragma unroll
    for (int i = 0; i < NC; ++i) red_o[y][(i / CV) * 64 + x * CV + i % CV] = o[i];
  }
  __syncthreads();
  if (pi != 0 || !on) return;
#pragma unroll 4
  for (int p = 1; p < ps; ++p) {
    l += red_l[p * rg + ri];
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] += red_o[p * rg + ri][(i / CV) * 64 + x * CV + i % CV];
  }
  int t, h;
  row_of(a, rt * a.rows + r, hg * a.hw + hi, t, h);
  const int64_t to = ((int64_t)b * a.T + t) * a.H + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (x == 0) a.lse[to] = l == 0.f ? -CUDART_INF_F : top * kTreeLn2 + logf(l);
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    T* row = reinterpret_cast<T*>(a.o) + to * DH + 64 * q + x * CV;
    const float* f = o + CV * q;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CV; i += 2) reinterpret_cast<float2*>(row)[i / 2] = make_float2(f[i] * inv, f[i + 1] * inv);
    } else if constexpr (CV == 4) {
      *reinterpret_cast<uint2*>(row) = make_uint2(pack_bf16(f[0] * inv, f[1] * inv), pack_bf16(f[2] * inv, f[3] * inv));
    } else {
      *reinterpret_cast<uint32_t*>(row) = pack_bf16(f[0] * inv, f[1] * inv);
    }
  }
}

// ------------------------------------------------------------------ plan of a tree
// One CTA a sequence, one thread a token.  Ancestors by doubling: after step i a token knows
// its 2^i nearest ancestors and the one beyond them.  Bound by its launch and eight rounds of
// barriers: 2.4 us for 16 trees of 64, 3.1 for 64 of 256.
constexpr int kPlanThreads = GCA_MAX_DRAFT;
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(TreePlanArgs a) {
  constexpr int W = GCA_MAX_DRAFT / 64;
  __shared__ unsigned long long anc[W][kPlanThreads];
  __shared__ int up[kPlanThreads], depth[kPlanThreads];  // depth < 0: padding
  const int b = blockIdx.x, t = threadIdx.x;
  int p = -2;
  if (t < a.T) {
    p = a.parents[(int64_t)b * a.T + t];
    if (p < -2 || p >= t) {
      flag_bad_index(a.err, p);
      p = -2;
    }
  }
  unsigned long long mine[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    mine[w] = w == (t >> 6) ? 1ull << (t & 63) : 0ull;
    anc[w][t] = mine[w];
  }
  int d = p == -2 ? INT32_MIN / 2 : (p == -1 ? 0 : 1);
  depth[t] = d;
  up[t] = p < 0 ? -1 : p;
  for (int step = 1; step < kPlanThreads; step <<= 1) {
    __syncthreads();
    const int q = up[t];
    int nu = q, nd = d;
    if (q >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) mine[w] |= anc[w][q];
      nd = depth[q] < 0 ? INT32_MIN / 2 : d + depth[q];
      nu = up[q];
    }
    __syncthreads();
    d = nd;
    depth[t] = nd;
    up[t] = nu;
#pragma unroll
    for (int w = 0; w < W; ++w) anc[w][t] = mine[w];
  }
  if (t >= a.T) return;
  const bool on = d >= 0;
  const int64_t at = (int64_t)b * a.T + t;
  const int len = a.lengths[b];
  if (t == 0 && len < 0) flag_bad_index(a.err, len);
  a.positions[at] = on ? (int)min((int64_t)max(len, 0) + d, (int64_t)INT32_MAX) : -1;
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < a.words) a.mask[at * a.words + w] = on ? mine[w] : 0ull;
}

// ------------------------------------------------------------------ launching
// Lead and least blocks of a share (see tree_sched.cuh).  Measured without and with the lead: 2 x 64K
// tokens, 128 rows, 47.8 and 41.3 us; 32 single tokens over 2K, dh 128, 38.5 and 36.9; where a share
// has a block or two the small kernel is better without (11.9 and 13.3 us).  Shares of one block
// and of four, 128 rows over 2K and 4K tokens: 15.6 and 13.7, 16.0 and 14.3 us.
constexpr int kLeadTc = 4, kLeadRows = 1;
constexpr int kJoinTc = 16, kJoinRows = 2;  // what partial results and their join cost, in blocks of a CTA
enum Kind { kRows, kTensor, kSimt };
struct Shape {
  Kind kind;
  int hw, rows, nrt;  // key heads and rows of a CTA, groups of rows
  int ctas;           // on the GPU at once
  int hl;             // CTAs of a share side by side over the key heads
  bool whole;         // a CTA finishes its tile
};
// Pages of a sequence that some row can see, at most.
int seen_pages(int width, int window) { return window > 0 ? std::min(width, window / kChunk + 2) : width; }
Shape shape_of(int B, int T, int g, int Hkv, int dh, int bf16, int width, int window) {
  const int R = T * g;
  Shape s{kSimt, 1, R <= 8 ? 8 : (R <= 16 ? 16 : 32), 1, (dh == 128 ? 2 : 4) * kSMs};
  const int seen = seen_pages(width, window), most = seen + (T + kChunk - 1) / kChunk;  // blocks of a tile, at most
  // Whole tiles: a CTA walks more blocks than a share would have, which must cost less than partial
  // results and their join.  Measured, joined against whole, in us: 16 trees of 48 tokens in a window
  // of 512, 12 heads, 19.4, 13.0; 4 of 32 over 1000 tokens 16.6, 14.1; with the small kernel 100 single
  // tokens over 300 25.9, 21.5, but 64 over 600 30.7, 35.6.  In float32 a block costs too much.
  auto whole = [&](int64_t tiles, int ctas, int join) { return tiles <= ctas && most * (ctas - tiles) <= (int64_t)join * ctas; };
  // bf16: 16 rows a warp without shared memory, or 128 rows a CTA on the tensor cores?  The
  // first starts and ends faster and re-reads the keys for each 16 rows; the second streams
  // better, has no join where its tiles are whole, and pays more for going on to another.
  // Measured, first against second, in us: 12 heads over 4000 tokens, one token: 10.1, 14.2; four
  // sequences over 2K: 15.2, 14.6; 4 heads of 128, 32 sequences over 2K: 36.0, 31.1; 64 sequences with a
  // window of 512: 27.7, 35.5; 16 of them (whole tiles) 14.2, 10.9; one over 600 tokens 8.6, 11.1, over
  // 130 8.4, 8.0 (4 heads of 128 10.5, 8.8); drafts of 64 over 1K tokens, four sequences: 18.1, 13.5.
  const int64_t work = (int64_t)B * Hkv * most * ((R + 15) / 16) * dh / 64;  // 8 KB blocks, once for each 16 rows
  bool few = (R <= 16 && seen < 32) || work <= 6 * kSMs;
  const int groups = (R + 127) / 128;
  if (whole((int64_t)B * Hkv * groups, 2 * kSMs, kJoinTc) && most <= 3 + dh / 32 + work / 190) few = false;
  int join = 0;
  if (bf16 && (few || dh == 32)) {
    s = Shape{kRows, Hkv % 4 == 0 ? 4 : (Hkv % 2 == 0 ? 2 : 1), 16, 1, kSMs * (dh == 32 ? 3 : 2)};
    join = kJoinRows;
  } else if (bf16) {
    s = Shape{kTensor, 1, 128, 1, 2 * kSMs};
    join = kJoinTc;
  }
  s.nrt = (R + s.rows - 1) / s.rows;
  s.whole = join > 0 && whole((int64_t)B * (Hkv / s.hw) * s.nrt, s.ctas, join);
  // As many heads walk together as leave nine shares or more (what does not divide the GPU's
  // CTAs stays idle: at most a tenth); where tiles are whole, all.
  s.hl = s.whole ? Hkv / s.hw : 1;
  for (int h = 1; h * s.hw <= Hkv && !s.whole; ++h)
    if (Hkv % (h * s.hw) == 0 && h * s.nrt * 9 <= s.ctas) s.hl = h;
  return s;
}
int shares_of(const Shape& s, int B) { return s.whole ? B : std::max(1, s.ctas / (s.nrt * s.hl)); }

template <int DH, int RT>
cudaError_t run_simt(const TreeArgs& a, cudaStream_t s) {
  cudaError_t e = allow_smem((const void*)tree_simt_kernel<DH, RT>, simt_smem<DH, RT>());
  if (e != cudaSuccess) return e;
  launch_begin("tree_simt", s);
  tree_simt_kernel<DH, RT><<<a.grid * a.hl * a.nrt, kSimtThreads, simt_smem<DH, RT>(), s>>>(a);
  return launch_end("tree_simt", s);
}
template <typename T, int DH>
cudaError_t run_dh(const TreeArgs& a, Kind kind, cudaStream_t s) {
  cudaError_t e;
  if constexpr (sizeof(T) == 2) e = kind == kRows ? launch_tree_rows(a, s) : launch_tree_tc(a, s);
  else e = a.rows == 8 ? run_simt<DH, 1>(a, s) : (a.rows == 16 ? run_simt<DH, 2>(a, s) : run_simt<DH, 4>(a, s));
  if (e != cudaSuccess || a.whole) return e;
  // Rows of a CTA: as many as leave a thread about four partials to walk (a tile has about
  // grid / tiles of them), and no more than there are.
  const int rows = a.hw * std::min(a.rows, a.T * a.g), tiles = a.Hkv / a.hw * a.nrt;
  const int64_t parts = (int64_t)a.grid * a.hl / ((int64_t)(a.Hkv / a.hw) * a.B) + 1;
  int rg = 16;
  while (rg > 1 && (rg / 2 >= rows || parts * rg > 64)) rg >>= 1;
  while (rg < 16 && (int64_t)tiles * a.B * ((rows + rg - 1) / rg) > kJoinCtas) rg <<= 1;
  launch_begin("tree_join", s);
  e = launch_after(tree_join_kernel<T, DH>, dim3(tiles, a.B, (rows + rg - 1) / rg), dim3(kJoinThreads), s, a, rg);
  const cudaError_t last = launch_end("tree_join", s);
  return e != cudaSuccess ? e : last;
}
template <typename T>
cudaError_t run(const TreeArgs& a, Kind kind, cudaStream_t s) {
  if (a.dh == 32) return run_dh<T, 32>(a, kind, s);
  if (a.dh == 64) return run_dh<T, 64>(a, kind, s);
  return run_dh<T, 128>(a, kind, s);
}

}  // namespace

size_t tree_scratch_bytes(int B, int T, int H, int Hkv, int dh, int bf16, int width, int window) {
  const Shape sh = shape_of(B, T, H / Hkv, Hkv, dh, bf16, width, window);
  if (sh.whole) return 256;  // nothing is kept there
  return (size_t)2 * shares_of(sh, B) * sh.nrt * sh.hl * sh.hw * sh.rows * (dh + 2) * 4;
}

cudaError_t launch_tree_attention(TreeArgs a, cudaStream_t s) {
  const Shape sh = shape_of(a.B, a.T, a.g, a.Hkv, a.dh, a.bf16, a.width, a.window);
  a.hw = sh.hw;
  a.rows = sh.rows;
  a.grid = shares_of(sh, a.B);
  a.whole = sh.whole;
  a.nrt = sh.nrt;
  a.hl = sh.hl;
  a.nd = (a.T + kChunk - 1) / kChunk;
  a.pieces = sh.kind == kTensor;
  // Each partial of a tile costs the join about 0.04 us and each block a share about 0.4: the best
  // number of blocks grows with the root of the tile's.  One key head, 64K tokens, 8 rows: shares of
  // four blocks 19.0 us, of eight 13.7; where 76 shares of each head walk, eight are no better.
  const int64_t many = (int64_t)400 * a.B * (a.Hkv / (a.hw * a.hl));
  a.least = sh.kind == kTensor ? 2 : 0;
  a.far = sh.kind == kTensor && a.grid >= kSMs ? (int)std::min<int64_t>(many, INT32_MAX) : INT32_MAX;
  const int64_t items = (int64_t)a.B * (a.Hkv / (a.hw * a.hl)) * (seen_pages(a.width, a.window) + a.nd);
  a.lead = sh.whole ? 0 : sh.kind == kTensor ? kLeadTc : (items > 2 * a.grid ? kLeadRows : 0);
  a.wide = (reinterpret_cast<uintptr_t>(a.kp) | reinterpret_cast<uintptr_t>(a.vp)) % 32 == 0;
  return a.bf16 ? run<bf16>(a, sh.kind, s) : run<float>(a, sh.kind, s);
}

cudaError_t launch_tree_plan(const TreePlanArgs& a, cudaStream_t s) {
  launch_begin("tree_plan", s);
  tree_plan_kernel<<<a.B, kPlanThreads, 0, s>>>(a);
  return launch_end("tree_plan", s);
}

}  // namespace gca
