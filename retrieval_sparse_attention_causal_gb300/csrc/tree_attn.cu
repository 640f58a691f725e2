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
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ partial results
// Slot s: [rows] maxima (of log2 e times the scaled logits), [rows] sums, [rows][dh] outputs.
struct Part {
  float* m; float* l; float* o;
};
__device__ __forceinline__ Part part_of(const TreeArgs& a, int64_t slot) {
  float* p = reinterpret_cast<float*>(a.part) + slot * a.rows * (a.dh + 2);
  return Part{p, p + a.rows, p + 2 * a.rows};
}

// Where row r of a tile goes: token t, query head h.
__device__ __forceinline__ void row_of(const TreeArgs& a, int r, int m, int& t, int& h) {
  t = r / a.g;
  h = m * a.g + (r - t * a.g);
}

// ------------------------------------------------------------------ CUDA-core kernel
// 128 threads; thread (ty, tx) owns rows ty RT .. ty RT + RT - 1, of a block's logits the
// keys tx + 16 j, and of the output DH / 16 columns.  K and V pass through shared memory
// in 32 bits.
constexpr int kSimtThreads = 128;
template <int DH, int RT>
constexpr int simt_smem() { return (8 * RT * (DH + 4) + 2 * 64 * (DH + 4) + 8 * RT * 68) * 4; }

template <typename T, int DH, int RT>
__global__ void __launch_bounds__(kSimtThreads) tree_simt_kernel(TreeArgs a) {
  constexpr int MT = 8 * RT, QS = DH + 4, CV = DH >= 64 ? 4 : 2, NC = DH / 16 / CV;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + MT * QS;
  float* Vs = Ks + 64 * QS;
  float* Ps = Vs + 64 * QS;
  __shared__ int64_t buf[kSimtThreads / 32 + 1];
  __shared__ Share sh_s;
  __shared__ int row_pos[MT];
  __shared__ unsigned long long used_s;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const Share sh = share_of<kSimtThreads>(a, blockIdx.x, -1, buf, &sh_s);
  const float sl2 = a.scale * kLog2e;
  const int R = a.T * a.g;
  int b = sh.b;
  int64_t off = sh.off, item = sh.lo;
  SeqBlocks sb = sh.lo < sh.hi ? seq_blocks(a, b, false) : SeqBlocks{};
  int slot = 0;
  while (item < sh.hi) {
    const int64_t tile = off / sb.nb;
    if (tile >= (int64_t)a.Hkv * a.nrt) {
      sb = seq_blocks(a, ++b, false);
      off = 0;
      continue;
    }
    const int m = (int)(tile / a.nrt), rt = (int)(tile % a.nrt);
    const int blk0 = (int)(off - tile * sb.nb), blk1 = (int)min((int64_t)sb.nb, blk0 + (sh.hi - item));
    const int rows = min(MT, R - rt * MT);
    __syncthreads();
    for (int i = tid; i < MT * DH; i += kSimtThreads) {
      const int r = i / DH, d = i - r * DH;
      float v = 0.f;
      if (r < rows) {
        int t, h;
        row_of(a, rt * MT + r, m, t, h);
        v = Elem<T>::ld(reinterpret_cast<const T*>(a.q) + b * a.q_bs + t * a.q_ts + h * a.q_hs + d);
      }
      Qs[r * QS + d] = v;
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
          lo = a.window > 0 ? max(0, sb.len - a.window + 1 - j0) : 0;
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
      if (tid == 0) used_s = ctx ? ~0ull : 0ull;
      __syncthreads();
      if (!ctx) {  // draft tokens that some row of the tile sees
        for (int k = tid; k < kChunk; k += kSimtThreads) {
          bool any = false;
          if (k < hi && token_position(a, b, j0 + k, sb.len) >= 0)
            for (int r = 0; r < rows && !any; r += 1) any = row_pos[r] >= 0 && sees_draft(a, b, (rt * MT + r) / a.g, j0 + k);
          if (any) atomicOr(&used_s, 1ull << k);
        }
        __syncthreads();
      }
      const unsigned long long used = used_s;
      // Rows that nobody sees are zeros: a weight of 0 times what lies there must stay 0.
      for (int i = tid; i < kChunk * DH; i += kSimtThreads) {
        const int r = i / DH, d = i - r * DH;
        const bool on = r >= lo && r < hi && ((used >> r) & 1);
        Ks[r * QS + d] = on ? Elem<T>::ld(kb + r * kts + d) : 0.f;
        Vs[r * QS + d] = on ? Elem<T>::ld(vb + r * vts + d) : 0.f;
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
        const int r = ty * RT + i, pos = row_pos[r];
        float top = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = tx + 16 * j;
          bool on = pos >= 0 && k >= lo && k < hi;
          if (ctx) {
            on = on && (a.window <= 0 || j0 + k > pos - a.window);
          } else if (on) {
            const int64_t up = token_position(a, b, j0 + k, sb.len);
            on = up >= 0 && sees_draft(a, b, (rt * MT + r) / a.g, j0 + k) && (a.window <= 0 || up > (int64_t)pos - a.window);
          }
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
    const Part part = part_of(a, 2 * (int64_t)blockIdx.x + slot);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty * RT + i;
      float sum = l[i];
#pragma unroll
      for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (r >= rows) continue;
      if (whole) {
        int t, h;
        row_of(a, rt * MT + r, m, t, h);
        const int64_t at = ((int64_t)b * a.T + t) * a.H + h;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // sum is 0 where the row saw nothing
        if (tx == 0) a.lse[at] = sum == 0.f ? -CUDART_INF_F : mx[i] * kLn2 + logf(sum);
#pragma unroll
        for (int c = 0; c < NC * CV; ++c)
          Elem<T>::st(reinterpret_cast<T*>(a.o) + at * DH + (c / CV) * 16 * CV + tx * CV + c % CV, o[i][c] * inv);
      } else {
        if (tx == 0) {
          part.m[r] = mx[i];
          part.l[r] = sum;
        }
#pragma unroll
        for (int c = 0; c < NC * CV; ++c) part.o[r * DH + (c / CV) * 16 * CV + tx * CV + c % CV] = o[i][c];
      }
    }
    slot = 1;
    off += blk1 - blk0;
    item += blk1 - blk0;
  }
}

// ------------------------------------------------------------------ joining the partials
// CTA (tile, sequence, row group): up to 8 rows, each by 16 threads over the columns and
// 256 / (16 rows) threads over the partials.
constexpr int kJoinThreads = 256;

template <typename T, int DH>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeArgs a, int rg) {
  constexpr int NC = DH / 16;
  __shared__ int64_t buf[kJoinThreads / 32 + 1];
  __shared__ Share sh_s;
  __shared__ float red_m[16][17], red_l[16];
  __shared__ float red_o[16][DH + 1];
  const int b = blockIdx.y, tile = blockIdx.x, m = tile / a.nrt, rt = tile % a.nrt;
  const Share sh = share_of<kJoinThreads>(a, 1, b, buf, &sh_s);
  const SeqBlocks sb = seq_blocks(a, b, false);
  const int64_t s0 = sh.lo + (int64_t)tile * sb.nb, s1 = s0 + sb.nb;
  const int64_t c0 = ((s0 + 1) * sh.G - 1) / sh.W, c1 = (s1 * sh.G - 1) / sh.W;  // CTAs of its first and last block
  if (c0 == c1) return;  // finished there
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4, ps = 16 / rg;
  const int ri = y % rg, pi = y / rg;
  const int r = blockIdx.z * rg + ri, rows = min(a.rows, a.T * a.g - rt * a.rows);
  const bool on = r < rows;
  float mx = -CUDART_INF_F;
  auto slot_of = [&](int64_t c) { return 2 * c + (sh.W * c / sh.G < s0 ? 1 : 0); };
  if (on)
    for (int64_t c = c0 + pi * 16 + x; c <= c1; c += 16 * ps) mx = fmaxf(mx, part_of(a, slot_of(c)).m[r]);
  red_m[y][x] = mx;
  __syncthreads();
  mx = -CUDART_INF_F;
  for (int p = 0; p < ps; ++p)
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, red_m[p * rg + ri][i]);
  const float base = mx == -CUDART_INF_F ? 0.f : mx;
  float l = 0.f, o[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) o[i] = 0.f;
  if (on) {
#pragma unroll 4
    for (int64_t c = c0 + pi; c <= c1; c += ps) {
      const Part p = part_of(a, slot_of(c));
      const float w = exp2f(p.m[r] - base);
      l = fmaf(p.l[r], w, l);
#pragma unroll
      for (int i = 0; i < NC; ++i) o[i] = fmaf(p.o[(int64_t)r * DH + x + 16 * i], w, o[i]);
    }
  }
  if (x == 0) red_l[y] = l;
#pragma unroll
  for (int i = 0; i < NC; ++i) red_o[y][x + 16 * i] = o[i];
  __syncthreads();
  if (pi != 0 || !on) return;
  for (int p = 1; p < ps; ++p) {
    l += red_l[p * rg + ri];
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] += red_o[p * rg + ri][x + 16 * i];
  }
  int t, h;
  row_of(a, rt * a.rows + r, m, t, h);
  const int64_t at = ((int64_t)b * a.T + t) * a.H + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (x == 0) a.lse[at] = l == 0.f ? -CUDART_INF_F : mx * kLn2 + logf(l);
#pragma unroll
  for (int i = 0; i < NC; ++i) Elem<T>::st(reinterpret_cast<T*>(a.o) + at * DH + x + 16 * i, o[i] * inv);
}

// ------------------------------------------------------------------ plan of a tree
// One CTA a sequence, one thread a token.  Ancestors by doubling: after step i a token knows
// its 2^i nearest ancestors and the one beyond them.
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
struct Shape {
  int rows, grid, min_blocks;
};
// Rows of a tile, CTAs, and the fewest blocks worth a CTA of their own.
Shape shape_of(int T, int g) {
  const int R = T * g;
  const int rows = R <= 8 ? 8 : (R <= 16 ? 16 : 32);
  return Shape{rows, kSMs * 2, 1};
}

template <typename T, int DH, int RT>
cudaError_t run_simt(const TreeArgs& a, cudaStream_t s) {
  cudaError_t e = allow_smem((const void*)tree_simt_kernel<T, DH, RT>, simt_smem<DH, RT>());
  if (e != cudaSuccess) return e;
  launch_begin("tree_attn", s);
  tree_simt_kernel<T, DH, RT><<<a.grid, kSimtThreads, simt_smem<DH, RT>(), s>>>(a);
  return launch_end("tree_attn", s);
}
template <typename T, int DH>
cudaError_t run_dh(const TreeArgs& a, cudaStream_t s) {
  cudaError_t e = a.rows == 8 ? run_simt<T, DH, 1>(a, s) : (a.rows == 16 ? run_simt<T, DH, 2>(a, s) : run_simt<T, DH, 4>(a, s));
  if (e != cudaSuccess) return e;
  const int most = std::min(a.rows, a.T * a.g);
  const int rg = most >= 8 ? 8 : (most >= 4 ? 4 : (most >= 2 ? 2 : 1));
  launch_begin("tree_join", s);
  tree_join_kernel<T, DH><<<dim3(a.Hkv * a.nrt, a.B, (most + rg - 1) / rg), kJoinThreads, 0, s>>>(a, rg);
  return launch_end("tree_join", s);
}
template <typename T>
cudaError_t run(const TreeArgs& a, cudaStream_t s) {
  if (a.dh == 32) return run_dh<T, 32>(a, s);
  if (a.dh == 64) return run_dh<T, 64>(a, s);
  return run_dh<T, 128>(a, s);
}

}  // namespace

size_t tree_scratch_bytes(int B, int T, int H, int Hkv, int dh, int bf16) {
  const Shape sh = shape_of(T, H / Hkv);
  return (size_t)2 * sh.grid * sh.rows * (dh + 2) * 4;
}

cudaError_t launch_tree_attention(TreeArgs a, cudaStream_t s) {
  const Shape sh = shape_of(a.T, a.g);
  a.rows = sh.rows;
  a.grid = sh.grid;
  a.min_blocks = sh.min_blocks;
  a.nrt = (a.T * a.g + a.rows - 1) / a.rows;
  a.nd = (a.T + kChunk - 1) / kChunk;
  return a.bf16 ? run<bf16>(a, s) : run<float>(a, s);
}

cudaError_t launch_tree_plan(const TreePlanArgs& a, cudaStream_t s) {
  launch_begin("tree_plan", s);
  tree_plan_kernel<<<a.B, kPlanThreads, 0, s>>>(a);
  return launch_end("tree_plan", s);
}

}  // namespace gca
