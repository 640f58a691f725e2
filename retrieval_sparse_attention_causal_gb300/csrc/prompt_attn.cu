// Causal attention over packed sequences with shared key heads, and its gradients: the launches, and
// the kernels for float32 on CUDA cores.
//
// Row t of a sequence sees its rows max(0, t - window + 1) .. t (window 0: 0 .. t):
//     s = scale <q, k>,   o = sum softmax(s) v,   lse = log sum exp(s)
//     D = <do, o>,  dS = P (<do, v> - D) scale,   dq = sum dS k,  dk = sum dS q,  dv = sum P do
// where dk and dv sum over the query heads of a key head.  Each gradient is summed by one CTA in a
// fixed order: the queries' side walks a tile's keys, the keys' side its queries and the heads that
// share it.  That costs a second product Q K^T and dO V^T, and needs no atomics.
//
// Float32 (prompt_tc.cu and prompt_bwd_tc.cu have bf16): tiles of 64 rows by 64 keys, operands in
// shared memory with rows padded by four floats, 16 x 16 threads with 4 x 4 logits and 4 x dh / 16
// outputs each.  Both products read two vectors of four floats for 16 multiplications, so the CUDA cores
// and shared memory are busy at about the same rate.  The next tile's loads run while this one is worked
// on.  Where the keys' tiles are too few to fill the GPU, the rows that see one are divided among CTAs,
// whose sums a last kernel adds in order.
// Measured: 4096 tokens of 8 heads of 64, 0.50 ms (35 TFLOP/s), gradients 1.87 (23); three sequences of 1142 tokens
// in all, 6 and 2 heads of 32, 34 us, a chain of up to nine tiles, and 86, of which 45 are dQ's chain.  Without the
// next tile's loads ahead 41 and 48.
#include <algorithm>

#include "prompt.cuh"

namespace gca {
namespace {

constexpr int kT = 64;        // rows and keys of a tile
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

template <int DH>
struct Simt {
  static constexpr int LD = DH + 4, LP = kT + 4;          // floats of a row in shared memory
  static constexpr int TILE = kT * LD, SCORES = kT * LP;  // floats
  static constexpr int CV = DH / 16;                      // columns of a thread's outputs
};

// Rows of a tile on their way: into registers, then into shared memory.  What lies behind the sequence counts
// as zeros.
template <int DH>
struct Rows {
  static constexpr int U = DH / 4, N = kT * U / kThreads;  // vectors of four floats of a row, and of a thread
  float4 x[N];
  __device__ __forceinline__ void fetch(const float* from, int64_t stride, int rows) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int u = threadIdx.x + n * kThreads, r = u / U, c = u % U * 4;
      x[n] = r < rows ? *reinterpret_cast<const float4*>(from + r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void put(float* to) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int u = threadIdx.x + n * kThreads, r = u / U, c = u % U * 4;
      *reinterpret_cast<float4*>(to + r * Simt<DH>::LD + c) = x[n];
    }
  }
};
template <int DH>
__device__ __forceinline__ void load_tile(float* to, const float* from, int64_t stride, int rows) {
  Rows<DH> r;
  r.fetch(from, stride, rows);
  r.put(to);
}

// s[i][j] = <A row ty + 16 i, B row tx + 16 j>.
template <int DH>
__device__ __forceinline__ void products(const float* A, const float* B, float (&s)[4][4]) {
  constexpr int LD = Simt<DH>::LD;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < DH; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * LD + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
  }
}

// The columns of a thread's outputs: runs of up to four, 64 apart.
template <int DH> __device__ __forceinline__ int column(int c) {
  constexpr int RUN = Simt<DH>::CV < 4 ? Simt<DH>::CV : 4;
  return (c / RUN) * 64 + (threadIdx.x & 15) * RUN + c % RUN;
}

// o[i][c] += sum over k of P[row ty + 16 i][k] V[k][column c].
template <int DH>
__device__ __forceinline__ void weighted(const float* P, const float* V, float (&o)[4][Simt<DH>::CV]) {
  constexpr int LD = Simt<DH>::LD, LP = Simt<DH>::LP, CV = Simt<DH>::CV, RUN = CV < 4 ? CV : 4;
  const int ty = threadIdx.x >> 4;
#pragma unroll 2
  for (int k = 0; k < kT; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty + 16 * i) * LP + k);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float v[CV];
#pragma unroll
      for (int c = 0; c < CV; c += RUN) {
        const float* at = V + (k + x) * LD + column<DH>(c);
        if constexpr (RUN == 4) {
          const float4 f = *reinterpret_cast<const float4*>(at);
          v[c] = f.x; v[c + 1] = f.y; v[c + 2] = f.z; v[c + 3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(at);
          v[c] = f.x; v[c + 1] = f.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = x == 0 ? p[i].x : x == 1 ? p[i].y : x == 2 ? p[i].z : p[i].w;
#pragma unroll
        for (int c = 0; c < CV; ++c) o[i][c] += w * v[c];
      }
    }
  }
}

// Of the 16 threads that share a row.
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The tile of this CTA and its head; false: there is none.
__device__ __forceinline__ bool my_tile(const PromptArgs& a, int heads, bool back, PromptTile& x, int& h) {
  __shared__ uint8_t keep[PromptTiles<kT>::kKeep];
  PromptTiles<kT>::fill(a, keep);
  __syncthreads();
  h = blockIdx.x % heads;
  PromptTiles<kT> tiles(a, keep);
  return prompt_tile(a, tiles, blockIdx.x / heads, back, x);
}
__device__ __forceinline__ bool sees(const PromptArgs& a, int t, int k) { return k <= t && (a.window == 0 || k > t - a.window); }
// The first tile of keys that rows t .. see, and behind the last tile of rows that see keys .. k.
__device__ __forceinline__ int first_keys(const PromptArgs& a, int t) { return a.window ? max(0, t - a.window + 1) / kT : 0; }
__device__ __forceinline__ int last_rows(const PromptArgs& a, int k, int len) {
  const int most = a.window ? (int)min((int64_t)len - 1, (int64_t)k + a.window - 1) : len - 1;
  return most / kT + 1;
}

template <int DH>
__global__ void __launch_bounds__(kThreads) prompt_simt_kernel(PromptArgs a) {
  using C = Simt<DH>;
  extern __shared__ float sm[];
  float *Q = sm, *K = Q + C::TILE, *V = K + C::TILE, *P = V + C::TILE;
  PromptTile x;
  int h;
  if (!my_tile(a, a.H, false, x, h)) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, t0 = x.tile * kT, m = h / a.g;
  load_tile<DH>(Q, reinterpret_cast<const float*>(a.q) + (int64_t)(x.off + t0) * a.q_ts + h * a.q_hs, a.q_ts, x.len - t0);
  const float* k = reinterpret_cast<const float*>(a.k) + (int64_t)x.off * a.k_ts + m * a.k_hs;
  const float* v = reinterpret_cast<const float*>(a.v) + (int64_t)x.off * a.v_ts + m * a.v_hs;
  float o[4][C::CV] = {}, mx[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mx[i] = -CUDART_INF_F;
    l[i] = 0.f;
  }
  const float sl2 = a.scale * kLog2e;
  Rows<DH> kr, vr;
  auto fetch = [&](int j) {
    kr.fetch(k + (int64_t)j * kT * a.k_ts, a.k_ts, x.len - j * kT);
    vr.fetch(v + (int64_t)j * kT * a.v_ts, a.v_ts, x.len - j * kT);
  };
  fetch(first_keys(a, t0));
  for (int j = first_keys(a, t0); j <= x.tile; ++j) {
    __syncthreads();
    kr.put(K);
    vr.put(V);
    __syncthreads();
    if (j < x.tile) fetch(j + 1);
    float s[4][4];
    products<DH>(Q, K, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + ty + 16 * i;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!sees(a, t, j * kT + tx + 16 * c)) s[i][c] = -CUDART_INF_F;
        top = fmaxf(top, s[i][c]);
      }
      top = fmaxf(mx[i], row_max(top));
      const float base = top == -CUDART_INF_F ? 0.f : top, f = exp2f((mx[i] - base) * sl2);
      mx[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = exp2f((s[i][c] - base) * sl2);
        sum += p;
        P[(ty + 16 * i) * C::LP + tx + 16 * c] = p;
      }
      l[i] = l[i] * f + row_sum(sum);
#pragma unroll
      for (int c = 0; c < C::CV; ++c) o[i][c] *= f;
    }
    __syncthreads();
    weighted<DH>(P, V, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty + 16 * i;
    if (t >= x.len) continue;
    const int64_t row = (int64_t)(x.off + t) * a.H + h;
    const float inv = 1.f / l[i];
#pragma unroll
    for (int c = 0; c < C::CV; ++c) reinterpret_cast<float*>(a.o)[row * DH + column<DH>(c)] = o[i][c] * inv;
    if (tx == 0) a.lse[row] = mx[i] * a.scale + logf(l[i]);
  }
}

// The first row of a row's sequence; false where it has none.  By a whole warp.
__device__ __forceinline__ bool sequence_of(const PromptArgs& a, int64_t row, int& off) {
  // The last that starts at the row or before (empty ones behind it start there too).
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= row) lo = mid;
    else hi = mid;
  }
  off = a.offsets[lo];
  if (row < off || row - off >= prompt_length(a, lo)) {
    // A row of no sequence; or offsets are out of order, and one that the search passed over has it.
    lo = a.B;
    for (int x = threadIdx.x & 31; x < a.B && lo == a.B; x += 32) {
      const int s = a.offsets[x], n = prompt_length(a, x);
      if (row >= s && row - s < n) lo = x;
    }
    lo = (int)__reduce_min_sync(0xffffffffu, (unsigned)lo);
    if (lo == a.B) return false;
    off = a.offsets[lo];
  }
  return true;
}

// What both sides of the backward pass need of a row, negative as they add it: D = <do, o>, and the
// log-sum-exp times log2(e); a head's rows side by side, [2][H][np] each (prompt_sums).  A warp takes a token, some of its heads
// at a time.  Bound by memory: 54 thousand tokens of 16 heads of 64 44 us (5.1 TB/s; with three heads of a lane on their
// way 50, with four 53: fewer warps fit).
template <typename T, int DH>
__global__ void __launch_bounds__(256) prompt_rows_kernel(PromptArgs a) {
  let_next();  // (in bf16.  float32's kernels, several CTAs an SM, are placed worse if they start early: 114 us for 86.)
  constexpr int V = Elem<T>::kVec, LANES = DH / V, SIDE = 32 / LANES, FLY = 2;  // lanes of a row, rows side by side
  const int lane = threadIdx.x & 31, at = lane % LANES, h0 = lane / LANES;
  const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (row >= a.N) return;
  int off;
  if (!sequence_of(a, row, off)) return;
  const T* o = reinterpret_cast<const T*>(a.o) + row * a.H * DH + at * V;
  const T* g = reinterpret_cast<const T*>(a.dout) + row * a.do_ts + at * V;
  const int64_t to = prompt_sums(a, off, 0) + row - off;
  for (int h = h0; h - h0 < a.H; h += FLY * SIDE) {  // the same for the whole warp: shuffles need every lane
    uint4 x[FLY], y[FLY];
    float l[FLY];
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      const int head = h + f * SIDE;
      x[f] = y[f] = make_uint4(0, 0, 0, 0);
      l[f] = 0.f;
      if (head >= a.H) continue;
      x[f] = *reinterpret_cast<const uint4*>(o + head * DH);
      y[f] = *reinterpret_cast<const uint4*>(g + head * a.do_hs);
      if (at == 0) l[f] = a.lse[row * a.H + head];
    }
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      float u[V], v[V], d = 0.f;
      unpack16(x[f], u, (const T*)nullptr);
      unpack16(y[f], v, (const T*)nullptr);
#pragma unroll
      for (int i = 0; i < V; ++i) d += u[i] * v[i];
#pragma unroll
      for (int m = LANES / 2; m >= 1; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
      const int head = h + f * SIDE;
      if (at == 0 && head < a.H) {
        a.nD[head * a.np + to] = -d;
        a.nlse[head * a.np + to] = -l[f] * kLog2e;
      }
    }
  }
}

// The same in bf16 where a window leaves a row few keys.  There D from the rounded output is off by as much as dS's own
// rounding, so it is made anew: the sum of P <do, v> over the row's keys, P from the log-sum-exp, in float32.  A warp takes a
// token, DH / 8 lanes a head.  (In a sequence's first 128 rows the queries' side finds D's error by itself, from dS of their
// one block; everywhere it does so for the keys' side.)
// Off by, dQ of rows behind the first 128, before and with this: a window of 2 3.7e-3 and 2.34e-3, of 4 3.0 and 2.34, of 8
// 2.7 and 2.35, of 16 2.54 and 2.36; of 24 2.49 without, of 64 2.43.  Bound by issue: all gradients of 46 thousand tokens of 12
// heads of 64 take 320 us by the rounded output, with this 349 in a window of 2, 400 of 8, 477 of 16; so wider ones go
// without.  (With four keys on their way, three CTAs an SM, 364, 407 and 482; with one 354, 410 and 494.)
constexpr int kFewKeys = 16;
template <int DH>
__global__ void __launch_bounds__(256, 4) prompt_few_rows_kernel(PromptArgs a) {
  let_next();
  using T = __nv_bfloat16;
  constexpr int V = 8, LANES = DH / V, SIDE = 32 / LANES, FLY = 2;  // keys on their way
  const int at = threadIdx.x % LANES, h0 = (threadIdx.x & 31) / LANES;
  const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (row >= a.N) return;
  int off;
  if (!sequence_of(a, row, off)) return;
  const int keys = (int)min(row - off + 1, (int64_t)a.window);
  const int64_t first = row - keys + 1, to = prompt_sums(a, off, 0) + row - off;
  const float sl2 = a.scale * kLog2e;
  auto pairs = [](const uint4& u, uint64_t (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = tc::f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  };
  auto product = [&](const uint64_t (&x)[4], const uint4& u) {
    uint64_t y[4];
    pairs(u, y);
    uint64_t s = tc::mul2(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = tc::fma2(x[i], y[i], s);
    float lo, hi;
    tc::uf2(s, lo, hi);
    return lo + hi;
  };
  for (int h = h0; h - h0 < a.H; h += SIDE) {  // the same for the whole warp: shuffles need every lane
    const bool on = h < a.H;
    const int head = on ? h : 0;
    const T* k = reinterpret_cast<const T*>(a.k) + first * a.k_ts + head / a.g * a.k_hs + at * V;
    const T* v = reinterpret_cast<const T*>(a.v) + first * a.v_ts + head / a.g * a.v_hs + at * V;
    uint4 x[FLY], y[FLY];
    auto fetch = [&](int j) {
#pragma unroll
      for (int f = 0; f < FLY; ++f) {
        const int n = min(j + f, keys - 1);
        x[f] = *reinterpret_cast<const uint4*>(k + n * a.k_ts);
        y[f] = *reinterpret_cast<const uint4*>(v + n * a.v_ts);
      }
    };
    fetch(0);
    uint64_t q[4], g[4];
    pairs(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + row * a.q_ts + head * a.q_hs + at * V), q);
    pairs(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.dout) + row * a.do_ts + head * a.do_hs + at * V), g);
    const float nl = -a.lse[row * a.H + head] * kLog2e;
    float d = 0.f;
    for (int j = 0; j < keys; j += FLY) {
      if (j) fetch(j);
#pragma unroll
      for (int f = 0; f < FLY; ++f) {
        if (j + f >= keys) break;  // (the same for the whole warp)
        float s = product(q, x[f]);
#pragma unroll
        for (int m = LANES / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        d += tc::ex2(s * sl2 + nl) * product(g, y[f]);  // (a lane's share of <do, v>)
      }
    }
#pragma unroll
    for (int m = LANES / 2; m >= 1; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
    if (at == 0 && on) {
      a.nD[head * a.np + to] = -d;
      a.nlse[head * a.np + to] = nl;
    }
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads) prompt_dq_simt_kernel(PromptArgs a) {
  using C = Simt<DH>;
  extern __shared__ float sm[];
  float *Q = sm, *G = Q + C::TILE, *K = G + C::TILE, *V = K + C::TILE, *S = V + C::TILE;
  PromptTile x;
  int h;
  if (!my_tile(a, a.H, false, x, h)) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, t0 = x.tile * kT, m = h / a.g;
  load_tile<DH>(Q, reinterpret_cast<const float*>(a.q) + (int64_t)(x.off + t0) * a.q_ts + h * a.q_hs, a.q_ts, x.len - t0);
  load_tile<DH>(G, reinterpret_cast<const float*>(a.dout) + (int64_t)(x.off + t0) * a.do_ts + h * a.do_hs, a.do_ts, x.len - t0);
  const float* k = reinterpret_cast<const float*>(a.k) + (int64_t)x.off * a.k_ts + m * a.k_hs;
  const float* v = reinterpret_cast<const float*>(a.v) + (int64_t)x.off * a.v_ts + m * a.v_hs;
  float dq[4][C::CV] = {}, nl[4], nd[4];
  const int64_t rows = prompt_sums(a, x.off, h) + t0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool on = t0 + ty + 16 * i < x.len;
    nl[i] = on ? a.nlse[rows + ty + 16 * i] : -CUDART_INF_F;  // rows that do not exist weigh nothing
    nd[i] = on ? a.nD[rows + ty + 16 * i] : 0.f;
  }
  const float sl2 = a.scale * kLog2e;
  Rows<DH> kr, vr;
  auto fetch = [&](int j) {
    kr.fetch(k + (int64_t)j * kT * a.k_ts, a.k_ts, x.len - j * kT);
    vr.fetch(v + (int64_t)j * kT * a.v_ts, a.v_ts, x.len - j * kT);
  };
  fetch(first_keys(a, t0));
  for (int j = first_keys(a, t0); j <= x.tile; ++j) {
    __syncthreads();
    kr.put(K);
    vr.put(V);
    __syncthreads();
    if (DH <= 64 && j < x.tile) fetch(j + 1);
    float s[4][4], dp[4][4];
    products<DH>(Q, K, s);
    products<DH>(G, V, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool on = sees(a, t0 + ty + 16 * i, j * kT + tx + 16 * c);
        S[(ty + 16 * i) * C::LP + tx + 16 * c] = on ? exp2f(s[i][c] * sl2 + nl[i]) * (dp[i][c] + nd[i]) : 0.f;
      }
    __syncthreads();
    weighted<DH>(S, K, dq);
    if (DH > 64 && j < x.tile) fetch(j + 1);  // (no registers for it before)
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty + 16 * i;
    if (t >= x.len) continue;
    float* to = reinterpret_cast<float*>(a.dq) + (int64_t)(x.off + t) * a.dq_ts + h * a.dq_hs;
#pragma unroll
    for (int c = 0; c < C::CV; ++c) to[column<DH>(c)] = dq[i][c] * a.scale;
  }
}

// Part blockIdx.y of gridDim.y of the rows that see a tile of keys: a run of (head, tile of rows), the tiles of the
// first head first.
template <int DH>
__global__ void __launch_bounds__(kThreads) prompt_dkv_simt_kernel(PromptArgs a) {
  using C = Simt<DH>;
  extern __shared__ float sm[];
  float *K = sm, *V = K + C::TILE, *Q = V + C::TILE, *G = Q + C::TILE, *P = G + C::TILE, *S = P + C::SCORES;
  PromptTile x;
  int m;
  if (!my_tile(a, a.Hkv, true, x, m)) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, k0 = x.tile * kT;
  load_tile<DH>(K, reinterpret_cast<const float*>(a.k) + (int64_t)(x.off + k0) * a.k_ts + m * a.k_hs, a.k_ts, x.len - k0);
  load_tile<DH>(V, reinterpret_cast<const float*>(a.v) + (int64_t)(x.off + k0) * a.v_ts + m * a.v_hs, a.v_ts, x.len - k0);
  float dk[4][C::CV] = {}, dv[4][C::CV] = {};
  const float sl2 = a.scale * kLog2e;
  const int tiles = last_rows(a, min(k0 + kT, x.len) - 1, x.len) - x.tile, steps = a.g * tiles;
  const int w0 = (int)((int64_t)steps * blockIdx.y / gridDim.y), w1 = (int)((int64_t)steps * (blockIdx.y + 1) / gridDim.y);
  Rows<DH> qr, gr;
  auto fetch = [&](int w) {
    const int h = m * a.g + w / tiles, i = x.tile + w % tiles;
    qr.fetch(reinterpret_cast<const float*>(a.q) + (int64_t)(x.off + i * kT) * a.q_ts + h * a.q_hs, a.q_ts, x.len - i * kT);
    gr.fetch(reinterpret_cast<const float*>(a.dout) + (int64_t)(x.off + i * kT) * a.do_ts + h * a.do_hs, a.do_ts, x.len - i * kT);
  };
  if (w0 < w1) fetch(w0);
  for (int w = w0; w < w1; ++w) {
    const int i = x.tile + w % tiles;
    const int64_t rows = prompt_sums(a, x.off, m * a.g + w / tiles);
    __syncthreads();
    qr.put(Q);
    gr.put(G);
    __syncthreads();
    if (DH <= 64 && w + 1 < w1) fetch(w + 1);
    float s[4][4], dp[4][4];
    products<DH>(K, Q, s);
    products<DH>(V, G, dp);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int t = i * kT + tx + 16 * c;
      const bool row = t < x.len;
      const float nl = row ? a.nlse[rows + t] : 0.f, nd = row ? a.nD[rows + t] : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool on = row && sees(a, t, k0 + ty + 16 * e);
        const float p = on ? exp2f(s[e][c] * sl2 + nl) : 0.f;
        P[(ty + 16 * e) * C::LP + tx + 16 * c] = p;
        S[(ty + 16 * e) * C::LP + tx + 16 * c] = on ? p * (dp[e][c] + nd) : 0.f;
      }
    }
    __syncthreads();
    weighted<DH>(P, G, dv);
    weighted<DH>(S, Q, dk);
    if (DH > 64 && w + 1 < w1) fetch(w + 1);  // (no registers for it before)
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int k = k0 + ty + 16 * e;
    if (k >= x.len) continue;
    if (gridDim.y == 1) {
      float* kt = reinterpret_cast<float*>(a.dk) + (int64_t)(x.off + k) * a.dk_ts + m * a.dk_hs;
      float* vt = reinterpret_cast<float*>(a.dv) + (int64_t)(x.off + k) * a.dv_ts + m * a.dv_hs;
#pragma unroll
      for (int c = 0; c < C::CV; ++c) {
        kt[column<DH>(c)] = dk[e][c] * a.scale;
        vt[column<DH>(c)] = dv[e][c];
      }
    } else {
      float* to = a.parts + (((int64_t)blockIdx.y * 2 * a.N + x.off + k) * a.Hkv + m) * DH;
#pragma unroll
      for (int c = 0; c < C::CV; ++c) {
        to[column<DH>(c)] = dk[e][c];
        to[a.N * a.Hkv * DH + column<DH>(c)] = dv[e][c];
      }
    }
  }
}

// The parts' sums of a tile of keys, added in order.
template <int DH>
__global__ void __launch_bounds__(kThreads) prompt_join_simt_kernel(PromptArgs a, int parts) {
  PromptTile x;
  int m;
  if (!my_tile(a, a.Hkv, true, x, m)) return;
  const int64_t part = a.N * a.Hkv * DH;  // floats of dK's, or dV's, part
  for (int u = threadIdx.x; u < kT * DH / 4; u += kThreads) {
    const int k = x.tile * kT + u / (DH / 4), c = u % (DH / 4) * 4;
    if (k >= x.len) break;
    const float* from = a.parts + ((int64_t)(x.off + k) * a.Hkv + m) * DH + c;
    float4 s[2] = {};
    for (int p = 0; p < parts; ++p)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float4 f = *reinterpret_cast<const float4*>(from + (2 * p + v) * part);
        s[v].x += f.x; s[v].y += f.y; s[v].z += f.z; s[v].w += f.w;
      }
    float* kt = reinterpret_cast<float*>(a.dk) + (int64_t)(x.off + k) * a.dk_ts + m * a.dk_hs + c;
    float* vt = reinterpret_cast<float*>(a.dv) + (int64_t)(x.off + k) * a.dv_ts + m * a.dv_hs + c;
    *reinterpret_cast<float4*>(kt) = make_float4(s[0].x * a.scale, s[0].y * a.scale, s[0].z * a.scale, s[0].w * a.scale);
    *reinterpret_cast<float4*>(vt) = s[1];
  }
}

// Tiles that the sequences can have: as many as whole tiles, and one that is not full each.
int64_t tiles_at_most(int64_t N, int B) { return N / kT + std::min<int64_t>(B, N); }
// Parts that the rows of a tile of keys are divided into: as many as bring the CTAs nearest to two an SM, eight at
// most.  (The keys' side and the join, in two parts and whole: 136 tiles 167 us and 301, 180 tiles 72 and 84, but 246
// tiles 100 and 84, 306 tiles 186 and 169; 40 tiles in seven parts 48, whole 178.)
int parts_of(int64_t N, int B, int Hkv) {
  const int64_t tiles = std::max<int64_t>(1, tiles_at_most(N, B) * Hkv);
  return (int)std::min<int64_t>(8, std::max<int64_t>(1, (2 * kSMs + tiles / 2) / tiles));
}

template <int DH>
cudaError_t forward_simt(const PromptArgs& a, cudaStream_t s) {
  using C = Simt<DH>;
  constexpr int smem = (3 * C::TILE + C::SCORES) * 4;
  cudaError_t e = allow_smem((const void*)prompt_simt_kernel<DH>, smem);
  if (e != cudaSuccess) return e;
  launch_begin("prompt_simt", s);
  prompt_simt_kernel<DH><<<(unsigned)(tiles_at_most(a.N, a.B) * a.H), kThreads, smem, s>>>(a);
  return launch_end("prompt_simt", s);
}

template <int DH>
cudaError_t backward_simt(const PromptArgs& a, cudaStream_t s) {
  using C = Simt<DH>;
  constexpr int sq = (4 * C::TILE + C::SCORES) * 4, skv = (4 * C::TILE + 2 * C::SCORES) * 4;
  cudaError_t e = allow_smem((const void*)prompt_dq_simt_kernel<DH>, sq);
  if (e == cudaSuccess) e = allow_smem((const void*)prompt_dkv_simt_kernel<DH>, skv);
  if (e != cudaSuccess) return e;
  const int64_t tiles = tiles_at_most(a.N, a.B);
  const int parts = parts_of(a.N, a.B, a.Hkv);
  launch_begin("prompt_dq_simt", s);
  prompt_dq_simt_kernel<DH><<<(unsigned)(tiles * a.H), kThreads, sq, s>>>(a);
  e = launch_end("prompt_dq_simt", s);
  if (e != cudaSuccess) return e;
  launch_begin("prompt_dkv_simt", s);
  prompt_dkv_simt_kernel<DH><<<dim3((unsigned)(tiles * a.Hkv), (unsigned)parts), kThreads, skv, s>>>(a);
  e = launch_end("prompt_dkv_simt", s);
  if (e != cudaSuccess || parts == 1) return e;
  launch_begin("prompt_join_simt", s);
  prompt_join_simt_kernel<DH><<<(unsigned)(tiles * a.Hkv), kThreads, 0, s>>>(a, parts);
  return launch_end("prompt_join_simt", s);
}

template <typename T>
void rows(const PromptArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.N + 7) / 8);
  if (a.bf16 && a.window > 0 && a.window <= kFewKeys) {
    if (a.dh == 32) prompt_few_rows_kernel<32><<<grid, 256, 0, s>>>(a);
    else if (a.dh == 64) prompt_few_rows_kernel<64><<<grid, 256, 0, s>>>(a);
    else prompt_few_rows_kernel<128><<<grid, 256, 0, s>>>(a);
    return;
  }
  if (a.dh == 32) prompt_rows_kernel<T, 32><<<grid, 256, 0, s>>>(a);
  else if (a.dh == 64) prompt_rows_kernel<T, 64><<<grid, 256, 0, s>>>(a);
  else prompt_rows_kernel<T, 128><<<grid, 256, 0, s>>>(a);
}

}  // namespace

int64_t prompt_scratch_rows(int64_t N) { return (N + kSumsOfTile + 3) / 4 * 4; }
size_t prompt_parts_bytes(int64_t N, int B, int Hkv, int dh, int bf16) {
  const int parts = bf16 ? 1 : parts_of(N, B, Hkv);
  return parts == 1 ? 0 : (size_t)parts * 2 * N * Hkv * dh * sizeof(float);
}

cudaError_t launch_prompt_forward(const PromptArgs& a, cudaStream_t s) {
  if (a.bf16) return launch_prompt_tc(a, s);
  return a.dh == 32 ? forward_simt<32>(a, s) : a.dh == 64 ? forward_simt<64>(a, s) : forward_simt<128>(a, s);
}

cudaError_t launch_prompt_backward(const PromptArgs& a, cudaStream_t s) {
  launch_begin("prompt_rows", s);
  if (a.bf16) rows<__nv_bfloat16>(a, s);
  else rows<float>(a, s);
  cudaError_t e = launch_end("prompt_rows", s);
  if (e != cudaSuccess) return e;
  if (a.bf16) return launch_prompt_bwd_tc(a, s);
  return a.dh == 32 ? backward_simt<32>(a, s) : a.dh == 64 ? backward_simt<64>(a, s) : backward_simt<128>(a, s);
}

}  // namespace gca
