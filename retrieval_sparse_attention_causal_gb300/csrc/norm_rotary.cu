// RMS norm of every head of queries and keys with the rotary positions in the same pass, and the
// gradients.
//
// With r = 1 / sqrt(mean(x^2) + eps) over a head's dh elements and R(p) the rotation of rotary.cu
// (its angles too):
//     y  = g R(p) (x r w)
//     u  = g R(-p) dy,   dw = sum over tokens and heads of u x r,
//     dx = r (w u - x r mean(w u x r))
//
// Bound by memory: x is read once and y written once, backward x and dy are read and dx written.  A
// group of lanes holds a head's row in registers from the loads over the sum of squares (shuffles) to
// the stores, so nothing is read twice.  A CTA computes the sines and cosines of some tokens once
// for all heads.  Backward, a CTA walks such pieces with the weights' gradients in registers and leaves
// one partial sum; a second kernel adds the CTAs' sums in order, so equal calls give equal results.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gca {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxAngles = 2048;  // sine and cosine pairs of a CTA (16 KB)

template <int BYTES> struct Raw;
template <> struct Raw<16> { using T = uint4; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<2> { using T = uint16_t; };

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack { T e[VEC]; };
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load(const T* p) {
  using R = typename Raw<sizeof(T) * VEC>::T;
  const R r = *reinterpret_cast<const R*>(p);
  return *reinterpret_cast<const Pack<T, VEC>*>(&r);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const Pack<T, VEC>& v) {
  using R = typename Raw<sizeof(T) * VEC>::T;
  *reinterpret_cast<R*>(p) = *reinterpret_cast<const R*>(&v);
}

// Where unit u of a head lies: VEC pairs (elements `at` and `at + step` on), or VEC elements behind them.
struct Unit {
  int at, step;
  bool turns, on;
};
template <int VEC>
__device__ __forceinline__ Unit unit_of(const NormRotaryArgs& a, int u) {
  const int half = a.rot >> 1, pairs = half / VEC;
  Unit x;
  x.on = u < pairs + (a.dh - a.rot) / VEC;
  x.turns = u < pairs;
  x.at = x.turns ? (a.paired ? 2 : 1) * u * VEC : a.rot + (u - pairs) * VEC;
  x.step = a.paired ? VEC : half;
  return x;
}

// Turns a unit's elements: x holds elements at .., y elements at + step ..; cs the unit's first pair.
template <int VEC>
__device__ __forceinline__ void rotate(bool paired, float (&x)[VEC], float (&y)[VEC], const float2* cs) {
  auto turn = [](float& p, float& q, float2 w) {
    const float a = p, b = q;
    p = a * w.x - b * w.y;
    q = a * w.y + b * w.x;
  };
  if (VEC > 1 && paired) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      turn(x[2 * i], x[2 * i + 1], cs[i]);
      turn(y[2 * i], y[2 * i + 1], cs[VEC / 2 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) turn(x[i], y[i], cs[i]);
  }
}

__device__ __forceinline__ float group_sum(float v, int G) {
  for (int d = G / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The piece's sines and cosines; the backward pass turns back (sgain < 0).
__device__ __forceinline__ void angles(const NormRotaryArgs& a, float2* turn, int b, int l0, int nt) {
  const int half = a.rot >> 1;
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int t = i / half, f = i - t * half;
    const int64_t p = a.pos ? a.pos[b * a.pos_bs + l0 + t] : l0 + t;
    const int32_t top = (int32_t)(uint32_t)(((uint64_t)p * a.freq[f]) >> 32);  // turns, 2^-32 each
    float s, c;
    sincospif((float)top * 0x1p-31f, &s, &c);
    turn[i] = make_float2(c * a.gain, s * a.sgain);
  }
}

// Rows of a piece of one side (queries or keys): row i is token i / heads, head i % heads.  FLY rows of a
// group are on their way at a time.
template <typename T, int VEC, int UPL, bool BWD>
__global__ void __launch_bounds__(kThreads, UPL > 1 ? 1 : BWD ? 4 : 6) norm_rotary_kernel(NormRotaryArgs a) {
  constexpr int FLY = UPL == 1 ? 2 : 1;
  extern __shared__ float2 turn[];  // [tokens][rot / 2], then the weights [2][dh], then backward [4 warps][dh]
  float* ws = reinterpret_cast<float*>(turn + (size_t)a.tokens * (a.rot >> 1));
  float* part = ws + 2 * a.dh;
  for (int i = threadIdx.x; i < 2 * a.dh; i += kThreads) ws[i] = i < a.dh ? a.qw[i] : (a.kw ? a.kw[i - a.dh] : 0.f);
  const int G = a.group, lane = threadIdx.x % G, first = threadIdx.x / G, groups = kThreads / G;
  const float inv = 1.f / (float)a.dh;
  Unit un[UPL];
#pragma unroll
  for (int j = 0; j < UPL; ++j) un[j] = unit_of<VEC>(a, lane + j * G);
  const int half = a.rot >> 1;
  float sum[2][BWD ? UPL : 1][2 * VEC];
  if (BWD) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < UPL; ++j)
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) sum[s][BWD ? j : 0][i] = 0.f;
  }
  const int per = (a.L + a.tokens - 1) / a.tokens;  // pieces of a sequence
  const int64_t pieces = (int64_t)per * a.B;
  for (int64_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
    const int b = (int)(piece / per), l0 = (int)(piece - (int64_t)b * per) * a.tokens, nt = min(a.tokens, a.L - l0);
    __syncthreads();  // the last piece's angles are no longer read; the weights are there
    angles(a, turn, b, l0, nt);
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const NormSide& s = side ? a.k : a.q;
      const int heads = side ? a.Hkv : a.H;
      if (heads == 0) continue;
      const float* w = ws + side * a.dh;
      const int rows = nt * heads;
      const T* in = reinterpret_cast<const T*>(s.in) + b * s.in_bs + l0 * s.in_ts;
      const T* dy = BWD ? reinterpret_cast<const T*>(s.dy) + b * s.dy_bs + l0 * s.dy_ts : nullptr;
      T* out = reinterpret_cast<T*>(s.out) + b * s.out_bs + l0 * s.out_ts;
      for (int r0 = 0; r0 < rows; r0 += FLY * groups) {  // the same for the whole CTA: shuffles need every lane
        Pack<T, VEC> xa[FLY][UPL], xb[FLY][UPL], da[FLY][UPL], db[FLY][UPL];
        int tok[FLY];
        bool on[FLY];
        int64_t hs_in[FLY], hs_dy[FLY], hs_out[FLY];
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const int row = r0 + f * groups + first;
          on[f] = row < rows;
          const int t = on[f] ? row / heads : 0, h = on[f] ? row - t * heads : 0;
          tok[f] = t;
          hs_in[f] = t * s.in_ts + h * s.in_hs;
          hs_out[f] = t * s.out_ts + h * s.out_hs;
          if (BWD) hs_dy[f] = t * s.dy_ts + h * s.dy_hs;
#pragma unroll
          for (int j = 0; j < UPL; ++j) {
            if (!on[f] || !un[j].on) continue;
            xa[f][j] = load<T, VEC>(in + hs_in[f] + un[j].at);
            if (un[j].turns) xb[f][j] = load<T, VEC>(in + hs_in[f] + un[j].at + un[j].step);
            if (BWD) {
              da[f][j] = load<T, VEC>(dy + hs_dy[f] + un[j].at);
              if (un[j].turns) db[f][j] = load<T, VEC>(dy + hs_dy[f] + un[j].at + un[j].step);
            }
          }
        }
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          float ss = 0.f, dot = 0.f;
          // Backward, the row's u takes the place of dy's values.
          float u1[BWD ? UPL : 1][VEC], u2[BWD ? UPL : 1][VEC];
#pragma unroll
          for (int j = 0; j < UPL; ++j) {
            if (!on[f] || !un[j].on) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float x = Elem<T>::ld(&xa[f][j].e[i]);
              ss += x * x;
              if (un[j].turns) {
                const float y = Elem<T>::ld(&xb[f][j].e[i]);
                ss += y * y;
              }
            }
            if (BWD) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                u1[BWD ? j : 0][i] = Elem<T>::ld(&da[f][j].e[i]);
                u2[BWD ? j : 0][i] = un[j].turns ? Elem<T>::ld(&db[f][j].e[i]) : 0.f;
              }
              if (un[j].turns) rotate<VEC>(a.paired, u1[BWD ? j : 0], u2[BWD ? j : 0], turn + tok[f] * half + (lane + j * G) * VEC);
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                dot += u1[BWD ? j : 0][i] * w[un[j].at + i] * Elem<T>::ld(&xa[f][j].e[i]);
                if (un[j].turns) dot += u2[BWD ? j : 0][i] * w[un[j].at + un[j].step + i] * Elem<T>::ld(&xb[f][j].e[i]);
              }
            }
          }
          ss = group_sum(ss, G);
          if (BWD) dot = group_sum(dot, G);
          const float r = rsqrtf(ss * inv + a.eps);
          const float c = dot * r * r * inv;  // mean(w u x r) r, the factor of x
#pragma unroll
          for (int j = 0; j < UPL; ++j) {
            if (!on[f] || !un[j].on) continue;
            float y1[VEC], y2[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float x1 = Elem<T>::ld(&xa[f][j].e[i]), x2 = un[j].turns ? Elem<T>::ld(&xb[f][j].e[i]) : 0.f;
              const float w1 = w[un[j].at + i], w2 = un[j].turns ? w[un[j].at + un[j].step + i] : 0.f;
              if (BWD) {
                const float d1 = u1[BWD ? j : 0][i], d2 = u2[BWD ? j : 0][i];
                y1[i] = r * (w1 * d1 - x1 * c);
                y2[i] = r * (w2 * d2 - x2 * c);
                sum[side][BWD ? j : 0][i] += d1 * (x1 * r);
                sum[side][BWD ? j : 0][VEC + i] += d2 * (x2 * r);
              } else {
                y1[i] = x1 * r * w1;
                y2[i] = x2 * r * w2;
              }
            }
            if (!BWD && un[j].turns) rotate<VEC>(a.paired, y1, y2, turn + tok[f] * half + (lane + j * G) * VEC);
            Pack<T, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) Elem<T>::st(&o.e[i], y1[i]);
            store<T, VEC>(out + hs_out[f] + un[j].at, o);
            if (un[j].turns) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) Elem<T>::st(&o.e[i], y2[i]);
              store<T, VEC>(out + hs_out[f] + un[j].at + un[j].step, o);
            }
          }
        }
      }
    }
  }
  if constexpr (BWD) {
    // The weights' gradients: over a warp's groups by shuffles, over the warps in shared memory.
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < UPL; ++j) {
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) {
          float v = sum[side][j][i];
          for (int d = G; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
          const bool second = i >= VEC;
          if ((threadIdx.x & 31) < G && un[j].on && (!second || un[j].turns))
            part[(threadIdx.x >> 5) * a.dh + un[j].at + (second ? un[j].step + i - VEC : i)] = v;
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < a.dh; i += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < kThreads / 32; ++x) v += part[x * a.dh + i];
        a.partial[((int64_t)side * gridDim.x + blockIdx.x) * a.dh + i] = v;
      }
    }
  }
}

// Element i of one side's weight gradient: 32 lanes of sums over the CTAs' partial sums, eight elements a CTA.
__global__ void __launch_bounds__(256) norm_weights_kernel(const float* partial, int ctas, int dh, float* dqw, float* dkw) {
  after_previous();
  const int e = threadIdx.x & 7, x = threadIdx.x >> 3, i = blockIdx.x * 8 + e;
  float* out = blockIdx.y ? dkw : dqw;
  const float* p = partial + (int64_t)blockIdx.y * ctas * dh;
  float v = 0.f;
  if (i < dh)
    for (int c = x; c < ctas; c += 32) v += p[(int64_t)c * dh + i];
  __shared__ float red[32][8];
  red[x][e] = v;
  __syncthreads();
  if (x == 0 && i < dh) {
    float s = 0.f;
    for (int c = 0; c < 32; ++c) s += red[c][e];
    out[i] = s;
  }
}

template <typename T, int VEC, int UPL>
cudaError_t launch(const NormRotaryArgs& a, int grid, size_t smem, cudaStream_t s) {
  if (a.backward) norm_rotary_kernel<T, VEC, UPL, true><<<grid, kThreads, smem, s>>>(a);
  else norm_rotary_kernel<T, VEC, UPL, false><<<grid, kThreads, smem, s>>>(a);
  return cudaSuccess;
}
template <typename T, int VEC>
cudaError_t launch(const NormRotaryArgs& a, int units, int grid, size_t smem, cudaStream_t s) {
  if constexpr (sizeof(T) * VEC < 16 || sizeof(T) == 4) {
    if (units > 32) return launch<T, VEC, 8>(a, grid, smem, s);
  }
  return launch<T, VEC, 1>(a, grid, smem, s);
}

}  // namespace

size_t norm_rotary_scratch_bytes(int dh) { return (size_t)kNormCtas * 2 * dh * sizeof(float); }

cudaError_t launch_norm_rotary(NormRotaryArgs a, cudaStream_t s) {
  const int esize = a.bf16 ? 2 : 4;
  int vec = 16 / esize;
  auto fits = [&](int v) {
    if ((a.rot / 2) % v || (a.dh - a.rot) % v) return false;
    for (const NormSide* x : {&a.q, &a.k}) {
      if (!x->in) continue;
      const int64_t all = x->in_bs | x->in_ts | x->in_hs | x->out_bs | x->out_ts | x->out_hs | x->dy_bs | x->dy_ts | x->dy_hs;
      const uintptr_t at = reinterpret_cast<uintptr_t>(x->in) | reinterpret_cast<uintptr_t>(x->out) | reinterpret_cast<uintptr_t>(x->dy);
      if (all % v || at % (v * esize)) return false;
    }
    return true;
  };
  while (vec > 1 && !fits(vec)) vec >>= 1;
  const int units = (a.rot / 2 + a.dh - a.rot) / vec;
  a.group = 1;
  while (a.group < units && a.group < 32) a.group <<= 1;
  // Tokens of a piece: enough rows for every group to have two sets on their way, while the GPU stays filled.
  const int groups = kThreads / a.group, heads = a.H + a.Hkv;
  int64_t nt = std::max(1, (4 * groups + heads - 1) / heads);
  nt = std::min<int64_t>(nt, ((int64_t)a.B * a.L + kSMs * 4 - 1) / (kSMs * 4));
  nt = std::max<int64_t>(1, std::min<int64_t>({nt, kMaxAngles / (a.rot / 2), (int64_t)a.L}));
  a.tokens = (int)nt;
  const int64_t pieces = (int64_t)((a.L + nt - 1) / nt) * a.B;
  const int grid = (int)std::min<int64_t>(pieces, a.backward ? kNormCtas : INT32_MAX);
  const size_t smem = (size_t)nt * (a.rot / 2) * sizeof(float2) + (size_t)(a.backward ? 2 + kThreads / 32 : 2) * a.dh * sizeof(float);
  launch_begin("norm_rotary", s);
  if (a.bf16) {
    using T = __nv_bfloat16;
    if (vec == 8) launch<T, 8>(a, units, grid, smem, s);
    else if (vec == 4) launch<T, 4>(a, units, grid, smem, s);
    else if (vec == 2) launch<T, 2>(a, units, grid, smem, s);
    else launch<T, 1>(a, units, grid, smem, s);
  } else {
    if (vec == 4) launch<float, 4>(a, units, grid, smem, s);
    else if (vec == 2) launch<float, 2>(a, units, grid, smem, s);
    else launch<float, 1>(a, units, grid, smem, s);
  }
  cudaError_t e = launch_end("norm_rotary", s);
  if (e != cudaSuccess || !a.backward) return e;
  launch_begin("norm_weights", s);
  e = launch_after(norm_weights_kernel, dim3((a.dh + 7) / 8, a.Hkv ? 2 : 1), dim3(256), s, (const float*)a.partial, grid, a.dh, a.dqw, a.dkw);
  const cudaError_t last = launch_end("norm_weights", s);
  return e != cudaSuccess ? e : last;
}

}  // namespace gca
