// Rotary positions for queries and keys, and the gradient.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) at position p turns by
// p w_i:  y1 = g (x1 cos - x2 sin),  y2 = g (x1 sin + x2 cos);  the gradient turns back.
// The elements from `rot` on pass through.
//
// The angle.  w_i arrives as f_i = round(2^64 w_i / 2 pi), so the angle in turns is the
// low 64 bits of p f_i: whole turns fall off as the integer overflows, and a position of
// any size costs one multiplication.  The error is |p| 2^-65 turns from f_i (2^-34 at
// p = 2^31), plus half a unit in the last place of the float that sincospif takes, at
// most 2^-26 of a turn.  A float product p w_i would be off by a radian at 16M tokens.
//
// Bound by memory: every element is read and written once, three operations each.  A CTA
// takes a few tokens, computes their sines and cosines once into shared memory (all heads
// share them), and streams the heads past them with the widest vectors that the sizes,
// strides and addresses allow.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gca {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;      // tokens of a CTA
constexpr int kMaxAngles = 4096;    // sine and cosine pairs of a CTA (32 KB)
constexpr int kRows = 4;            // head rows that a thread keeps in flight

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

template <typename T, int VEC, bool PAIRED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
  extern __shared__ float2 turn[];  // [tokens][rot / 2]: cos, sin
  __shared__ int2 place[kMaxTokens];
  const int64_t n0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, (int64_t)a.B * a.L - n0);
  const int half = a.rot >> 1;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const int64_t n = n0 + t;
    const int b = (int)(n / a.L), l = (int)(n - (int64_t)b * a.L);
    const int64_t p = a.pos ? a.pos[b * a.pos_bs + l] : l;
    const int32_t top = (int32_t)(uint32_t)(((uint64_t)p * a.freq[f]) >> 32);  // turns, 2^-32 each, in [-1/2, 1/2)
    float s, c;
    sincospif((float)top * 0x1p-31f, &s, &c);
    turn[i] = make_float2(c * a.gain, s * a.sgain);
    if (f == 0) place[t] = make_int2(b, l);
  }
  // Threads = (row slot, unit): unit u of a head is VEC pairs, the units behind them copy VEC elements.
  const int units = half / VEC + a.tail / VEC, slots = kThreads / units;
  const int u = threadIdx.x % units, slot = threadIdx.x / units;
  const int heads = a.H + a.Hkv, rows = nt * heads;
  const bool turns = u < half / VEC;
  const int ea = turns ? (PAIRED ? 2 : 1) * u * VEC : a.rot + (u - half / VEC) * VEC;
  const int eb = PAIRED ? ea + VEC : ea + half;
  __syncthreads();
  if (slot >= slots) return;
  for (int r0 = slot; r0 < rows; r0 += kRows * slots) {
    Pack<T, VEC> x[kRows], y[kRows];
    T* out[kRows];
    int tok[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = r0 + k * slots;
      if (r >= rows) continue;
      const int t = r / heads, h = r - t * heads;
      const bool isq = h < a.H;
      const RotarySide& s = isq ? a.q : a.k;
      const int hh = isq ? h : h - a.H;
      const T* in = reinterpret_cast<const T*>(s.in) + place[t].x * s.in_bs + place[t].y * s.in_ts + hh * s.in_hs;
      out[k] = reinterpret_cast<T*>(s.out) + place[t].x * s.out_bs + place[t].y * s.out_ts + hh * s.out_hs;
      tok[k] = t;
      x[k] = load<T, VEC>(in + ea);
      if (turns) y[k] = load<T, VEC>(in + eb);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (r0 + k * slots >= rows) continue;
      if (turns) {
        const float2* cs = turn + tok[k] * half + u * VEC;
        auto rotate = [](T& p, T& q, float2 w) {
          const float x1 = Elem<T>::ld(&p), x2 = Elem<T>::ld(&q);
          Elem<T>::st(&p, x1 * w.x - x2 * w.y);
          Elem<T>::st(&q, x1 * w.y + x2 * w.x);
        };
        if constexpr (PAIRED && VEC > 1) {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) {
            rotate(x[k].e[2 * e], x[k].e[2 * e + 1], cs[e]);
            rotate(y[k].e[2 * e], y[k].e[2 * e + 1], cs[VEC / 2 + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) rotate(x[k].e[e], y[k].e[e], cs[e]);
        }
        store<T, VEC>(out[k] + eb, y[k]);
      }
      store<T, VEC>(out[k] + ea, x[k]);
    }
  }
}

template <typename T, int VEC>
void launch(const RotaryArgs& a, unsigned grid, size_t smem, cudaStream_t s) {
  if (a.paired) rotary_kernel<T, VEC, true><<<grid, kThreads, smem, s>>>(a);
  else rotary_kernel<T, VEC, false><<<grid, kThreads, smem, s>>>(a);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, cudaStream_t s) {
  // The widest vector that divides the pairs of a head, what lies behind them, every
  // stride and every address.
  const int esize = a.bf16 ? 2 : 4;
  int vec = 16 / esize;
  auto fits = [&](int v) {
    if ((a.rot / 2) % v || a.tail % v) return false;
    for (const RotarySide* x : {&a.q, &a.k}) {
      if (!x->in) continue;
      const int64_t all = x->in_bs | x->in_ts | x->in_hs | x->out_bs | x->out_ts | x->out_hs;
      const uintptr_t at = reinterpret_cast<uintptr_t>(x->in) | reinterpret_cast<uintptr_t>(x->out);
      if (all % v || at % (v * esize)) return false;
    }
    return true;
  };
  while (vec > 1 && !fits(vec)) vec >>= 1;
  if ((a.rot / 2 + a.tail) / vec > kThreads) return cudaErrorInvalidValue;
  // Enough tokens to give every thread its rows in flight, while the GPU stays filled.
  const int64_t tokens = (int64_t)a.B * a.L;
  const int per_token = ((a.rot / 2 + a.tail) / vec) * (a.H + a.Hkv);
  int nt = (kThreads * kRows + per_token - 1) / per_token;
  nt = (int)std::min<int64_t>(nt, (tokens + kSMs * 4 - 1) / (kSMs * 4));
  nt = std::max(1, std::min({nt, kMaxTokens, kMaxAngles / (a.rot / 2)}));
  a.tokens = nt;
  const unsigned grid = (unsigned)((tokens + nt - 1) / nt);
  const size_t smem = (size_t)nt * (a.rot / 2) * sizeof(float2);
  launch_begin("rotary", s);
  if (a.bf16) {
    using T = __nv_bfloat16;
    if (vec == 8) launch<T, 8>(a, grid, smem, s);
    else if (vec == 4) launch<T, 4>(a, grid, smem, s);
    else if (vec == 2) launch<T, 2>(a, grid, smem, s);
    else launch<T, 1>(a, grid, smem, s);
  } else {
    if (vec == 4) launch<float, 4>(a, grid, smem, s);
    else if (vec == 2) launch<float, 2>(a, grid, smem, s);
    else launch<float, 1>(a, grid, smem, s);
  }
  return launch_end("rotary", s);
}

}  // namespace gca
