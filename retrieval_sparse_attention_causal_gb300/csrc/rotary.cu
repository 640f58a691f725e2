// Rotary positions for queries and keys, and the gradient.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) at position p turns by
// p w_i:  y1 = g (x1 cos - x2 sin),  y2 = g (x1 sin + x2 cos);  the gradient turns back.
// The elements from `rot` on pass through.
//
// The angle.  w_i arrives as f_i = round(2^64 w_i / 2 pi), so the angle in turns is the
// low 64 bits of p f_i: whole turns fall off as the integer overflows, and a position of
// any size costs one multiplication, which is exact.  What is off, in radians: f_i, computed in
// double precision, by |p| 2^-49 at most (2^-25 at 16M tokens; at 2^31, 2^-18, which is the
// largest term there); the cut to the top 32 bits by 2 pi 2^-32; half a unit in the last place of
// the float that sincospif takes, pi 2^-25.  A float product p w_i would be off by a radian at
// 16M tokens.
//
// Bound by memory: every element is read and written once, three operations each.  A CTA
// takes some tokens of one sequence, computes their sines and cosines once into shared memory
// (all heads share them), and a thread then walks one place of one head (the widest vectors
// that the sizes, strides and addresses allow) down the tokens, so that nothing but the
// rotation itself is computed per element.  A thread asks for its first tokens before the
// angles are computed; small CTAs (about 128 threads, 64 registers, three tokens in flight a
// thread) keep enough loads on their way while others compute.  Measured: 4 x 16384 tokens of
// 24 heads of 64, bf16, 62 us (6.5 TB/s); with 256 threads 65, with four tokens in flight (97
// registers) 76, with the loads behind the angles 119.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gca {
namespace {

constexpr int kThreads = 128;       // of a CTA, about
constexpr int kMaxThreads = 512;
constexpr int kMaxAngles = 2048;    // sine and cosine pairs of a CTA (16 KB)
constexpr int kFly = 3;             // tokens that a thread keeps in flight

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
__global__ void __launch_bounds__(kMaxThreads, 2) rotary_kernel(RotaryArgs a) {
  extern __shared__ float2 turn[];  // [tokens][rot / 2]: cos, sin
  const int b = blockIdx.y, l0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.L - l0);
  const int half = a.rot >> 1;
  // Unit u of a head is VEC pairs; the units behind the pairs copy VEC elements.
  const int units = half / VEC + a.tail / VEC, places = units * (a.H + a.Hkv);
  const int first = threadIdx.x / places, step = max(1, (int)blockDim.x / places);  // tokens side by side
  const T* in = nullptr;
  T* out = nullptr;
  int64_t in_ts = 0, out_ts = 0;
  bool turns = false;
  int u = 0, eb = 0;
  auto place = [&](int e) {
    const int h = e / units;
    u = e - h * units;
    turns = u < half / VEC;
    const bool isq = h < a.H;
    const RotarySide& s = isq ? a.q : a.k;
    const int64_t hh = isq ? h : h - a.H;
    const int ea = turns ? (PAIRED ? 2 : 1) * u * VEC : a.rot + (u - half / VEC) * VEC;
    eb = PAIRED ? VEC : half;  // from the pairs' first elements to their second
    in = reinterpret_cast<const T*>(s.in) + b * s.in_bs + l0 * s.in_ts + hh * s.in_hs + ea;
    out = reinterpret_cast<T*>(s.out) + b * s.out_bs + l0 * s.out_ts + hh * s.out_hs + ea;
    in_ts = s.in_ts;
    out_ts = s.out_ts;
  };
  Pack<T, VEC> x[kFly], y[kFly];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      const int t = t0 + k * step;
      if (t >= nt) continue;
      x[k] = load<T, VEC>(in + t * in_ts);
      if (turns) y[k] = load<T, VEC>(in + t * in_ts + eb);
    }
  };
  const int e0 = threadIdx.x - first * places;
  const bool works = first < step && e0 < places;
  if (works) {
    place(e0);
    fetch(first);  // on their way while the angles are computed
  }
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int t = i / half, f = i - t * half;
    const int64_t p = a.pos ? a.pos[b * a.pos_bs + l0 + t] : l0 + t;
    const int32_t top = (int32_t)(uint32_t)(((uint64_t)p * a.freq[f]) >> 32);  // turns, 2^-32 each, in [-1/2, 1/2)
    float s, c;
    sincospif((float)top * 0x1p-31f, &s, &c);
    turn[i] = make_float2(c * a.gain, s * a.sgain);
  }
  __syncthreads();
  if (!works) return;
  for (int e = e0;;) {
    for (int t0 = first; t0 < nt;) {
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const int t = t0 + k * step;
        if (t >= nt) continue;
        if (turns) {
          const float2* cs = turn + t * half + u * VEC;
          auto rotate = [](T& p, T& q, float2 w) {
            const float x1 = Elem<T>::ld(&p), x2 = Elem<T>::ld(&q);
            Elem<T>::st(&p, x1 * w.x - x2 * w.y);
            Elem<T>::st(&q, x1 * w.y + x2 * w.x);
          };
          if constexpr (PAIRED && VEC > 1) {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
              rotate(x[k].e[2 * i], x[k].e[2 * i + 1], cs[i]);
              rotate(y[k].e[2 * i], y[k].e[2 * i + 1], cs[VEC / 2 + i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) rotate(x[k].e[i], y[k].e[i], cs[i]);
          }
          store<T, VEC>(out + t * out_ts + eb, y[k]);
        }
        store<T, VEC>(out + t * out_ts, x[k]);
      }
      t0 += kFly * step;
      if (t0 < nt) fetch(t0);
    }
    e += blockDim.x;
    if (e >= places) return;
    place(e);
    fetch(first);
  }
}

template <typename T, int VEC>
void launch(const RotaryArgs& a, dim3 grid, int threads, size_t smem, cudaStream_t s) {
  if (a.paired) rotary_kernel<T, VEC, true><<<grid, threads, smem, s>>>(a);
  else rotary_kernel<T, VEC, false><<<grid, threads, smem, s>>>(a);
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
  const int places = ((a.rot / 2 + a.tail) / vec) * (a.H + a.Hkv);
  // Tokens of a CTA: enough to give every thread its tokens in flight, while the GPU stays filled.
  const int side = std::max(1, kThreads / places);
  int64_t nt = std::min<int64_t>(4 * kFly * side, ((int64_t)a.B * a.L + kSMs * 4 - 1) / (kSMs * 4));
  nt = std::max<int64_t>(1, std::min<int64_t>({nt, kMaxAngles / (a.rot / 2), (int64_t)a.L}));
  a.tokens = (int)nt;
  const int threads = std::min(kMaxThreads, (places * std::min<int>(side, (int)nt) + 31) / 32 * 32);
  const dim3 grid((unsigned)((a.L + nt - 1) / nt), (unsigned)a.B);
  const size_t smem = (size_t)nt * (a.rot / 2) * sizeof(float2);
  launch_begin("rotary", s);
  if (a.bf16) {
    using T = __nv_bfloat16;
    if (vec == 8) launch<T, 8>(a, grid, threads, smem, s);
    else if (vec == 4) launch<T, 4>(a, grid, threads, smem, s);
    else if (vec == 2) launch<T, 2>(a, grid, threads, smem, s);
    else launch<T, 1>(a, grid, threads, smem, s);
  } else {
    if (vec == 4) launch<float, 4>(a, grid, threads, smem, s);
    else if (vec == 2) launch<float, 2>(a, grid, threads, smem, s);
    else launch<float, 1>(a, grid, threads, smem, s);
  }
  return launch_end("rotary", s);
}

}  // namespace gca
