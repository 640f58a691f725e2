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
// group of lanes owns a token: it computes the token's sines and cosines (each lane those of the pairs it
// holds, so none twice), with its weights, into registers, and then walks the token's heads of one side
// (queries or keys), a few heads' loads on their way at a time.  A head's row stays in registers from the
// loads over the sum of squares (shuffles) to the stores; shared memory and barriers are not used.  Few
// tokens are split further, by heads.  The arithmetic goes two numbers an instruction (f32x2): one by one,
// with weights, norm and rotation apart, it was 23 instructions an element, and issue took as long as memory.
// Backward, CTAs walk tokens with the weights' gradients in registers and leave one partial sum each; a
// second kernel adds them in order, so equal calls give equal results.
// Measured, bf16: 4 x 16384 tokens of 24 heads of 64, 68 us (5.9 TB/s), their gradients 112 (5.4); 8 x 16384 tokens
// of 20 heads, half of each turned, pairs side by side, gradients 182 (5.5 TB/s); the first in float32 121 (6.6), gradients 186
// (6.5).  With two heads of a token on
// their way in place of four 80 us, with vectors of 8 bytes 84; gradients with two in place of three 115, in
// two rounds of CTAs too many (kNormRows of 16 an SM) 125.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace gca {
namespace {

constexpr int kThreads = 128;

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

// Numbers of a vector in pairs (a vector of one: with a zero).
template <int VEC> constexpr int kPairs = VEC > 1 ? VEC / 2 : 1;
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& v, uint64_t (&x)[kPairs<VEC>]) {
#pragma unroll
  for (int i = 0; i < kPairs<VEC>; ++i) {
    if constexpr (VEC == 1) {
      x[i] = tc::f2(Elem<T>::ld(&v.e[0]), 0.f);
    } else if constexpr (sizeof(T) == 2) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[i];
      x[i] = tc::f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
      x[i] = tc::f2(v.e[2 * i], v.e[2 * i + 1]);
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack(const uint64_t (&x)[kPairs<VEC>]) {
  Pack<T, VEC> v;
#pragma unroll
  for (int i = 0; i < kPairs<VEC>; ++i) {
    float lo, hi;
    tc::uf2(x[i], lo, hi);
    if constexpr (VEC == 1) Elem<T>::st(&v.e[0], lo);
    else if constexpr (sizeof(T) == 2) reinterpret_cast<uint32_t*>(&v)[i] = pack_bf16(lo, hi);
    else v.e[2 * i] = lo, v.e[2 * i + 1] = hi;
  }
  return v;
}
__device__ __forceinline__ uint64_t swapped(uint64_t x) {
  float lo, hi;
  tc::uf2(x, lo, hi);
  return tc::f2(hi, lo);
}
__device__ __forceinline__ float both(uint64_t x) {
  float lo, hi;
  tc::uf2(x, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ uint64_t twice(float x) { return tc::f2(x, x); }

// Unit u of a head: two vectors, at `at` and `at + step`.  They are VEC pairs that turn (with PAIRED, VEC / 2
// pairs each), or elements behind them; of those the second vector may be missing.
struct Unit {
  int at, step;
  bool on, two, turns;
};
template <int VEC, bool PAIRED>
__device__ __forceinline__ Unit unit_of(const NormRotaryArgs& a, int u) {
  const int half = a.rot >> 1, pairs = half / VEC, tail = (a.dh - a.rot) / VEC;
  Unit x;
  x.turns = u < pairs;
  const int v = 2 * (u - pairs);  // of the vectors behind the pairs
  x.on = x.turns || v < tail;
  x.two = x.turns || v + 1 < tail;
  x.at = x.turns ? (PAIRED ? 2 : 1) * u * VEC : a.rot + v * VEC;
  x.step = x.turns && !PAIRED ? half : VEC;
  return x;
}

__device__ __forceinline__ float group_sum(float v, int G) {
  for (int d = G / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// grid: (CTAs over the tokens, parts of the heads: first those of q, then those of k).  UPL: units of a lane.
template <typename T, int VEC, int UPL, bool PAIRED, bool BWD>
__global__ void __launch_bounds__(kThreads, UPL > 1 ? 1 : BWD ? 3 : 4) norm_rotary_kernel(NormRotaryArgs a) {
  constexpr int FLY = UPL > 1 ? 1 : BWD ? 3 : 4;  // heads whose loads are on their way
  constexpr int P = kPairs<VEC>;
  const int G = a.group, lane = threadIdx.x % G, groups = kThreads / G;
  const int side = (int)blockIdx.y >= a.q_parts, y = blockIdx.y - (side ? a.q_parts : 0);
  const NormSide& s = side ? a.k : a.q;
  const int heads = side ? a.Hkv : a.H, h0 = y * a.per, h1 = min(heads, h0 + a.per);
  const float inv = 1.f / (float)a.dh;
  Unit un[UPL];
  uint64_t w1[UPL][P], w2[UPL][P];  // the weights of its elements
  const float* w = side ? a.kw : a.qw;
#pragma unroll
  for (int j = 0; j < UPL; ++j) {
    un[j] = unit_of<VEC, PAIRED>(a, lane + j * G);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float* at = w + un[j].at + 2 * i;
      w1[j][i] = un[j].on ? tc::f2(at[0], VEC > 1 ? at[1] : 0.f) : 0;
      at += un[j].step;
      w2[j][i] = un[j].two ? tc::f2(at[0], VEC > 1 ? at[1] : 0.f) : 0;
    }
  }
  uint64_t sum1[BWD ? UPL : 1][P], sum2[BWD ? UPL : 1][P];
  if constexpr (BWD) {
#pragma unroll
    for (int j = 0; j < UPL; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) sum1[j][i] = sum2[j][i] = 0;
  }
  const int64_t tokens = (int64_t)a.B * a.L;
  for (int64_t t0 = (int64_t)blockIdx.x * groups; t0 < tokens; t0 += (int64_t)gridDim.x * groups) {
    const int64_t t = t0 + threadIdx.x / G;
    const bool there = t < tokens;
    const int64_t b = there ? t / a.L : 0, l = there ? t - b * a.L : 0;
    const T* in = reinterpret_cast<const T*>(s.in) + b * s.in_bs + l * s.in_ts;
    const T* dy = BWD ? reinterpret_cast<const T*>(s.dy) + b * s.dy_bs + l * s.dy_ts : nullptr;
    T* out = reinterpret_cast<T*>(s.out) + b * s.out_bs + l * s.out_ts;
    Pack<T, VEC> xa[FLY][UPL], xb[FLY][UPL], da[BWD ? FLY : 1][UPL], db[BWD ? FLY : 1][UPL];
    auto fetch = [&](int f, int h) {
      if (h >= h1) return;
#pragma unroll
      for (int j = 0; j < UPL; ++j) {
        const int64_t from = h * s.in_hs + un[j].at;
        if (there && un[j].on) xa[f][j] = load<T, VEC>(in + from);
        if (there && un[j].two) xb[f][j] = load<T, VEC>(in + from + un[j].step);
        if constexpr (BWD) {
          const int64_t at = h * s.dy_hs + un[j].at;
          if (there && un[j].on) da[f][j] = load<T, VEC>(dy + at);
          if (there && un[j].two) db[f][j] = load<T, VEC>(dy + at + un[j].step);
        }
      }
    };
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
#pragma unroll
      for (int j = 0; j < UPL; ++j) {  // what a lane lacks counts as zeros
        xa[f][j] = xb[f][j] = Pack<T, VEC>{};
        if constexpr (BWD) da[f][j] = db[f][j] = Pack<T, VEC>{};
      }
      fetch(f, h0 + f);  // on their way while the angles are computed
    }
    // The turned vectors are  a: A x_a + B partner_a,  b: C x_b + D partner_b, where a partner is the unit's other
    // vector, or with PAIRED the same vector with its pairs swapped.  Forward the weights are in the factors.
    uint64_t A[UPL][P], B[UPL][P], C[UPL][P], D[UPL][P];
    const int64_t p = !there ? 0 : a.pos ? a.pos[b * a.pos_bs + l] : l;
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      float c[VEC], n[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        c[i] = 1.f;
        n[i] = 0.f;
        if (un[j].turns) {
          const int32_t top = (int32_t)(uint32_t)(((uint64_t)p * a.freq[(lane + j * G) * VEC + i]) >> 32);  // turns, 2^-32 each
          sincospif((float)top * 0x1p-31f, &n[i], &c[i]);
          c[i] *= a.gain;
          n[i] *= a.sgain;
        }
      }
      constexpr bool OWN = PAIRED && VEC > 1;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if constexpr (OWN) {
          A[j][i] = twice(c[i]);
          B[j][i] = tc::f2(-n[i], n[i]);
          C[j][i] = twice(c[P + i]);
          D[j][i] = tc::f2(-n[P + i], n[P + i]);
        } else {
          const float n1 = VEC > 1 ? n[2 * i + (VEC > 1)] : 0.f;
          A[j][i] = C[j][i] = tc::f2(c[2 * i], VEC > 1 ? c[2 * i + (VEC > 1)] : 0.f);
          B[j][i] = tc::f2(-n[2 * i], -n1);
          D[j][i] = tc::f2(n[2 * i], n1);
        }
        if constexpr (!BWD) {
          A[j][i] = tc::mul2(A[j][i], w1[j][i]);
          B[j][i] = tc::mul2(B[j][i], OWN ? swapped(w1[j][i]) : w2[j][i]);
          C[j][i] = tc::mul2(C[j][i], w2[j][i]);
          D[j][i] = tc::mul2(D[j][i], OWN ? swapped(w2[j][i]) : w1[j][i]);
        }
      }
    }
    auto turn = [&](int j, const uint64_t (&x)[P], const uint64_t (&z)[P], uint64_t (&y1)[P], uint64_t (&y2)[P]) {
      constexpr bool OWN = PAIRED && VEC > 1;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        y1[i] = tc::fma2(A[j][i], x[i], tc::mul2(B[j][i], OWN ? swapped(x[i]) : z[i]));
        y2[i] = tc::fma2(C[j][i], z[i], tc::mul2(D[j][i], OWN ? swapped(z[i]) : x[i]));
      }
    };
    for (int h = h0; h < h1; h += FLY) {  // the same for the whole warp: shuffles need every lane
#pragma unroll
      for (int f = 0; f < FLY; ++f) {
        if (h + f >= h1) break;
        uint64_t x1[UPL][P], x2[UPL][P], u1[UPL][P], u2[UPL][P];  // u: the turned row, backward dy turned back
        uint64_t ss = 0, dot = 0;
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
          unpack<T, VEC>(xa[f][j], x1[j]);
          unpack<T, VEC>(xb[f][j], x2[j]);
#pragma unroll
          for (int i = 0; i < P; ++i) ss = tc::fma2(x2[j][i], x2[j][i], tc::fma2(x1[j][i], x1[j][i], ss));
          if constexpr (BWD) {
            uint64_t d1[P], d2[P];
            unpack<T, VEC>(da[f][j], d1);
            unpack<T, VEC>(db[f][j], d2);
            turn(j, d1, d2, u1[j], u2[j]);
#pragma unroll
            for (int i = 0; i < P; ++i)
              dot = tc::fma2(tc::mul2(u2[j][i], w2[j][i]), x2[j][i], tc::fma2(tc::mul2(u1[j][i], w1[j][i]), x1[j][i], dot));
          } else {
            turn(j, x1[j], x2[j], u1[j], u2[j]);
          }
        }
        fetch(f, h + FLY + f);  // the next head in the place of this one
        const float rms = rsqrtf(group_sum(both(ss), G) * inv + a.eps);
        const float r = there ? rms : 0.f;  // (a token that is not there may give an infinity where eps is 0)
        const uint64_t r2 = twice(r);
        uint64_t c2 = 0;
        if constexpr (BWD) c2 = twice(-group_sum(both(dot), G) * r * r * r * inv);  // -mean(w u x r) r^2, the factor of x
        T* to = out + (h + f) * s.out_hs;
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if constexpr (BWD) {
              sum1[j][i] = tc::fma2(u1[j][i], tc::mul2(x1[j][i], r2), sum1[j][i]);
              sum2[j][i] = tc::fma2(u2[j][i], tc::mul2(x2[j][i], r2), sum2[j][i]);
              u1[j][i] = tc::fma2(tc::mul2(u1[j][i], w1[j][i]), r2, tc::mul2(x1[j][i], c2));
              u2[j][i] = tc::fma2(tc::mul2(u2[j][i], w2[j][i]), r2, tc::mul2(x2[j][i], c2));
            } else {
              u1[j][i] = tc::mul2(u1[j][i], r2);
              u2[j][i] = tc::mul2(u2[j][i], r2);
            }
          }
          if (there && un[j].on) store<T, VEC>(to + un[j].at, pack<T, VEC>(u1[j]));
          if (there && un[j].two) store<T, VEC>(to + un[j].at + un[j].step, pack<T, VEC>(u2[j]));
        }
      }
    }
  }
  if constexpr (BWD) {
    // The weights' gradients: over a warp's groups by shuffles, over the warps in shared memory.
    __shared__ float part[kThreads / 32][256];
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v, other;
          tc::uf2(e < 2 ? sum1[j][i] : sum2[j][i], v, other);
          if (e & 1) v = other;
          for (int d = G; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
          if ((threadIdx.x & 31) < G && (e < 2 ? un[j].on : un[j].two) && (VEC > 1 || !(e & 1)))
            part[threadIdx.x >> 5][un[j].at + (e < 2 ? 0 : un[j].step) + 2 * i + (e & 1)] = v;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.dh; i += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int x = 0; x < kThreads / 32; ++x) v += part[x][i];
      a.partial[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.dh + i] = v;
    }
  }
}

// One side's weight gradient: its CTAs' partial sums, 32 lanes of sums an element, eight elements a CTA.
__global__ void __launch_bounds__(256) norm_weights_kernel(const float* partial, int q_rows, int k_rows, int dh, float* dqw, float* dkw) {
  after_previous();
  const int e = threadIdx.x & 7, x = threadIdx.x >> 3, i = blockIdx.x * 8 + e;
  float* out = blockIdx.y ? dkw : dqw;
  const float* p = partial + (blockIdx.y ? (int64_t)q_rows * dh : 0);
  const int rows = blockIdx.y ? k_rows : q_rows;
  float v = 0.f;
  if (i < dh)
#pragma unroll 4
    for (int c = x; c < rows; c += 32) v += p[(int64_t)c * dh + i];
  __shared__ float red[32][8];
  red[x][e] = v;
  __syncthreads();
  if (x == 0 && i < dh) {
    float s = 0.f;
    for (int c = 0; c < 32; ++c) s += red[c][e];
    out[i] = s;
  }
}

template <typename T, int VEC, int UPL, bool PAIRED>
void launch(const NormRotaryArgs& a, dim3 grid, cudaStream_t s) {
  if (a.backward) norm_rotary_kernel<T, VEC, UPL, PAIRED, true><<<grid, kThreads, 0, s>>>(a);
  else norm_rotary_kernel<T, VEC, UPL, PAIRED, false><<<grid, kThreads, 0, s>>>(a);
}
template <typename T, int VEC>
void launch(const NormRotaryArgs& a, dim3 grid, cudaStream_t s) {
  if constexpr (VEC == 1) {  // a vector of one turns the same either way; a head has up to 128 units
    if (a.paired) launch<T, 1, 4, true>(a, grid, s);
    else launch<T, 1, 4, false>(a, grid, s);
  } else {
    if (a.paired) launch<T, VEC, 1, true>(a, grid, s);
    else launch<T, VEC, 1, false>(a, grid, s);
  }
}

}  // namespace

size_t norm_rotary_scratch_bytes(int dh) { return (size_t)kNormRows * dh * sizeof(float); }

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
  // Vectors of 16 or 8 bytes, else of one element: a head of up to 256 elements has 32 units of 8 elements or more.
  // (4 x 16384 tokens of 24 heads of 64, bf16: 68 us in vectors of 16 bytes, rot 36 by single elements 633, gradients 1229.)
  while (vec > 1 && !fits(vec)) vec >>= 1;
  auto units_of = [&](int v) { return a.rot / 2 / v + ((a.dh - a.rot) / v + 1) / 2; };
  if (vec * esize < 8 || units_of(vec) > 32) vec = 1;
  const int units = units_of(vec);
  a.group = 1;
  while (a.group < units && a.group < 32) a.group <<= 1;
  // Heads of a CTA: all of a side, or fewer where the tokens alone do not fill the GPU.
  const int groups = kThreads / a.group, most = std::max(a.H, a.Hkv);
  const int64_t ctas = ((int64_t)a.B * a.L + groups - 1) / groups, full = a.backward ? kNormRows : kSMs * 8;
  const int64_t parts = std::min<int64_t>(most, std::max<int64_t>(1, full / (2 * ctas)));
  a.per = (int)((most + parts - 1) / parts);
  a.q_parts = (a.H + a.per - 1) / a.per;
  const int k_parts = (a.Hkv + a.per - 1) / a.per;
  dim3 grid((unsigned)std::min<int64_t>(ctas, INT32_MAX), (unsigned)(a.q_parts + k_parts));
  if (a.backward) grid.x = (unsigned)std::min<int64_t>(ctas, std::max(1, kNormRows / (a.q_parts + k_parts)));
  launch_begin("norm_rotary", s);
  if (a.bf16) {
    using T = __nv_bfloat16;
    if (vec == 8) launch<T, 8>(a, grid, s);
    else if (vec == 4) launch<T, 4>(a, grid, s);
    else launch<T, 1>(a, grid, s);
  } else {
    if (vec == 4) launch<float, 4>(a, grid, s);
    else if (vec == 2) launch<float, 2>(a, grid, s);
    else launch<float, 1>(a, grid, s);
  }
  cudaError_t e = launch_end("norm_rotary", s);
  if (e != cudaSuccess || !a.backward) return e;
  launch_begin("norm_weights", s);
  e = launch_after(norm_weights_kernel, dim3((a.dh + 7) / 8, a.Hkv ? 2 : 1), dim3(256), s, (const float*)a.partial, (int)(a.q_parts * grid.x),
                   (int)(k_parts * grid.x), a.dh, a.dqw, a.dkw);
  const cudaError_t last = launch_end("norm_weights", s);
  return e != cudaSuccess ? e : last;
}

}  // namespace gca
