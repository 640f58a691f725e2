// A cache that holds its keys and values in 8 bits: rows quantised as they are appended, and chunks
// read back.
//
// A token's row is heads x dh numbers in e4m3, then one byte a head, up to a multiple of 16 bytes.  With
// a head's largest magnitude m, the byte is e + 127 for the least e >= -120 with m <= 448 * 2^e, and a
// number is x 2^-e rounded to e4m3.  Powers of two make both directions plain: scaling rounds nothing,
// a number is off by half a step of e4m3 (2^-4 of it, or 2^-10 * 2^e where that is more), and what is
// read back is exact, in bf16 too.  A scale of any other kind would win no precision: e4m3 rounds
// relative to the number.  An infinity or NaN becomes NaN, and does not count for m.
//
// The pages, their table and counts are those of cache.cu, whose operations move rows as bytes.
// Bound by memory: each row is read and written once.  Measured, 12 heads of 64 in bf16: eight prompts of 67
// thousand tokens in all, 59 us with the plan of their pages (5.2 TB/s); 80 tokens of 32 sequences 6.4; 16 x 8 chunks
// read 9.2, 16 x 128 chunks 103 (5.9 TB/s).  In float32: 79 thousand tokens 102 us (5.9 TB/s), chunks 16.4 and 206 (4.9).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include <cuda_fp8.h>

namespace gca {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;      // numbers of a thread: 16 bytes of a row
constexpr int kParts = 2;      // CTAs of a page that is written (with 4 the prompts take 61 us, with 8 75)
constexpr int kReadParts = 8;  // ... that is read: few chunks are read at a time
constexpr int kLowest = -120, kBias = 127;

template <typename T> struct In;
template <> struct In<__nv_bfloat16> {
  static constexpr int kVecs = 2;
  static __device__ __forceinline__ void unpack(const uint4 (&u)[2], float (&x)[kPer]) {
    unpack16(u[0], x, (const __nv_bfloat16*)nullptr);
    unpack16(u[1], x + 8, (const __nv_bfloat16*)nullptr);
  }
  static __device__ __forceinline__ void pack(const float (&x)[kPer], uint4 (&u)[2]) {
    u[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    u[1] = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
  }
};
template <> struct In<float> {
  static constexpr int kVecs = 4;
  static __device__ __forceinline__ void unpack(const uint4 (&u)[4], float (&x)[kPer]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack16(u[i], x + 4 * i, (const float*)nullptr);
  }
  static __device__ __forceinline__ void pack(const float (&x)[kPer], uint4 (&u)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
  }
};

__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

// The exponent that holds magnitudes up to m (finite, >= 0): m = 1.f * 2^x with 448 = 1.75 * 2^8.
__device__ __forceinline__ int exponent_for(float m) {
  const uint32_t bits = __float_as_uint(m);
  return max((int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), kLowest);  // m below 2^-126: the lowest
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 16 numbers of a head, the `lanes` threads of the head side by side: their e4m3 numbers and exponent.
__device__ __forceinline__ uint4 quantise(float (&x)[kPer], int lanes, int& e) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = fmaxf(m, fabsf(x[i]));  // (passes over NaN)
  for (int d = lanes / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (__any_sync(0xffffffffu, m == CUDART_INF_F)) {  // infinities do not count, and become NaN
    m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (fabsf(x[i]) == CUDART_INF_F) x[i] = CUDART_NAN_F;
      m = fmaxf(m, fabsf(x[i]));
    }
    for (int d = lanes / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  e = exponent_for(m);
  const float f = two_to(-e);
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] *= f;
  return make_uint4(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]), e4m3x4(x[8], x[9], x[10], x[11]),
                    e4m3x4(x[12], x[13], x[14], x[15]));
}

// CTA (page step of the call, part of its rows).  The plan counted the pages that each entry touches.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantise_rows_kernel(AppendArgs a) {
  using I = In<T>;
  const CacheArgs& c = a.c;
  after_previous();
  const int step = blockIdx.x / kParts, part = blockIdx.x % kParts;
  int i = 0;  // entries whose pages all lie before this step
  for (int j0 = 0; j0 < c.n; j0 += kThreads) i += __syncthreads_count(j0 + (int)threadIdx.x < c.n && a.steps[j0 + threadIdx.x] <= step);
  if (i >= c.n) return;
  const int4 rec = reinterpret_cast<const int4*>(a.rec)[i];
  const int old = rec.x, now = old + rec.y, slot = rec.w;
  const int p = old / kChunk + step - (i ? a.steps[i - 1] : 0);
  constexpr int per = kChunk / kParts;
  const int r0 = part * per, lanes = a.dh / kPer, units = a.heads * lanes;
  const int held = old - p * kChunk;  // rows of the page that were there before
  const int first = max(r0, held), end = min(r0 + per, now - p * kChunk);
  const int64_t start = a.offsets ? a.offsets[i] : 0;
  // A thread's unit on its way: the first is fetched before the page is known, the next before one is written.
  uint4 kin[I::kVecs], vin[I::kVecs];
  bool on;
  auto fetch = [&](int u) {
    on = u < end * units;
    const int r = u / units, x = u - r * units, t = r - held;
    int64_t row = t;
    if (a.path && on) {
      row = a.path[(int64_t)i * a.T + t];
      if (row < 0 || row >= a.T) {
        if (x == 0) flag_bad_index(c.err, (int)row);
        on = false;
      }
    }
    const uint4* k = reinterpret_cast<const uint4*>(a.kn + i * a.kn_bs + (start + row) * a.kn_ts) + x * I::kVecs;
    const uint4* v = reinterpret_cast<const uint4*>(a.vn + i * a.vn_bs + (start + row) * a.vn_ts) + x * I::kVecs;
#pragma unroll
    for (int n = 0; n < I::kVecs; ++n) {
      kin[n] = on ? k[n] : make_uint4(0, 0, 0, 0);
      vin[n] = on ? v[n] : make_uint4(0, 0, 0, 0);
    }
  };
  fetch(first * units + threadIdx.x);
  const int64_t page = c.table[(int64_t)slot * c.width + p];
  unsigned char *kto = c.kp + page * kChunk * c.token_bytes, *vto = c.vp + page * kChunk * c.token_bytes;
  if (rec.z >= 0 && held > r0) {      // a shared last page: its rows move to this one
    const int words = (int)(c.token_bytes / 16), to = min(r0 + per, held) * words;
    const uint4* kfrom = reinterpret_cast<const uint4*>(c.kp + (int64_t)rec.z * kChunk * c.token_bytes);
    const uint4* vfrom = reinterpret_cast<const uint4*>(c.vp + (int64_t)rec.z * kChunk * c.token_bytes);
    for (int u = r0 * words + threadIdx.x; u < to; u += kThreads) {
      const uint4 x = kfrom[u], y = vfrom[u];
      reinterpret_cast<uint4*>(kto)[u] = x;
      reinterpret_cast<uint4*>(vto)[u] = y;
    }
  }
  // Whole warps go round together, for the heads' maxima.
  for (int u0 = first * units; u0 < end * units; u0 += kThreads) {
    const int u = u0 + threadIdx.x;
    const bool mine = on;
    float f[kPer], g[kPer];
    int ke, ve;
    I::unpack(kin, f);
    I::unpack(vin, g);
    if (u0 + kThreads < end * units) fetch(u + kThreads);
    const uint4 kq = quantise(f, lanes, ke);
    const uint4 vq = quantise(g, lanes, ve);
    if (!mine) continue;
    const int r = u / units, x = u - r * units, h = x / lanes;
    const int64_t at = (int64_t)r * c.token_bytes;
    *reinterpret_cast<uint4*>(kto + at + x * kPer) = kq;
    *reinterpret_cast<uint4*>(vto + at + x * kPer) = vq;
    if (x % lanes == 0) {
      const int64_t eat = at + a.heads * a.dh + h;
      kto[eat] = (unsigned char)(ke + kBias);
      vto[eat] = (unsigned char)(ve + kBias);
      if (h == a.heads - 1)  // whole sectors: nothing has to be read to fill them
        for (int z = a.heads; z % 16; ++z) kto[at + a.heads * a.dh + z] = vto[at + a.heads * a.dh + z] = 0;
    }
  }
}

// CTA (chunk of an entry, part of its rows): a thread reads 16 numbers of K and of V and writes them as T.
template <typename T>
__global__ void __launch_bounds__(kThreads) read_chunks_kernel(ReadArgs a) {
  using I = In<T>;
  const CacheArgs& c = a.c;
  const int i = blockIdx.y, e = blockIdx.x / kReadParts, part = blockIdx.x % kReadParts;
  const int s = c.slot ? c.slot[i] : i, j = a.idx[(int64_t)i * a.per + e];
  int page = -1, len = 0;
  if (s < 0 || s >= c.slots) {
    if (part == 0 && threadIdx.x == 0) flag_bad_index(c.err, s);
  } else if (j < -1 || j >= c.width) {
    if (part == 0 && threadIdx.x == 0) flag_bad_index(c.err, j);
  } else if (j >= 0) {
    page = c.table[(int64_t)s * c.width + j];
    len = c.lengths[s];
    if (page < -1 || page >= c.pages) {
      if (part == 0 && threadIdx.x == 0) flag_bad_index(c.err, page);
      page = -1;
    }
  }
  if (part == 0 && threadIdx.x == 0 && a.local) a.local[(int64_t)i * a.per + e] = page < 0 ? -1 : e;
  const int lanes = a.dh / kPer, units = a.heads * lanes;
  constexpr int per = kChunk / kReadParts;
  const int have = page < 0 ? 0 : min(kChunk, max(0, len - j * kChunk));  // rows that hold tokens
  const unsigned char *kp = c.kp + max(page, 0) * (int64_t)kChunk * c.token_bytes, *vp = c.vp + max(page, 0) * (int64_t)kChunk * c.token_bytes;
  const int64_t to = ((int64_t)i * a.per + e) * kChunk * units;
  auto widen = [](const uint4& q, int x, uint4 (&out)[I::kVecs]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    // Two to the exponent; below 2^-126 by halves (no row that was written here has one).
    const float f = x > 0 ? __uint_as_float((uint32_t)x << 23) : 0x1p-127f;
    float y[kPer];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[n / 2] >> (16 * (n & 1))), __NV_E4M3);
      const float2 p = __half22float2(__half2(h));
      y[2 * n] = p.x * f;
      y[2 * n + 1] = p.y * f;
    }
    I::pack(y, out);
  };
  for (int u = part * per * units + threadIdx.x; u < (part + 1) * per * units; u += kThreads) {
    uint4 ko[I::kVecs], vo[I::kVecs];
#pragma unroll
    for (int n = 0; n < I::kVecs; ++n) ko[n] = vo[n] = make_uint4(0, 0, 0, 0);
    const int r = u / units, x = u - r * units;
    if (r < have) {
      const int64_t at = (int64_t)r * c.token_bytes;
      const uint4 kq = *reinterpret_cast<const uint4*>(kp + at + x * kPer), vq = *reinterpret_cast<const uint4*>(vp + at + x * kPer);
      const int ke = kp[at + a.heads * a.dh + x / lanes], ve = vp[at + a.heads * a.dh + x / lanes];
      widen(kq, ke, ko);
      widen(vq, ve, vo);
    }
    uint4* k = reinterpret_cast<uint4*>(a.k) + (to + u) * I::kVecs;
    uint4* v = reinterpret_cast<uint4*>(a.v) + (to + u) * I::kVecs;
#pragma unroll
    for (int n = 0; n < I::kVecs; ++n) {
      k[n] = ko[n];
      v[n] = vo[n];
    }
  }
}

}  // namespace

cudaError_t launch_quantise_rows(const AppendArgs& a, cudaStream_t s) {
  launch_begin("cache_quantise_rows", s);
  const dim3 grid((unsigned)(a.most_steps * kParts));
  cudaError_t e = a.src_bf16 ? launch_after(quantise_rows_kernel<__nv_bfloat16>, grid, dim3(kThreads), s, a)
                             : launch_after(quantise_rows_kernel<float>, grid, dim3(kThreads), s, a);
  const cudaError_t last = launch_end("cache_quantise_rows", s);
  return e != cudaSuccess ? e : last;
}

cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t s) {
  launch_begin("cache_read", s);
  const dim3 grid((unsigned)(a.per * kReadParts), (unsigned)a.c.n);
  if (a.bf16) read_chunks_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else read_chunks_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return launch_end("cache_read", s);
}

}  // namespace gca
