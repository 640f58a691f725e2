// Row-per-thread Tensor Memory access and 2-D TMA loads, for M = 128 tiles.
//
// With M = 128 the accumulator's row r (and the A operand's row r, when A sits in TMEM)
// lives in TMEM lane r.  A warp may touch only the 32 lanes of its quarter (warp id % 4),
// so thread t of a warp in quarter q owns row 32 q + t; the 32x32b shapes below give
// that thread consecutive 32-bit columns of its own lane.
#pragma once

#include <stdint.h>

#include "tc.cuh"

namespace gca {
namespace tc {

// 32 consecutive columns of the thread's lane, starting at `taddr` (lane base of the
// warp's quarter in bits 16+, column in bits 0-15).
__device__ __forceinline__ void ld32x32b_x32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// 16 consecutive columns of the thread's lane.
__device__ __forceinline__ void ld32x32b_x16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
// Wait for outstanding tcgen05.ld, tied to the loaded registers so that no use of them
// moves above the wait.
__device__ __forceinline__ void ld_wait_row(float (&v)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
        "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
        "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
        "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void ld_wait_row(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15]));
}
// 8 consecutive 32-bit columns of the thread's lane.
__device__ __forceinline__ void st32x32b_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// One 32-bit column of the thread's lane.
__device__ __forceinline__ void st32x32b_x1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void ld32x32b_x1(uint32_t taddr, float& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(taddr));
}
__device__ __forceinline__ void ld_wait_row(float (&v)[1]) { asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(v[0])); }

// Rows in registers, one a lane, U units of 16 bytes each, to memory with U lanes a row: lane i's unit j becomes lane j's
// unit i.  (Each lane its own row, an instruction touches 32 lines: the forward attention over prompts was 5 to 9 %
// slower.)  `to` is unit 0 of row 0, `pos` the lane's row; rows from `len` on and units from `units` on are left out.
template <int U>
__device__ __forceinline__ void store_rows(uint4 (&x)[U], uint4* to, int64_t stride, int pos, int len, int units) {
#pragma unroll
  for (int d = 1; d < U; d <<= 1) {
    const bool up = threadIdx.x & d;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i & d) continue;
      uint4 &lo = x[i], &hi = x[i | d], v;
      v.x = __shfl_xor_sync(0xffffffffu, up ? lo.x : hi.x, d);
      v.y = __shfl_xor_sync(0xffffffffu, up ? lo.y : hi.y, d);
      v.z = __shfl_xor_sync(0xffffffffu, up ? lo.z : hi.z, d);
      v.w = __shfl_xor_sync(0xffffffffu, up ? lo.w : hi.w, d);
      if (up) lo = v;
      else hi = v;
    }
  }
  const int at = threadIdx.x & (U - 1), first = pos - at, rows = at < units ? len - first : 0;
  to += first * stride + at;
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (i < rows) to[i * stride] = x[i];
}

// Announcement of `bytes`, and a 4-D TMA tile load, by one elected lane of a converged warp that
// calls with the same operands (a one-lane branch around them costs about twice the issue time).
__device__ __forceinline__ void mbar_expect_tx_warp(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(su32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_warp(void* dst, const void* tmap, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n}\n" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(su32(bar))
      : "memory");
}

// TMA tile load of a 2-D tensor map (x innermost; x times the element size must be a
// multiple of 16 bytes), completing on `bar`.
__device__ __forceinline__ void tma_load_2d(void* dst, const void* tmap, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(su32(bar))
      : "memory");
}

// TMA tile load of a 3-D tensor map (x innermost, same alignment rule), completing on `bar`.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(su32(bar))
      : "memory");
}

// TMA tile store of a 2-D tensor map from shared memory (bulk-group completion); rows or
// columns outside the tensor are not written.  x and y must not be negative.
__device__ __forceinline__ void tma_store_2d(const void* tmap, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(su32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Wait until at most N bulk groups of this thread still read their shared-memory source.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// Wait until every bulk group of this thread has completed (its writes performed).
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace tc
}  // namespace gca
