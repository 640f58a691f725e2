// Pages of a K/V cache: appending rows, forking, trimming and compacting.
//
// A pool holds pages of 64 tokens (the chunks of the retrieval store); table[slot][p] is the
// page with the slot's tokens 64 p .. 64 p + 63, or -1; refs[page] counts the slots that
// hold it, 0 for a free page.  refs is the only record of what is free: a call takes the
// free pages with the lowest numbers, in the order of its entries, so that equal states and
// calls give equal states whatever the timing.
//
// Bound by memory where rows move (every byte is read and written once), by launch and
// dependent loads where only the tables change.  Measured: 4 prompts of 16K tokens of 12 heads of
// 64 into fresh pages, 65 us (6.2 TB/s, 91 % of a plain copy); a pool of 16384 pages
// of which half are held and 4096 move down, 160 us (90 %); 64 slots' five tokens, 4.2 us; 32 forks of 64 pages, 2.5; 64
// trims, 1.7; 2048 pages given back, 2.7; 64 x 8 lookups, 1.6.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gca {
namespace {

constexpr int kPlanThreads = kCacheEntries;  // one thread an entry

__device__ __forceinline__ void flag_full(ErrWord* e) {
  if (e) atomicOr(&e->flags, kErrFull);
}

// The slot of entry i; entries whose slot is out of range, or was named by an earlier
// entry, are flagged and left out (-1).  `all` holds every entry's slot as given.
__device__ __forceinline__ int given_slot(const CacheArgs& c, int i) { return c.slot ? c.slot[i] : i; }
__device__ __forceinline__ int checked_slot(const CacheArgs& c, const int* all, int i) {
  const int s = all[i];
  bool bad = s < 0 || s >= c.slots;
  if (c.slot)
    for (int j = 0; j < i && !bad; ++j) bad = all[j] == s;
  if (bad) flag_bad_index(c.err, s);
  return bad ? -1 : s;
}

// Inclusive sum over the block's 1024 threads; `red` holds 32 values.
__device__ __forceinline__ int block_scan(int v, int* red, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) red[warp] = v;
  __syncthreads();
  int w = red[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int base = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  __syncthreads();
  return v + (warp ? base : 0);
}

// ------------------------------------------------------------------ append
// One CTA, one thread an entry: what each entry needs, the free pages in order, the tables.  One
// CTA, because an entry's pages depend on what all before it took; the chain of its loads (slot,
// length, last page, its count, the counts of the pool) is most of the 3 us it takes.
__global__ void __launch_bounds__(kPlanThreads) append_plan_kernel(AppendArgs a) {
  const CacheArgs& c = a.c;
  let_next();
  __shared__ int all[kCacheEntries], start[kCacheEntries], first[kCacheEntries];
  __shared__ int red[32];
  const int i = threadIdx.x;
  all[i] = i < c.n ? given_slot(c, i) : -1;
  __syncthreads();
  int slot = -1, old = 0, take = 0, hold = -1, span = 0;
  if (a.offsets) {  // rows offsets[i] .. offsets[i + 1] - 1 of a packed tensor of T rows
    const int from = i < c.n ? a.offsets[i] : 0, to = i < c.n ? a.offsets[i + 1] : 0;
    const bool bad = from < 0 || to < from || to > a.T;
    if (bad) flag_bad_index(c.err, from < 0 || from > a.T ? from : to);
    // Out of order, they could ask for more rows than there are, and for more pages than the scratch holds.
    span = __syncthreads_or(bad) ? 0 : to - from;
  }
  if (i < c.n) {
    slot = checked_slot(c, all, i);
    if (slot >= 0) {
      take = a.offsets ? span : a.counts[i];
      old = c.lengths[slot];
      if (take < 0 || take > a.T) {
        flag_bad_index(c.err, take);
        take = 0;
      }
      if (old < 0 || old > (int64_t)c.width * kChunk) {
        flag_bad_index(c.err, old);
        take = 0;
      } else if ((int64_t)old + take > (int64_t)c.width * kChunk) {
        flag_full(c.err);
        take = 0;
      }
      if (take > 0 && old % kChunk) {
        hold = c.table[(int64_t)slot * c.width + old / kChunk];
        if (hold < 0 || hold >= c.pages) {
          flag_bad_index(c.err, hold);
          take = 0;
          hold = -1;
        }
      }
    }
  }
  // A last page that several slots hold is copied for each entry that writes to it (its
  // readers of this call and those that keep it see the rows as they are).
  const bool copy = hold >= 0 && c.refs[hold] > 1;
  const int f = copy ? old / kChunk : (old + kChunk - 1) / kChunk;
  const int need = take > 0 ? (old + take + kChunk - 1) / kChunk - f : 0;
  int total;
  const int incl = block_scan(need, red, total);
  start[i] = incl - need;
  first[i] = f;
  __syncthreads();
  // The first `total` free pages, in order.
  int found = 0;
  for (int64_t p0 = 0; p0 < c.pages && found < total; p0 += 4 * kPlanThreads) {
    const int64_t p = p0 + 4 * i;
    int r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = p + k < c.pages ? c.refs[p + k] : 1;
    const int mine = (r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0);
    int got;
    int at = found + block_scan(mine, red, got) - mine;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r[k] == 0) {
        if (at < total) a.fresh[at] = (int)(p + k);
        ++at;
      }
    found += got;
  }
  found = min(found, total);
  __syncthreads();
  // Entries are served in order; from the first that the free pages do not reach, none is.
  const bool served = take > 0 && start[i] + need <= found;
  if (take > 0 && !served) flag_full(c.err);
  int hand;
  block_scan(served ? need : 0, red, hand);  // pages that are handed out: entries are a prefix
  for (int k = i; k < hand; k += kPlanThreads) {
    int lo = 0, hi = c.n - 1;  // the last entry whose pages start at k or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= k) lo = mid;
      else hi = mid - 1;
    }
    const int page = a.fresh[k];
    c.table[(int64_t)all[lo] * c.width + first[lo] + k - start[lo]] = page;
    c.refs[page] = 1;
  }
  if (served) {
    if (copy) atomicSub(&c.refs[hold], 1);
    c.lengths[slot] = old + take;
  }
  if (i < c.n) {
    int4* rec = reinterpret_cast<int4*>(a.rec) + i;
    *rec = make_int4(old, served ? take : 0, served && copy ? hold : -1, slot);
  }
  if (a.steps) {  // pages that the entries up to this one write to
    int all_steps;
    const int sum = block_scan(served ? (old + take - 1) / kChunk - old / kChunk + 1 : 0, red, all_steps);
    if (i < c.n) a.steps[i] = sum;
  }
}

// CTA (page step, entry): the rows of one page, a quarter of them a CTA.  A thread has the
// loads of kFly units of K and of V on their way before it stores the first.  Bound by memory
// (a prompt: 6.2 TB/s read and written).
constexpr int kRowParts = 4;
constexpr int kFly = 3;
__global__ void __launch_bounds__(256) append_rows_kernel(AppendArgs a) {
  const CacheArgs& c = a.c;
  after_previous();
  const int i = blockIdx.y, step = blockIdx.x / kRowParts, part = blockIdx.x % kRowParts;
  const int4 rec = reinterpret_cast<const int4*>(a.rec)[i];
  const int old = rec.x, now = old + rec.y, slot = rec.w;
  const int p = old / kChunk + step;
  if (rec.y == 0 || (int64_t)p * kChunk >= now) return;
  const int64_t page = c.table[(int64_t)slot * c.width + p];
  const int units = (int)(c.token_bytes / 16), per = kChunk / kRowParts, r0 = part * per;
  const bool copied = rec.z >= 0 && step == 0;
  // Rows first .. end - 1 of this part are written.
  const int first = copied ? r0 : max(r0, old - p * kChunk), end = min(r0 + per, now - p * kChunk);
  for (int u0 = first * units + threadIdx.x; u0 < end * units; u0 += kFly * blockDim.x) {
    uint4 kv[kFly], vv[kFly];
    bool on[kFly];
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int u = u0 + f * blockDim.x;
      on[f] = u < end * units;
      if (!on[f]) continue;
      const int r = u / units, x = u - r * units, t = p * kChunk + r - old;  // row of the page; token of the entry
      const unsigned char *k, *v;
      if (t >= 0) {
        int row = t;
        if (a.path) {
          row = a.path[(int64_t)i * a.T + t];
          if (row < 0 || row >= a.T) {
            if (x == 0) flag_bad_index(c.err, row);
            on[f] = false;
            continue;
          }
        }
        k = a.kn + i * a.kn_bs + row * a.kn_ts + x * 16;
        v = a.vn + i * a.vn_bs + row * a.vn_ts + x * 16;
      } else {
        const int64_t from = ((int64_t)rec.z * kChunk + r) * c.token_bytes + x * 16;
        k = c.kp + from;
        v = c.vp + from;
      }
      kv[f] = *reinterpret_cast<const uint4*>(k);
      vv[f] = *reinterpret_cast<const uint4*>(v);
    }
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      if (!on[f]) continue;
      const int64_t to = page * kChunk * c.token_bytes + (int64_t)(u0 + f * blockDim.x) * 16;
      *reinterpret_cast<uint4*>(c.kp + to) = kv[f];
      *reinterpret_cast<uint4*>(c.vp + to) = vv[f];
    }
  }
}

// ------------------------------------------------------------------ fork
// One CTA a pair.  A pair whose destination is not empty, is named by an earlier pair, or
// whose source is a destination of the call, is flagged and left out.
__global__ void __launch_bounds__(1024) fork_kernel(CacheArgs c, const int32_t* dst) {
  const int i = blockIdx.x;
  const int s = c.slot[i], d = dst[i];
  bool bad = s < 0 || s >= c.slots || d < 0 || d >= c.slots;
  for (int j = threadIdx.x; j < c.n; j += blockDim.x) bad = bad || dst[j] == s || (j < i && dst[j] == d);
  if (!bad) bad = c.lengths[d] != 0;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag_bad_index(c.err, d);
    return;
  }
  for (int p = threadIdx.x; p < c.width; p += blockDim.x) {
    int t = c.table[(int64_t)s * c.width + p];
    if (t < -1 || t >= c.pages) {
      flag_bad_index(c.err, t);
      t = -1;
    }
    if (t >= 0) atomicAdd(&c.refs[t], 1);
    c.table[(int64_t)d * c.width + p] = t;
  }
  if (threadIdx.x == 0) c.lengths[d] = c.lengths[s];
}

// ------------------------------------------------------------------ trim
// One CTA an entry: keeps tokens begin .. end - 1; pages that lie outside are given back.
__global__ void __launch_bounds__(1024) trim_kernel(CacheArgs c, const int32_t* begin, const int32_t* end, int release) {
  const int i = blockIdx.x;
  const int s = given_slot(c, i);
  bool bad = s < 0 || s >= c.slots;
  if (c.slot)
    for (int j = threadIdx.x; j < i; j += blockDim.x) bad = bad || c.slot[j] == s;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag_bad_index(c.err, s);
    return;
  }
  const int len = max(c.lengths[s], 0);
  const int hi = release ? 0 : (end ? min(max(end[i], 0), len) : len);
  const int lo = begin ? min(max(begin[i], 0), hi) : 0;
  __syncthreads();  // every thread has read the length
  for (int p = threadIdx.x; p < c.width; p += blockDim.x) {
    const int64_t j = (int64_t)p * kChunk;
    if (j + kChunk > lo && j < hi) continue;
    int32_t* at = c.table + (int64_t)s * c.width + p;
    const int t = *at;
    if (t == -1) continue;
    *at = -1;
    if (t < -1 || t >= c.pages) {
      flag_bad_index(c.err, t);
    } else if (atomicSub(&c.refs[t], 1) <= 0) {  // not counted for this slot
      atomicAdd(&c.refs[t], 1);
      flag_bad_index(c.err, t);
    }
  }
  if (threadIdx.x == 0) c.lengths[s] = hi;
}

// ------------------------------------------------------------------ compact
// With n pages in use, those numbered n and above move, in order, to the free numbers
// below n, in order: no other choice moves fewer.  Three launches: uses per part of the
// pool; the two lists, and for every page its rank (-1: free; n and above: its place among those
// that move); the rows and the tables.  A pool of up to kSmallPool pages takes two: one
// CTA makes the lists.
__global__ void __launch_bounds__(256) compact_count_kernel(CompactArgs a) {
  let_next();
  const int64_t per = (a.c.pages + kCompactParts - 1) / kCompactParts;
  const int64_t p0 = min(blockIdx.x * per, a.c.pages), p1 = min(p0 + per, a.c.pages);
  int n = 0;
  for (int64_t p = p0 + threadIdx.x; p < p1; p += blockDim.x) n += a.c.refs[p] > 0;
  __shared__ int sum;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  if ((threadIdx.x & 31) == 0) atomicAdd(&sum, n);
  __syncthreads();
  if (threadIdx.x == 0) a.counts[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(1024) compact_lists_kernel(CompactArgs a) {
  __shared__ int red[32];
  __shared__ int extra;
  after_previous();
  let_next();
  const int64_t per = (a.c.pages + kCompactParts - 1) / kCompactParts;
  if (threadIdx.x == 0) extra = 0;
  __syncthreads();
  // Pages in use: all, before this part, and below page n in whole parts (each warp for itself).
  auto uses = [&](int parts) {
    int sum = 0;
    for (int k = threadIdx.x & 31; k < parts; k += 32) sum += a.counts[k];
    return __reduce_add_sync(0xffffffffu, sum);
  };
  const int n = uses(kCompactParts);
  int before = uses(blockIdx.x);
  const int whole = (int)(n / per);
  int below = uses(whole);
  int mine = 0;
  for (int64_t p = whole * per + threadIdx.x; p < n; p += blockDim.x) mine += a.c.refs[p] > 0;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
  if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&extra, mine);
  __syncthreads();
  below += extra;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.live[0] = n;
    a.counts[kCompactParts] = n - below;  // pages that move
  }
  const int64_t q0 = min(blockIdx.x * per, a.c.pages), q1 = min(q0 + per, a.c.pages);
  for (int64_t base = q0; base < q1; base += blockDim.x) {
    const int64_t p = base + threadIdx.x;
    const int used = p < q1 && a.c.refs[p] > 0;
    int got;
    const int rank = before + block_scan(used, red, got) - used;  // uses before page p
    before += got;
    if (p >= q1) continue;
    if (used && p >= n) a.movers[rank - below] = (int)p;
    if (!used && p < n) a.holes[p - rank] = (int)p;
    a.rank[p] = used ? max(rank - below, 0) : -1;
  }
}

// One CTA, eight pages in a row a thread.  With nothing to move, two launches against three: 1024
// pages 3.4 and 7.8 us, 8192 pages 6.0 and 8.0.
constexpr int kSmallPages = 8, kSmallPool = 1024 * kSmallPages;
__global__ void __launch_bounds__(1024) compact_small_kernel(CompactArgs a) {
  __shared__ int red[32];
  __shared__ int below;
  let_next();
  const int pages = (int)a.c.pages, p0 = threadIdx.x * kSmallPages;
  uint32_t used = 0;
#pragma unroll
  for (int k = 0; k < kSmallPages; ++k)
    if (p0 + k < pages && a.c.refs[p0 + k] > 0) used |= 1u << k;
  int n;
  const int before = block_scan(__popc(used), red, n) - __popc(used);  // uses before page p0
  auto rank = [&](int k) { return before + __popc(used & ((1u << k) - 1)); };
  if (n - p0 >= 0 && n - p0 < kSmallPages) below = rank(n - p0);
  if (threadIdx.x == 0 && n == kSmallPool) below = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    a.live[0] = n;
    a.counts[kCompactParts] = n - below;  // pages that move
  }
#pragma unroll
  for (int k = 0; k < kSmallPages; ++k) {
    const int p = p0 + k;
    if (p >= pages) break;
    const bool on = (used >> k) & 1;
    if (on && p >= n) a.movers[rank(k) - below] = p;
    if (!on && p < n) a.holes[p - rank(k)] = p;
    a.rank[p] = on ? max(rank(k) - below, 0) : -1;
  }
}

constexpr int kMoveParts = 8;
__global__ void __launch_bounds__(256) compact_move_kernel(CompactArgs a) {
  const CacheArgs& c = a.c;
  after_previous();
  const int n = a.live[0], moves = a.counts[kCompactParts];
  const int64_t page16 = kChunk * c.token_bytes / 16, per16 = page16 / kMoveParts;
  for (int64_t w = blockIdx.x; w < (int64_t)moves * kMoveParts; w += gridDim.x) {
    const int k = (int)(w / kMoveParts), part = (int)(w % kMoveParts);
    const int64_t src = a.movers[k] * page16 + part * per16, dst = a.holes[k] * page16 + part * per16;
    const uint4 *ks = reinterpret_cast<const uint4*>(c.kp) + src, *vs = reinterpret_cast<const uint4*>(c.vp) + src;
    uint4 *kd = reinterpret_cast<uint4*>(c.kp) + dst, *vd = reinterpret_cast<uint4*>(c.vp) + dst;
    for (int64_t u = threadIdx.x; u < per16; u += kFly * blockDim.x) {
      uint4 x[kFly], y[kFly];
#pragma unroll
      for (int f = 0; f < kFly; ++f) {
        if (u + f * blockDim.x >= per16) continue;
        x[f] = ks[u + f * blockDim.x];
        y[f] = vs[u + f * blockDim.x];
      }
#pragma unroll
      for (int f = 0; f < kFly; ++f) {
        if (u + f * blockDim.x >= per16) continue;
        kd[u + f * blockDim.x] = x[f];
        vd[u + f * blockDim.x] = y[f];
      }
    }
    if (part == 0 && threadIdx.x == 0) {
      c.refs[a.holes[k]] = c.refs[a.movers[k]];
      c.refs[a.movers[k]] = 0;
    }
  }
  const int64_t all = (int64_t)c.slots * c.width;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < all; e += (int64_t)gridDim.x * blockDim.x) {
    const int t = c.table[e];
    if (t == -1) continue;
    // A free page's number is no one's: it may be the new place of a page that moves.  (Its rank tells; the
    // counts change while this runs.)
    const int k = t >= 0 && t < c.pages ? a.rank[t] : -1;
    if (k < 0) {
      flag_bad_index(c.err, t);
      c.table[e] = -1;
    } else if (t >= n) {
      c.table[e] = a.holes[k];
    }
  }
}

// ------------------------------------------------------------------ lookup
__global__ void __launch_bounds__(256) lookup_kernel(CacheArgs c, const int32_t* idx, int per, int32_t* out) {
  const int i = blockIdx.y, e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= per) return;
  const int64_t at = (int64_t)i * per + e;
  const int s = given_slot(c, i), j = idx[at];
  int page = -1;
  if (s < 0 || s >= c.slots) flag_bad_index(c.err, s);
  else if (j < -1 || j >= c.width) flag_bad_index(c.err, j);
  else if (j >= 0) page = c.table[(int64_t)s * c.width + j];
  out[at] = page;
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  launch_begin("cache_append_plan", s);
  append_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
  cudaError_t e = launch_end("cache_append_plan", s);
  if (e != cudaSuccess) return e;
  if (a.steps) return launch_quantise_rows(a, s);
  const int steps = (a.T + kChunk - 1) / kChunk + 1;
  launch_begin("cache_append_rows", s);
  e = launch_after(append_rows_kernel, dim3(steps * kRowParts, a.c.n), dim3(256), s, a);
  const cudaError_t last = launch_end("cache_append_rows", s);
  return e != cudaSuccess ? e : last;
}

cudaError_t launch_cache_fork(const CacheArgs& c, const int32_t* dst, cudaStream_t s) {
  launch_begin("cache_fork", s);
  fork_kernel<<<c.n, 1024, 0, s>>>(c, dst);
  return launch_end("cache_fork", s);
}

cudaError_t launch_cache_trim(const CacheArgs& c, const int32_t* begin, const int32_t* end, int release, cudaStream_t s) {
  launch_begin("cache_trim", s);
  trim_kernel<<<c.n, 1024, 0, s>>>(c, begin, end, release);
  return launch_end("cache_trim", s);
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t s) {
  cudaError_t e, last;
  if (a.c.pages <= kSmallPool) {
    launch_begin("cache_compact_small", s);
    compact_small_kernel<<<1, 1024, 0, s>>>(a);
    e = launch_end("cache_compact_small", s);
    if (e != cudaSuccess) return e;
  } else {
    launch_begin("cache_compact_count", s);
    compact_count_kernel<<<kCompactParts, 256, 0, s>>>(a);
    e = launch_end("cache_compact_count", s);
    if (e != cudaSuccess) return e;
    launch_begin("cache_compact_lists", s);
    e = launch_after(compact_lists_kernel, dim3(kCompactParts), dim3(1024), s, a);
    last = launch_end("cache_compact_lists", s);
    if (e != cudaSuccess || last != cudaSuccess) return e != cudaSuccess ? e : last;
  }
  launch_begin("cache_compact_move", s);
  e = launch_after(compact_move_kernel, dim3(kSMs * 6), dim3(256), s, a);
  last = launch_end("cache_compact_move", s);
  return e != cudaSuccess ? e : last;
}

cudaError_t launch_cache_lookup(const CacheArgs& c, const int32_t* idx, int per, int32_t* out, cudaStream_t s) {
  launch_begin("cache_lookup", s);
  lookup_kernel<<<dim3((per + 255) / 256, c.n), 256, 0, s>>>(c, idx, per, out);
  return launch_end("cache_lookup", s);
}

}  // namespace gca
