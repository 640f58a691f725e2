// C ABI entry points of the GCA library: argument validation, workspace carving, kernel
// launches, the device error word and launch instrumentation.  The operations
// themselves are documented in include/gca.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "../../include/gca.h"
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace gca {
namespace {

thread_local std::string t_detail;

gca_status fail(gca_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gca_status fail(gca_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_detail = buf;
  return s;
}

gca_status cuda_fail(cudaError_t e, const char* where) {
  return fail(GCA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// ---------------------------------------------------------------- instrumentation
std::atomic<uint64_t> g_launches{0};
std::mutex g_mu;
bool g_prof = false;
struct Rec {
  const char* name;
  cudaEvent_t a, b;
};
std::vector<Rec> g_open;      // recorded, not yet collected
std::vector<cudaEvent_t> g_pool;
struct Row {
  std::string name;
  int launches;
  double ms;
};
std::vector<Row> g_table;

cudaEvent_t take_event() {
  if (!g_pool.empty()) {
    cudaEvent_t e = g_pool.back();
    g_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  cudaEventCreate(&e);
  return e;
}

}  // namespace

void launch_begin(const char* name, cudaStream_t s) {
  if (!g_prof) return;
  std::lock_guard<std::mutex> lk(g_mu);
  Rec r{name, take_event(), take_event()};
  cudaEventRecord(r.a, s);
  g_open.push_back(r);
}

cudaError_t launch_end(const char* name, cudaStream_t s) {
  cudaError_t e = cudaGetLastError();
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (g_prof) {
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto it = g_open.rbegin(); it != g_open.rend(); ++it) {
      if (it->name == name) {
        cudaEventRecord(it->b, s);
        break;
      }
    }
  }
  return e;
}

int set_error_detail(const char* msg) {
  t_detail = msg;
  return 0;
}

cudaError_t allow_smem(const void* fn, int bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  struct Done {
    const void* fn;
    int dev, bytes;
  };
  static std::mutex mu;
  static std::vector<Done> done;  // largest limit set so far per (function, device)
  std::lock_guard<std::mutex> lk(mu);
  for (auto& d : done)
    if (d.fn == fn && d.dev == dev) {
      if (d.bytes >= bytes) return cudaSuccess;
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e == cudaSuccess) d.bytes = bytes;
      return e;
    }
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.push_back(Done{fn, dev, bytes});
  return e;
}

}  // namespace gca

using namespace gca;

// ==================================================================== common
extern "C" const char* gca_status_string(gca_status s) {
  switch (s) {
    case GCA_OK: return "GCA_OK";
    case GCA_ERR_INVALID_ARG: return "GCA_ERR_INVALID_ARG";
    case GCA_ERR_UNSUPPORTED: return "GCA_ERR_UNSUPPORTED";
    case GCA_ERR_WORKSPACE: return "GCA_ERR_WORKSPACE";
    case GCA_ERR_CUDA: return "GCA_ERR_CUDA";
    case GCA_ERR_DEVICE_INDEX: return "GCA_ERR_DEVICE_INDEX";
    case GCA_ERR_TIMEOUT: return "GCA_ERR_TIMEOUT";
    case GCA_ERR_CACHE_FULL: return "GCA_ERR_CACHE_FULL";
  }
  return "unknown gca_status";
}

extern "C" const char* gca_last_error_detail(void) { return t_detail.c_str(); }

static gca_status check_ws(void* ws, size_t have, size_t need) {
  if (ws == nullptr) return fail(GCA_ERR_WORKSPACE, "workspace pointer is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255) return fail(GCA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (have < need) return fail(GCA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return GCA_OK;
}

static gca_status check_landmarks(const void* q, int64_t q_rs, int64_t q_bs, const void* k, int64_t k_bs,
                                  gca_dtype dt, int B, int nQ, int nC, int D, int topk) {
  if (dt != GCA_F32 && dt != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (!q || !k) return fail(GCA_ERR_INVALID_ARG, "landmark pointer is NULL");
  if (B < 1 || nQ < 1 || nC < 1) return fail(GCA_ERR_INVALID_ARG, "B, nQ and nC must be >= 1 (got %d, %d, %d)", B, nQ, nC);
  if (B > 65535) return fail(GCA_ERR_INVALID_ARG, "B must be <= 65535");
  if (topk < 1 || topk > GCA_MAX_TOPK) return fail(GCA_ERR_UNSUPPORTED, "topk must be in 1..16 (got %d)", topk);
  const int epv = dt == GCA_BF16 ? 8 : 4;
  if (dt == GCA_BF16 && (D < 64 || D > 1024 || D % 64))
    return fail(GCA_ERR_UNSUPPORTED, "bf16 landmark dim must be a multiple of 64 in 64..1024 (got %d)", D);
  if (dt == GCA_F32 && (D < 32 || D > 512 || D % 32))
    return fail(GCA_ERR_UNSUPPORTED, "f32 landmark dim must be a multiple of 32 in 32..512 (got %d)", D);
  if (!aligned16(q) || !aligned16(k)) return fail(GCA_ERR_INVALID_ARG, "landmark pointers must be 16-byte aligned");
  if (q_rs < D || q_rs % epv) return fail(GCA_ERR_INVALID_ARG, "q_row_stride must be >= D and a multiple of %d", epv);
  if (q_bs < 0 || q_bs % epv) return fail(GCA_ERR_INVALID_ARG, "q_batch_stride must be >= 0 and a multiple of %d", epv);
  if (B > 1 && q_bs < (int64_t)(nQ - 1) * q_rs + D)
    return fail(GCA_ERR_INVALID_ARG, "q_batch_stride too small for nQ rows");
  if (k_bs != 0 && (k_bs < (int64_t)nC * D || k_bs % epv))
    return fail(GCA_ERR_INVALID_ARG, "k_batch_stride must be 0 or >= nC*D and a multiple of %d", epv);
  return GCA_OK;
}

// ==================================================================== retrieval
extern "C" size_t gca_retrieve_workspace_size(int B, int nQ, int nC, int topk, int causal_offset) {
  if (B < 1 || nQ < 1 || nC < 1 || topk < 1 || causal_offset < 0) return kErrBytes;
  RetrievePlan p = retrieve_plan(B, nQ, nC, topk, causal_offset);
  return kErrBytes + align256(p.part_bytes);
}

gca_status gca::check_retrieve_args(const void* q_lmk, int64_t q_row_stride, int64_t q_batch_stride,
                                    const void* k_lmk, int64_t k_batch_stride, gca_dtype dtype, int B, int nQ,
                                    int nC, int D, int topk, int causal_offset, int use_gumbel, int group,
                                    const int32_t* idx, const float* scores) {
  gca_status st = check_landmarks(q_lmk, q_row_stride, q_batch_stride, k_lmk, k_batch_stride, dtype, B, nQ,
                                  nC, D, topk);
  if (st != GCA_OK) return st;
  if (!idx || !scores) return fail(GCA_ERR_INVALID_ARG, "idx/scores pointer is NULL");
  if (causal_offset < 0) return fail(GCA_ERR_INVALID_ARG, "causal_offset must be >= 0");
  if (use_gumbel && (B > 256 || nQ > (1 << 24) || nC > (1 << 24) || group < 0 || group > 255))
    return fail(GCA_ERR_INVALID_ARG, "Gumbel noise needs B <= 256, nQ, nC <= 2^24, 0 <= group < 256");
  return GCA_OK;
}

static gca_status retrieve_topk_impl(const void* q_lmk, int64_t q_row_stride, int64_t q_batch_stride,
                                     const void* k_lmk, int64_t k_batch_stride, gca_dtype dtype, int B, int nQ,
                                     int nC, int D, int topk, int causal_offset, int use_gumbel, uint64_t seed,
                                     const uint64_t* seed_dev, int group, int32_t* idx, float* scores, void* ws,
                                     size_t ws_bytes, gca_stream_t stream) {
  gca_status st = check_retrieve_args(q_lmk, q_row_stride, q_batch_stride, k_lmk, k_batch_stride, dtype, B, nQ,
                                      nC, D, topk, causal_offset, use_gumbel, group, idx, scores);
  if (st != GCA_OK) return st;
  if ((st = check_ws(ws, ws_bytes, gca_retrieve_workspace_size(B, nQ, nC, topk, causal_offset))) != GCA_OK)
    return st;
  RetrievePlan p = retrieve_plan(B, nQ, nC, topk, causal_offset);
  RetrieveArgs a{};
  a.q = q_lmk; a.q_rs = q_row_stride; a.q_bs = q_batch_stride;
  a.k = k_lmk; a.k_bs = k_batch_stride;
  a.bf16 = dtype == GCA_BF16;
  a.B = B; a.nQ = nQ; a.nC = nC; a.D = D; a.topk = topk; a.off = causal_offset;
  a.gumbel = use_gumbel ? 1 : 0; a.seed = seed; a.group = group; a.seed_dev = seed_dev;
  a.idx = idx; a.scores = scores;
  a.err = reinterpret_cast<ErrWord*>(ws);
  a.part = static_cast<unsigned char*>(ws) + kErrBytes;
  cudaError_t e = launch_retrieve(a, p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_retrieve_topk launch");
  return GCA_OK;
}

extern "C" gca_status gca_retrieve_topk(const void* q_lmk, int64_t q_row_stride, int64_t q_batch_stride,
                                        const void* k_lmk, int64_t k_batch_stride, gca_dtype dtype, int B,
                                        int nQ, int nC, int D, int topk, int causal_offset, int use_gumbel,
                                        uint64_t seed, int group, int32_t* idx, float* scores, void* ws,
                                        size_t ws_bytes, gca_stream_t stream) {
  return retrieve_topk_impl(q_lmk, q_row_stride, q_batch_stride, k_lmk, k_batch_stride, dtype, B, nQ, nC, D, topk,
                            causal_offset, use_gumbel, seed, nullptr, group, idx, scores, ws, ws_bytes, stream);
}

extern "C" gca_status gca_retrieve_topk_dseed(const void* q_lmk, int64_t q_row_stride, int64_t q_batch_stride,
                                              const void* k_lmk, int64_t k_batch_stride, gca_dtype dtype, int B,
                                              int nQ, int nC, int D, int topk, int causal_offset, int use_gumbel,
                                              const uint64_t* seed, int group, int32_t* idx, float* scores,
                                              void* ws, size_t ws_bytes, gca_stream_t stream) {
  if (!seed || (reinterpret_cast<uintptr_t>(seed) & 7))
    return fail(GCA_ERR_INVALID_ARG, "seed must be a non-NULL, 8-byte aligned device pointer");
  return retrieve_topk_impl(q_lmk, q_row_stride, q_batch_stride, k_lmk, k_batch_stride, dtype, B, nQ, nC, D, topk,
                            causal_offset, use_gumbel, 0, seed, group, idx, scores, ws, ws_bytes, stream);
}

// ==================================================================== GCA forward
static gca_status check_gca(const void* q, const void* k, const void* v, gca_dtype dt, int B, int nQ, int nC,
                            int H, int dh, const int32_t* idx, const float* scores, int topk, int shift,
                            bool need_scores = true) {
  if (dt != GCA_F32 && dt != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (!q || !k || !v || !idx || (need_scores && !scores)) return fail(GCA_ERR_INVALID_ARG, "input pointer is NULL");
  if (B < 1 || nQ < 1 || nC < 1 || H < 1) return fail(GCA_ERR_INVALID_ARG, "B, nQ, nC, H must be >= 1");
  if (B > 65535 || H > 65535) return fail(GCA_ERR_INVALID_ARG, "B and H must be <= 65535");
  if ((int64_t)nQ * 64 > INT32_MAX || (int64_t)nC * 64 > INT32_MAX)
    return fail(GCA_ERR_INVALID_ARG, "sequence too long");
  if (dh != 32 && dh != 64) return fail(GCA_ERR_UNSUPPORTED, "head dim must be 32 or 64 (got %d)", dh);
  if (topk < 1 || topk > GCA_MAX_TOPK) return fail(GCA_ERR_UNSUPPORTED, "topk must be in 1..16 (got %d)", topk);
  if (shift != 0 && shift != 1) return fail(GCA_ERR_INVALID_ARG, "shift must be 0 or 1");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return fail(GCA_ERR_INVALID_ARG, "q/k/v must be 16-byte aligned");
  return GCA_OK;
}

extern "C" size_t gca_forward_workspace_size(void) { return kErrBytes; }

extern "C" gca_status gca_forward(const void* q, const void* k, const void* v, int64_t kv_batch_stride,
                                  gca_dtype dtype, int B, int nQ, int nC, int H, int dh, const int32_t* idx,
                                  const float* scores, int topk, int shift, void* o, float* lse, void* ws,
                                  size_t ws_bytes, gca_stream_t stream) {
  gca_status st = check_gca(q, k, v, dtype, B, nQ, nC, H, dh, idx, scores, topk, shift);
  if (st != GCA_OK) return st;
  if (!o || !lse) return fail(GCA_ERR_INVALID_ARG, "o/lse pointer is NULL");
  if (!aligned16(o) || !aligned16(lse)) return fail(GCA_ERR_INVALID_ARG, "o/lse must be 16-byte aligned");
  const int64_t per_seq = (int64_t)nC * 64 * H * dh;
  if (kv_batch_stride != 0 && (kv_batch_stride < per_seq || kv_batch_stride % 8))
    return fail(GCA_ERR_INVALID_ARG, "kv_batch_stride must be 0 or >= nC*64*H*dh and a multiple of 8");
  if ((st = check_ws(ws, ws_bytes, gca_forward_workspace_size())) != GCA_OK) return st;
  FwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.kv_bs = kv_batch_stride;
  a.bf16 = dtype == GCA_BF16; a.B = B; a.nQ = nQ; a.nC = nC; a.H = H; a.dh = dh;
  a.idx = idx; a.scores = scores; a.topk = topk; a.shift = shift;
  a.o = o; a.lse = lse; a.err = reinterpret_cast<ErrWord*>(ws);
  cudaError_t e = launch_forward(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_forward launch");
  return GCA_OK;
}

// ==================================================================== window attention and CCA
extern "C" gca_status gca_window_forward(const void* q, const void* k, const void* v, gca_dtype dtype, int B,
                                         int L, int H, int dh, int window, void* o, float* lse, int accumulate,
                                         void* ws, size_t ws_bytes, gca_stream_t stream) {
  if (dtype != GCA_F32 && dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (B < 1 || H < 1 || L < 64 || L % 64) return fail(GCA_ERR_INVALID_ARG, "B, H >= 1 and L a positive multiple of 64");
  if (dh != 32 && dh != 64) return fail(GCA_ERR_UNSUPPORTED, "dh must be 32 or 64");
  if (window < 64 || window % 64 || window > 63 * 64)
    return fail(GCA_ERR_UNSUPPORTED, "window must be a multiple of 64 in 64..4032");
  if (L / 64 > 65535 || B > 65535 || H > 65535) return fail(GCA_ERR_UNSUPPORTED, "L/64, B and H must be <= 65535");
  if (!q || !k || !v || !o || !lse) return fail(GCA_ERR_INVALID_ARG, "a pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(GCA_ERR_INVALID_ARG, "q, k, v, o, lse must be 16-byte aligned");
  gca_status st;
  if ((st = check_ws(ws, ws_bytes, gca_forward_workspace_size())) != GCA_OK) return st;
  BlockAttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.kv_bs = (int64_t)L * H * dh;
  a.bf16 = dtype == GCA_BF16; a.B = B; a.nQ = L / 64; a.nC = L / 64; a.H = H; a.dh = dh;
  a.mode = 0; a.window = window; a.o = o; a.lse = lse; a.accumulate = accumulate ? 1 : 0;
  a.err = reinterpret_cast<ErrWord*>(ws);
  cudaError_t e = launch_block_attn(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_window_forward launch");
  return GCA_OK;
}

extern "C" size_t gca_window_backward_workspace_size(int B, int L, int H) {
  if (B < 1 || L < 64 || H < 1) return kErrBytes;
  return kErrBytes + align256((size_t)B * (L / 64) * H * 64 * 4);
}

extern "C" gca_status gca_window_backward(const void* q, const void* k, const void* v, const void* o,
                                          const void* dout, const float* lse, gca_dtype dtype, int B, int L, int H,
                                          int dh, int window, void* dq, void* dk, void* dv, int accumulate,
                                          void* ws, size_t ws_bytes, gca_stream_t stream) {
  if (dtype != GCA_F32 && dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (B < 1 || H < 1 || L < 64 || L % 64) return fail(GCA_ERR_INVALID_ARG, "B, H >= 1 and L a positive multiple of 64");
  if (dh != 32 && dh != 64) return fail(GCA_ERR_UNSUPPORTED, "dh must be 32 or 64");
  if (window < 64 || window % 64 || window > 63 * 64)
    return fail(GCA_ERR_UNSUPPORTED, "window must be a multiple of 64 in 64..4032");
  if (L / 64 > 65535 || B > 65535 || H > 65535) return fail(GCA_ERR_UNSUPPORTED, "L/64, B and H must be <= 65535");
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return fail(GCA_ERR_INVALID_ARG, "a pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(lse) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(GCA_ERR_INVALID_ARG, "all tensors must be 16-byte aligned");
  gca_status st;
  if ((st = check_ws(ws, ws_bytes, gca_window_backward_workspace_size(B, L, H))) != GCA_OK) return st;
  WindowBwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.lse = lse;
  a.Dbuf = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kErrBytes);
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.bf16 = dtype == GCA_BF16; a.B = B; a.nQ = L / 64; a.H = H; a.dh = dh; a.window = window;
  a.mode = 0; a.nC = a.nQ;
  a.accumulate = accumulate ? 1 : 0;
  a.err = reinterpret_cast<ErrWord*>(ws);
  cudaError_t e = launch_window_backward(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_window_backward launch");
  return GCA_OK;
}

extern "C" gca_status gca_cca_forward(const void* q, const void* k, const void* v, int64_t kv_batch_stride,
                                      gca_dtype dtype, int B, int nQ, int nC, int H, int dh, const int32_t* idx,
                                      int topk, int shift, void* o, float* lse, int accumulate, void* ws,
                                      size_t ws_bytes, gca_stream_t stream) {
  gca_status st = check_gca(q, k, v, dtype, B, nQ, nC, H, dh, idx, nullptr, topk, shift, false);
  if (st != GCA_OK) return st;
  if (!o || !lse) return fail(GCA_ERR_INVALID_ARG, "o/lse pointer is NULL");
  if (!aligned16(o) || !aligned16(lse)) return fail(GCA_ERR_INVALID_ARG, "o/lse must be 16-byte aligned");
  const int64_t per_seq = (int64_t)nC * 64 * H * dh;
  if (kv_batch_stride != 0 && (kv_batch_stride < per_seq || kv_batch_stride % 8))
    return fail(GCA_ERR_INVALID_ARG, "kv_batch_stride must be 0 or >= nC*64*H*dh and a multiple of 8");
  if ((st = check_ws(ws, ws_bytes, gca_forward_workspace_size())) != GCA_OK) return st;
  BlockAttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.kv_bs = kv_batch_stride;
  a.bf16 = dtype == GCA_BF16; a.B = B; a.nQ = nQ; a.nC = nC; a.H = H; a.dh = dh;
  a.mode = 1; a.idx = idx; a.topk = topk; a.shift = shift;
  a.o = o; a.lse = lse; a.accumulate = accumulate ? 1 : 0;
  a.err = reinterpret_cast<ErrWord*>(ws);
  cudaError_t e = launch_block_attn(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cca_forward launch");
  return GCA_OK;
}

// ==================================================================== CCA backward
extern "C" size_t gca_cca_backward_workspace_size(int B, int nQ, int nC, int H, int topk) {
  if (B < 1 || nQ < 1 || nC < 1 || H < 1 || topk < 1) return kErrBytes;
  return kErrBytes + align256((size_t)B * nQ * H * 64 * 4) + align256((size_t)B * (nC + 1) * 4) +
         align256((size_t)B * nQ * topk * 4) + align256((size_t)B * nC * 4);
}

extern "C" gca_status gca_cca_backward(const void* q, const void* k, const void* v, const void* o, const void* dout,
                                       const float* lse, gca_dtype dtype, int B, int nQ, int nC, int H, int dh,
                                       const int32_t* idx, int topk, int shift, void* dq, void* dk, void* dv,
                                       int accumulate, void* ws, size_t ws_bytes, gca_stream_t stream) {
  gca_status st = check_gca(q, k, v, dtype, B, nQ, nC, H, dh, idx, nullptr, topk, shift, false);
  if (st != GCA_OK) return st;
  if (!o || !dout || !lse || !dq || !dk || !dv) return fail(GCA_ERR_INVALID_ARG, "a pointer is NULL");
  if (!aligned16(o) || !aligned16(dout) || !aligned16(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(GCA_ERR_INVALID_ARG, "all tensors must be 16-byte aligned");
  if ((st = check_ws(ws, ws_bytes, gca_cca_backward_workspace_size(B, nQ, nC, H, topk))) != GCA_OK) return st;
  unsigned char* base = static_cast<unsigned char*>(ws) + kErrBytes;
  WindowBwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.lse = lse;
  a.Dbuf = reinterpret_cast<float*>(base);
  base += align256((size_t)B * nQ * H * 64 * 4);
  a.csr_off = reinterpret_cast<int32_t*>(base);
  base += align256((size_t)B * (nC + 1) * 4);
  a.csr_ent = reinterpret_cast<int32_t*>(base);
  base += align256((size_t)B * nQ * topk * 4);
  a.csr_cur = reinterpret_cast<int32_t*>(base);
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.bf16 = dtype == GCA_BF16; a.B = B; a.nQ = nQ; a.H = H; a.dh = dh; a.window = 64;
  a.mode = 1; a.nC = nC; a.idx = idx; a.topk = topk; a.shift = shift;
  a.accumulate = accumulate ? 1 : 0;
  a.err = reinterpret_cast<ErrWord*>(ws);
  cudaError_t e = launch_window_backward(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cca_backward launch");
  return GCA_OK;
}

// ==================================================================== chunk encoder
extern "C" size_t gca_chunk_encoder_workspace_size(int B, int nC, int d) {
  if (B < 1 || nC < 1 || d < 1) return kErrBytes;
  const size_t M = (size_t)B * nC * 65;
  return kErrBytes + 2 * align256(M * d * 2) + align256(M * 4 * d * 2);
}

extern "C" gca_status gca_chunk_encoder_forward(const void* x, gca_dtype dtype, int B, int nC, int d, int H,
                                                const gca_encoder_weights* w, void* y, void* k, void* v,
                                                void* k_lmk, void* ws, size_t ws_bytes, gca_stream_t stream) {
  if (dtype != GCA_F32 && dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (dtype != GCA_BF16) return fail(GCA_ERR_UNSUPPORTED, "the encoder runs in bf16 only");
  if (B < 1 || nC < 1 || H < 1) return fail(GCA_ERR_INVALID_ARG, "B, nC, H must be >= 1");
  if (d % 128 || d < 128 || d > 1024) return fail(GCA_ERR_UNSUPPORTED, "d must be a multiple of 128 in 128..1024");
  if (d != 64 * H) return fail(GCA_ERR_UNSUPPORTED, "the encoder's head dim d / H must be 64");
  if ((int64_t)B * nC > (int64_t)INT32_MAX / 65) return fail(GCA_ERR_UNSUPPORTED, "B * nC * 65 must fit in int32");
  if (!w) return fail(GCA_ERR_INVALID_ARG, "weights pointer is NULL");
  const void* ptrs[] = {x, y, k, v, k_lmk, w->ln1_g, w->ln1_b, w->w_qkv, w->b_qkv, w->w_o, w->b_o,
                        w->ln2_g, w->ln2_b, w->w_1, w->b_1, w->w_2, w->b_2, w->w_kv};
  for (const void* p : ptrs) {
    if (!p) return fail(GCA_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned16(p)) return fail(GCA_ERR_INVALID_ARG, "all tensors must be 16-byte aligned");
  }
  gca_status st;
  if ((st = check_ws(ws, ws_bytes, gca_chunk_encoder_workspace_size(B, nC, d))) != GCA_OK) return st;
  const size_t M = (size_t)B * nC * 65;
  unsigned char* base = static_cast<unsigned char*>(ws) + kErrBytes;
  EncoderArgs a{};
  a.x = x; a.B = B; a.nC = nC; a.d = d; a.H = H;
  a.ln1_g = w->ln1_g; a.ln1_b = w->ln1_b; a.b_qkv = w->b_qkv; a.b_o = w->b_o;
  a.ln2_g = w->ln2_g; a.ln2_b = w->ln2_b; a.b_1 = w->b_1; a.b_2 = w->b_2;
  a.w_qkv = w->w_qkv; a.w_o = w->w_o; a.w_1 = w->w_1; a.w_2 = w->w_2; a.w_kv = w->w_kv;
  a.y = y; a.k = k; a.v = v; a.k_lmk = k_lmk;
  a.bufA = base;
  a.bufU = base + align256(M * d * 2);
  a.bufF = base + 2 * align256(M * d * 2);
  a.err = reinterpret_cast<ErrWord*>(ws);
  cudaError_t e = launch_chunk_encoder(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_chunk_encoder_forward launch");
  return GCA_OK;
}

// ==================================================================== chunk gather
extern "C" size_t gca_gather_workspace_size(void) { return kErrBytes; }

extern "C" gca_status gca_gather_chunks(const void* k_src, const void* v_src, int64_t src_batch_stride,
                                        gca_dtype dtype, int B, int nQ, int nC, int H, int dh,
                                        const int32_t* idx, int topk, void* k_dst, void* v_dst,
                                        int32_t* idx_local, void* ws, size_t ws_bytes, gca_stream_t stream) {
  if (dtype != GCA_F32 && dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (B < 1 || nQ < 1 || nC < 1 || H < 1) return fail(GCA_ERR_INVALID_ARG, "B, nQ, nC, H must be >= 1");
  if (topk < 1 || topk > kMaxTopk) return fail(GCA_ERR_UNSUPPORTED, "topk must be in 1..%d", kMaxTopk);
  if (dh != 32 && dh != 64) return fail(GCA_ERR_UNSUPPORTED, "dh must be 32 or 64");
  if (!k_src || !v_src || !idx || !k_dst || !v_dst || !idx_local)
    return fail(GCA_ERR_INVALID_ARG, "a pointer is NULL");
  if (!aligned16(k_src) || !aligned16(v_src) || !aligned16(k_dst) || !aligned16(v_dst))
    return fail(GCA_ERR_INVALID_ARG, "k/v source and destination must be 16-byte aligned");
  const int64_t per_seq = (int64_t)nC * 64 * H * dh;
  if (src_batch_stride != 0 && (src_batch_stride < per_seq || src_batch_stride % 8))
    return fail(GCA_ERR_INVALID_ARG, "src_batch_stride must be 0 or >= nC*64*H*dh and a multiple of 8");
  if ((int64_t)nQ * topk > 65535 || B > 65535) return fail(GCA_ERR_UNSUPPORTED, "nQ*topk and B must be <= 65535");
  gca_status st;
  if ((st = check_ws(ws, ws_bytes, gca_gather_workspace_size())) != GCA_OK) return st;
  GatherArgs a{};
  a.k_src = k_src; a.v_src = v_src; a.src_bs = src_batch_stride;
  a.esize = dtype == GCA_BF16 ? 2 : 4; a.B = B; a.nQ = nQ; a.nC = nC; a.H = H; a.dh = dh; a.topk = topk;
  a.idx = idx; a.k_dst = k_dst; a.v_dst = v_dst; a.idx_local = idx_local;
  a.err = reinterpret_cast<ErrWord*>(ws);
  cudaError_t e = launch_gather(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_gather_chunks launch");
  return GCA_OK;
}

// ==================================================================== GCA backward
namespace {
struct BwdLayout {
  size_t D, dwp, off, ent, cur, wrow, ctr, total;
};
BwdLayout bwd_layout(int B, int nQ, int nC, int H, int topk) {
  BwdLayout L{};
  size_t p = kErrBytes;
  L.D = p; p += align256((size_t)B * nQ * H * topk * 64 * 4);
  L.dwp = p; p += align256((size_t)B * nQ * H * topk * 4);
  L.off = p; p += align256((size_t)B * (nC + 1) * 4);
  L.ent = p; p += align256((size_t)B * nQ * topk * 4);
  L.cur = p; p += align256((size_t)B * nC * 4);
  L.wrow = p; p += align256((size_t)B * nQ * topk * 4);
  L.ctr = p; p += 256;
  L.total = p;
  return L;
}
}  // namespace

extern "C" size_t gca_backward_workspace_size(int B, int nQ, int nC, int H, int topk) {
  if (B < 1 || nQ < 1 || nC < 1 || H < 1 || topk < 1) return kErrBytes;
  return bwd_layout(B, nQ, nC, H, topk).total;
}

extern "C" gca_status gca_backward(const void* q, const void* k, const void* v, gca_dtype dtype, int B, int nQ,
                                   int nC, int H, int dh, const int32_t* idx, const float* scores, int topk,
                                   int shift, const void* dout, const float* lse, void* dq, void* dk, void* dv,
                                   float* dscores, int accumulate_dkv, void* ws, size_t ws_bytes,
                                   gca_stream_t stream) {
  gca_status st = check_gca(q, k, v, dtype, B, nQ, nC, H, dh, idx, scores, topk, shift);
  if (st != GCA_OK) return st;
  if (!dout || !lse || !dq || !dk || !dv || !dscores) return fail(GCA_ERR_INVALID_ARG, "output/gradient pointer is NULL");
  if (!aligned16(dout) || !aligned16(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(GCA_ERR_INVALID_ARG, "dout/lse/dq/dk/dv must be 16-byte aligned");
  if ((st = check_ws(ws, ws_bytes, gca_backward_workspace_size(B, nQ, nC, H, topk))) != GCA_OK) return st;
  BwdLayout L = bwd_layout(B, nQ, nC, H, topk);
  unsigned char* w = static_cast<unsigned char*>(ws);
  BwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.bf16 = dtype == GCA_BF16;
  a.B = B; a.nQ = nQ; a.nC = nC; a.H = H; a.dh = dh;
  a.idx = idx; a.scores = scores; a.topk = topk; a.shift = shift;
  a.dout = dout; a.lse = lse; a.dq = dq; a.dk = dk; a.dv = dv; a.dscores = dscores;
  a.acc_dkv = accumulate_dkv ? 1 : 0;
  a.err = reinterpret_cast<ErrWord*>(ws);
  a.Dbuf = reinterpret_cast<float*>(w + L.D);
  a.dwp = reinterpret_cast<float*>(w + L.dwp);
  a.csr_off = reinterpret_cast<int32_t*>(w + L.off);
  a.csr_ent = reinterpret_cast<int32_t*>(w + L.ent);
  a.csr_cur = reinterpret_cast<int32_t*>(w + L.cur);
  a.wrow = reinterpret_cast<float*>(w + L.wrow);
  a.kv_ctr = reinterpret_cast<int32_t*>(w + L.ctr);
  cudaError_t e = launch_backward(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_backward launch");
  return GCA_OK;
}

// ==================================================================== landmark gradients
namespace {
struct SbLayout {
  size_t off, ent, cur, total;
};
SbLayout sb_layout(int B, int nQ, int nC, int topk) {
  SbLayout L{};
  size_t p = kErrBytes;
  L.off = p; p += align256((size_t)B * (nC + 1) * 4);
  L.ent = p; p += align256((size_t)B * nQ * topk * 4);
  L.cur = p; p += align256((size_t)B * nC * 4);
  L.total = p;
  return L;
}
}  // namespace

extern "C" size_t gca_scores_backward_workspace_size(int B, int nQ, int nC, int topk) {
  if (B < 1 || nQ < 1 || nC < 1 || topk < 1) return kErrBytes;
  return sb_layout(B, nQ, nC, topk).total;
}

extern "C" gca_status gca_scores_backward(const void* q_lmk, int64_t q_row_stride, int64_t q_batch_stride,
                                          const void* k_lmk, int64_t k_batch_stride, gca_dtype dtype, int B,
                                          int nQ, int nC, int D, const int32_t* idx, const float* dscores,
                                          int topk, void* dq_lmk, gca_dtype dq_dtype, int64_t dq_row_stride,
                                          int64_t dq_batch_stride, int dq_accumulate, float* dk_lmk, void* ws,
                                          size_t ws_bytes, gca_stream_t stream) {
  gca_status st = check_landmarks(q_lmk, q_row_stride, q_batch_stride, k_lmk, k_batch_stride, dtype, B, nQ,
                                  nC, D, topk);
  if (st != GCA_OK) return st;
  if (k_batch_stride == 0 && B > 1) return fail(GCA_ERR_INVALID_ARG, "k_batch_stride may not be 0 here");
  if (!idx || !dscores || !dq_lmk || !dk_lmk) return fail(GCA_ERR_INVALID_ARG, "pointer is NULL");
  if (dq_dtype != GCA_F32 && dq_dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dq_dtype must be GCA_F32 or GCA_BF16");
  if (dq_row_stride < D || dq_batch_stride < 0) return fail(GCA_ERR_INVALID_ARG, "dq strides out of range");
  if ((st = check_ws(ws, ws_bytes, gca_scores_backward_workspace_size(B, nQ, nC, topk))) != GCA_OK) return st;
  SbLayout L = sb_layout(B, nQ, nC, topk);
  unsigned char* w = static_cast<unsigned char*>(ws);
  ScoresBwdArgs a{};
  a.q = q_lmk; a.q_rs = q_row_stride; a.q_bs = q_batch_stride;
  a.k = k_lmk; a.k_bs = k_batch_stride;
  a.bf16 = dtype == GCA_BF16; a.B = B; a.nQ = nQ; a.nC = nC; a.D = D;
  a.idx = idx; a.ds = dscores; a.topk = topk;
  a.dq = dq_lmk; a.dq_bf16 = dq_dtype == GCA_BF16; a.dq_rs = dq_row_stride; a.dq_bs = dq_batch_stride;
  a.dq_acc = dq_accumulate ? 1 : 0; a.dk = dk_lmk;
  a.err = reinterpret_cast<ErrWord*>(ws);
  a.csr_off = reinterpret_cast<int32_t*>(w + L.off);
  a.csr_ent = reinterpret_cast<int32_t*>(w + L.ent);
  a.csr_cur = reinterpret_cast<int32_t*>(w + L.cur);
  cudaError_t e = launch_scores_backward(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_scores_backward launch");
  return GCA_OK;
}

// ==================================================================== rotary positions
extern "C" gca_status gca_rotary_frequencies(int rot, double base, gca_rotary_scaling scaling, double factor,
                                             double context, double low, double high, uint64_t* freq) {
  if (rot < 2 || rot > 256 || rot % 2) return fail(GCA_ERR_INVALID_ARG, "rot must be even in 2..256 (got %d)", rot);
  if (!freq) return fail(GCA_ERR_INVALID_ARG, "freq is NULL");
  if (!(base >= 1.0) || !std::isfinite(base)) return fail(GCA_ERR_INVALID_ARG, "base must be finite and >= 1");
  if (scaling < GCA_ROTARY_PLAIN || scaling > GCA_ROTARY_PARTS) return fail(GCA_ERR_INVALID_ARG, "unknown scaling %d", (int)scaling);
  if (scaling != GCA_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(GCA_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (scaling == GCA_ROTARY_PARTS && (!(context >= 1.0) || !std::isfinite(context) || !(high > low) || !std::isfinite(high - low)))
    return fail(GCA_ERR_INVALID_ARG, "parts needs a finite context >= 1 and high > low");
  const double two_pi = 6.283185307179586476925;
  double bs = base;
  if (scaling == GCA_ROTARY_NTK && rot > 2) bs *= std::pow(factor, (double)rot / (rot - 2));
  for (int i = 0; i < rot / 2; ++i) {
    double w = std::pow(bs, -2.0 * i / rot);
    if (scaling == GCA_ROTARY_LINEAR) w /= factor;
    if (scaling == GCA_ROTARY_PARTS) {
      const double c = std::min(1.0, std::max(0.0, (context * w / two_pi - low) / (high - low)));
      w = w * c + w / factor * (1.0 - c);
    }
    freq[i] = (uint64_t)std::llrint(w / two_pi * 18446744073709551616.0);  // w <= 1: below 2^62
  }
  return GCA_OK;
}

// A written tensor's elements must not share addresses: with the axes in the order of their
// strides, each must step over everything the ones before it span.
static bool strides_overlap(const gca_heads& t, int64_t B, int64_t L, int64_t H, int64_t dh) {
  std::pair<int64_t, int64_t> ax[3] = {{t.batch_stride, B}, {t.token_stride, L}, {t.head_stride, H}};
  std::sort(ax, ax + 3);
  int64_t span = dh;
  for (auto& x : ax) {
    if (x.second == 1) continue;
    if (x.first < span) return true;
    span += x.first * (x.second - 1);
  }
  return false;
}

// Runs of bytes that a tensor has: `run` at p + s[0] i + s[1] j + s[2] k, for i < n[0] and so on.
struct Runs {
  const void* p;
  int64_t run, n[3], s[3];
};
static Runs runs_of(const gca_heads& t, int64_t B, int64_t L, int64_t H, int64_t dh, int esize) {
  return Runs{t.data, dh * esize, {B, L, H}, {t.batch_stride * esize, t.token_stride * esize, t.head_stride * esize}};
}
static Runs runs_of(const void* p, int64_t bytes) { return Runs{p, bytes, {1, 1, 1}, {0, 0, 0}}; }

// Whether two tensors share a byte.  Their runs do where the distance of two of them, a sum of multiples of both
// tensors' strides, lies in (-b.run, a.run).  Looked for from the largest stride down, with the multiples by which
// the rest can still reach that range: one to three where the strides nest, as those of views of one tensor do.
// (Strides of two tensors that do not nest could take long: after a million steps they count as sharing.)
static bool share_bytes(const Runs& a, const Runs& b) {
  using Wide = __int128;
  auto span = [](const Runs& x) {
    Wide n = x.run;
    for (int i = 0; i < 3; ++i) n += (Wide)x.s[i] * (x.n[i] - 1);
    return n;
  };
  const Wide apart = (Wide)reinterpret_cast<intptr_t>(b.p) - (Wide)reinterpret_cast<intptr_t>(a.p);
  if (apart >= span(a) || -apart >= span(b)) return false;
  struct Term { Wide s, lo, hi; };  // s x, lo <= x <= hi
  Term t[6];
  int m = 0;
  auto add = [&](Wide s, Wide lo, Wide hi) {
    if (s == 0 || lo == hi) return;
    for (int i = 0; i < m; ++i)
      if (t[i].s == s) {
        t[i].lo += lo;
        t[i].hi += hi;
        return;
      }
    t[m++] = Term{s, lo, hi};
  };
  for (int i = 0; i < 3; ++i) {
    add(b.s[i], 0, b.n[i] - 1);
    add(a.s[i], 1 - a.n[i], 0);
  }
  std::sort(t, t + m, [](const Term& x, const Term& y) { return x.s > y.s; });
  Wide lo[7], hi[7];  // what the terms from i on can add
  lo[m] = hi[m] = 0;
  for (int i = m - 1; i >= 0; --i) {
    lo[i] = lo[i + 1] + t[i].s * t[i].lo;
    hi[i] = hi[i + 1] + t[i].s * t[i].hi;
  }
  auto floored = [](Wide x, Wide y) -> Wide {  // y > 0
    if (x == (int64_t)x && y == (int64_t)y) return (int64_t)x / (int64_t)y - ((int64_t)x % (int64_t)y < 0);  // (the wide division is slow)
    return x / y - (x % y < 0);
  };
  int steps = 1 << 20;
  auto reach = [&](auto& self, int i, Wide d) -> bool {
    if (d + hi[i] <= -b.run || d + lo[i] >= a.run) return false;
    if (i == m || --steps < 0) return true;
    const Wide from = -floored(d + hi[i + 1] + b.run - 1, t[i].s), to = floored(a.run - 1 - lo[i + 1] - d, t[i].s);
    for (Wide x = std::max(from, t[i].lo); x <= std::min(to, t[i].hi); ++x)
      if (self(self, i + 1, d + x * t[i].s)) return true;
    return false;
  };
  return reach(reach, 0, apart);
}

// What gca_rotary and gca_norm_rotary ask of their tensors and sizes.
static gca_status check_turned(const gca_heads* q, const gca_heads* k, const gca_heads* q_out, const gca_heads* k_out,
                               gca_dtype dtype, int B, int L, int H, int Hkv, int dh, int rot, const uint64_t* freq,
                               int64_t position_batch_stride) {
  if (dtype != GCA_F32 && dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (!q || !q_out || !q->data || !q_out->data) return fail(GCA_ERR_INVALID_ARG, "q or q_out is NULL");
  if (!k != !k_out || (k && (!k->data || !k_out->data))) return fail(GCA_ERR_INVALID_ARG, "k and k_out must both be given");
  if (B < 1 || L < 1 || H < 1 || Hkv < (k ? 1 : 0) || (!k && Hkv != 0))
    return fail(GCA_ERR_INVALID_ARG, "B, L, H must be >= 1, and Hkv >= 1 with k, 0 without (got %d, %d, %d, %d)", B, L, H, Hkv);
  if (H > 65535 || Hkv > 65535) return fail(GCA_ERR_INVALID_ARG, "H and Hkv must be <= 65535");
  if ((int64_t)B * L > INT32_MAX || B > 65535) return fail(GCA_ERR_INVALID_ARG, "B * L must be below 2^31, B at most 65535");
  if (dh < 2 || dh > 256) return fail(GCA_ERR_UNSUPPORTED, "head dim must be in 2..256 (got %d)", dh);
  if (rot < 2 || rot > dh || rot % 2) return fail(GCA_ERR_INVALID_ARG, "rot must be even in 2..dh (got %d)", rot);
  if (!freq || (reinterpret_cast<uintptr_t>(freq) & 7)) return fail(GCA_ERR_INVALID_ARG, "freq must be 8-byte aligned and not NULL");
  if (position_batch_stride < 0) return fail(GCA_ERR_INVALID_ARG, "position_batch_stride must be >= 0");
  const int esize = dtype == GCA_BF16 ? 2 : 4;
  for (const gca_heads* t : {q, k, q_out, k_out}) {
    if (!t) continue;
    if (reinterpret_cast<uintptr_t>(t->data) % esize) return fail(GCA_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
    if (t->batch_stride < 0 || t->token_stride < 0 || t->head_stride < 0) return fail(GCA_ERR_INVALID_ARG, "strides must be >= 0");
  }
  if (strides_overlap(*q_out, B, L, H, dh) || (k && strides_overlap(*k_out, B, L, Hkv, dh)))
    return fail(GCA_ERR_INVALID_ARG, "output strides make elements overlap");
  return GCA_OK;
}

extern "C" gca_status gca_rotary(const gca_heads* q, const gca_heads* k, const gca_heads* q_out,
                                 const gca_heads* k_out, gca_dtype dtype, int B, int L, int H, int Hkv, int dh, int rot,
                                 int interleaved, int backward, const uint64_t* freq, const int32_t* positions,
                                 int64_t position_batch_stride, float gain, gca_stream_t stream) {
  gca_status st = check_turned(q, k, q_out, k_out, dtype, B, L, H, Hkv, dh, rot, freq, position_batch_stride);
  if (st != GCA_OK) return st;
  auto same = [](const gca_heads* a, const gca_heads* b) {
    return a->data == b->data && a->batch_stride == b->batch_stride && a->token_stride == b->token_stride &&
           a->head_stride == b->head_stride;
  };
  auto side = [](const gca_heads* i, const gca_heads* o) {
    return RotarySide{i->data, i->batch_stride, i->token_stride, i->head_stride,
                      o->data, o->batch_stride, o->token_stride, o->head_stride};
  };
  RotaryArgs a{};
  a.q = side(q, q_out);
  if (k) a.k = side(k, k_out);
  a.bf16 = dtype == GCA_BF16; a.B = B; a.L = L; a.H = H; a.Hkv = Hkv; a.dh = dh; a.rot = rot;
  a.paired = interleaved ? 1 : 0;
  a.tail = same(q, q_out) && (!k || same(k, k_out)) ? 0 : dh - rot;
  a.freq = freq; a.pos = positions; a.pos_bs = position_batch_stride;
  a.gain = gain; a.sgain = backward ? -gain : gain;
  cudaError_t e = launch_rotary(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_rotary launch");
  return GCA_OK;
}

// ==================================================================== norms with rotary positions
namespace {
gca_status check_weights(const gca_heads* k, float eps, const float* q_weight, const float* k_weight) {
  if (!q_weight || (k && !k_weight)) return fail(GCA_ERR_INVALID_ARG, "a weight is NULL");
  for (const float* w : {q_weight, k_weight})
    if (reinterpret_cast<uintptr_t>(w) & 3) return fail(GCA_ERR_INVALID_ARG, "weights must be 4-byte aligned");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(GCA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return GCA_OK;
}
// Written tensors share no byte with each other, nor with a read one, but that a lane may write each element where it
// read it: of the tensors read in `own`, one may be the written one itself (same pointer and strides).
struct Written {
  const gca_heads* t;
  int heads;
  const gca_heads* own[2];
};
gca_status check_written(std::initializer_list<Written> written, std::initializer_list<Runs> read, int B, int L, int dh, int esize) {
  auto runs = [&](const gca_heads* t, int heads) { return runs_of(*t, B, L, heads, dh, esize); };
  auto itself = [&](const gca_heads* a, const gca_heads* b, int heads) {
    return a->data == b->data && (B == 1 || a->batch_stride == b->batch_stride) && (L == 1 || a->token_stride == b->token_stride) &&
           (heads == 1 || a->head_stride == b->head_stride);
  };
  for (const Written& x : written) {
    if (!x.t) continue;
    const Runs out = runs(x.t, x.heads);
    for (const Runs& y : read)
      if (y.p && share_bytes(out, y)) return fail(GCA_ERR_INVALID_ARG, "an output must not overlap an input");
    for (const Written& y : written) {
      if (!y.t) continue;
      if (&y != &x && share_bytes(out, runs(y.t, y.heads))) return fail(GCA_ERR_INVALID_ARG, "two outputs overlap");
      for (const gca_heads* in : y.own)
        if (in && !(&y == &x && itself(x.t, in, x.heads)) && share_bytes(out, runs(in, y.heads)))
          return fail(GCA_ERR_INVALID_ARG, "an output must be its input itself or not overlap it");
    }
  }
  return GCA_OK;
}
Runs runs_of_positions(const int32_t* positions, int B, int L, int64_t batch_stride) {
  return Runs{positions, (int64_t)L * 4, {B, 1, 1}, {batch_stride * 4, 0, 0}};
}
NormSide norm_side(const gca_heads* in, const gca_heads* dy, const gca_heads* out) {
  NormSide x{};
  x.in = in->data; x.in_bs = in->batch_stride; x.in_ts = in->token_stride; x.in_hs = in->head_stride;
  if (dy) { x.dy = dy->data; x.dy_bs = dy->batch_stride; x.dy_ts = dy->token_stride; x.dy_hs = dy->head_stride; }
  x.out = out->data; x.out_bs = out->batch_stride; x.out_ts = out->token_stride; x.out_hs = out->head_stride;
  return x;
}
}  // namespace

extern "C" gca_status gca_norm_rotary(const gca_heads* q, const gca_heads* k, const gca_heads* q_out, const gca_heads* k_out,
                                      gca_dtype dtype, int B, int L, int H, int Hkv, int dh, int rot, int interleaved,
                                      float eps, const float* q_weight, const float* k_weight, const uint64_t* freq,
                                      const int32_t* positions, int64_t position_batch_stride, float gain,
                                      gca_stream_t stream) {
  gca_status st = check_turned(q, k, q_out, k_out, dtype, B, L, H, Hkv, dh, rot, freq, position_batch_stride);
  if (st != GCA_OK) return st;
  if ((st = check_weights(k, eps, q_weight, k_weight)) != GCA_OK) return st;
  st = check_written({{q_out, H, {q, nullptr}}, {k_out, Hkv, {k, nullptr}}},
                     {runs_of(q_weight, dh * 4), runs_of(k_weight, dh * 4), runs_of(freq, rot * 4), runs_of_positions(positions, B, L, position_batch_stride)},
                     B, L, dh, dtype == GCA_BF16 ? 2 : 4);
  if (st != GCA_OK) return st;
  NormRotaryArgs a{};
  a.q = norm_side(q, nullptr, q_out);
  if (k) a.k = norm_side(k, nullptr, k_out);
  a.bf16 = dtype == GCA_BF16; a.B = B; a.L = L; a.H = H; a.Hkv = Hkv; a.dh = dh; a.rot = rot; a.paired = interleaved ? 1 : 0;
  a.qw = q_weight; a.kw = k_weight; a.freq = freq; a.pos = positions; a.pos_bs = position_batch_stride;
  a.gain = gain; a.sgain = gain; a.eps = eps;
  cudaError_t e = launch_norm_rotary(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_norm_rotary launch");
  return GCA_OK;
}

extern "C" size_t gca_norm_rotary_backward_scratch_size(int dh) {
  return dh < 2 || dh > 256 ? 256 : align256(norm_rotary_scratch_bytes(dh));
}

static gca_status check_scratch(const void* p, size_t have, size_t need) {
  if (p == nullptr) return fail(GCA_ERR_WORKSPACE, "scratch pointer is NULL");
  if (reinterpret_cast<uintptr_t>(p) & 255) return fail(GCA_ERR_WORKSPACE, "scratch is not 256-byte aligned");
  if (have < need) return fail(GCA_ERR_WORKSPACE, "scratch has %zu bytes, needs %zu", have, need);
  return GCA_OK;
}

extern "C" gca_status gca_norm_rotary_backward(const gca_heads* q, const gca_heads* k, const gca_heads* dq_out,
                                               const gca_heads* dk_out, const gca_heads* dq, const gca_heads* dk,
                                               gca_dtype dtype, int B, int L, int H, int Hkv, int dh, int rot,
                                               int interleaved, float eps, const float* q_weight, const float* k_weight,
                                               const uint64_t* freq, const int32_t* positions, int64_t position_batch_stride,
                                               float gain, float* dq_weight, float* dk_weight, void* scratch,
                                               size_t scratch_bytes, gca_stream_t stream) {
  gca_status st = check_turned(q, k, dq, dk, dtype, B, L, H, Hkv, dh, rot, freq, position_batch_stride);
  if (st != GCA_OK) return st;
  if ((st = check_turned(dq_out, dk_out, dq, dk, dtype, B, L, H, Hkv, dh, rot, freq, position_batch_stride)) != GCA_OK) return st;
  if ((st = check_weights(k, eps, q_weight, k_weight)) != GCA_OK) return st;
  if (!dq_weight || (k && !dk_weight)) return fail(GCA_ERR_INVALID_ARG, "a weight's gradient is NULL");
  for (const float* w : {dq_weight, dk_weight})
    if (reinterpret_cast<uintptr_t>(w) & 3) return fail(GCA_ERR_INVALID_ARG, "weights' gradients must be 4-byte aligned");
  if ((st = check_scratch(scratch, scratch_bytes, gca_norm_rotary_backward_scratch_size(dh))) != GCA_OK) return st;
  st = check_written({{dq, H, {q, dq_out}}, {dk, Hkv, {k, dk_out}}},
                     {runs_of(q_weight, dh * 4), runs_of(k_weight, dh * 4), runs_of(freq, rot * 4), runs_of_positions(positions, B, L, position_batch_stride),
                      runs_of(dq_weight, dh * 4), runs_of(dk_weight, dh * 4)},
                     B, L, dh, dtype == GCA_BF16 ? 2 : 4);
  if (st != GCA_OK) return st;
  if (dk_weight && share_bytes(runs_of(dq_weight, dh * 4), runs_of(dk_weight, dh * 4)))
    return fail(GCA_ERR_INVALID_ARG, "the weights' gradients overlap");
  NormRotaryArgs a{};
  a.q = norm_side(q, dq_out, dq);
  if (k) a.k = norm_side(k, dk_out, dk);
  a.bf16 = dtype == GCA_BF16; a.backward = 1; a.B = B; a.L = L; a.H = H; a.Hkv = Hkv; a.dh = dh; a.rot = rot;
  a.paired = interleaved ? 1 : 0;
  a.qw = q_weight; a.kw = k_weight; a.freq = freq; a.pos = positions; a.pos_bs = position_batch_stride;
  a.gain = gain; a.sgain = -gain; a.eps = eps;
  a.partial = static_cast<float*>(scratch); a.dqw = dq_weight; a.dkw = dk_weight;
  cudaError_t e = launch_norm_rotary(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_norm_rotary_backward launch");
  return GCA_OK;
}

// ==================================================================== attention over prompts
namespace {
// A packed tensor whose rows are read (or written) in 16-byte units.
gca_status check_packed(const gca_heads* t, int esize, int N, int heads, const char* what) {
  if (!t || !t->data) return fail(GCA_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned16(t->data)) return fail(GCA_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  if (N > 1 && t->token_stride <= 0) return fail(GCA_ERR_INVALID_ARG, "%s: the token stride must be > 0", what);
  // (in a tensor map a stride has 40 bits of bytes)
  for (int64_t s : {N > 1 ? t->token_stride : 0, heads > 1 ? t->head_stride : 0})
    if (s < 0 || s * esize % 16 || s >= (int64_t)1 << 36)
      return fail(GCA_ERR_INVALID_ARG, "%s: strides must be >= 0, multiples of 16 bytes and below 2^36", what);
  return GCA_OK;
}
gca_status check_prompt(const gca_heads* q, const gca_heads* k, const gca_heads* v, gca_dtype dtype, int N, int B, int H,
                        int Hkv, int dh, const int32_t* offsets, int window, float scale, const void* o, const float* lse) {
  if (dtype != GCA_F32 && dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (N < 0 || N > 1 << 30) return fail(GCA_ERR_INVALID_ARG, "N must be in 0..2^30 (got %d)", N);
  if (B < 1 || B > GCA_MAX_SEQUENCES) return fail(GCA_ERR_INVALID_ARG, "B must be in 1..%d (got %d)", GCA_MAX_SEQUENCES, B);
  if (Hkv < 1 || H < Hkv || H % Hkv || H > 65535) return fail(GCA_ERR_INVALID_ARG, "H must be a multiple of Hkv, at most 65535 (got %d, %d)", H, Hkv);
  if (dh != 32 && dh != 64 && dh != 128) return fail(GCA_ERR_UNSUPPORTED, "head dim must be 32, 64 or 128 (got %d)", dh);
  if (((int64_t)N / 64 + B) * H > INT32_MAX) return fail(GCA_ERR_UNSUPPORTED, "N, B and H are too large together");
  if (window < 0) return fail(GCA_ERR_INVALID_ARG, "window must be >= 0");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(GCA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!offsets || (reinterpret_cast<uintptr_t>(offsets) & 3)) return fail(GCA_ERR_INVALID_ARG, "offsets must be 4-byte aligned and not NULL");
  if (N == 0) return GCA_OK;  // no row: no address is used
  gca_status st;
  const int esize = dtype == GCA_BF16 ? 2 : 4;
  if ((st = check_packed(q, esize, N, H, "q")) != GCA_OK) return st;
  if ((st = check_packed(k, esize, N, Hkv, "k")) != GCA_OK) return st;
  if ((st = check_packed(v, esize, N, Hkv, "v")) != GCA_OK) return st;
  if (!o || !lse || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3))
    return fail(GCA_ERR_INVALID_ARG, "o and lse must not be NULL, o 16-byte aligned");
  return GCA_OK;
}
PromptArgs prompt_args(const gca_heads* q, const gca_heads* k, const gca_heads* v, gca_dtype dtype, int N, int B, int H, int Hkv,
                       int dh, const int32_t* offsets, int window, float scale, const void* o, const float* lse, void* ws) {
  PromptArgs a{};
  auto ts = [&](const gca_heads* t) { return N > 1 ? t->token_stride : 0; };
  a.q = q->data; a.q_ts = ts(q); a.q_hs = H > 1 ? q->head_stride : 0;
  a.k = k->data; a.k_ts = ts(k); a.k_hs = Hkv > 1 ? k->head_stride : 0;
  a.v = v->data; a.v_ts = ts(v); a.v_hs = Hkv > 1 ? v->head_stride : 0;
  a.offsets = offsets; a.N = N; a.bf16 = dtype == GCA_BF16; a.B = B; a.H = H; a.Hkv = Hkv; a.g = H / Hkv; a.dh = dh;
  a.window = window; a.scale = scale;
  a.o = const_cast<void*>(o); a.lse = const_cast<float*>(lse);
  a.err = reinterpret_cast<ErrWord*>(ws);
  return a;
}
}  // namespace

extern "C" gca_status gca_prompt_attention(const gca_heads* q, const gca_heads* k, const gca_heads* v, gca_dtype dtype, int N,
                                           int B, int H, int Hkv, int dh, const int32_t* offsets, int window, float scale,
                                           void* o, float* lse, void* ws, size_t ws_bytes, gca_stream_t stream) {
  gca_status st = check_prompt(q, k, v, dtype, N, B, H, Hkv, dh, offsets, window, scale, o, lse);
  if (st != GCA_OK) return st;
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  if (N == 0) return GCA_OK;
  // Rows are written before others are read.
  const int esize = dtype == GCA_BF16 ? 2 : 4;
  const Runs out[] = {runs_of(o, (int64_t)N * H * dh * esize), runs_of(lse, (int64_t)N * H * 4)};
  const Runs in[] = {runs_of(*q, 1, N, H, dh, esize), runs_of(*k, 1, N, Hkv, dh, esize), runs_of(*v, 1, N, Hkv, dh, esize),
                     runs_of(offsets, ((int64_t)B + 1) * 4)};
  for (const Runs& x : out)
    for (const Runs& y : in)
      if (share_bytes(x, y)) return fail(GCA_ERR_INVALID_ARG, "o and lse must not overlap an input");
  if (share_bytes(out[0], out[1])) return fail(GCA_ERR_INVALID_ARG, "o and lse overlap");
  const PromptArgs a = prompt_args(q, k, v, dtype, N, B, H, Hkv, dh, offsets, window, scale, o, lse, ws);
  cudaError_t e = launch_prompt_forward(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_prompt_attention launch");
  return GCA_OK;
}

extern "C" size_t gca_prompt_attention_backward_scratch_size(int N, int B, int H, int Hkv, int dh, gca_dtype dtype) {
  if (N < 1 || B < 1 || H < 1 || Hkv < 1 || dh < 1) return 256;
  return 2 * align256((size_t)prompt_scratch_rows(N) * 2 * H * sizeof(float)) + align256(prompt_parts_bytes(N, B, Hkv, dh, dtype == GCA_BF16));
}

extern "C" gca_status gca_prompt_attention_backward(const gca_heads* q, const gca_heads* k, const gca_heads* v, const void* o,
                                                    const gca_heads* dout, const float* lse, gca_dtype dtype, int N, int B,
                                                    int H, int Hkv, int dh, const int32_t* offsets, int window, float scale,
                                                    const gca_heads* dq, const gca_heads* dk, const gca_heads* dv, void* ws,
                                                    size_t ws_bytes, void* scratch, size_t scratch_bytes,
                                                    gca_stream_t stream) {
  gca_status st = check_prompt(q, k, v, dtype, N, B, H, Hkv, dh, offsets, window, scale, o, lse);
  if (st != GCA_OK) return st;
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  if (N == 0) return GCA_OK;
  const int esize = dtype == GCA_BF16 ? 2 : 4;
  const struct { const gca_heads* t; int heads; const char* what; } all[] = {{dout, H, "dout"}, {dq, H, "dq"}, {dk, Hkv, "dk"}, {dv, Hkv, "dv"}};
  for (auto& x : all)
    if ((st = check_packed(x.t, esize, N, x.heads, x.what)) != GCA_OK) return st;
  if (strides_overlap(*dq, 1, N, H, dh) || strides_overlap(*dk, 1, N, Hkv, dh) || strides_overlap(*dv, 1, N, Hkv, dh))
    return fail(GCA_ERR_INVALID_ARG, "output strides make elements overlap");
  if ((st = check_scratch(scratch, scratch_bytes, gca_prompt_attention_backward_scratch_size(N, B, H, Hkv, dh, dtype))) != GCA_OK) return st;
  // Each gradient is written before the last input is read.
  const Runs in[] = {runs_of(*q, 1, N, H, dh, esize), runs_of(*k, 1, N, Hkv, dh, esize), runs_of(*v, 1, N, Hkv, dh, esize),
                     runs_of(o, (int64_t)N * H * dh * esize), runs_of(*dout, 1, N, H, dh, esize), runs_of(lse, (int64_t)N * H * 4),
                     runs_of(offsets, ((int64_t)B + 1) * 4)};
  const Runs out[] = {runs_of(*dq, 1, N, H, dh, esize), runs_of(*dk, 1, N, Hkv, dh, esize), runs_of(*dv, 1, N, Hkv, dh, esize)};
  for (int i = 0; i < 3; ++i) {
    for (const Runs& x : in)
      if (share_bytes(out[i], x)) return fail(GCA_ERR_INVALID_ARG, "a gradient must not overlap an input");
    if (share_bytes(out[i], out[(i + 1) % 3])) return fail(GCA_ERR_INVALID_ARG, "two gradients are one tensor, or overlap");
  }
  PromptArgs a = prompt_args(q, k, v, dtype, N, B, H, Hkv, dh, offsets, window, scale, o, lse, ws);
  a.dout = dout->data; a.do_ts = N > 1 ? dout->token_stride : 0; a.do_hs = H > 1 ? dout->head_stride : 0;
  a.dq = dq->data; a.dq_ts = dq->token_stride; a.dq_hs = dq->head_stride;
  a.dk = dk->data; a.dk_ts = dk->token_stride; a.dk_hs = dk->head_stride;
  a.dv = dv->data; a.dv_ts = dv->token_stride; a.dv_hs = dv->head_stride;
  a.np = prompt_scratch_rows(N);
  a.nlse = static_cast<float*>(scratch);
  const size_t rows = align256((size_t)a.np * 2 * H * sizeof(float));
  a.nD = reinterpret_cast<float*>(static_cast<unsigned char*>(scratch) + rows);
  a.parts = reinterpret_cast<float*>(static_cast<unsigned char*>(scratch) + 2 * rows);
  cudaError_t e = launch_prompt_backward(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_prompt_attention_backward launch");
  return GCA_OK;
}

// ==================================================================== paged cache
namespace {
// Bytes of a token's row: a quantised one has a byte a head behind its numbers, up to a multiple of 16.
int64_t row_bytes(gca_dtype dtype, int heads, int dh) {
  const int64_t n = (int64_t)heads * dh;
  return dtype == GCA_E4M3 ? n + ((int64_t)heads + 15) / 16 * 16 : n * (dtype == GCA_BF16 ? 2 : 4);
}
// The page operations take pages of any kind (`any`); what reads or writes numbers takes its own.
gca_status check_cache(const gca_cache* c, bool need_refs, bool any = false) {
  if (!c) return fail(GCA_ERR_INVALID_ARG, "cache is NULL");
  if (c->dtype != GCA_F32 && c->dtype != GCA_BF16 && !(any && c->dtype == GCA_E4M3))
    return fail(GCA_ERR_INVALID_ARG, any ? "dtype must be GCA_F32, GCA_BF16 or GCA_E4M3" : "dtype must be GCA_F32 or GCA_BF16");
  if (!c->k_pages || !c->v_pages || !c->table || !c->lengths || (need_refs && !c->refs))
    return fail(GCA_ERR_INVALID_ARG, "a cache pointer is NULL");
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return fail(GCA_ERR_INVALID_ARG, "pages must be 16-byte aligned");
  // (The page operations may be given a quantised row as one head of what is left beside its exponents.)
  if (c->heads < 1 || c->heads > 65535 || c->dh < 1 || (c->dh > 65535 && c->dtype != GCA_E4M3) || c->pages < 1 || c->slots < 1 || c->width < 1)
    return fail(GCA_ERR_INVALID_ARG, "heads, dh, pages, slots and width must be >= 1 (heads, dh <= 65535)");
  if ((int64_t)c->width * 64 > INT32_MAX) return fail(GCA_ERR_INVALID_ARG, "table too wide: 64 * width must be below 2^31");
  if (row_bytes(c->dtype, c->heads, c->dh) % 16)
    return fail(GCA_ERR_INVALID_ARG, "a token's row (heads * dh elements) must be a multiple of 16 bytes");
  return GCA_OK;
}
gca_status check_quantised(const gca_cache* c, gca_dtype dtype) {
  gca_status st = check_cache(c, false, true);
  if (st != GCA_OK) return st;
  if (c->dtype != GCA_E4M3) return fail(GCA_ERR_INVALID_ARG, "the cache must hold GCA_E4M3");
  if (dtype != GCA_F32 && dtype != GCA_BF16) return fail(GCA_ERR_INVALID_ARG, "dtype must be GCA_F32 or GCA_BF16");
  if (c->dh != 32 && c->dh != 64 && c->dh != 128) return fail(GCA_ERR_UNSUPPORTED, "head dim must be 32, 64 or 128 (got %d)", c->dh);
  return GCA_OK;
}
gca_status check_entries(const gca_cache* c, int n, bool listed) {
  if (n < 1 || n > GCA_MAX_CACHE_ENTRIES) return fail(GCA_ERR_INVALID_ARG, "n must be in 1..%d (got %d)", GCA_MAX_CACHE_ENTRIES, n);
  if (!listed && n > c->slots) return fail(GCA_ERR_INVALID_ARG, "n must be at most the number of slots where no slots are named");
  return GCA_OK;
}
CacheArgs cache_args(const gca_cache* c, int n, const int32_t* slot, void* ws) {
  CacheArgs a{};
  a.kp = static_cast<unsigned char*>(c->k_pages);
  a.vp = static_cast<unsigned char*>(c->v_pages);
  a.pages = c->pages;
  a.token_bytes = row_bytes(c->dtype, c->heads, c->dh);
  a.table = c->table; a.slots = c->slots; a.width = c->width; a.lengths = c->lengths; a.refs = c->refs;
  a.n = n; a.slot = slot;
  a.err = reinterpret_cast<ErrWord*>(ws);
  return a;
}
// A tensor whose rows are read in 16-byte units.
gca_status check_vectors(const gca_heads* t, int esize, const char* what) {
  if (!t || !t->data) return fail(GCA_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned16(t->data)) return fail(GCA_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  for (int64_t s : {t->batch_stride, t->token_stride, t->head_stride})
    if (s < 0 || s * esize % 16) return fail(GCA_ERR_INVALID_ARG, "%s: strides must be >= 0 and multiples of 16 bytes", what);
  return GCA_OK;
}
}  // namespace

extern "C" size_t gca_cache_append_scratch_size(int n, int T) {
  if (n < 1 || T < 1) return 256;
  return align256((size_t)n * kAppendRec * 4) + align256((size_t)n * ((size_t)T / 64 + 2) * 4);
}

extern "C" gca_status gca_cache_append(const gca_cache* cache, const gca_heads* k_new, const gca_heads* v_new, int n,
                                       int T, const int32_t* slot_ids, const int32_t* counts, const int32_t* path,
                                       void* ws, size_t ws_bytes, void* scratch, size_t scratch_bytes,
                                       gca_stream_t stream) {
  gca_status st;
  if ((st = check_cache(cache, true)) != GCA_OK) return st;
  if ((st = check_entries(cache, n, slot_ids != nullptr)) != GCA_OK) return st;
  if (T < 1 || T > INT32_MAX / 2) return fail(GCA_ERR_INVALID_ARG, "T must be in 1..2^30");
  if ((int64_t)n * (T / 64 + 2) > INT32_MAX) return fail(GCA_ERR_INVALID_ARG, "n and T are too large together");
  if (!counts) return fail(GCA_ERR_INVALID_ARG, "counts is NULL");
  const int esize = cache->dtype == GCA_BF16 ? 2 : 4;
  if ((st = check_vectors(k_new, esize, "k_new")) != GCA_OK) return st;
  if ((st = check_vectors(v_new, esize, "v_new")) != GCA_OK) return st;
  if (cache->heads > 1 && (k_new->head_stride != cache->dh || v_new->head_stride != cache->dh))
    return fail(GCA_ERR_INVALID_ARG, "the heads of a new token must be contiguous (head stride dh)");
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  if ((st = check_scratch(scratch, scratch_bytes, gca_cache_append_scratch_size(n, T))) != GCA_OK) return st;
  AppendArgs a{};
  a.c = cache_args(cache, n, slot_ids, ws);
  a.kn = static_cast<const unsigned char*>(k_new->data);
  a.kn_bs = k_new->batch_stride * esize; a.kn_ts = k_new->token_stride * esize;
  a.vn = static_cast<const unsigned char*>(v_new->data);
  a.vn_bs = v_new->batch_stride * esize; a.vn_ts = v_new->token_stride * esize;
  a.counts = counts; a.path = path; a.T = T;
  a.rec = static_cast<int32_t*>(scratch);
  a.fresh = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(scratch) + align256((size_t)n * kAppendRec * 4));
  cudaError_t e = launch_cache_append(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cache_append launch");
  return GCA_OK;
}

extern "C" size_t gca_cache_row_bytes(gca_dtype dtype, int heads, int dh) {
  return heads < 1 || dh < 1 ? 0 : (size_t)row_bytes(dtype, heads, dh);
}

// Pages that the entries of a quantised append can write to: those of n times T rows, or of T rows in all.
static int64_t most_pages(int n, int T, bool packed) { return packed ? T / 64 + 2 * (int64_t)n : n * ((int64_t)T / 64 + 2); }

extern "C" size_t gca_cache_append_quantised_scratch_size(int n, int T, int packed) {
  if (n < 1 || T < 1) return 256;
  return align256((size_t)n * kAppendRec * 4) + align256((size_t)n * 4) + align256((size_t)most_pages(n, T, packed != 0) * 4);
}

extern "C" gca_status gca_cache_append_quantised(const gca_cache* cache, const gca_heads* k_new, const gca_heads* v_new,
                                                 gca_dtype dtype, int n, int T, const int32_t* slot_ids, const int32_t* counts,
                                                 const int32_t* path, const int32_t* offsets, void* ws, size_t ws_bytes,
                                                 void* scratch, size_t scratch_bytes, gca_stream_t stream) {
  gca_status st;
  if ((st = check_quantised(cache, dtype)) != GCA_OK) return st;
  if (!cache->refs) return fail(GCA_ERR_INVALID_ARG, "a cache pointer is NULL");
  if ((st = check_entries(cache, n, slot_ids != nullptr)) != GCA_OK) return st;
  if (T < 1 || T > INT32_MAX / 2) return fail(GCA_ERR_INVALID_ARG, "T must be in 1..2^30");
  if (most_pages(n, T, offsets != nullptr) > INT32_MAX / 4) return fail(GCA_ERR_INVALID_ARG, "n and T are too large together");
  if (!counts == !offsets) return fail(GCA_ERR_INVALID_ARG, "counts or offsets must be given, not both");
  if (offsets && path) return fail(GCA_ERR_INVALID_ARG, "a packed append has no path");
  const int esize = dtype == GCA_BF16 ? 2 : 4;
  if ((st = check_vectors(k_new, esize, "k_new")) != GCA_OK) return st;
  if ((st = check_vectors(v_new, esize, "v_new")) != GCA_OK) return st;
  if (cache->heads > 1 && (k_new->head_stride != cache->dh || v_new->head_stride != cache->dh))
    return fail(GCA_ERR_INVALID_ARG, "the heads of a new token must be contiguous (head stride dh)");
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  if ((st = check_scratch(scratch, scratch_bytes, gca_cache_append_quantised_scratch_size(n, T, offsets != nullptr))) != GCA_OK) return st;
  AppendArgs a{};
  a.c = cache_args(cache, n, slot_ids, ws);
  a.kn = static_cast<const unsigned char*>(k_new->data);
  a.kn_bs = offsets ? 0 : k_new->batch_stride * esize; a.kn_ts = k_new->token_stride * esize;
  a.vn = static_cast<const unsigned char*>(v_new->data);
  a.vn_bs = offsets ? 0 : v_new->batch_stride * esize; a.vn_ts = v_new->token_stride * esize;
  a.counts = counts; a.path = path; a.T = T; a.offsets = offsets;
  a.heads = cache->heads; a.dh = cache->dh; a.src_bf16 = dtype == GCA_BF16;
  a.most_steps = most_pages(n, T, offsets != nullptr);
  unsigned char* p = static_cast<unsigned char*>(scratch);
  a.rec = reinterpret_cast<int32_t*>(p); p += align256((size_t)n * kAppendRec * 4);
  a.steps = reinterpret_cast<int32_t*>(p); p += align256((size_t)n * 4);
  a.fresh = reinterpret_cast<int32_t*>(p);
  cudaError_t e = launch_cache_append(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cache_append_quantised launch");
  return GCA_OK;
}

extern "C" gca_status gca_cache_read(const gca_cache* cache, int n, int per, const int32_t* slot_ids, const int32_t* idx,
                                     gca_dtype dtype, void* k_out, void* v_out, int32_t* idx_local, void* ws, size_t ws_bytes,
                                     gca_stream_t stream) {
  gca_status st;
  if ((st = check_quantised(cache, dtype)) != GCA_OK) return st;
  if ((st = check_entries(cache, n, slot_ids != nullptr)) != GCA_OK) return st;
  if (per < 1 || per > INT32_MAX / 256) return fail(GCA_ERR_INVALID_ARG, "per must be in 1..2^23 (got %d)", per);
  if (!idx || !k_out || !v_out) return fail(GCA_ERR_INVALID_ARG, "a pointer is NULL");
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(GCA_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  ReadArgs a{};
  a.c = cache_args(cache, n, slot_ids, ws);
  a.idx = idx; a.per = per; a.heads = cache->heads; a.dh = cache->dh; a.bf16 = dtype == GCA_BF16;
  a.k = k_out; a.v = v_out; a.local = idx_local;
  cudaError_t e = launch_cache_read(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cache_read launch");
  return GCA_OK;
}

extern "C" gca_status gca_cache_fork(const gca_cache* cache, int n, const int32_t* src, const int32_t* dst, void* ws,
                                     size_t ws_bytes, gca_stream_t stream) {
  gca_status st;
  if ((st = check_cache(cache, true, true)) != GCA_OK) return st;
  if (!src || !dst) return fail(GCA_ERR_INVALID_ARG, "src or dst is NULL");
  if ((st = check_entries(cache, n, true)) != GCA_OK) return st;
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  cudaError_t e = launch_cache_fork(cache_args(cache, n, src, ws), dst, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cache_fork launch");
  return GCA_OK;
}

extern "C" gca_status gca_cache_trim(const gca_cache* cache, int n, const int32_t* slot_ids, const int32_t* begin,
                                     const int32_t* end, int release, void* ws, size_t ws_bytes, gca_stream_t stream) {
  gca_status st;
  if ((st = check_cache(cache, true, true)) != GCA_OK) return st;
  if ((st = check_entries(cache, n, slot_ids != nullptr)) != GCA_OK) return st;
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  cudaError_t e = launch_cache_trim(cache_args(cache, n, slot_ids, ws), begin, end, release ? 1 : 0,
                                    reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cache_trim launch");
  return GCA_OK;
}

extern "C" size_t gca_cache_compact_scratch_size(int pages) {
  if (pages < 1) return 256;
  return align256((kCompactParts + 1) * 4) + 3 * align256((size_t)pages * 4);
}

extern "C" gca_status gca_cache_compact(const gca_cache* cache, int32_t* live, void* ws, size_t ws_bytes,
                                        void* scratch, size_t scratch_bytes, gca_stream_t stream) {
  gca_status st;
  if ((st = check_cache(cache, true, true)) != GCA_OK) return st;
  if (!live) return fail(GCA_ERR_INVALID_ARG, "live is NULL");
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  if ((st = check_scratch(scratch, scratch_bytes, gca_cache_compact_scratch_size(cache->pages))) != GCA_OK) return st;
  CompactArgs a{};
  a.c = cache_args(cache, cache->slots, nullptr, ws);
  a.live = live;
  unsigned char* p = static_cast<unsigned char*>(scratch);
  const size_t list = align256((size_t)cache->pages * 4);
  a.counts = reinterpret_cast<int32_t*>(p); p += align256((kCompactParts + 1) * 4);
  a.movers = reinterpret_cast<int32_t*>(p); p += list;
  a.holes = reinterpret_cast<int32_t*>(p); p += list;
  a.rank = reinterpret_cast<int32_t*>(p);
  cudaError_t e = launch_cache_compact(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cache_compact launch");
  return GCA_OK;
}

extern "C" gca_status gca_cache_lookup(const gca_cache* cache, int n, int per, const int32_t* slot_ids,
                                       const int32_t* idx, int32_t* pages_out, void* ws, size_t ws_bytes,
                                       gca_stream_t stream) {
  gca_status st;
  if ((st = check_cache(cache, false, true)) != GCA_OK) return st;
  if ((st = check_entries(cache, n, slot_ids != nullptr)) != GCA_OK) return st;
  if (per < 1) return fail(GCA_ERR_INVALID_ARG, "per must be >= 1");
  if (!idx || !pages_out) return fail(GCA_ERR_INVALID_ARG, "idx or pages_out is NULL");
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  cudaError_t e = launch_cache_lookup(cache_args(cache, n, slot_ids, ws), idx, per, pages_out,
                                      reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_cache_lookup launch");
  return GCA_OK;
}

// ==================================================================== attention of drafted tokens
extern "C" gca_status gca_tree_plan(const int32_t* parents, const int32_t* lengths, int B, int T, uint64_t* mask,
                                    int32_t* positions, void* ws, size_t ws_bytes, gca_stream_t stream) {
  if (!parents || !lengths || !mask || !positions) return fail(GCA_ERR_INVALID_ARG, "a pointer is NULL");
  if (B < 1 || B > 65535) return fail(GCA_ERR_INVALID_ARG, "B must be in 1..65535 (got %d)", B);
  if (T < 1 || T > GCA_MAX_DRAFT) return fail(GCA_ERR_UNSUPPORTED, "T must be in 1..%d (got %d)", GCA_MAX_DRAFT, T);
  if (reinterpret_cast<uintptr_t>(mask) & 7) return fail(GCA_ERR_INVALID_ARG, "mask must be 8-byte aligned");
  gca_status st;
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  TreePlanArgs a{parents, lengths, B, T, (T + 63) / 64, mask, positions, reinterpret_cast<ErrWord*>(ws)};
  cudaError_t e = launch_tree_plan(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_tree_plan launch");
  return GCA_OK;
}

extern "C" size_t gca_tree_attention_scratch_size(int B, int T, int H, int heads, int dh, int width, int window, gca_dtype dtype) {
  if (B < 1 || T < 1 || T > GCA_MAX_DRAFT || heads < 1 || H < heads || H % heads || dh < 1 || width < 1 || window < 0) return 256;
  return align256(tree_scratch_bytes(B, T, H, heads, dh, dtype == GCA_BF16, width, window));
}

extern "C" gca_status gca_tree_attention(const gca_heads* q, const gca_heads* k_new, const gca_heads* v_new,
                                         const gca_cache* cache, int B, int T, int H, const uint64_t* mask,
                                         const int32_t* positions, int window, float scale, void* o, float* lse,
                                         void* ws, size_t ws_bytes, void* scratch, size_t scratch_bytes,
                                         gca_stream_t stream) {
  gca_status st;
  if ((st = check_cache(cache, false)) != GCA_OK) return st;
  const int esize = cache->dtype == GCA_BF16 ? 2 : 4;
  if ((st = check_vectors(q, esize, "q")) != GCA_OK) return st;
  if ((st = check_vectors(k_new, esize, "k_new")) != GCA_OK) return st;
  if ((st = check_vectors(v_new, esize, "v_new")) != GCA_OK) return st;
  if (B < 1 || B > cache->slots || B > 65535) return fail(GCA_ERR_INVALID_ARG, "B must be in 1..slots, at most 65535 (got %d)", B);
  if (T < 1 || T > GCA_MAX_DRAFT) return fail(GCA_ERR_UNSUPPORTED, "T must be in 1..%d (got %d)", GCA_MAX_DRAFT, T);
  if (H < cache->heads || H % cache->heads || H > 65535)
    return fail(GCA_ERR_INVALID_ARG, "H must be a multiple of the cache's heads (got %d, %d)", H, cache->heads);
  if (cache->dh != 32 && cache->dh != 64 && cache->dh != 128)
    return fail(GCA_ERR_UNSUPPORTED, "head dim must be 32, 64 or 128 (got %d)", cache->dh);
  if (window < 0) return fail(GCA_ERR_INVALID_ARG, "window must be >= 0");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(GCA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (mask && (reinterpret_cast<uintptr_t>(mask) & 7)) return fail(GCA_ERR_INVALID_ARG, "mask must be 8-byte aligned");
  if ((T > 1 && k_new->token_stride == 0) || (T > 1 && v_new->token_stride == 0))
    return fail(GCA_ERR_UNSUPPORTED, "k_new and v_new may not repeat one token (token stride 0)");
  if ((int64_t)cache->width * 64 + GCA_MAX_DRAFT > INT32_MAX)
    return fail(GCA_ERR_UNSUPPORTED, "table too wide: positions behind 64 * width tokens must stay below 2^31");
  // All blocks of 64 keys are numbered in 32 bits.
  if ((double)B * cache->heads * ((double)cache->width + 16) > INT32_MAX)
    return fail(GCA_ERR_UNSUPPORTED, "B, H, T and the table's width are too large together");
  if (!o || !lse || !aligned16(o)) return fail(GCA_ERR_INVALID_ARG, "o and lse must not be NULL, o 16-byte aligned");
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  if ((st = check_scratch(scratch, scratch_bytes, gca_tree_attention_scratch_size(B, T, H, cache->heads, cache->dh, cache->width, window, cache->dtype))) != GCA_OK)
    return st;
  TreeArgs a{};
  a.q = q->data; a.q_bs = q->batch_stride; a.q_ts = q->token_stride; a.q_hs = q->head_stride;
  a.kn = k_new->data; a.kn_bs = k_new->batch_stride; a.kn_ts = k_new->token_stride; a.kn_hs = k_new->head_stride;
  a.vn = v_new->data; a.vn_bs = v_new->batch_stride; a.vn_ts = v_new->token_stride; a.vn_hs = v_new->head_stride;
  a.kp = cache->k_pages; a.vp = cache->v_pages; a.pages = cache->pages;
  a.table = cache->table; a.width = cache->width; a.lengths = cache->lengths;
  a.mask = mask; a.words = (T + 63) / 64; a.positions = positions;
  a.o = o; a.lse = lse;
  a.bf16 = cache->dtype == GCA_BF16; a.B = B; a.T = T; a.H = H; a.Hkv = cache->heads; a.g = H / cache->heads;
  a.dh = cache->dh; a.window = window; a.scale = scale;
  a.err = reinterpret_cast<ErrWord*>(ws);
  a.part = static_cast<unsigned char*>(scratch);
  cudaError_t e = launch_tree_attention(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_tree_attention launch");
  return GCA_OK;
}

// ==================================================================== errors, instrumentation
extern "C" gca_status gca_check_error(void* ws, gca_stream_t stream, int* bad_value) {
  if (!ws) return fail(GCA_ERR_WORKSPACE, "workspace pointer is NULL");
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gca_check_error sync");
  ErrWord h{};
  e = cudaMemcpy(&h, ws, sizeof h, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "gca_check_error read");
  if (h.flags == 0) return GCA_OK;
  // One kind a call, what makes results unusable first: it is cleared, the others stay for the next.
  const int kind = h.flags & kErrTimeout ? kErrTimeout : h.flags & kErrIndex ? kErrIndex : h.flags;
  ErrWord left = h;
  left.flags &= ~kind;
  if (kind == kErrTimeout) left.wait_sites = left.first[0] = left.first[1] = left.first[2] = left.first[3] = 0;
  else left.bad_value = 0;
  e = cudaMemcpy(ws, &left, sizeof left, cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "gca_check_error clear");
  const char* more = left.flags ? "; more is flagged: check again" : "";
  if (kind == kErrTimeout)
    return fail(GCA_ERR_TIMEOUT,
                "a bounded wait for tensor-core or copy completion ran out (wait sites 0x%x; first: site %d, "
                "CTA %d, tile %d, slot %d)%s",
                (unsigned)h.wait_sites, h.first[0] - 1, h.first[1], h.first[2], h.first[3], more);
  if (kind != kErrIndex)
    return fail(GCA_ERR_CACHE_FULL, "a cache had too few free pages, or too narrow a table, for an append");
  if (bad_value) *bad_value = h.bad_value;
  return fail(GCA_ERR_DEVICE_INDEX, "a kernel met index %d out of range (a retrieved chunk outside [-1, nC), or a page, slot, "
              "count or token)%s", h.bad_value, more);
}

// ==================================================================== wait self-test
namespace gca {
namespace {
constexpr int kSelftestSite = 30;

// One CTA waits on an mbarrier that nothing arrives at, with the same bounded wait the
// kernels use for tensor-core and copy completion: the wait runs out, every thread records
// the timeout in the error word, and the CTA exits normally.
__global__ void __launch_bounds__(32) selftest_timeout_kernel(ErrWord* err, uint32_t spins) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bar, 1);
    tc::fence_mbar_init();
  }
  __syncwarp();
  if (!tc::mbar_wait(&bar, 0, spins)) flag_timeout(err, kSelftestSite, blockIdx.x, -1, threadIdx.x);
}
}  // namespace
}  // namespace gca

extern "C" gca_status gca_selftest_timeout(void* ws, size_t ws_bytes, uint32_t spins, gca_stream_t stream) {
  gca_status st;
  if ((st = check_ws(ws, ws_bytes, kErrBytes)) != GCA_OK) return st;
  if (spins < 1 || spins > (1u << 20)) return fail(GCA_ERR_INVALID_ARG, "spins must be in 1..2^20");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  launch_begin("selftest_timeout", s);
  gca::selftest_timeout_kernel<<<1, 32, 0, s>>>(reinterpret_cast<ErrWord*>(ws), spins);
  cudaError_t e = launch_end("selftest_timeout", s);
  if (e != cudaSuccess) return cuda_fail(e, "gca_selftest_timeout launch");
  return GCA_OK;
}

extern "C" uint64_t gca_launch_count(void) { return g_launches.load(); }

extern "C" gca_status gca_profile_begin(void) {
  std::lock_guard<std::mutex> lk(g_mu);
  g_prof = true;
  return GCA_OK;
}

extern "C" int gca_profile_end(void) {
  std::lock_guard<std::mutex> lk(g_mu);
  g_prof = false;
  g_table.clear();
  for (auto& r : g_open) {
    float ms = 0.f;
    cudaEventSynchronize(r.b);
    cudaEventElapsedTime(&ms, r.a, r.b);
    Row* row = nullptr;
    for (auto& t : g_table)
      if (t.name == r.name) row = &t;
    if (!row) {
      g_table.push_back(Row{r.name, 0, 0.0});
      row = &g_table.back();
    }
    row->launches += 1;
    row->ms += ms;
    g_pool.push_back(r.a);
    g_pool.push_back(r.b);
  }
  g_open.clear();
  return (int)g_table.size();
}

extern "C" gca_status gca_profile_row(int i, const char** name, int* launches, double* total_ms) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (i < 0 || i >= (int)g_table.size()) return fail(GCA_ERR_INVALID_ARG, "profile row out of range");
  if (name) *name = g_table[i].name.c_str();
  if (launches) *launches = g_table[i].launches;
  if (total_ms) *total_ms = g_table[i].ms;
  return GCA_OK;
}
