/*
 * gca.h - C ABI of the GB300 (sm_103a) library for Grouped Cross-Attention (GCA) with
 * causal chunk retrieval.
 *
 * The method (paper "Efficient Length-Generalizable Attention via Causal Retrieval for
 * Long-Context Language Modeling"; sources cited below):
 *   - a sequence is cut into chunks of S = 64 tokens, each chunk summarised by a
 *     landmark vector (Paper-Notes page, section 整体框架 / framework);
 *   - retrieval: the landmark of chunk i scores every earlier chunk's landmark and keeps
 *     the top-k (Paper-Notes page, 关键设计 / key design, "causal retrieval"; OpenReview
 *     forum page, abstract); during training Gumbel noise perturbs the selection
 *     (Paper-Notes page, 关键设计, "Gumbel top-k");
 *   - fusion: every token of the NEXT chunk attends to each retrieved chunk with its own
 *     softmax and the k results are summed with softmax(retrieval score) weights, so
 *     the scores receive gradient (Paper-Notes page, 关键设计, "Grouped Cross-Attention"
 *     and 亮点与洞察 / insights).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library never
 *     allocates, frees or retains them.  Every call is asynchronous on `stream`.
 *   - Sizes: S = 64 tokens per chunk (fixed).  B sequences, nQ query chunks, nC key
 *     chunks, H heads of size dh, landmark dimension D, top-k = `topk`.
 *   - Layouts are row-major with the last index contiguous.  "elements" strides count
 *     elements of the tensor's own dtype.
 *   - `ws` is caller-owned device workspace of at least the size returned by the
 *     matching *_workspace_size function, 256-byte aligned.  Its first 256 bytes are a
 *     sticky device error word: zero it once after allocation; kernels only ever set
 *     bits in it; gca_check_error() reports and clears them.  Different concurrent calls
 *     must use different workspaces.
 *   - Errors: argument problems are reported synchronously (nothing is launched).
 *     A bad retrieved index met by a kernel (outside [-1, nC)) is treated as an empty
 *     slot and flagged in the error word; call gca_check_error() to see it.
 */
#ifndef GCA_H
#define GCA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define GCA_API __attribute__((visibility("default")))
#else
#define GCA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; NULL means the legacy default stream. */
typedef struct CUstream_st* gca_stream_t;

typedef enum {
  GCA_OK = 0,
  GCA_ERR_INVALID_ARG = 1,  /* a pointer, size, stride or flag is out of range          */
  GCA_ERR_UNSUPPORTED = 2,  /* valid but not provided (e.g. dh not 32/64, topk > 16)    */
  GCA_ERR_WORKSPACE = 3,    /* ws is NULL, misaligned or smaller than required          */
  GCA_ERR_CUDA = 4,         /* a CUDA runtime call failed; see gca_last_error_detail()  */
  GCA_ERR_DEVICE_INDEX = 5, /* (gca_check_error) a kernel met idx outside [-1, nC)      */
  GCA_ERR_TIMEOUT = 6,      /* (gca_check_error) a bounded wait inside a kernel ran out  */
  GCA_ERR_CACHE_FULL = 7    /* (gca_check_error) a cache had no room for an append       */
} gca_status;

typedef enum { GCA_F32 = 0, GCA_BF16 = 1, GCA_E4M3 = 2 /* pages of a quantised cache only */ } gca_dtype;

enum { GCA_CHUNK = 64, GCA_MAX_TOPK = 16, GCA_MAX_DRAFT = 256, GCA_MAX_CACHE_ENTRIES = 1024, GCA_MAX_SEQUENCES = 1024 };

/* Human-readable name of a status. */
GCA_API const char* gca_status_string(gca_status s);
/* Text of the last error raised on the calling host thread ("" if none). */
GCA_API const char* gca_last_error_detail(void);

/* ---------------------------------------------------------------------------------
 * gca_retrieve_topk - causal landmark scoring + per-row top-k.
 *
 * Paper-Notes page, 关键设计 (causal retrieval; Gumbel top-k); OpenReview abstract.
 * For every sequence b and query row i, with candidates j = 0 .. n_i - 1 where
 * n_i = min(nC, i + causal_offset):
 *     s_ij   = <q_lmk[b,i,:], k_lmk[b,j,:]> / sqrt(D)       (float32 accumulation)
 *     key_ij = s_ij + g_ij   if use_gumbel, else s_ij       (float32)
 *     g_ij   = -log(-log U),  U = ((h >> 41) + 0.5) / 2^23,
 *     h      = splitmix64 output number (ctr + 1) from state `seed`,
 *     ctr    = group << 56 | b << 48 | i << 24 | j.
 * The min(topk, n_i) candidates with the largest keys are written in descending key
 * order (equal keys: lower j first).  Unused slots get idx = -1 and score = -inf.
 * The call picks its kernels from the shape (a streaming scan for up to 8 query rows;
 * tensor-core score tiles with the selection in their epilogue for large bf16 problems;
 * 64-row tiles otherwise).  All apply the same order and tie rule; their float32 sums
 * may round differently, so only keys within that rounding of each other can be
 * ordered differently by different kernels.  A given shape always takes the same
 * kernels, and its result does not depend on how the candidates are split.
 *
 *   q_lmk   [B][nQ][D] at q_row_stride / q_batch_stride elements (row stride >= D,
 *           a multiple of 8 elements for bf16 and 4 for f32; strides allow reading the
 *           landmark rows straight out of a larger tensor).
 *   k_lmk   [B][nC][D], rows contiguous, batch stride k_batch_stride (>= nC*D, or 0 to
 *           share one landmark set among all sequences).
 *   dtype   GCA_F32 or GCA_BF16 (both landmark tensors).
 *   D       bf16: a multiple of 64 in 64..1024; f32: a multiple of 32 in 32..512.
 *   topk    1 .. 16.   causal_offset >= 0 (0 in training; nC at decode).
 *   use_gumbel: requires B <= 256, nQ, nC <= 2^24 and 0 <= group < 256.
 *   idx     [B][nQ][topk] int32 out.   scores [B][nQ][topk] float32 out (clean s).
 *   ws      >= gca_retrieve_workspace_size(B, nQ, nC, topk, causal_offset) bytes.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_retrieve_workspace_size(int B, int nQ, int nC, int topk, int causal_offset);
GCA_API gca_status gca_retrieve_topk(const void* q_lmk, int64_t q_row_stride, int64_t q_batch_stride,
                             const void* k_lmk, int64_t k_batch_stride, gca_dtype dtype,
                             int B, int nQ, int nC, int D, int topk, int causal_offset,
                             int use_gumbel, uint64_t seed, int group, int32_t* idx,
                             float* scores, void* ws, size_t ws_bytes, gca_stream_t stream);
/* gca_retrieve_topk_dseed - gca_retrieve_topk with the noise seed in device memory: the
 * kernels read the one uint64 at `seed` when they run, not when the call is made.  A
 * captured CUDA graph of a training step can then draw fresh noise on every replay (a
 * kernel in the graph, or a copy before each replay, writes the next seed).  `seed` is a
 * device pointer, 8-byte aligned, that the caller keeps alive while the work runs; it is
 * only read.  Every other argument, the results and the errors are those of
 * gca_retrieve_topk with that seed value; a NULL or misaligned `seed` returns
 * GCA_ERR_INVALID_ARG before anything is launched. */
GCA_API gca_status gca_retrieve_topk_dseed(const void* q_lmk, int64_t q_row_stride,
                                   int64_t q_batch_stride, const void* k_lmk,
                                   int64_t k_batch_stride, gca_dtype dtype, int B, int nQ,
                                   int nC, int D, int topk, int causal_offset, int use_gumbel,
                                   const uint64_t* seed, int group, int32_t* idx,
                                   float* scores, void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_retrieve_topk_noalloc - gca_retrieve_topk for callers that cannot allocate.
 *
 * The paper has no counterpart: this is a convenience of the library.  Some callers
 * cannot allocate device memory where they retrieve: a plug-in inside a host
 * application whose allocator already owns all of the GPU's memory, a latency-bound
 * decode loop where a cudaMalloc would synchronise the device and stall other streams,
 * or a plain C caller with no device allocator of its own.  This entry point takes the
 * arguments of gca_retrieve_topk without the workspace and keeps its scratch (the
 * per-split candidate lists and an error word) in one static device array of
 * gca_retrieve_noalloc_max_scratch() = 4 MiB (+256 bytes), which every GPU that loads
 * the library holds until the process exits.
 *   - A problem whose candidate scratch is larger (gca_retrieve_workspace_size() minus
 *     256 bytes above 4 MiB) returns GCA_ERR_UNSUPPORTED with an explanation: decode
 *     at 16M context with up to 16 sequences and training-size problems fit, a
 *     1M-token prefill does not.
 *   - Nothing is allocated (no cudaMalloc or cudaFree).  The first call on a device
 *     looks up the array's device address (cudaGetSymbolAddress) with that device
 *     current; make that first call before any stream capture.
 *   - Every call shares the one array, which keeps the last call's contents.  Calls
 *     that can overlap on the GPU (several streams or host threads) race on it; issue
 *     them on one stream.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_retrieve_noalloc_max_scratch(void);
GCA_API gca_status gca_retrieve_topk_noalloc(const void* q_lmk, int64_t q_row_stride,
                                     int64_t q_batch_stride, const void* k_lmk,
                                     int64_t k_batch_stride, gca_dtype dtype, int B, int nQ,
                                     int nC, int D, int topk, int causal_offset,
                                     int use_gumbel, uint64_t seed, int group, int32_t* idx,
                                     float* scores, gca_stream_t stream);
/* gca_retrieve_noalloc_check_error - gca_check_error() for the static array of
 * gca_retrieve_topk_noalloc on the current device: synchronises `stream`, reads and clears
 * the array's device error word.  Returns GCA_OK, GCA_ERR_TIMEOUT (a bounded wait ran out:
 * the idx/scores of that call are not valid), GCA_ERR_DEVICE_INDEX or GCA_ERR_CUDA.  Each
 * gca_retrieve_topk_noalloc call clears the word when it starts, so check after a call and
 * before the next one.  Argument errors of a rejected call are returned by that call and
 * leave the word untouched. */
GCA_API gca_status gca_retrieve_noalloc_check_error(gca_stream_t stream, int* bad_value);
/* Test hook: gca_selftest_timeout() run against the same array's error word (a wait on a
 * barrier that nothing arrives at runs out after `spins` probes and records
 * GCA_ERR_TIMEOUT; no fault or hang), so that a test can see the error reach
 * gca_retrieve_noalloc_check_error(). */
GCA_API gca_status gca_retrieve_noalloc_selftest_timeout(uint32_t spins, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_forward - grouped cross-attention over the retrieved chunks.
 *
 * Paper-Notes page, 关键设计 ("Grouped Cross-Attention"): each retrieved chunk gets its
 * own softmax; the k outputs are fused with softmax-normalised retrieval scores.
 * Query chunk c uses retrieval row r = c - shift (shift = 1: the next-chunk rule of
 * training, where row r's landmark sits at the end of chunk r; shift = 0: decode).
 * For each valid slot m of row r (j = idx[b,r,m] >= 0) and head h:
 *     A_m = softmax(Q_c K_j^T / sqrt(dh)) V_j      (64 x 64 logits, no mask)
 *     O_c = sum_m w_m A_m,   w = softmax over valid slots of scores[b,r,:]
 * Chunks with r < 0 or without a valid slot get O = 0.
 *
 *   q, o    [B][nQ*64][H][dh] contiguous, dtype `dtype`.
 *   k, v    [B][nC*64][H][dh]; kv_batch_stride elements between sequences
 *           (nC*64*H*dh when contiguous; 0 = all sequences share one store).
 *   idx, scores [B][nQ][topk] (idx in [-1, nC); scores float32).
 *   lse     [B][nQ][H][topk][64] float32 out: log-sum-exp of each slot's scaled
 *           logits (natural log), -inf for slots that are not valid; kept for backward.
 *   dh      32 or 64.   topk 1..16.   shift 0 or 1.
 *   ws      >= gca_forward_workspace_size() bytes (error word only).
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_forward_workspace_size(void);
GCA_API gca_status gca_forward(const void* q, const void* k, const void* v, int64_t kv_batch_stride,
                       gca_dtype dtype, int B, int nQ, int nC, int H, int dh,
                       const int32_t* idx, const float* scores, int topk, int shift,
                       void* o, float* lse, void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_window_forward - sliding-window causal self-attention.
 *
 * Paper-Notes page, 损失函数/训练策略 (training strategy): the attention block runs
 * sliding-window self-attention (W = 512) beside the top-k retrieval.  Token t attends to
 * tokens t - window + 1 .. t of its own sequence (fewer at the start) with one softmax of
 * the dh^-1/2-scaled logits.  With accumulate != 0 the result is added to o (the block's
 * sum of this sublayer and gca_forward's output); otherwise o is overwritten.
 *
 *   q, k, v, o [B][L][H][dh] contiguous, dtype `dtype`; L a multiple of 64.
 *   lse     [B][L/64][H][64] float32 out: log-sum-exp of each row's scaled logits.
 *   window  a multiple of 64 in 64..4032.   dh 32 or 64.
 *   ws      >= gca_forward_workspace_size() bytes (error word only).
 * ------------------------------------------------------------------------------- */
GCA_API gca_status gca_window_forward(const void* q, const void* k, const void* v, gca_dtype dtype, int B,
                              int L, int H, int dh, int window, void* o, float* lse, int accumulate,
                              void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_window_backward - gradients of gca_window_forward.
 *
 * With P the masked row softmax (from the saved LSE) and D = rowsum(dO * O):
 *     dS = P * (dO V^T - D),  dQ = dS K / sqrt(dh),  dK = dS^T Q / sqrt(dh),  dV = P^T dO.
 * Deterministic (no atomics): a query-side and a key-side pass.
 *
 *   q, k, v, lse, window: as passed to / produced by gca_window_forward.
 *   o       [B][L][H][dh] the window attention's own output (before any accumulation
 *           onto another sublayer's output; that sum is linear, so dout is the same).
 *   dout    [B][L][H][dh] gradient of o.
 *   dq, dk, dv [B][L][H][dh] out (accumulate != 0: added to).
 *   ws      >= gca_window_backward_workspace_size(B, L, H) bytes.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_window_backward_workspace_size(int B, int L, int H);
GCA_API gca_status gca_window_backward(const void* q, const void* k, const void* v, const void* o,
                               const void* dout, const float* lse, gca_dtype dtype, int B, int L,
                               int H, int dh, int window, void* dq, void* dk, void* dv,
                               int accumulate, void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_cca_forward - chunked cross-attention over the retrieved chunks (ablation).
 *
 * Paper-Notes page, 关键设计 ("Grouped Cross-Attention"): the variant GCA is contrasted
 * with.  The valid retrieved chunks of row r = c - shift are concatenated and query chunk
 * c attends to them with ONE softmax; the retrieval scores take no part.  Chunks without a
 * valid slot get O = 0 (unchanged when accumulating) and LSE = -inf.
 *
 *   q, k, v, kv_batch_stride, idx, topk, shift: as for gca_forward (no scores).
 *   o       [B][nQ*64][H][dh] out (accumulate != 0: added to).
 *   lse     [B][nQ][H][64] float32 out.
 *   ws      >= gca_forward_workspace_size() bytes (error word; idx outside [-1, nC) is
 *           flagged there and skipped).
 * ------------------------------------------------------------------------------- */
GCA_API gca_status gca_cca_forward(const void* q, const void* k, const void* v, int64_t kv_batch_stride,
                           gca_dtype dtype, int B, int nQ, int nC, int H, int dh, const int32_t* idx,
                           int topk, int shift, void* o, float* lse, int accumulate, void* ws,
                           size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_selftest_timeout - exercise the device error path of a wait that runs out.
 *
 * Launches one CTA that waits, with the library's bounded mbarrier wait limited to
 * `spins` probes, on a barrier that nothing ever arrives at.  The wait runs out, the CTA
 * records GCA_ERR_TIMEOUT (wait site 30) in the error word of `ws` and exits; no fault,
 * trap or hang.  gca_check_error(ws) then returns GCA_ERR_TIMEOUT and clears the word, and
 * the context stays usable.  For tests of the failure path.
 *
 *   ws      >= 256 bytes (the error word).   spins in 1..2^20.
 * ------------------------------------------------------------------------------- */
GCA_API gca_status gca_selftest_timeout(void* ws, size_t ws_bytes, uint32_t spins, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_cca_backward - gradients of gca_cca_forward.
 *
 * With P the joint row softmax of a query chunk over its valid retrieved chunks (from the
 * saved LSE) and D = rowsum(dO * O):  dS = P * (dO V^T - D),  dQ = dS K / sqrt(dh),
 * dK_j += dS^T Q / sqrt(dh),  dV_j += P^T dO  for every retrieved chunk j.  The scores take
 * no part in CCA, so there is no score gradient.  Deterministic (no atomics): a query-side
 * pass, and a key-side pass over each chunk's consumers in entry order.
 *
 *   q, k, v, idx, topk, shift, lse: as passed to / produced by gca_cca_forward (K/V
 *           contiguous per sequence: no shared store).
 *   o       [B][nQ*64][H][dh] CCA's own output (before any accumulation).
 *   dout    [B][nQ*64][H][dh] gradient of o.
 *   dq [B][nQ*64][H][dh], dk, dv [B][nC*64][H][dh] out (accumulate != 0: added to).  Query
 *           chunks without a valid slot get dq = 0, chunks never retrieved dk = dv = 0.
 *   ws      >= gca_cca_backward_workspace_size(B, nQ, nC, H, topk) bytes (error word,
 *           D rows, consumer lists); idx outside [-1, nC) is flagged there and skipped.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_cca_backward_workspace_size(int B, int nQ, int nC, int H, int topk);
GCA_API gca_status gca_cca_backward(const void* q, const void* k, const void* v, const void* o,
                            const void* dout, const float* lse, gca_dtype dtype, int B, int nQ,
                            int nC, int H, int dh, const int32_t* idx, int topk, int shift,
                            void* dq, void* dk, void* dv, int accumulate, void* ws,
                            size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_chunk_encoder_forward - the chunk / landmark encoder and the shared K/V transform.
 *
 * Paper-Notes page, 整体框架 (framework): the lower layers' output, with an LMK token
 * closing every 64-token chunk, passes a bidirectional Transformer encoder that yields
 * the chunk representations and the landmark representations shared by the upper
 * layers; 关键设计 / GCA: one K/V transform serves all of them.  Read as one pre-LN
 * encoder layer applied to every chunk on its own (the pages give neither depth nor
 * form), with dh = d / H:
 *     u = x + MHA(LN1(x)) W_o^T + b_o     attention over the chunk's 65 rows, no mask,
 *                                         logits scaled by dh^-1/2;
 *     y = u + GELU(LN2(u) W_1^T + b_1) W_2^T + b_2      (erf GELU, LayerNorm eps 1e-5);
 *     k_lmk = y at the LMK rows;   K, V = (y at the token rows) W_K^T, W_V^T.
 *
 *   x       [B][nC*65][d] bf16: per chunk its 64 token rows, then its LMK row.
 *   w       weights: matrices bf16 [out][in] row-major (w_qkv [3d][d] with the Q, K, V
 *           blocks in that order and heads contiguous inside each; w_o [d][d]; w_1 [4d][d];
 *           w_2 [d][4d]; w_kv [2d][d], K rows first); biases and LayerNorm gains/shifts
 *           float32 ([3d], [d], [4d], [d]; [d]).  Caller-owned device memory.
 *   y       [B][nC*65][d] bf16 out: the encoder's output rows.
 *   k, v    [B][nC*64][d] bf16 out: GCA's keys and values, i.e. [B][L][H'][dh'] for any
 *           head split H' dh' = d of the upper layers.
 *   k_lmk   [B][nC][d] bf16 out: the landmark representations (retrieval's k_lmk, D = d).
 *   dtype   GCA_BF16 (GCA_ERR_UNSUPPORTED otherwise).   d a multiple of 128 in 128..1024,
 *           H = d / 64 (encoder head dim 64).  All pointers 16-byte aligned.
 *   ws      >= gca_chunk_encoder_workspace_size(B, nC, d) bytes: the error word and the
 *           intermediate rows (B*nC*65 x 6d bf16).
 * ------------------------------------------------------------------------------- */
typedef struct {
  const float* ln1_g; const float* ln1_b;
  const void* w_qkv;  const float* b_qkv;
  const void* w_o;    const float* b_o;
  const float* ln2_g; const float* ln2_b;
  const void* w_1;    const float* b_1;
  const void* w_2;    const float* b_2;
  const void* w_kv;
} gca_encoder_weights;
GCA_API size_t gca_chunk_encoder_workspace_size(int B, int nC, int d);
GCA_API gca_status gca_chunk_encoder_forward(const void* x, gca_dtype dtype, int B, int nC, int d, int H,
                                     const gca_encoder_weights* w, void* y, void* k, void* v, void* k_lmk,
                                     void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_gather_chunks - copy the retrieved chunks' keys and values into a compact buffer.
 *
 * Paper-Notes page, 关键设计 / key design (inference memory offload): the past chunks'
 * K/V may live in host memory; only the k retrieved chunks are brought to the GPU.  The
 * copy is a GPU kernel driven by the device-side idx, so nothing returns to the host.
 * For each (b, r, m) with j = idx[b,r,m] in [0, nC): chunk j of the store (64 tokens x H
 * x dh of K and of V) goes to slot s = r*topk + m of the destination, and
 * idx_local[b,r,m] = s; other slots get idx_local = -1 and are left untouched.
 * gca_forward(q, k_dst, v_dst, kv_batch_stride = nQ*topk*64*H*dh, nC' = nQ*topk,
 * idx_local, scores, ...) then gives the same result as on the full store.
 *
 *   k_src, v_src [B][nC*64][H][dh] (src_batch_stride elements between sequences, 0 = one
 *           store shared by all).  Any memory the device can read: device memory, or
 *           pinned host memory (read directly by the GPU over its host link).
 *   k_dst, v_dst [B][nQ*topk*64][H][dh] device memory.   idx, idx_local [B][nQ][topk].
 *   dtype   GCA_F32 or GCA_BF16.   dh 32 or 64.   topk 1..16.   Pointers 16-byte aligned.
 *   ws      >= gca_gather_workspace_size() bytes (error word only); idx outside [-1, nC)
 *           is flagged there (GCA_ERR_DEVICE_INDEX) and treated as -1.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_gather_workspace_size(void);
GCA_API gca_status gca_gather_chunks(const void* k_src, const void* v_src, int64_t src_batch_stride,
                             gca_dtype dtype, int B, int nQ, int nC, int H, int dh,
                             const int32_t* idx, int topk, void* k_dst, void* v_dst,
                             int32_t* idx_local, void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_backward - gradients of gca_forward: dQ, dK, dV and the retrieval scores.
 *
 * The score gradient is what lets the retriever learn from the language-model loss
 * (Paper-Notes page, 研究背景与动机 / motivation and 亮点与洞察 / insights).  With
 * D_m[t] = <dO[t], A_m[t]> and dw_m = sum over tokens and heads of D_m:
 *     dscores[b,r,m] = w_m (dw_m - sum_n w_n dw_n)
 *     dS_m = w_m P_m * (dO V_j^T - D_m) / sqrt(dh)
 *     dQ_c = sum_m dS_m K_j,   dK_j += dS_m^T Q_c,   dV_j += w_m P_m^T dO_c
 *
 *   q, k, v, idx, scores, lse: as passed to / produced by gca_forward (K/V contiguous).
 *   dout    [B][nQ*64][H][dh] gradient of o.
 *   dq      [B][nQ*64][H][dh] out (chunks without a valid slot get 0).
 *   dk, dv  [B][nC*64][H][dh] out; every chunk is written (0 if never retrieved), or,
 *           with accumulate_dkv = 1, the gradient is added to their current contents.
 *   dscores [B][nQ][topk] float32 out, aligned with idx (0 for unused slots and rows).
 *   ws      >= gca_backward_workspace_size(B, nQ, nC, H, topk) bytes.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_backward_workspace_size(int B, int nQ, int nC, int H, int topk);
GCA_API gca_status gca_backward(const void* q, const void* k, const void* v, gca_dtype dtype, int B,
                        int nQ, int nC, int H, int dh, const int32_t* idx, const float* scores,
                        int topk, int shift, const void* dout, const float* lse, void* dq,
                        void* dk, void* dv, float* dscores, int accumulate_dkv, void* ws,
                        size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_scores_backward - gradient of the scaled dot-product scores into the landmarks.
 *
 *     dq_lmk[b,i] (+)= sum_m dscores[b,i,m] k_lmk[b, idx[b,i,m]] / sqrt(D)
 *     dk_lmk[b,j]   = sum_{(i,m): idx[b,i,m] = j} dscores[b,i,m] q_lmk[b,i] / sqrt(D)
 * The Gumbel noise only chose the slots and carries no gradient.
 *
 *   q_lmk, k_lmk, dtype, strides: as for gca_retrieve_topk (k_batch_stride may not be 0).
 *   idx, dscores [B][nQ][topk].
 *   dq_lmk  output with its own dtype, row and batch strides (elements); with
 *           dq_accumulate = 1 the gradient is added to the current contents (used to
 *           push a second group's landmark gradient into the first group's output
 *           gradient at each chunk's last token).
 *   dk_lmk  [B][nC][D] float32 out, overwritten.
 *   ws      >= gca_scores_backward_workspace_size(B, nQ, nC, topk) bytes.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_scores_backward_workspace_size(int B, int nQ, int nC, int topk);
GCA_API gca_status gca_scores_backward(const void* q_lmk, int64_t q_row_stride, int64_t q_batch_stride,
                               const void* k_lmk, int64_t k_batch_stride, gca_dtype dtype,
                               int B, int nQ, int nC, int D, const int32_t* idx,
                               const float* dscores, int topk, void* dq_lmk,
                               gca_dtype dq_dtype, int64_t dq_row_stride,
                               int64_t dq_batch_stride, int dq_accumulate, float* dk_lmk,
                               void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_rotary - rotary positions for queries and keys, and (backward != 0) their gradient.
 *
 * For the window attention, or the cached attention below, beside the retrieval.  Pair i of
 * a head is elements (i, i + rot/2), or (2i, 2i+1) with interleaved != 0, for i < rot/2; at
 * position p it turns by p w_i:
 *     y1 = gain (x1 cos - x2 sin),   y2 = gain (x1 sin + x2 cos)
 * and by -p w_i with backward != 0 (inputs are then the gradients of y, outputs those of
 * x).  Elements rot .. dh-1 are copied.  The angle is off by
 * |p| 2^-49 + 2^-23 radians at most (2^-22 up to 16M tokens).
 *
 *   q, k    [B][L][H][dh] and [B][L][Hkv][dh] with free strides (views of a fused
 *           projection; 0 repeats); k may be NULL (Hkv = 0).  dtype of all four tensors.
 *   q_out, k_out  like them; may be the inputs themselves (same pointer and strides), but
 *           must not overlap them otherwise.  Their strides may not make elements overlap.
 *   dh 2..256, rot even in 2..dh.   B <= 65535, B * L < 2^31.
 *   freq    [rot/2] device, w_i in units of 2^-64 turns per position, as written by
 *           gca_rotary_frequencies.
 *   positions [B][L] int32 device (>= 0 or not), position_batch_stride elements between
 *           sequences (0: shared by all); NULL: token l is at position l.
 *
 * gca_rotary_frequencies writes freq on the HOST: w_i = base^(-2i/rot), then with
 *   GCA_ROTARY_LINEAR  w_i / factor;
 *   GCA_ROTARY_NTK     base factor^(rot/(rot-2)) in the place of base (rot > 2);
 *   GCA_ROTARY_PARTS   (1 - c_i) w_i / factor + c_i w_i, where
 *                      c_i = clamp((context w_i / 2 pi - low) / (high - low), 0, 1): pairs that
 *                      turn more than `high` times in `context` tokens keep their speed, those
 *                      below `low` turns are stretched.
 * ------------------------------------------------------------------------------- */
typedef struct {
  void* data;
  int64_t batch_stride, token_stride, head_stride; /* elements; unit stride inside a head */
} gca_heads;
typedef enum { GCA_ROTARY_PLAIN = 0, GCA_ROTARY_LINEAR = 1, GCA_ROTARY_NTK = 2, GCA_ROTARY_PARTS = 3 } gca_rotary_scaling;
GCA_API gca_status gca_rotary_frequencies(int rot, double base, gca_rotary_scaling scaling, double factor,
                                  double context, double low, double high, uint64_t* freq);
GCA_API gca_status gca_rotary(const gca_heads* q, const gca_heads* k, const gca_heads* q_out, const gca_heads* k_out,
                      gca_dtype dtype, int B, int L, int H, int Hkv, int dh, int rot, int interleaved,
                      int backward, const uint64_t* freq, const int32_t* positions,
                      int64_t position_batch_stride, float gain, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_norm_rotary - RMS norm of every head of queries and keys, and their rotary positions, in one pass.
 *
 *     y = gain R(p) (x w / sqrt(mean(x^2) + eps))       for each token and head of q and of k
 * with the mean over the head's dh elements, the weights w [dh] shared by the heads, and R(p), freq,
 * rot, interleaved, positions and gain as in gca_rotary: elements rot .. dh-1 are normed, but neither
 * turned nor multiplied by gain.
 *
 *   q, k, q_out, k_out, dtype and sizes: as in gca_rotary; q_out may be q itself and k_out k (same
 *           pointer and strides), but no output may share a byte with an input or an output otherwise.
 *   q_weight, k_weight [dh] float32 device (k_weight may be NULL without k).   eps >= 0, finite.
 *
 * gca_norm_rotary_backward - its gradients.  q, k are its inputs, dq_out, dk_out the gradients of its
 * outputs; written are dq, dk (they may be dq_out, dk_out or q, k themselves) and dq_weight, dk_weight [dh]
 * float32, sums over all tokens and heads.  Deterministic (no atomics).
 *   scratch >= gca_norm_rotary_backward_scratch_size(dh) bytes, 256-byte aligned, any contents; one for
 *           each call that can overlap another.
 * ------------------------------------------------------------------------------- */
GCA_API gca_status gca_norm_rotary(const gca_heads* q, const gca_heads* k, const gca_heads* q_out, const gca_heads* k_out,
                           gca_dtype dtype, int B, int L, int H, int Hkv, int dh, int rot, int interleaved, float eps,
                           const float* q_weight, const float* k_weight, const uint64_t* freq, const int32_t* positions,
                           int64_t position_batch_stride, float gain, gca_stream_t stream);
GCA_API size_t gca_norm_rotary_backward_scratch_size(int dh);
GCA_API gca_status gca_norm_rotary_backward(const gca_heads* q, const gca_heads* k, const gca_heads* dq_out,
                                    const gca_heads* dk_out, const gca_heads* dq, const gca_heads* dk, gca_dtype dtype, int B,
                                    int L, int H, int Hkv, int dh, int rot, int interleaved, float eps, const float* q_weight,
                                    const float* k_weight, const uint64_t* freq, const int32_t* positions,
                                    int64_t position_batch_stride, float gain, float* dq_weight, float* dk_weight,
                                    void* scratch, size_t scratch_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_prompt_attention - causal attention over packed sequences, with shared key heads.
 *
 * The window sublayer and the lower layers on prompts or documents of any lengths, one behind the
 * other in one tensor.  Sequence b is rows offsets[b] .. offsets[b+1]-1; query head h reads key head
 * h / (H / Hkv).  Row t of a sequence sees its rows t - window + 1 .. t (window 0: 0 .. t):
 *     s = scale <q, k>,   o = sum softmax(s) v,   lse = log sum exp(s)
 *
 *   q [N][H][dh], k, v [N][Hkv][dh]: token and head strides of gca_heads (batch_stride is not used),
 *           16-byte aligned, strides multiples of 16 bytes (a head stride of 0 repeats a head; no
 *           token stride of 0).
 *   offsets [B+1] int32 device, 0 <= offsets[0] <= .. <= offsets[B] <= N; a sequence may be empty.  One
 *           whose offsets are out of order or of range is left out and flagged (GCA_ERR_DEVICE_INDEX);
 *           others that then share rows get any values (o and lse in the rows that they share, dq, dk and
 *           dv in all of theirs), those that share none are as ever.
 *   N 0 .. 2^30 rows.   B 1 .. 1024.   H a multiple of Hkv.   dh 32, 64 or 128.   window >= 0.   scale > 0.
 *   o [N][H][dh] contiguous, 16-byte aligned.   lse [N][H] float32.   Neither may share a byte with an
 *           input or the other.  Rows of no sequence are left as they were.
 *   ws      >= gca_forward_workspace_size() bytes (error word only).
 * No sequence sees another: rows of others, and behind the last, may hold anything.  An infinity or
 * NaN of a sequence can reach all its own rows (a weight of 0 times it is NaN).  bf16: as in
 * gca_tree_attention, products accumulate in float32 and softmax weights are rounded to bf16 for the
 * product with v.
 *
 * gca_prompt_attention_backward - its gradients:
 *     D = <dout, o>,  dS = P (<dout, v> - D) scale,  dq = sum dS k,  dk = sum dS q,  dv = sum P dout
 * with P from lse; dk, dv sum over the query heads that share a key head.  Deterministic (no atomics).
 * bf16: P and dS are rounded to bf16 for their products.  D, of the rounded o, is corrected by the sums
 * of dS, which ought to be 0, for dk everywhere and for dq in a sequence's first 128 rows; under a window
 * of 16 or less it is summed from the keys, for both.  (In wider windows dq of later rows is off by 2.5e-3 of its size
 * at most, elsewhere dq and dk by 2.4e-3: normal inputs.)
 *   o, lse  from the forward call.   dout [N][H][dh]: like q.
 *   dq [N][H][dh], dk, dv [N][Hkv][dh]: written, strides like q's but none may make elements overlap;
 *           no byte of one may be another's or an input's (views of one tensor that lie between each other may).
 *   scratch >= gca_prompt_attention_backward_scratch_size() bytes, 256-byte aligned, any contents; one
 *           for each call that can overlap another.
 * ------------------------------------------------------------------------------- */
GCA_API gca_status gca_prompt_attention(const gca_heads* q, const gca_heads* k, const gca_heads* v, gca_dtype dtype, int N,
                                int B, int H, int Hkv, int dh, const int32_t* offsets, int window, float scale, void* o,
                                float* lse, void* ws, size_t ws_bytes, gca_stream_t stream);
GCA_API size_t gca_prompt_attention_backward_scratch_size(int N, int B, int H, int Hkv, int dh, gca_dtype dtype);
GCA_API gca_status gca_prompt_attention_backward(const gca_heads* q, const gca_heads* k, const gca_heads* v, const void* o,
                                         const gca_heads* dout, const float* lse, gca_dtype dtype, int N, int B, int H,
                                         int Hkv, int dh, const int32_t* offsets, int window, float scale,
                                         const gca_heads* dq, const gca_heads* dk, const gca_heads* dv, void* ws,
                                         size_t ws_bytes, void* scratch, size_t scratch_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * A paged K/V cache.
 *
 * Pages are the method's chunks: 64 tokens of every key head, in the layout of the K/V
 * store that gca_forward reads (kv_batch_stride = 0, nC = pages, idx = page numbers from
 * gca_cache_lookup, where heads = H and dh is 32 or 64).  Slot s holds lengths[s] tokens;
 * tokens 64p .. 64p+63 lie in page table[s][p], -1 where no page is held (behind the length,
 * or given back by gca_cache_trim).  refs[page] counts the slots that hold a page; 0 is free.
 * All arrays are device memory of the caller; pools 16-byte aligned, a token's row
 * (heads * dh elements) a multiple of 16 bytes.
 *
 * What the operations have in common: they run on the device without a copy to the host, so
 * a captured graph follows the cache's state; they change the state in the order of the
 * stream, and two of them on one cache must not overlap.  `slot_ids` [n] (n <= 1024) names the
 * slots of the call's entries, NULL: entry i is slot i.  An entry whose slot, count or page
 * is out of range, or whose slot an earlier entry names, is left out and flagged in the
 * error word (GCA_ERR_DEVICE_INDEX).  Free pages are taken lowest number first, in the order
 * of the entries: equal states and calls give equal states.
 *   ws      >= gca_forward_workspace_size() bytes (error word only).
 *   scratch >= the matching *_scratch_size() bytes, 256-byte aligned, any contents; one for
 *           each call that can overlap another.
 * ------------------------------------------------------------------------------- */
typedef struct {
  void* k_pages; void* v_pages; /* [pages][64][heads][dh] */
  gca_dtype dtype; int heads, dh, pages;
  int32_t* table; int slots, width; /* [slots][width] */
  int32_t* lengths;                 /* [slots] */
  int32_t* refs;                    /* [pages]; may be NULL for attention and lookup */
} gca_cache;

/* gca_cache_append - counts[i] new tokens for each entry's slot, behind its last.
 *   k_new, v_new [n][T][heads][dh] (16-byte aligned, head stride dh, other strides multiples
 *           of 16 bytes); counts [n] int32 in 0..T; path [n][T] int32 (NULL: row t): the
 *           row of k_new that token t of the entry comes from, e.g. the accepted nodes of a
 *           draft, in order.  A row outside 0..T-1 is flagged and leaves its token unwritten.
 * A last page that other slots hold too is first copied to a fresh page (its rows in use;
 * the others are left as they were) and given back.  Entries are served in order: from the
 * first that the free pages do not reach, none is, and their slots stay as they were; one
 * that the table has no room for is left out.  Both are flagged (GCA_ERR_CACHE_FULL). */
GCA_API size_t gca_cache_append_scratch_size(int n, int T);
GCA_API gca_status gca_cache_append(const gca_cache* cache, const gca_heads* k_new, const gca_heads* v_new, int n, int T,
                            const int32_t* slot_ids, const int32_t* counts, const int32_t* path, void* ws,
                            size_t ws_bytes, void* scratch, size_t scratch_bytes, gca_stream_t stream);
/* gca_cache_fork - slot dst[i] becomes a copy of slot src[i] that shares its pages.  Left
 * out and flagged: a destination that is not empty, or that an earlier pair names; a source
 * that is a destination of the call. */
GCA_API gca_status gca_cache_fork(const gca_cache* cache, int n, const int32_t* src, const int32_t* dst, void* ws,
                          size_t ws_bytes, gca_stream_t stream);
/* gca_cache_trim - keeps the tokens begin[i] .. end[i]-1 of each entry's slot and gives back
 * the pages that lie wholly outside: end below the length takes the last tokens back, begin
 * above 0 lets go of those that a window has passed (the length stays; their table entries
 * become -1).  NULL begin: 0; NULL end: the length; both are clamped to the tokens there
 * are.  release != 0 frees the slots (begin and end are not used). */
GCA_API gca_status gca_cache_trim(const gca_cache* cache, int n, const int32_t* slot_ids, const int32_t* begin,
                          const int32_t* end, int release, void* ws, size_t ws_bytes, gca_stream_t stream);
/* gca_cache_compact - moves pages so that those in use are numbers 0 .. live-1, with their
 * counts, and renames them in every table.  With live pages in use, the k-th page in use at
 * or above `live` moves to the k-th free number below it; the rest stay.  live [1] int32
 * device out.  Table entries that name a free page become -1 (flagged). */
GCA_API size_t gca_cache_compact_scratch_size(int pages);
GCA_API gca_status gca_cache_compact(const gca_cache* cache, int32_t* live, void* ws, size_t ws_bytes, void* scratch,
                             size_t scratch_bytes, gca_stream_t stream);
/* gca_cache_lookup - the page of chunk idx[i][e] of each entry's slot: pages_out [n][per].
 * -1 stays -1; outside [-1, width) or in a bad slot is flagged and gives -1. */
GCA_API gca_status gca_cache_lookup(const gca_cache* cache, int n, int per, const int32_t* slot_ids, const int32_t* idx,
                            int32_t* pages_out, void* ws, size_t ws_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * A quantised cache: pages of dtype GCA_E4M3, half the bytes of bf16.
 *
 * A token's row in a page is heads * dh numbers in e4m3, then one byte a head, filled up with zeros to a
 * multiple of 16 bytes: gca_cache_row_bytes().  A number is its e4m3 value times 2^(byte - 127).  The byte
 * is the least exponent, -120 or more, by which the head's largest finite magnitude is 448 at most, so
 * a number is off by 2^-4 of itself or 2^-10 times the scale at most, whichever is more.  Infinities and
 * NaN become NaN; what rounds to 2^128 reads as an infinity.  gca_cache_fork, _trim, _compact and _lookup work on such pages as on others;
 * gca_cache_append, gca_tree_attention and gca_forward do not read them.  dh 32, 64 or 128, heads * dh a
 * multiple of 16.
 *
 * gca_cache_append_quantised - gca_cache_append of rows in `dtype` (GCA_BF16 or GCA_F32), quantised as they
 * are written.  With offsets [n+1] int32 instead of counts, k_new and v_new are packed tensors of T rows
 * (batch_stride is not used, path NULL) and entry i takes rows offsets[i] .. offsets[i+1]-1; offsets that
 * are not in order within 0 .. T are flagged and nothing is appended.
 *
 * gca_cache_read - chunks of a quantised cache, widened to `dtype` (exactly).  Chunk idx[i][e] of entry i's
 * slot goes to rows 64e .. 64e+63 of its outputs and idx_local[i][e] = e, so that gca_forward(q, k_out,
 * v_out, kv_batch_stride = per * 64 * heads * dh, nC = per, idx_local, ...) attends to them.  Rows at or
 * behind the slot's length are zeros.  A chunk of -1, or one whose page is not held, is zeros with
 * idx_local -1; one outside [-1, width), or in a bad slot, is that and flagged (GCA_ERR_DEVICE_INDEX).
 *   k_out, v_out [n][per * 64][heads][dh], 16-byte aligned.   idx, idx_local [n][per] int32 (idx_local may
 *           be NULL).   per >= 1.
 * ------------------------------------------------------------------------------- */
GCA_API size_t gca_cache_row_bytes(gca_dtype dtype, int heads, int dh);
GCA_API size_t gca_cache_append_quantised_scratch_size(int n, int T, int packed);
GCA_API gca_status gca_cache_append_quantised(const gca_cache* cache, const gca_heads* k_new, const gca_heads* v_new,
                                      gca_dtype dtype, int n, int T, const int32_t* slot_ids, const int32_t* counts,
                                      const int32_t* path, const int32_t* offsets, void* ws, size_t ws_bytes, void* scratch,
                                      size_t scratch_bytes, gca_stream_t stream);
GCA_API gca_status gca_cache_read(const gca_cache* cache, int n, int per, const int32_t* slot_ids, const int32_t* idx,
                          gca_dtype dtype, void* k_out, void* v_out, int32_t* idx_local, void* ws, size_t ws_bytes,
                          gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_tree_attention - attention of newly drafted tokens over a paged cache.
 *
 * The decoding form of the window attention: T new tokens of each sequence (one token, a
 * run of tokens, or a tree of drafted candidates) attend with one softmax to the cache's
 * tokens and to each other.  Query head h reads key head h / (H / heads).
 *     s = scale <q, k>,   o = sum softmax(s) v,   lse = log sum exp(s)
 * over the cache's tokens j < lengths[b] of slot b, and the draft's tokens u whose bit is set
 * in token t's mask; with window > 0 only those with position > position_t - window, where
 * token j of the cache is at position j.  A token that sees nothing, and padding, gets o = 0
 * and lse = -inf.  A page number outside [0, pages) is left out (flagged unless it is -1).
 *
 *   q [B][T][H][dh], k_new, v_new [B][T][heads][dh]: free strides, 16-byte aligned, strides
 *           multiples of 16 bytes (0 repeats a sequence or a head; in k_new, v_new not a token).  B <= cache->slots: sequence b is slot b.
 *   mask    [B][T][ceil(T/64)] uint64: bit u % 64 of word u / 64 of row t: t sees u.  NULL: t
 *           sees the tokens u <= t.  Tokens of the cache or the draft that no row sees may hold
 *           anything; an infinity or NaN that some row sees can reach the sequence's other rows
 *           (a weight of 0 times it is NaN).
 *   positions [B][T] int32: -1 for padding (seen by none and seeing none), else the token's
 *           position, taken as lengths[b] where it is lower.  NULL: lengths[b] + t.
 *   window  0 (everything) or more.   scale > 0.   T 1..256.   dh 32, 64 or 128.   A table of
 *           64 * width + 256 < 2^31.
 *   o       [B][T][H][dh] contiguous, 16-byte aligned.   lse [B][T][H] float32.
 *   ws      >= gca_forward_workspace_size() bytes (error word only).
 *   scratch >= gca_tree_attention_scratch_size() bytes, 256-byte aligned, any contents; one for
 *           each call that can overlap another.
 * bf16 products accumulate in float32; their softmax weights are rounded to bf16 for the product
 * with v (relative to each weight, 2^-8 at most), as in gca_window_forward.
 *
 * gca_tree_plan - mask and positions of a tree, once for all layers of a step.
 *   parents [B][T] int32: the earlier token of the draft that token t follows, -1 for the
 *           cache's last token, -2 for padding.  Any other value is flagged and read as -2;
 *           what follows padding is padding.  lengths [B].
 *   mask, positions: as above (a token sees itself and its ancestors; its position is
 *           lengths[b] plus the number of its ancestors).
 * ------------------------------------------------------------------------------- */
GCA_API gca_status gca_tree_plan(const int32_t* parents, const int32_t* lengths, int B, int T, uint64_t* mask,
                         int32_t* positions, void* ws, size_t ws_bytes, gca_stream_t stream);
GCA_API size_t gca_tree_attention_scratch_size(int B, int T, int H, int heads, int dh, int width, int window, gca_dtype dtype);
GCA_API gca_status gca_tree_attention(const gca_heads* q, const gca_heads* k_new, const gca_heads* v_new,
                              const gca_cache* cache, int B, int T, int H, const uint64_t* mask,
                              const int32_t* positions, int window, float scale, void* o, float* lse, void* ws,
                              size_t ws_bytes, void* scratch, size_t scratch_bytes, gca_stream_t stream);

/* ---------------------------------------------------------------------------------
 * gca_check_error - synchronise `stream`, read the device error word of `ws` and clear what
 * is reported: one kind a call, in the order below, so that the next call reports the next.
 * Returns GCA_OK, GCA_ERR_TIMEOUT (a tensor-core completion wait gave up instead of
 * hanging; the results of that call are not valid), GCA_ERR_DEVICE_INDEX (with the
 * offending index in *bad_value when bad_value != NULL), GCA_ERR_CACHE_FULL or GCA_ERR_CUDA.
 * ------------------------------------------------------------------------------- */
GCA_API gca_status gca_check_error(void* ws, gca_stream_t stream, int* bad_value);

/* ---------------------------------------------------------------------------------
 * Instrumentation (host side, process-wide).
 *   gca_launch_count  - number of kernels this library has launched so far.
 *   gca_profile_begin - from now on, bracket every kernel launch with CUDA events on
 *                       its own stream (adds ~1 us per launch).
 *   gca_profile_end   - stop recording, wait for the events, and fill a table of
 *                       (kernel name, launches, total milliseconds); returns the number
 *                       of rows, reads them with gca_profile_row(i, ...).
 * ------------------------------------------------------------------------------- */
GCA_API uint64_t gca_launch_count(void);
GCA_API gca_status gca_profile_begin(void);
GCA_API int gca_profile_end(void);
GCA_API gca_status gca_profile_row(int i, const char** name, int* launches, double* total_ms);

#ifdef __cplusplus
}
#endif

#endif /* GCA_H */
