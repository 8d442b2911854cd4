/* ggufdq.h -- C ABI of the GB300 GGUF block-dequant GEMV / MoE library.
 *
 * The library computes matrix-vector products over GGUF block-quantized weights that stay
 * in their raw GGUF block layout in device memory and are decoded inside the product, plus
 * the mixture-of-experts step built on them.  The operations follow the engine pages of the
 * diskformer npm package:
 *   - qwen3_moe_ssd.js (diskformer 0.0.1 -> 0.3.0): header comment (Q8_0 blocks kept
 *     bit-exact, dot products equal llama.cpp's up to summation order); WGSL kernels
 *     matmulQ8, matmulF32, topk, expertQ8, siluMulMoe, moeAccum.
 *   - qwen35_moe_ssd.js (diskformer 0.5.4 -> 0.6.6): BATCH_KERNELS matmulQ8T (token-major
 *     batches, one weight read serves several tokens), topkB, expertQ8B, siluMul2B.
 *   - gemma4_moe_ssd.js (diskformer 0.5.4 -> 0.6.6): Q4_0 layout (Q4DOT comment), Q6_K
 *     layout (Q6P comment), matmulQ4, matmulQ6K.
 *   - ternary_bonsai_2_dflash.js (diskformer 0.5.4 -> 0.6.6): the K-quant block layouts
 *     ("Layouts follow ggml-quants.c"), dequantQ4K / dequantQ6K, WG_GEMM_Q4K / WG_GEMM_Q6K.
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library never
 *     allocates device memory, never synchronises the stream and keeps no host state; all
 *     work is enqueued on `stream` (NULL = the legacy default stream).
 *   - Weights `w` are raw GGUF blocks, row-major: row m of an [M][N] tensor is N / QK
 *     consecutive blocks.  Block layouts (QK elements, bytes):
 *       QG_TYPE_Q8_0  (32, 34):  f16 d, int8 q[32];            w = d * q
 *       QG_TYPE_Q4_0  (32, 18):  f16 d, u8 qs[16];  byte j holds element j (low nibble)
 *                                and j + 16 (high nibble);      w = (nibble - 8) * d
 *       QG_TYPE_Q4_K (256, 144): f16 d, f16 dmin, u8 scales[12] (8 packed 6-bit scales and
 *                                mins), u8 qs[128];             w = d*sc*q - dmin*m
 *       QG_TYPE_Q6_K (256, 210): u8 ql[128], u8 qh[64], int8 scales[16], f16 d;
 *                                                               w = d * scale * (q - 32)
 *   - Activations and outputs are f32, token-major: x[t][k] at x + t*N + k, y[t][m] at
 *     y + t*M + m.  Accumulation is f32; results equal the exact products up to f32
 *     summation order.
 *   - Alignment: `w`, every f32 tensor and every expert base must be 16-byte aligned;
 *     expert strides must be multiples of 16 bytes.
 *   - Errors: argument checks run on the host before anything is enqueued and return a
 *     non-zero qg_status with nothing launched.  QG_ECUDA reports a launch failure
 *     (cudaGetLastError).  Kernels never trap: a device-side check that fails (an expert
 *     id out of range, a bounded wait that expired) sets a device status word that
 *     qg_device_status() reads, and the affected outputs are undefined.
 *   - Outputs never alias inputs, except x_inout in moe_combine / moe_layer.
 */
#ifndef GGUFDQ_H
#define GGUFDQ_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define QG_API __attribute__((visibility("default")))
#else
#define QG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; the header does not need the CUDA headers. */
typedef struct CUstream_st *qg_stream_t;

/* ggml type ids of the supported block formats */
enum {
  QG_TYPE_Q4_0 = 2,
  QG_TYPE_Q8_0 = 8,
  QG_TYPE_Q4_K = 12,
  QG_TYPE_Q6_K = 14
};

typedef enum qg_status {
  QG_OK = 0,
  QG_EINVAL_SHAPE = 1,  /* a size is out of range or not a multiple of the block size */
  QG_EINVAL_PTR = 2,    /* a required pointer is NULL */
  QG_EALIGN = 3,        /* a pointer or stride is not 16-byte aligned */
  QG_EUNSUPPORTED = 4,  /* block type not supported by this call */
  QG_ECUDA = 5,         /* a CUDA call or kernel launch failed */
  QG_EDEVICE_ID = 6,    /* device status bit: an expert id or slot was out of range */
  QG_ETIMEOUT = 7,      /* device status bit: a bounded wait inside a kernel expired */
  QG_EWORKSPACE = 8     /* workspace pointer NULL or smaller than the size query says */
} qg_status;

/* Library ABI version (incremented on incompatible changes). */
QG_API int qg_version(void);

/* Short description of a status code; never NULL. */
QG_API const char *qg_strerror(int status);

/* Elements and bytes per block of `type`; returns QG_EUNSUPPORTED for other types. */
QG_API qg_status qg_block_shape(int type, int *qk, int *block_bytes);

/* Device status word of the current device: a bitwise OR of (1 << QG_EDEVICE_ID) and
 * (1 << QG_ETIMEOUT) for every kernel that detected such a condition since the last clear.
 * Synchronises the device.  When `clear` is non-zero the word is reset to 0. */
QG_API qg_status qg_device_status(uint32_t *status_out, int clear);

/* Static weights, a setting of one stream (off by default).  Every launch of this library
 * waits for the preceding kernel in its stream (programmatic dependent launch) before it
 * touches memory.  A caller whose weight buffers are immutable model parameters - written
 * once, before any GEMV that reads them, and never by a kernel enqueued ahead of a GEMV in
 * the same stream - may call qg_set_static_weights(stream, 1): the dense GEMVs (qgemv_*,
 * qgemv_t, qgemv_multi) and the one-token MoE layer enqueued on that stream then start
 * streaming their first weight tiles while the preceding kernel drains, and only the
 * activations and outputs wait for it.  Leave it off when a kernel in the stream may write
 * the weights (quantise-in-place, a loader that copies through a kernel): the GEMV could read
 * stale bytes.  Host-to-device copies are ordered either way.
 *   - The setting belongs to the (device, stream handle) pair that is current at the call,
 *     and other streams and other users of the library in the process are not affected.
 *     Clear it before destroying the stream: a new stream may reuse the handle.
 *   - It takes effect for launches enqueued (or captured) after the call.
 *   - Returns the previous setting of that stream (0 or 1), or -1 when 256 streams already
 *     hold the setting. */
QG_API int qg_set_static_weights(qg_stream_t stream, int enable);

/* ---- dense quantized GEMV, one token ----------------------------------------------------
 * y[m] = sum_k W[m][k] * x[k] for m < M  (matmulQ8 / matmulQ4 / matmulQ6K on the pages, and
 * the Q4_K row dot of WG_GEMM_Q4K).  w: M*N/QK raw blocks; x: f32[N]; y: f32[M].
 * N must be a positive multiple of QK (32 for Q8_0 / Q4_0, 256 for Q4_K / Q6_K), M >= 0
 * (M == 0 enqueues nothing), M, N <= 2^31 - 1. */
QG_API qg_status qgemv_q8_0(const void *w, const float *x, float *y, int64_t M, int64_t N, qg_stream_t stream);
QG_API qg_status qgemv_q4_0(const void *w, const float *x, float *y, int64_t M, int64_t N, qg_stream_t stream);
QG_API qg_status qgemv_q4_k(const void *w, const float *x, float *y, int64_t M, int64_t N, qg_stream_t stream);
QG_API qg_status qgemv_q6_k(const void *w, const float *x, float *y, int64_t M, int64_t N, qg_stream_t stream);

/* ---- dense quantized GEMV over T token columns, one weight pass ---------------------------
 * Y[t][m] = sum_k W[m][k] * X[t][k] for t < T, m < M  (matmulQ8T in qwen35_moe_ssd.js: every
 * weight byte read serves all T tokens).  x: f32[T][N]; y: f32[T][M]; 1 <= T <= 16.
 * Same shape rules as above. */
QG_API qg_status qgemv_t(int type, const void *w, const float *x, float *y, int64_t M, int64_t N, int T,
                  qg_stream_t stream);

/* ---- several matrices over the same activations, one launch ------------------------------
 * Y_j[t][m] = sum_k W_j[m][k] * X[t][k] for j < n (n <= 4), every W_j of the same type and row
 * length N, X shared.  The decode steps whose projections read one normalised input (q, k and
 * v of attention; gate and up of the FFN) stream all their rows in a single pass of the
 * kernel instead of one launch each.  w, y and M are HOST arrays of n entries (device pointers
 * to raw blocks and f32 [T][M_j] outputs, row counts); a matrix with M_j == 0 is skipped.
 * Same shape and alignment rules as qgemv_t. */
QG_API qg_status qgemv_multi(int type, int n, const void *const *w, float *const *y, const int64_t *M, int64_t N,
                      const float *x, int T, qg_stream_t stream);

/* ---- prefill dequant-GEMM, T >= 17 token rows --------------------------------------------
 * Y[t][m] = sum_k W[m][k] * X[t][k] with W decoded to bf16 and X rounded to bf16 for the
 * tensor cores, f32 accumulation (the tiled matmulQ8T generalised to a prefill chunk).
 * Workspace: at least qgemm_workspace_size(type, M, N, T) bytes of device memory, 16-byte
 * aligned, used for the bf16 copy of X; may be NULL when the size is 0.  T >= 1 is
 * accepted (T <= 16 is routed to qgemv_t, which is exact in f32). */
QG_API size_t qgemm_workspace_size(int type, int64_t M, int64_t N, int64_t T);
QG_API qg_status qgemm(int type, const void *w, const float *x, float *y, int64_t M, int64_t N, int64_t T,
                void *workspace, size_t workspace_bytes, qg_stream_t stream);

/* ---- MoE step ----------------------------------------------------------------------------
 * Shapes: T tokens, hidden size H, expert FFN size F, E router experts, k picks per token.
 * Limits: 1 <= k <= 32, k <= E <= 256 (the pages' topk limits), H and F multiples of the
 * block QK, H % 4 == 0.
 * Expert weights: expert e lives in pool slot s = slots[e] (slots == NULL: s = e); its gate
 * rows (F x H), up rows (F x H) and down rows (H x F) are raw blocks at
 * w_gate + s*expert_stride, w_up + s*expert_stride, w_down + s*expert_stride.  This covers
 * the pages' per-expert record (gate || up || down contiguous, expertQ8 with
 * rowsPerExpert) and GGUF's separate ffn_{gate,up,down}_exps tensors.  0 <= s < n_slots.
 * ids / weights: int32 [T][k] expert ids in pick order and f32 [T][k] combine weights.
 * Pairs z = t*k + j index the per-pick buffers (act is f32 [T*k][F]).
 *
 * Workspace: moe_workspace_size(T, k, E, H, F) bytes of device memory, 16-byte aligned,
 * zero-filled by the caller once before its first use.  Its first 260 KB are a fixed header
 * whose words keep their meaning from call to call: the one-token layer's grid-barrier
 * counter and call counter (64-bit words that every moe_layer call at T = 1 advances), its
 * logits tagged with the call, and the router's per-tile tickets (every call leaves them at
 * zero again).  Their offsets do not depend on the
 * call's shape, so one workspace sized for the largest shape it will serve (the largest T, k,
 * E, H, F) may serve any call whose moe_workspace_size is not larger.  The rest holds scratch
 * that each call rewrites: the router logits, the per-pick down rows and, for more than 16
 * tokens, the grouped bf16 rows.  A NULL, misaligned or too small workspace returns
 * QG_EWORKSPACE (QG_EALIGN when misaligned) with nothing launched.  Calls that share a
 * workspace must not run concurrently. */
QG_API size_t moe_workspace_size(int T, int k, int E, int H, int F);

/* Router (matmulF32 + topk / topkB): logits l[t][e] = sum_h wr[e][h] * xn[t][h] (f32
 * weights), softmax over the E logits, k greedy picks of the largest (ties to the lowest
 * expert id), weights p_j / sum of the picked p (norm_topk_prob).  Picks are taken on the
 * logits, which gives the same order as taking them on the softmax probabilities.
 * xn: f32 [T][H]; wr: f32 [E][H]; ids: int32 [T][k]; weights: f32 [T][k];
 * logits_out: optional f32 [T][E] copy of the logits (NULL to skip). */
QG_API qg_status moe_route_topk(const float *xn, const float *wr, int T, int H, int E, int k, int32_t *ids,
                         float *weights, float *logits_out, void *workspace, size_t workspace_bytes,
                         qg_stream_t stream);

/* The router of moe_route_topk for callers that cannot hand the library a workspace: for
 * instance a host engine whose device memory is entirely reserved by its own allocator before
 * it calls in, or a binding that exposes only input and output tensors.  The library keeps a
 * fixed 68 KB scratch area in device memory (1024 ticket words, then 16384 logits) and
 * allocates nothing (no cudaMalloc, no allocating library call).
 *   - Limits: T * E <= 16384 and T <= 16384 (at most 1024 tiles of 16 tokens); larger shapes
 *     return QG_EWORKSPACE.  Every other argument check is moe_route_topk's, and all of them
 *     run before anything is enqueued.
 *   - The scratch address is looked up once per device, on the first call with that device
 *     current; make that first call before any stream capture.
 *   - Each call clears the tickets of its shape on `stream` (one memset) before the router
 *     runs; with logits_out == NULL the logits live in the scratch area.
 *   - One scratch area per device: calls that overlap (other streams, other host threads)
 *     race on it and must be serialised by the caller.
 * Results are the same as moe_route_topk's.  The engine pages have no counterpart: their
 * router buffers are allocated by the engine. */
QG_API qg_status moe_route_topk_noalloc(const float *xn, const float *wr, int T, int H, int E, int k, int32_t *ids,
                                 float *weights, float *logits_out, qg_stream_t stream);

/* Gate/up expert rows with SwiGLU (expertQ8 with a shared input, then siluMulMoe): for each
 * pair z = t*k + j with expert e = ids[z]:  g = Wg[s] . xn[t],  u = Wu[s] . xn[t]  (F rows
 * each),  act[z][i] = g_i / (1 + exp(-g_i)) * u_i.  Experts are grouped so that each picked
 * expert's rows are read once for all its tokens.  An id outside [0, E) or a slot outside
 * [0, n_slots) sets QG_EDEVICE_ID in the device status and that pair's act row is zero. */
QG_API qg_status moe_expert_swiglu(int type, const void *w_gate, const void *w_up, int64_t expert_stride,
                            const int32_t *slots, int n_slots, int E, const int32_t *ids, const float *xn,
                            int T, int k, int H, int F, float *act, void *workspace, size_t workspace_bytes,
                            qg_stream_t stream);

/* Down expert rows and the weighted combine (expertQ8 with a per-pick input, then
 * moeAccum):  x_inout[t][h] = (add_residual ? x_inout[t][h] : 0)
 *                              + sum_j weights[t][j] * (Wd[s_j] . act[t*k + j])[h].
 * The expert sum is formed first and the residual added last, as the pages order it. */
QG_API qg_status moe_combine(int type, const void *w_down, int64_t expert_stride, const int32_t *slots, int n_slots,
                      int E, const int32_t *ids, const float *weights, const float *act, int T, int k, int H,
                      int F, float *x_inout, int add_residual, void *workspace, size_t workspace_bytes,
                      qg_stream_t stream);

/* The whole MoE step: moe_route_topk, moe_expert_swiglu, moe_combine (add_residual = 1).
 * xn: router / expert input [T][H]; x_inout: residual stream [T][H], updated in place;
 * ids, weights, act: caller buffers that receive the intermediates. */
QG_API qg_status moe_layer(int type, const float *xn, const float *wr, const void *w_gate, const void *w_up,
                    const void *w_down, int64_t expert_stride, const int32_t *slots, int n_slots, int T, int H,
                    int F, int E, int k, int32_t *ids, float *weights, float *act, float *x_inout,
                    void *workspace, size_t workspace_bytes, qg_stream_t stream);

/* ---- the steps on either side of a GEMV chain ----------------------------------------------
 * Embedding row gather (embedQ8 in qwen3_moe_ssd.js, embedQ6K in gemma4_moe_ssd.js):
 *   out[i][k] = w(ids[i], k) * scale   for i < n, k < N,
 * w(r, .) the dequantized row r of the [V][N] table in raw blocks of `type` (any of the four),
 * decoded by the GEMV's own decoders; the product is one f32 rounding (scale = 1 is exact;
 * embedQ6K's page multiplies by sqrt(H)).  table: device, 16-byte aligned, V*N/QK blocks;
 * ids: device int32[n]; out: device f32[n][N], 16-byte aligned.  N a positive multiple of QK,
 * 1 <= V, 0 <= n (n == 0 enqueues nothing).  An id outside [0, V) gives a zero row and sets
 * QG_EDEVICE_ID in the device status. */
QG_API qg_status qg_embed_rows(int type, const void *table, int64_t V, int64_t N, const int32_t *ids, int n,
                               float scale, float *out, qg_stream_t stream);

/* RMSNorm (rmsnorm in qwen3_moe_ssd.js, rmsnormB for a token batch; with a factor, rmsnormK
 * of gemma4_moe_ssd.js, the MoE router's input with k = 1/sqrt(H)):
 *   y[t][i] = ((x[t][i] * s_t) * k) * w[i],   s_t = 1 / sqrt(mean_i x[t][i]^2 + eps),
 * sums in f32; k = 1 is plain RMSNorm.  x, y: device f32[T][N]; w: device f32[N]; all 16-byte
 * aligned; y may be x.  N a positive multiple of 4, 0 <= T <= 65535, eps >= 0. */
QG_API qg_status qg_rmsnorm(const float *x, const float *w, int T, int64_t N, float eps, float k, float *y,
                            qg_stream_t stream);

/* argmax per row (argmax in qwen3_moe_ssd.js, argmaxRows in qwen35_dense.js): ids[t] = the
 * lowest index of the largest value of row t of logits[T][n]; NaN is never picked and a row
 * with nothing but NaN gives 0.  logits, ids: device, 4-byte aligned; 0 <= T <= 8191.  Each
 * row is scanned by a cluster of 8 CTAs whose partial picks meet in distributed shared memory. */
QG_API qg_status qg_argmax_rows(const float *logits, int T, int64_t n, int32_t *ids, qg_stream_t stream);

/* Tied head and greedy pick in one call (encodeHead of qwen3_moe_ssd.js: the head GEMV over
 * the vocabulary, then argmax): logits[t][m] = sum_k W[m][k] * x[t][k] as qgemv_t, then
 * ids[t] = argmax_m logits[t][m] as qg_argmax_rows.  logits: device f32[T][M] (caller
 * buffer, written); ids: device int32[T]; 1 <= T <= 16; other rules as qgemv_t.  A caller
 * that wants only the tokens reads back T ids instead of T * M logits. */
QG_API qg_status qg_head_argmax(int type, const void *w, int64_t M, int64_t N, const float *x, int T, float *logits,
                                int32_t *ids, qg_stream_t stream);

/* ---- MoE variants on the same kernels -----------------------------------------------------
 * The Gemma 4 MoE (gemma4_moe_ssd.js: Q4_0 experts, geglu, moeSum's per-expert down scale; its
 * router input is qg_rmsnorm with k = 1/sqrt(H)) and the Qwen3.5/3.6 MoE (qwen35_moe_ssd.js:
 * moeAccumShared, the sigmoid-gated shared expert) differ from the Qwen3 MoE above only in the
 * expert activation and the combine.  A variant is a HOST struct; NULL is the Qwen3 MoE. */
#define QG_ACT_SILU 0      /* act = SiLU(g) * u                         (siluMulMoe) */
#define QG_ACT_GELU_TANH 1 /* act = GELU(g) * u, tanh form, argument clamped to [-10, 10] (geglu) */
typedef struct qg_moe_variant {
  int act;                  /* QG_ACT_SILU or QG_ACT_GELU_TANH */
  const float *down_scale;  /* NULL, or device f32[E]: pick j's down row is scaled by down_scale[id_j] */
  const float *shared_out;  /* NULL, or device f32[T][H] (16-byte aligned): the shared expert's output */
  const float *shared_gate; /* with shared_out: device f32[T], the shared expert's gate logit */
} qg_moe_variant;

/* moe_expert_swiglu with the variant's activation (act[z][i] = SiLU or GELU of gate, times up). */
QG_API qg_status moe_expert_act(int type, const void *w_gate, const void *w_up, int64_t expert_stride,
                                const int32_t *slots, int n_slots, int E, const int32_t *ids, const float *xn, int T,
                                int k, int H, int F, const qg_moe_variant *variant, float *act, void *workspace,
                                size_t workspace_bytes, qg_stream_t stream);

/* moe_combine with the variant's combine (moeSum, then moeAccumShared):
 *   x_inout[t][h] = (add_residual ? x_inout[t][h] : 0)
 *                   + (sum_j (dn_j[h] * down_scale[id_j]) * weights[t][j]  +  shared_out[t][h] * s(shared_gate[t])),
 * dn_j = Wd[s_j] . act[t*k + j], s the logistic function, the expert sum in pick order first,
 * the shared term next, the residual last. */
QG_API qg_status moe_combine_ex(int type, const void *w_down, int64_t expert_stride, const int32_t *slots,
                                int n_slots, int E, const int32_t *ids, const float *weights, const float *act, int T,
                                int k, int H, int F, const qg_moe_variant *variant, float *x_inout, int add_residual,
                                void *workspace, size_t workspace_bytes, qg_stream_t stream);

/* moe_layer with a variant: router with top-k, moe_expert_act, moe_combine_ex (add_residual =
 * 1).  A NULL or default variant is moe_layer itself (one launch at T = 1); other variants run
 * the three steps at every T.  A variant with shared_out and no shared_gate (or the reverse)
 * returns QG_EINVAL_PTR, an unknown act QG_EINVAL_SHAPE, all before anything is enqueued. */
QG_API qg_status moe_layer_ex(int type, const float *xn, const float *wr, const void *w_gate, const void *w_up,
                              const void *w_down, int64_t expert_stride, const int32_t *slots, int n_slots, int T,
                              int H, int F, int E, int k, const qg_moe_variant *variant, int32_t *ids, float *weights,
                              float *act, float *x_inout, void *workspace, size_t workspace_bytes,
                              qg_stream_t stream);

/* ---- paged key/value cache ------------------------------------------------------------------
 * The steps between a layer's q/k/v projections and its output projection, and the beam search
 * that follows the head (qkNormRope, kvStore, attnScore / softmax / attnOut and their batched
 * forms on the pages; the pages keep one sequence in one f16 buffer, this cache keeps many in
 * pages).  A cache is a pool of n_pages pages for the keys and one for the values of a layer;
 * token s of a sequence lives in row s % page_size of page table[s / page_size].
 *   - Element (page p, row r, head h, i) is at p*page_stride + r*token_stride + h*head_stride + i
 *     (strides in elements, the same for k and v), so token-major and head-major pools and
 *     pools interleaved in one allocation are all described.
 *   - k, v 16-byte aligned, strides multiples of 8 elements and not negative, page_size a power
 *     of two up to 65536, head_dim 64, 128 or 256.  Distinct elements must not overlap.
 * Both structs are HOST structs, read during the call. */
enum { QG_DT_F32 = 0, QG_DT_F16 = 1, QG_DT_BF16 = 2 };

typedef struct qg_kv_cache {
  void *k, *v;       /* device */
  int dtype;         /* QG_DT_F16 or QG_DT_BF16 */
  int n_pages, page_size, n_heads, head_dim;
  int64_t page_stride, token_stride, head_stride;
} qg_kv_cache;

/* A batch of n_seqs sequences with n_tokens new tokens in all.  The new tokens of sequence b
 * are rows q_start[b] .. q_start[b+1]-1 of the token tensors (q_start NULL: one token per
 * sequence, n_tokens == n_seqs); kv_len[b] counts the sequence's own cached tokens WITH the new
 * ones, so new token i of n sits in slot kv_len[b] - n + i of the sequence's page list.
 * Groups (n_groups 0: none) share a prefix: sequences group_start[g] .. group_start[g+1]-1 are
 * preceded by the prefix_len[g] tokens of prefix_pages[g], stored once.  A token's position is
 * (its group's prefix length) + (its slot).
 *   - pages: int32 [n_seqs][max_pages]; prefix_pages: int32 [n_groups][max_prefix_pages].
 *   - q_start and group_start rise and start at 0; all arrays are device memory, 4-byte
 *     aligned, and read by the kernels (a captured graph sees later contents).
 *   - Lengths past the page lists, negative lengths, page ids outside [0, n_pages) and new tokens
 *     without a slot set QG_EDEVICE_ID in the device status; nothing out of range is accessed,
 *     whatever the arrays hold.
 * Limits: n_seqs, n_groups <= 65535, n_groups <= n_seqs, n_tokens <= 2^24.  A call on a batch
 * without tokens (without sequences for qg_beam_reorder) enqueues nothing. */
typedef struct qg_kv_batch {
  int n_seqs, n_tokens, n_groups, max_pages, max_prefix_pages;
  const int32_t *q_start;      /* [n_seqs + 1] or NULL */
  const int32_t *kv_len;       /* [n_seqs]; written by qg_kv_fork and qg_kv_reserve only */
  int32_t *pages;              /* written by these and qg_beam_reorder only */
  const int32_t *group_start;  /* [n_groups + 1] */
  const int32_t *prefix_len;   /* [n_groups] */
  const int32_t *prefix_pages; /* qg_kv_append does not read it */
} qg_kv_batch;

/* Position-rotation table for qg_kv_append: out[i] = round(2^64 * f_i / (2 pi)), the turns per
 * position of pair i < rot/2 as a 64-bit fraction, f_i = theta^(-2 i / rot) / factors[i] (HOST
 * arrays; factors NULL: 1; theta > 1, rot even and positive).  A position times such an entry,
 * modulo 2^64, is the pair's angle as a fraction of a turn, exact to 2^-64 turns per position
 * at any distance, without 64-bit floating point in the kernel.  An f_i above 2 pi is refused. */
QG_API qg_status qg_rope_freqs(int rot, double theta, const float *factors, uint64_t *out);

/* Rotate and append (qkNormRope, then kvStore): for each new token t of the batch, with q, k, v
 * its f32 projection rows (head h of q at q + t*q_stride + h*D, and so on; strides in floats),
 *   x <- x / sqrt(mean_D x^2 + eps) * w     per head of q and k, where q_norm / k_norm (f32[D]) are given
 *   (x_a, x_b) <- (x_a c - x_b s, x_a s + x_b c)   c, s of angle position * f_i, for the pairs i < rot/2:
 *     rope_pairs 0: a = i, b = i + rot/2;  rope_pairs 1: a = 2i, b = 2i + 1; the rest of a head unchanged
 * then the rotated k and the v go to the token's row of the cache and the rotated q to
 * q_out[t][h][D] (the cache's type), each rounded once from f32.  q may be NULL (with q_out NULL
 * and Hq 0): append only.  freqs: device, rot/2 entries of qg_rope_freqs (may be NULL when rot
 * is 0).  Hq a multiple of the cache's heads; 0 <= rot <= D, rot % 8 == 0; row strides multiples of 4
 * floats that hold a row; f32 pointers and q_out 16-byte aligned, freqs 8-byte. */
QG_API qg_status qg_kv_append(const qg_kv_cache *cache, const qg_kv_batch *batch, int Hq, const float *q,
                              int64_t q_stride, const float *k, int64_t k_stride, const float *v, int64_t v_stride,
                              const float *q_norm, const float *k_norm, float eps, const uint64_t *freqs, int rot,
                              int rope_pairs, void *q_out, qg_stream_t stream);

/* Causal attention over the cache: for new token t at position p and query head h,
 *   out[t][h] = sum_j softmax_j(scale * q[t][h] . K[j][h / (Hq / n_heads)]) V[j][..],
 * j over the positions 0 .. p of its group's prefix and its own tokens.  A group's prefix is read
 * once for all its sequences.  A token that sees no key (p < 0), or only scores of -inf, gets zeros; one
 * that sees a NaN or +inf score gets NaN.
 *   - q: device, the cache's type, head h of token t at q + t*q_stride + h*D (q_stride in elements,
 *     a multiple of 8, at least Hq*D), 16-byte aligned.
 *   - out: device [n_tokens][Hq][D], 16-byte aligned, of out_dtype: QG_DT_F32 or the cache's type.
 *     Scores and sums are f32.  The tensor cores take the softmax weights in the cache's type:
 *     one rounding (2^-9 of a weight in bf16, 2^-12 in f16) for a 16-bit output, and for an f32
 *     output two terms, which leave 2^-18 (bf16) or 2^-24 (f16).  Their sums over n keys are n / 16 additions
 *     (n / 8 with two terms), each within 2^-23 of the sum: at most 0.8e-3 (1.5e-3) of it at 10^5 keys.
 *   - Rows past a sequence's length are never read: whatever they hold has no effect.  Nor do the keys and
 *     values of positions after a token's own.  An infinite or NaN value that a token sees makes that
 *     element of its output infinite or NaN.
 * Hq a multiple of n_heads, at most 16 query heads per cached head.  Workspace: qg_attn_workspace_size
 * bytes, 16-byte aligned, contents irrelevant; one call at a time may use it. */
QG_API size_t qg_attn_workspace_size(const qg_kv_cache *cache, const qg_kv_batch *batch, int Hq);
QG_API qg_status qg_attn_paged(const qg_kv_cache *cache, const qg_kv_batch *batch, int Hq, const void *q,
                               int64_t q_stride, float scale, void *out, int out_dtype, void *workspace,
                               size_t workspace_bytes, qg_stream_t stream);

/* ---- beam search -------------------------------------------------------------------------------
 * One selection: for each of N requests with W beams, the K best of the W*V continuations
 *   score[w] + log softmax(logits[w])[v]
 * in falling order, equal ones by the lowest w*V + v.  logits: f32 [N*W][V]; scores: f32 [N*W], sums of
 * log-probabilities so far (-inf: a beam that must not be continued).  An ended beam (done[w] != 0;
 * done may be NULL) has one continuation, the token eos at its score unchanged.
 *   - out_scores f32 [N][K], parents int32 [N][K] (w of the pick), tokens int32 [N][K], done_out
 *     u8 [N][K] or NULL: the parent had ended or the token is eos (eos < 0: no end token).
 *   - NaN logits and NaN or +inf scores count as -inf; a row whose largest logit is infinite has no
 *     distribution, its continuations are -inf.  Sums over the vocabulary are f32;
 *     candidates are ranked in 64 bits.
 * 1 <= W <= 64, 1 <= K <= 64, K <= W*V, V <= 2^20, 0 <= N, N*W <= 65535.  Outputs may be the arrays of the
 * next call's inputs, not of this one's.  Workspace: beam_workspace_size bytes, 16-byte aligned. */
QG_API size_t qg_beam_workspace_size(int N, int W, int K, int64_t V);
QG_API qg_status qg_beam_select(const float *logits, const float *scores, const uint8_t *done, int eos, int N, int W,
                                int K, int64_t V, float *out_scores, int32_t *parents, int32_t *tokens,
                                uint8_t *done_out, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/* The matching reorder of the cached states: beam i of request n continues the tokens of beam
 * parents[n][i] (int32 [N][W], several i may name one parent).  Per request, with len = kv_len (equal for its W
 * sequences n*W .. n*W+W-1; otherwise QG_EDEVICE_ID and the request is left as it is):
 *   - the first len / page_size columns of the W page lists are permuted: full pages are shared;
 *   - the len % page_size rows begun in the next page are copied, in every layer, from the parent's
 *     page to the beam's own page, all beams as if at once.
 * Every beam must have its own page in the column being filled; full pages must not be written
 * again.  caches: HOST array of n_layers (<= 128) caches with one geometry.  batch: n_seqs (= N*W), kv_len,
 * pages, max_pages; the rest is ignored.  1 <= W <= 32.  A parent outside [0, W) sets QG_EDEVICE_ID and the
 * beam keeps its own state; a page id outside the pool in the column being filled, of any of the W beams,
 * sets it and leaves the request as it is. */
QG_API qg_status qg_beam_reorder(const qg_kv_cache *caches, int n_layers, const qg_kv_batch *batch, int W,
                                 const int32_t *parents, qg_stream_t stream);

/* ---- drafted decode ----------------------------------------------------------------------------
 * The steps of a server that drafts tokens, verifies them with the target model and branches its contexts,
 * and the recurrent layers of hybrid decoders (gdnStep / gdnStepR and the DFlash runner on the pages).
 *
 * The gated delta rule of a linear-attention layer.  Every value head h of a sequence has a state matrix
 * S [Dk][Dv]; a token with query q, key k, value v, log decay g and step beta does
 *   S <- e^g S,   u = beta (v - S^T k),   S <- S + k u^T,   out = scale S^T q.
 *   - Value head h takes the query and key of key head h / (Hv / Hk) (QG_HEADS_GROUPED) or h % Hk
 *     (QG_HEADS_TILED).  Hv a multiple of Hk, Hv <= 1024; Dk 64 or 128; Dv a multiple of 32 up to 1024.
 *   - a, b: with a_scale and a_bias (f32[Hv] each), g = a_scale[h] softplus(a + a_bias[h]) and beta =
 *     sigmoid(b); with neither, g = a and beta = b.  g may be positive.  Log decays below -110, -inf among them, count as -110: their e^g is 0.
 *   - l2norm: q and k are first divided by sqrt(sum of squares + eps), eps >= 0.
 *   - Rows: head h of token t's q at q + t*q_stride + h*Dk (k alike; v and out with Dv; a and b one float per value
 *     head), strides in floats.  q, k, v, out 16-byte aligned with strides a multiple of 4; a and b 4-byte aligned.
 *   - States live in n_slots slots; slot s, value head h, row i, column j is at
 *     states[s*slot_stride + (h*Dk + i)*Dv + j] (16-byte aligned, slot_stride a multiple of 4).  Sequence
 *     b starts from slot state_in[b], or from zeros where that is -1 (state_in NULL: all from zeros), and leaves
 *     its last state in slot state_out[b], or nowhere (-1; NULL: none does).  state_each, NULL or int32[n_tokens],
 *     names a slot for the state after each single token (-1: not kept): a server that drafts takes the one after the
 *     last token it keeps as the next call's state_in.  A slot may be read and then written by the same sequence;
 *     no slot may be written by one sequence and used by another in one call.  A sequence without tokens writes none.
 *   - out and the states overlap no other array of the call.
 *   - q_start: device int32[n_seqs + 1], the first token row of each sequence, rising from 0 (NULL: one token each,
 *     n_tokens == n_seqs).  Rows behind the last sequence are left as they are.
 *   - max_new: the most tokens that a sequence of the call has, as far as the caller knows (0: not known).  It
 *     chooses between kernels; results are right whatever it says.
 *   - A slot outside [-1, n_slots) sets QG_EDEVICE_ID: a state_in of that kind counts as -1, the others as not kept.
 *   - A NaN or an infinity in a token's inputs, or one that finite inputs make of its update or state, reaches the tokens from that one
 *     on, never earlier ones nor other sequences or heads, and one in column j of v only column j of the outputs.
 * All sums and states are f32; in chunks, state entries below 2^-126 become 0.  Prompts go through the tensor cores 32 tokens at a
 * time: keys, queries, states and what a chunk adds to them as sums of two f16 terms with a power of two per key, query and column of a
 * state (22 bits of its largest), everything else as three bf16 terms (24 bits).  So a token's error is that of its own and its
 * column's size, whatever comes behind it and whatever has been forgotten before.  Workspace: qg_delta_workspace_size bytes, 16-byte
 * aligned, contents irrelevant, NULL where that is 0; one call at a time may use it.  args is a HOST struct.
 * Limits: n_seqs <= 65535, n_tokens <= 2^24. */
enum { QG_HEADS_GROUPED = 0, QG_HEADS_TILED = 1 };

typedef struct qg_delta_args {
  int n_seqs, n_tokens, max_new;
  int Hk, Hv, Dk, Dv;
  int head_order;                      /* QG_HEADS_GROUPED or QG_HEADS_TILED */
  int l2norm;                          /* 0 or 1 */
  int n_slots;
  float eps, scale;
  const int32_t *q_start;              /* [n_seqs + 1] or NULL */
  const float *q, *k, *v, *a, *b;
  int64_t q_stride, k_stride, v_stride, a_stride, b_stride;
  const float *a_scale, *a_bias;       /* both or neither */
  float *states;
  int64_t slot_stride;
  const int32_t *state_in, *state_out; /* [n_seqs] or NULL */
  const int32_t *state_each;           /* [n_tokens] or NULL */
  float *out;
  int64_t out_stride;
} qg_delta_args;

QG_API size_t qg_delta_workspace_size(const qg_delta_args *args);
QG_API qg_status qg_delta_rule(const qg_delta_args *args, void *workspace, size_t workspace_bytes,
                               qg_stream_t stream);

/* Probabilities of the next token: probs[t] = softmax(logits[t] / temperature[t]) over V values, f32.
 *   - temperature: device f32[T], or NULL for 1 everywhere.  A temperature that is not above 0 (0, negative, NaN)
 *     gives 1 to the lowest index of the largest logit and 0 to the rest; an infinite one, equal shares of all
 *     finite logits.
 *   - NaN logits count as -inf; a row whose largest logit is infinite has no distribution and gets zeros.
 * Rows are contiguous; probs may be logits.  Pointers 16-byte aligned; 1 <= V <= 2^20, 0 <= T <= 65535. */
QG_API qg_status qg_token_probs(const float *logits, const float *temperature, int T, int64_t V, float *probs,
                                qg_stream_t stream);

/* Verification of drafted tokens (the accept step of the DFlash and FlashMap runners, for sampled tokens).  Rows
 * q_start[b] .. q_start[b+1]-1 belong to sequence b: tokens[] there are its pending token and then its drafts, and row t of
 * probs (f32 [n_rows][V]) is the target's distribution of the token AFTER row t.  draft_probs, of the same shape,
 * is what the drafter drew the token after row t from (its last row per sequence is not read); NULL: the drafts were
 * certain.  With x = tokens[t + 1], q = draft_probs[t][x] (or 1), p = probs[t][x], a draft is accepted while
 *   u[t] q < p.
 * At the first row where it is not, the next token is drawn from max(probs - draft_probs, 0) (in f32; for certain drafts
 * probs less 1 at x); if all are accepted, from the last row's probs; where nothing is left of the difference, from probs.
 * The draw is the lowest v with  sum of r[w], w <= v,  >  u_next[b] * (sum of all r)  and r[v] > 0, or the last v with r[v]
 * > 0 where there is none; sums and comparisons carry at least 40 bits.
 *   - accepted int32[n_seqs]: how many drafts; next_token int32[n_seqs]: the drawn token, -1 where the row has no mass.
 *   - kv_len, kept_len (both or neither; int32[n_seqs]): kept_len[b] = kv_len[b] - (drafts not accepted), what qg_kv_fork
 *     is to leave of a cache that holds all of the step's rows.  They may be one array.
 *   - Negative and NaN probabilities count as 0, those above 2^100 as 2^100, NaN and negative random numbers as
 *     0.  A drafted token outside [0, V) is not accepted and sets QG_EDEVICE_ID: with draft_probs the next token is drawn from
 *     max(probs - draft_probs, 0) as for any other draft, and where drafts are certain from probs, of which nothing is taken.
 *   - A sequence without rows gets 0, -1 and its kv_len.  q_start NULL: one row each (a sampler; tokens and u may be NULL).
 * probs, draft_probs 16-byte aligned, the rest 4-byte.  1 <= V <= 2^20, n_seqs <= 65535, n_rows <= 2^24. */
QG_API qg_status qg_draft_verify(const float *probs, const float *draft_probs, const int32_t *tokens, const float *u,
                                 const float *u_next, const int32_t *q_start, int n_seqs, int n_rows, int64_t V,
                                 int32_t *accepted, int32_t *next_token, const int32_t *kv_len, int32_t *kept_len,
                                 qg_stream_t stream);

/* Pages with holders.  refs (device int32[n_pages]) counts the sequences whose page lists hold each page; a page
 * with 0 is free.  The batch's sequences are rows of its tables: kv_len and pages are READ AND WRITTEN; q_start and
 * groups are ignored.  A sequence holds the first (kv_len + page_size - 1) / page_size pages of its row; what lies behind
 * in a row stays as it is.  Counting is by integer atomics on whole calls, so results do not depend on any order.
 *
 * Fork, truncate, free: sequence b becomes the first keep[b] tokens of sequence src[b].
 *   - src[b] == b (src NULL: everywhere): truncated; src[b] == -1: freed, as with keep[b] 0; another src[b]: what b
 *     held is released and it shares the source's pages, the last one too if it is begun.  keep NULL, keep[b] -1 or above
 *     the source's length: all of it.
 *   - A sequence that others take as their source must stay as it is in that call, with src its own number and keep -1 (or
 *     NULL); a src[b] that does not, or one outside [-1, n_seqs), a keep[b] below -1, and lengths past the page lists set
 *     QG_EDEVICE_ID and leave b as it is.  A page id
 *     outside [0, n_pages) sets it and is not counted; nor does a count fall below 0.
 * cache: any layer's (the number of pages and their size count). */
QG_API qg_status qg_kv_fork(const qg_kv_cache *cache, const qg_kv_batch *batch, int32_t *refs, const int32_t *src,
                            const int32_t *keep, qg_stream_t stream);

/* Room for new tokens: kv_len[b] grows by add[b] (int32[n_seqs]), for qg_kv_append to fill.
 *   - A sequence whose last page is begun and had more than one holder when the call began gets a page of its own
 *     in its place, with the begun rows copied, in every layer; then follow the pages that the new length needs.  New pages are
 *     the lowest free ones, in the order of the sequences and their columns, each with one holder.
 *   - missing (device int32[1]): 0, or how many free pages were too few (at most 2^31 - 1); then the call changes nothing else. A batch
 *     without sequences enqueues nothing and leaves missing as it was.
 *   - add[b] 0 leaves b as it is, whatever its length and pages.  A negative add[b], a length that is negative or would pass the
 *     page list, and a begun page outside the pool set QG_EDEVICE_ID and leave b as it is.
 * caches: HOST array of n_layers (<= 128) caches of one geometry.  Workspace: qg_kv_reserve_workspace_size bytes,
 * 16-byte aligned, contents irrelevant; one call at a time may use it. */
QG_API size_t qg_kv_reserve_workspace_size(const qg_kv_cache *caches, const qg_kv_batch *batch);
QG_API qg_status qg_kv_reserve(const qg_kv_cache *caches, int n_layers, const qg_kv_batch *batch, int32_t *refs,
                               const int32_t *add, int32_t *missing, void *workspace, size_t workspace_bytes,
                               qg_stream_t stream);

/* Compaction: slot i of sequence b receives the cached token in slot keep[keep_start[b] + i] of sequence src[b], in every
 * layer, for i < keep_start[b+1] - keep_start[b]; src[b] -1: nothing.  keep_start: int32[n_seqs + 1], rising from 0 to at
 * most n_keep, the length of keep.  Keys stay rotated as they are.
 *   - The receiving pages must hold nothing that the call reads (pages from qg_kv_reserve, for instance); src[b] == b,
 *     src[b] outside [-1, n_seqs), more tokens than b's kv_len, slots outside the source's kv_len and pages outside
 *     the pool set QG_EDEVICE_ID, and those tokens are not copied.
 * caches as in qg_kv_reserve.  n_keep <= 2^24. */
QG_API qg_status qg_kv_compact(const qg_kv_cache *caches, int n_layers, const qg_kv_batch *batch, const int32_t *src,
                               const int32_t *keep_start, const int32_t *keep, int n_keep, qg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GGUFDQ_H */
