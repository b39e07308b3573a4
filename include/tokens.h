/*
 * tokens.h -- C ABI of the operators for sequences of tokens (MI355X, gfx950),
 * part of the same library as voxelize.h and sharing its return codes and
 * conventions (host-side argument checks, caller-owned device memory on the
 * current device, work enqueued on `stream` without synchronising, nothing
 * allocated on the device, no state kept between calls).
 *
 * A detector that treats pillars (voxelize.h) or the points of a scan
 * (spherical.h) as tokens needs, next to the binning:
 *   - an embedding lookup: every token takes a row of a table (the learned
 *     row of its cell, or the feature row of its pillar by the point map),
 *     and the gradient of that table;
 *   - attention between the tokens of a frame, with a bias that falls with
 *     their distance on the grid, forward and backward;
 *   - a gated linear recurrence along an order of the tokens, forward and
 *     backward.
 * Frames are packed one after another: token tensors are [T, ...] and an
 * int32 array of `docs + 1` offsets on the device says where each frame
 * (document) starts and ends. Tokens before the first offset or from the last
 * one on belong to no document, so a buffer of a fixed capacity may be passed
 * with the offsets of what it holds. The offsets are device data: they are
 * clamped to [0, T] and a decreasing pair is an empty document, so a wrong
 * array gives wrong results but no access outside the tensors.
 *
 * Results do not depend on the order in which blocks run: no floating-point
 * atomics are used and every sum is added in a fixed order, so the same call
 * on the same inputs gives the same bits.
 */
#ifndef TOKENS_H
#define TOKENS_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "voxelize.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define TOK_F32 0
#define TOK_BF16 1
#define TOK_F16 2

/* ---- embedding ------------------------------------------------------------
 *
 * out[i, :] = scale * table[ids[i], :] for i in [0, n), computed in float32
 * and rounded once to the table's type; a row of zeros where ids[i] is not in
 * [0, rows) (the library marks a point without a pillar with -1). ids is
 * int32 (id_bytes 4) or int64 (id_bytes 8), contiguous. Rows of `width`
 * elements, table rows `row_stride` elements apart, out contiguous.
 * Limits: 0 <= n <= 2^31 - 1, 1 <= rows <= 2^31 - 1, 1 <= width <= 65536.
 */
int tok_embed(const void* table, int64_t rows, int64_t width, int64_t row_stride, int32_t dtype,
              const void* ids, int32_t id_bytes, int64_t n, float scale, void* out,
              hipStream_t stream);

/*
 * Gradient of the table: out[r, :] = scale * (sum of grad[i, :] over the i
 * with ids[i] == r), every row written (zeros where no token has the row),
 * [rows, width] contiguous, in grad's type. Sums are held in float32: the
 * tokens of a row are added in token order inside runs of a fixed length, and
 * the runs in order. grad rows are `grad_stride` elements apart.
 * Limits: 0 <= n <= 2^27, 1 <= rows <= 2^24, 1 <= width <= 65536.
 * The workspace (0 bytes: NULL will do) needs no initial contents, 256-byte
 * aligned.
 */
int64_t tok_embed_grad_workspace_bytes(int64_t n, int64_t rows, int64_t width);
int tok_embed_grad(const void* grad, int64_t grad_stride, int32_t dtype, const void* ids,
                   int32_t id_bytes, int64_t n, int64_t rows, int64_t width, float scale,
                   void* out, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* ---- attention ------------------------------------------------------------
 *
 * q [tq, heads, width], k and v [tk, kv_heads, width], bf16 or fp16, packed by
 * q_offsets and k_offsets [docs + 1]. Query head h reads key head
 * h / (heads / kv_heads). For query i and key j of the same document (both
 * counted from its start, lq and lk its lengths):
 *   z = scale * q.k;  if cap > 0: z = cap * tanh(z / cap)
 *   if axes > 0: z -= slopes[h] * sum over the axes of |q_pos[i] - k_pos[j]|
 *   key j is visible to query i when mask is 0, or j <= i + (lk - lq), or
 *   j < prefix[document] (prefix NULL: 0)
 *   out = sum over visible j of softmax(z)[j] * v[j];  lse = log sum exp z
 * A query that sees no key gets zeros and lse = -inf, and passes no gradient.
 * Scores, softmax statistics and sums are held in float32; the softmax
 * weights and the score gradients are rounded to the tensors' type before
 * they enter the second products, with powers of two taken out first where
 * fp16 would not hold them. Keys of other documents, and rows of no
 * document, never enter a result whatever they hold; inside a document a
 * value that is not finite may reach every query of it.
 * Positions are int32 in [0, 65535] (values outside are clamped), 1 to 3 axes,
 * any strides. width: a multiple of 8, at most 128. Token and head strides of
 * q, k, v are multiples of 8 elements, the token strides below 2^25 elements
 * and the bases 16-byte aligned; out,
 * lse [tq, heads] and the gradients are contiguous, grad_out as q.
 */
typedef struct tok_attention {
    int32_t dtype;              /* TOK_BF16 or TOK_F16 */
    int32_t heads, kv_heads;    /* heads a multiple of kv_heads */
    int32_t width;
    int64_t tq, tk;             /* tokens; tq * heads, tk * kv_heads <= 2^31 - 2048 */
    int32_t docs;               /* >= 1, at most 2^20; (docs + 2) * kv_heads <= 2^30 */
    int32_t mask;               /* 0: every key of the document; 1: causal / prefix */
    const int32_t* q_offsets;   /* device [docs + 1]; NULL: one document of all tokens */
    const int32_t* k_offsets;
    const int32_t* prefix;      /* device [docs] or NULL */
    float scale;                /* in [1e-30, 1e30] */
    float cap;                  /* 0: none; else in [2^-126, 2^127] */
    const float* slopes;        /* device [heads]; NULL when axes is 0. slopes and, without a
                                   cap, slopes / scale: magnitudes below 2^100 */
    const int32_t* q_pos;       /* device [tq, axes] */
    const int32_t* k_pos;       /* device [tk, axes] */
    int32_t axes;               /* 0 (no bias) to 3 */
    int32_t reserved;           /* 0 */
    int64_t q_stride[2], k_stride[2], v_stride[2], g_stride[2]; /* token, head; g: grad_out */
    int64_t q_pos_stride[2], k_pos_stride[2];                   /* token, axis */
} tok_attention;

/* Bytes of workspace for tok_attend / tok_attend_grad (0: NULL will do), or
 * VOX_EINVAL. The workspace needs no initial contents, 256-byte aligned. */
int64_t tok_attend_workspace_bytes(const tok_attention* args);
int64_t tok_attend_grad_workspace_bytes(const tok_attention* args);

/* lse may be NULL. */
int tok_attend(const tok_attention* args, const void* q, const void* k, const void* v, void* out,
               float* lse, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Gradients of q, k and v from the forward's out and lse. */
int tok_attend_grad(const tok_attention* args, const void* q, const void* k, const void* v,
                    const void* out, const float* lse, const void* grad_out, void* grad_q,
                    void* grad_k, void* grad_v, void* workspace, int64_t workspace_bytes,
                    hipStream_t stream);

/* ---- gated recurrence -----------------------------------------------------
 *
 * gate and x [t, width] (float32, bf16 or fp16, contiguous), packed by
 * offsets [docs + 1]; state [docs, width] float32 or NULL (zeros). Along each
 * document, from its first token (reverse 0) or its last (reverse 1):
 *   a = 1 / (1 + exp(-gate));  h = a * h + (1 - a) * x;  y[t] = h
 * starting from the document's state; last_state [docs, width] float32 (or
 * NULL) receives h after its last step (the state itself for a document of no
 * tokens). Tokens of no document get y = 0 and no gradient. The state is held
 * in float32. carry (or NULL) receives the state before each run of
 * TOK_SCAN_RUN tokens, [tok_scan_runs(t), width] float32, for tok_scan_grad.
 * The workspace (0 bytes: NULL will do) needs no initial contents, 256-byte
 * aligned.
 * Limits: 0 <= t <= 2^31 - 2048, 1 <= width <= 65536, 1 <= docs <= 2^20.
 */
#define TOK_SCAN_RUN 16
int64_t tok_scan_runs(int64_t t);
int64_t tok_scan_workspace_bytes(int64_t t, int64_t width);
int tok_scan(const void* gate, const void* x, int32_t dtype, int64_t t, int64_t width,
             const int32_t* offsets, int32_t docs, int32_t reverse, const float* state, void* y,
             float* last_state, float* carry, void* workspace, int64_t workspace_bytes,
             hipStream_t stream);

/* Gradients of gate, x and state (grad_state, or NULL) from those of y and of
 * last_state (grad_last, or NULL: zeros). The workspace is of
 * tok_scan_workspace_bytes. */
int tok_scan_grad(const void* grad_y, const void* gate, const void* x, const float* carry,
                  int32_t dtype, int64_t t, int64_t width, const int32_t* offsets, int32_t docs,
                  int32_t reverse, const float* state, const float* grad_last, void* grad_gate,
                  void* grad_x, float* grad_state, void* workspace, int64_t workspace_bytes,
                  hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TOKENS_H */
