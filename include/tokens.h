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
 *     backward;
 *   - rotary positions: queries and keys turned by their places, and turned
 *     back;
 *   - attention with decay, whose cost grows with the tokens alone, forward,
 *     backward and token by token;
 *   - the loss of predicting a row of the table (the next pillar's cell), and
 *     its gradients.
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

/* ---- rotary positions -------------------------------------------------------
 *
 * x [tokens, heads, width] (float32, bf16 or fp16), strides in elements, an
 * element's 1. The first 2 * axes * pairs elements of a head are turned, axis
 * by axis of the positions [tokens, axes] (int32, any value, 1 to 3 axes, strides
 * in elements): pair p of axis c, elements (u, v), by the angle
 * pos[t, c] * freqs[c, p]:
 *   (u cos - v sin, u sin + v cos);  inverse 1: by the opposite angle.
 * Axis c has the elements from 2 * c * pairs on; its pair p is the elements
 * (p, pairs + p) of them, or interleaved (2 p, 2 p + 1). The rest of the head is
 * copied. freqs [axes, pairs] is float64 (radians a position), contiguous: the
 * angle is reduced to a turn in 64 bits, with what their roundings leave, and is
 * right to 2^-25 of a turn however far the position. Sines, cosines and products
 * are in float32, rounded once to x's type. out is contiguous. The gradient of x
 * is the gradient of out turned back.
 * Limits: 0 <= tokens <= 2^31 - 1, 1 <= heads, width <= 65536; a finite
 * frequency's product with a position below 2^52 turns.
 */
int tok_rotate(const void* x, int64_t tokens, int64_t heads, int64_t width, int64_t token_stride,
               int64_t head_stride, int32_t dtype, const int32_t* pos, int64_t pos_stride,
               int64_t axis_stride, int32_t axes, const double* freqs, int64_t pairs,
               int32_t interleaved, int32_t inverse, void* out, hipStream_t stream);

/* ---- attention with decay ---------------------------------------------------
 *
 * q [t, heads, width], k and v [t, kv_heads, width], bf16 or fp16, packed by
 * offsets [docs + 1]; query head h reads key head h / (heads / kv_heads) and has a
 * state S [width, width] of its own. Along each document, from its first token
 * (reverse 0) or its last (reverse 1):
 *   S = exp(-decay[h]) S + k v^T;  out[t] = scale * q S
 * from the document's state (state [docs, heads, width, width] float32, S[i, j]
 * of k's element i and v's j; NULL: zeros); last_state of the same shape (or NULL)
 * receives S after its last step (the state itself for a document of no tokens).
 * Tokens of no document get zeros and no gradient. decay is float32 on the device;
 * negative values (and NaN) are taken as 0 and values over 1000 as 1000. States and
 * sums are float32; documents of more than a token or two are taken in chunks of 32
 * tokens on matrix instructions, for which the copy of a state that q is multiplied
 * with is rounded to the tensors' type (in fp16 after a power of two that brings the
 * largest of 32 columns to about 1; under 2^-14 of it bits are lost). A value that is
 * not finite may reach every token of its chunk of 32 and of the document after it,
 * and none of another one.
 * carry receives what tok_decay_attend_grad needs besides: tok_decay_carry_rows()
 * states [heads, width, width] float32 (0: NULL will do). It is needed without
 * gradients too: it is the call's workspace.
 * Limits: t * heads and t at most 2^31 - 4096, 1 <= docs <= 2^20,
 * (docs + 2) * heads <= 2^30; width a multiple of 8, at most 128; strides multiples of
 * 8, the token strides below 2^25; all bases 16-byte aligned; scale in [1e-30, 1e30].
 */
typedef struct tok_decay {
    int32_t dtype;              /* TOK_BF16 or TOK_F16 */
    int32_t heads, kv_heads;    /* heads a multiple of kv_heads */
    int32_t width;
    int64_t t;                  /* tokens */
    int32_t docs, reverse;
    const int32_t* offsets;     /* device [docs + 1]; NULL: one document of all tokens */
    const float* decay;         /* device [heads] */
    float scale;
    int32_t reserved;           /* 0 */
    int64_t q_stride[2], k_stride[2], v_stride[2], g_stride[2]; /* token, head; g: grad_out */
} tok_decay;

/* Or VOX_EINVAL. */
int64_t tok_decay_carry_rows(const tok_decay* args);
int64_t tok_decay_grad_workspace_bytes(const tok_decay* args);

int tok_decay_attend(const tok_decay* args, const void* q, const void* k, const void* v,
                     const float* state, void* out, float* last_state, float* carry,
                     hipStream_t stream);

/* Gradients of q, k, v and state (grad_state, or NULL) from those of out and of
 * last_state (grad_last, or NULL: zeros), with the carry of the forward call.
 * Gradients of shared key heads are summed over their query heads in float32, whose
 * parts are in the workspace: 8 bytes an element of q. */
int tok_decay_attend_grad(const tok_decay* args, const void* q, const void* k, const void* v,
                          const void* grad_out, const float* state, const float* carry,
                          const float* grad_last, void* grad_q, void* grad_k, void* grad_v,
                          float* grad_state, void* workspace, int64_t workspace_bytes,
                          hipStream_t stream);

/* ---- loss over a table's rows -----------------------------------------------
 *
 * x [t, width] and table [rows, width], bf16 or fp16, rows x_stride and
 * table_stride elements apart; ids [t] int32 (id_bytes 4) or int64 (8):
 *   lse[i]  = log sum over r of exp(scale * x[i].table[r])
 *   loss[i] = lse[i] - scale * x[i].table[ids[i]]
 * both float32; 0 where ids[i] is not in [0, rows), and then nothing of x[i] is
 * used. lse may be NULL. Logits are not kept: they are summed as they are made,
 * and made again for the gradients, in pieces of the rows. Logits, maxima and sums
 * are float32.
 *
 * The gradients, with w[i, r] = (exp(scale * x[i].table[r] - lse[i]) - [r is
 * ids[i]]) * grad[i] for the gradient grad [t] float32 of the loss:
 *   grad_x[i] = scale * sum over r of w[i, r] table[r]        [t, width]
 *   grad_table[r] = scale * sum over i of w[i, r] x[i]        [rows, width]
 * contiguous, in x's type, every row written; one of the two may be NULL and is not
 * computed then. w is rounded to that type (fp16:
 * after a power of two that brings the largest |grad| to 2^14; under 2^-28 of that
 * bits are lost), of up to 256 tokens in two parts; sums are float32.
 * Limits: 0 <= t <= 2^25, 1 <= rows <= 2^31 - 2048; width a multiple of 8, at most
 * 65536; strides multiples of 8 below 2^22; all bases 16-byte aligned; scale in
 * [1e-30, 1e30]. The workspace needs no initial contents, 256-byte aligned. It holds x once (a width
 * over 128 rounded up to whole 256s; forward only then, and of more than 32 tokens), for gradients x in
 * float32 besides and an eighth of x where tokens are more than 2^19, 12 bytes a token, and up to 768 MiB
 * that do not grow with the tokens (three times as much at widths over 4096).
 */
int64_t tok_row_loss_workspace_bytes(int64_t t, int64_t rows, int64_t width);
int tok_row_loss(const void* x, int64_t x_stride, const void* table, int64_t table_stride,
                 int32_t dtype, int64_t t, int64_t rows, int64_t width, const void* ids,
                 int32_t id_bytes, float scale, float* loss, float* lse, void* workspace,
                 int64_t workspace_bytes, hipStream_t stream);

int64_t tok_row_loss_grad_workspace_bytes(int64_t t, int64_t rows, int64_t width);
int tok_row_loss_grad(const float* grad, const void* x, int64_t x_stride, const void* table,
                      int64_t table_stride, int32_t dtype, int64_t t, int64_t rows, int64_t width,
                      const void* ids, int32_t id_bytes, const float* lse, float scale,
                      void* grad_x, void* grad_table, void* workspace, int64_t workspace_bytes,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TOKENS_H */
