/*
 * tbe_lm.h — language-model operators beside the table-batched embedding.
 *
 *   token    lookup of one token table with a scale, and the table's dense
 *            gradient
 *   expert   assignments of tokens to experts sorted by expert, the rows sent
 *            there (dispatch) and back with weights (combine), and the
 *            gradients of both
 *   distill  distillation loss of a student's logits against a teacher's top
 *            logits, and its gradient
 *
 * Conventions are those of tbe.h: the caller owns every buffer, nothing is
 * allocated, work is enqueued on `stream` (a hipStream_t, NULL = the null
 * stream) and the call returns without waiting, argument errors are found on
 * the host before anything is enqueued, TBE_ERR_HIP reports a failed launch
 * (tbe_last_error has the text). Every call may be captured into a HIP graph
 * (kernels only). Results are the same bits from call to call: no sum's order
 * depends on the order in which workgroups run.
 *
 * Matrices are row-major with unit column stride and a row stride `ld...` in
 * elements. An output's row stride is at least its width; an input's may be
 * any value >= 0 (0: every row is the same row). Rows need only their
 * element's alignment. Element offsets are 64-bit. Unless stated, an output
 * must not overlap an input.
 *
 * Element types are tbe_dtype; sums, softmax statistics and losses are float32
 * and every 16-bit result is rounded once, to nearest even.
 *
 * Ids are int32 or int64 (`idx64`), device memory, dense.
 */
#ifndef TBE_LM_H
#define TBE_LM_H

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- token table ---------------------------------------------------------
 *   forward    out[n, :] = scale * W[ids[n], :]
 *   backward   gW[v, :]  = scale * sum over n with ids[n] = v of g[n, :]
 * An id outside [0, V) is padding: its output row is zero and it adds nothing
 * to gW. The backward writes all V rows of gW (zeros where no token has the
 * id). 1 <= V <= 1047552 (1023 * 1024), N < 2^30, 1 <= D <= 2^28 (else
 * TBE_ERR_ARG or TBE_ERR_UNSUPPORTED). */
typedef struct {
    int64_t N;            /* tokens, >= 0 */
    int64_t V;            /* rows of the table */
    int32_t D;            /* columns */
    tbe_dtype wdtype;     /* element type of W and gW */
    tbe_dtype xdtype;     /* element type of out and g */
    int32_t idx64;        /* 0: int32 ids, 1: int64 ids */
    float scale;
} tbe_token_desc;

/* W: device [V, D], read only. out: device [N, D], overwritten. */
tbe_status tbe_token_forward(const tbe_token_desc* desc, const void* W, int64_t ldw,
                             const void* ids, void* out, int64_t ldo, void* stream);

/* Bytes of the backward's workspace (0 on a bad description). Scratch device
 * memory, 256-byte aligned; its contents need not be preserved. Host only. */
size_t tbe_token_workspace_bytes(const tbe_token_desc* desc);

/* g: device [N, D], read only. gW: device [V, D], overwritten. */
tbe_status tbe_token_backward(const tbe_token_desc* desc, const void* g, int64_t ldg,
                              const void* ids, void* gW, int64_t ldgw, void* ws, size_t ws_bytes,
                              void* stream);

/* ---- experts --------------------------------------------------------------
 * Assignment j = n*K + k sends token n to expert ids[n, k]; ids outside
 * [0, E) are dropped. The plan sorts the M = N*K assignments by expert,
 * stably, dropped ones last:
 *   offsets[e]  first place of expert e; offsets[E] = assignments kept
 *   order[p]    the assignment at place p
 *   slots[j]    the place of assignment j; ~place (negative) when dropped
 * The other calls read only `slots`. They take a slot outside [-M, M) for a
 * dropped assignment without a place: it is neither read nor written.
 * 1 <= E <= 1023, 1 <= K <= 64, 1 <= D <= 2^28, N*K < 2^31 - 1. */
typedef struct {
    int64_t N;            /* tokens, >= 0 */
    int32_t K;            /* assignments per token */
    int32_t E;            /* experts */
    int32_t D;            /* columns of a row */
    tbe_dtype dtype;      /* element type of every matrix of rows */
    int32_t idx64;        /* 0: int32 ids, 1: int64 ids */
} tbe_expert_desc;

/* Bytes of tbe_expert_plan's workspace (0 on a bad description), as above. */
size_t tbe_expert_workspace_bytes(const tbe_expert_desc* desc);

/* ids: device [N, K]. offsets int32 [E+1], order int32 [M], slots int32 [M]:
 * device, overwritten. */
tbe_status tbe_expert_plan(const tbe_expert_desc* desc, const void* ids, int32_t* offsets,
                           int32_t* order, int32_t* slots, void* ws, size_t ws_bytes,
                           void* stream);

/* xs[place of (n,k), :] = x[n, :]; places of dropped assignments get zeros.
 * x: device [N, D]. xs: device [M, D], overwritten. */
tbe_status tbe_expert_dispatch(const tbe_expert_desc* desc, const void* x, int64_t ldx,
                               const int32_t* slots, void* xs, int64_t ldxs, void* stream);

/* dx[n, :] = sum over kept k of dxs[place of (n,k), :]. */
tbe_status tbe_expert_dispatch_backward(const tbe_expert_desc* desc, const void* dxs,
                                        int64_t lddxs, const int32_t* slots, void* dx,
                                        int64_t lddx, void* stream);

/* out[n, :] = sum over kept k of w[n, k] * ys[place of (n,k), :].
 * w: device float32 [N, K], dense. A dropped assignment's weight and row are
 * not used (NaN there is harmless). */
tbe_status tbe_expert_combine(const tbe_expert_desc* desc, const void* ys, int64_t ldys,
                              const int32_t* slots, const float* w, void* out, int64_t ldo,
                              void* stream);

/* dys[place of (n,k), :] = w[n, k] * dout[n, :] (zeros where dropped);
 * dw[n, k] = <dout[n, :], ys[place of (n,k), :]> (0 where dropped).
 * dys may be ys itself (the same address and row stride). dw: device float32
 * [N, K], dense. */
tbe_status tbe_expert_combine_backward(const tbe_expert_desc* desc, const void* dout,
                                       int64_t lddo, const void* ys, int64_t ldys,
                                       const int32_t* slots, const float* w, void* dys,
                                       int64_t lddys, float* dw, void* stream);

/* ---- distillation -----------------------------------------------------------
 * Row n has a student's logits x[n, 0..V) and a teacher's K logits t[n, k] at
 * the vocabulary places ids[n, k]. With tau the temperature:
 *   p = softmax over the row's entries of t[n, k] / tau
 *   q = softmax over the vocabulary of x[n, v] / tau
 *   loss[n]   = tau^2 * sum over k of p_k * (log p_k - log q[ids[n, k]])
 *   gx[n, v]  = gl[n] * tau * (q[v] - sum over k with ids[n, k] = v of p_k)
 * which is gl[n] times the gradient of loss[n]. Entries with an id outside
 * [0, V) or with t = -inf take no part. A row with no entry left has loss 0
 * and a zero gradient whatever its logits are, which are then not read. The
 * same id may occur more than once in a row. Logits of -inf have q = 0 (a
 * teacher's entry there with p > 0 makes the loss +inf); a row with a NaN or
 * +inf logit, or none but -inf, gives NaN.
 * 1 <= V < 2^31 - 1, 1 <= K <= 1024, tau finite and > 0 (TBE_ERR_UNSUPPORTED
 * below 4.24e-39, where log2(e) / tau is no float32). */
typedef struct {
    int64_t N;            /* rows, >= 0 */
    int64_t V;            /* vocabulary */
    int32_t K;            /* teacher's entries per row */
    tbe_dtype dtype;      /* element type of x and gx */
    tbe_dtype tdtype;     /* element type of t */
    int32_t idx64;        /* 0: int32 ids, 1: int64 ids */
    float temperature;
} tbe_distill_desc;

/* Bytes of the workspace of the forward and the step (0 on a bad
 * description), as above. Both calls require it; the kernels of this version
 * need no scratch memory and leave it as it is, so its size is one alignment
 * unit whatever the description. */
size_t tbe_distill_workspace_bytes(const tbe_distill_desc* desc);

/* x: device [N, V]. ids, t: device [N, K], dense. loss: device float32 [N],
 * overwritten. stats: device float32 [N, 2], overwritten: the row's largest
 * logit and the sum of exp((x - largest) / tau), for the backward (0 and 0
 * for a row without a teacher). */
tbe_status tbe_distill_forward(const tbe_distill_desc* desc, const void* x, int64_t ldx,
                               const void* ids, const void* t, float* loss, float* stats,
                               void* ws, size_t ws_bytes, void* stream);

/* gl: device float32 [N], upstream gradient of loss. gx: device [N, V],
 * overwritten; may be x itself (the same address and row stride). */
tbe_status tbe_distill_backward(const tbe_distill_desc* desc, const void* x, int64_t ldx,
                                const void* ids, const void* t, const float* stats,
                                const float* gl, void* gx, int64_t ldgx, void* stream);

/* Forward and backward in one call, for a training step that knows gl
 * beforehand. gx may be x itself (the same address and row stride). */
tbe_status tbe_distill_step(const tbe_distill_desc* desc, const void* x, int64_t ldx,
                            const void* ids, const void* t, const float* gl, float* loss,
                            void* gx, int64_t ldgx, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_LM_H */
