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
 *   norm     layer norm of rows, and its gradients
 *   ffn      the experts' gated feed-forward products over rows sorted by
 *            expert, and their gradients
 *   adamw    one AdamW step over many tensors, moments in 32 or in 8 bits
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

/* ---- layer norm -------------------------------------------------------------
 *   mean[n] = mean over d of x[n, d]
 *   rstd[n] = 1 / sqrt(mean over d of (x[n, d] - mean[n])^2 + eps)
 *   xh[n, d] = (x[n, d] - mean[n]) * rstd[n]
 *   y[n, d]  = xh[n, d] * w[d] + b[d]
 * and with a[n, d] = dy[n, d] * w[d]
 *   dx[n, d] = rstd[n] * (a - mean over d of a - xh * mean over d of a * xh)
 *   dw[d] = sum over n of dy * xh          db[d] = sum over n of dy
 * A NULL w stands for ones, a NULL b for zeros. 1 <= D <= 2^28, N < 2^31 - 1,
 * eps finite and >= 0 (with eps 0 a row of equal values gives NaN). */
typedef struct {
    int64_t N;            /* rows, >= 0 */
    int32_t D;            /* columns */
    tbe_dtype dtype;      /* element type of x, y and their gradients */
    tbe_dtype wdtype;     /* element type of w, b and their gradients */
    float eps;
} tbe_norm_desc;

/* x: device [N, D]. w, b: device [D], dense, each may be NULL. y: device
 * [N, D], overwritten. stats: device float32 [N, 2], overwritten: mean and
 * rstd of each row, for the backward. */
tbe_status tbe_norm_forward(const tbe_norm_desc* desc, const void* x, int64_t ldx, const void* w,
                            const void* b, void* y, int64_t ldy, float* stats, void* stream);

/* Bytes of the backward's workspace (0 on a bad description), as above. */
size_t tbe_norm_workspace_bytes(const tbe_norm_desc* desc);

/* dy: device [N, D]. dx: device [N, D], overwritten. dw, db: device [D],
 * dense, overwritten (zeros when N = 0); each may be NULL, which leaves it
 * out. Where the mean's rounding to float32 matters (|mean| far above the
 * deviation) the call corrects it from x. */
tbe_status tbe_norm_backward(const tbe_norm_desc* desc, const void* dy, int64_t lddy,
                             const void* x, int64_t ldx, const void* w, const float* stats,
                             void* dx, int64_t lddx, void* dw, void* db, void* ws,
                             size_t ws_bytes, void* stream);

/* ---- experts' gated feed-forward ---------------------------------------------
 * Row r of xs belongs to expert e when offsets[e] <= r < offsets[e + 1]
 * (tbe_expert_plan's offsets, tbe_expert_dispatch's rows). With its matrices
 *   g = xs[r, :] gate[e]^T      u = xs[r, :] up[e]^T       [F]
 *   h = act(g) * u              ys[r, :] = h down[e]^T     [D]
 * One expert and offsets 0, M make it a dense gated feed-forward block.
 * Rows that belong to no expert are not read, and left as they are in every
 * output. Offsets are read on the device; one below its predecessor or outside
 * [0, M] is taken for the nearest that is neither.
 * Products accumulate in float32. In 16-bit types pre, h and the gradients of
 * g and u are rounded to the type between the products that use them.
 * 1 <= E <= 1023, 1 <= D, F <= 65536, M * max(D, 2 F) <= 2^36,
 * E * D * F <= 2^36, M < 2^31 - 1024. */
typedef enum { TBE_ACT_SILU = 0, TBE_ACT_GELU = 1 } tbe_act;   /* GELU by the error function */

typedef struct {
    int64_t M;            /* rows, >= 0 */
    int32_t E;            /* experts */
    int32_t D;            /* columns of a row */
    int32_t F;            /* columns between the products */
    tbe_dtype dtype;      /* element type of every matrix */
    int32_t act;          /* tbe_act */
} tbe_ffn_desc;

/* E matrices: element (r, c) of matrix e is data[e * stride + r * ld + c].
 * An input's ld and stride may be any values >= 0; an output's rows and
 * matrices must not overlap (ld >= columns, stride >= rows * ld where E > 1). */
typedef struct {
    void* data;
    int64_t ld;
    int64_t stride;
} tbe_stack;

/* Bytes of the workspace of both calls (0 on a bad description), as above. */
size_t tbe_ffn_workspace_bytes(const tbe_ffn_desc* desc);

/* xs: device [M, D]. offsets: device int32 [E + 1]. gate, up: [E] of [F, D],
 * down: [E] of [D, F], device, read only. pre: device [M, 2 F], overwritten
 * with g and u beside each other, for the backward; may be NULL. ys: device
 * [M, D], overwritten. */
tbe_status tbe_ffn_forward(const tbe_ffn_desc* desc, const void* xs, int64_t ldxs,
                           const int32_t* offsets, const tbe_stack* gate, const tbe_stack* up,
                           const tbe_stack* down, void* pre, int64_t ldpre, void* ys,
                           int64_t ldys, void* ws, size_t ws_bytes, void* stream);

/* dys: device [M, D]; pre as the forward left it. dxs: device [M, D],
 * overwritten. dgate, dup: [E] of [F, D], ddown: [E] of [D, F], device,
 * overwritten (zeros for an expert without rows). */
tbe_status tbe_ffn_backward(const tbe_ffn_desc* desc, const void* dys, int64_t lddys,
                            const void* xs, int64_t ldxs, const int32_t* offsets,
                            const tbe_stack* gate, const tbe_stack* up, const tbe_stack* down,
                            const void* pre, int64_t ldpre, void* dxs, int64_t lddxs,
                            const tbe_stack* dgate, const tbe_stack* dup, const tbe_stack* ddown,
                            void* ws, size_t ws_bytes, void* stream);

/* ---- AdamW ------------------------------------------------------------------
 * With g the gradient times *scale, t = *step (counted from 1; less is taken
 * for 1) and *lr, element by element over all tensors of the call:
 *   m = beta1 m + (1 - beta1) g       v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in float32, p rounded once to its type. step, lr and scale are device memory
 * and read by the kernels, so a captured step follows them.
 * bits = 32: m and v are float32. bits = 8: each moment is an e4m3 number (4
 * exponent and 3 mantissa bits, up to 448) times the float32 scale of its
 * block of 256 elements, counted from the tensor's start; the scale is the
 * block's largest magnitude times the float32 nearest to 1 / 448, the number
 * the nearest to the value divided by it, ties to even. m holds the moment, v
 * the root of the second moment, both from the formulas above with every
 * operation rounded to float32 by itself (constants beforehand, v's second term
 * as ((1 - beta2) g) g): they are the same bits wherever the formulas are
 * evaluated so. A root above zero is held as at least the smallest number, so
 * that no update is divided by eps alone. Blocks whose largest magnitude is
 * below 2^-100 are held as zeros, a moment that is not finite as NaN (its
 * block's others keep theirs). All buffers zero is the state before step 1. */
typedef struct {
    tbe_dtype pdtype;     /* element type of the parameters */
    tbe_dtype gdtype;     /* of the gradients */
    int32_t cdtype;       /* of the copies: TBE_F16 or TBE_BF16 with float32 parameters, -1: none */
    int32_t bits;         /* 32 or 8 */
    double beta1, beta2;  /* in [0, 1) */
    double eps;           /* >= 0, finite; TBE_ERR_UNSUPPORTED above 0 and below 2^-126.
                             With eps 0 an element whose gradients are all zero gives NaN. */
    double weight_decay;  /* >= 0, finite */
} tbe_adamw_desc;

/* One tensor of n elements, dense, any start (8-bit moments: a multiple of 8
 * bytes). Nothing that is written may overlap; a parameter that overlaps
 * another parameter, or a copy another copy, is refused. */
typedef struct {
    void* p;              /* parameters, updated */
    const void* g;        /* gradients */
    void* m;              /* moments, updated */
    void* v;
    float* mscale;        /* [(n + 255) / 256], updated; bits = 8 only */
    float* vscale;
    void* c;              /* the new parameters rounded to cdtype, overwritten; cdtype >= 0 only */
    int64_t n;            /* elements, >= 0 */
} tbe_adamw_tensor;

/* tensors: HOST array of `count`, read during the call. step: device int64.
 * lr: device float32. scale: device float32, NULL for 1. count < 2^24,
 * n < 2^40. */
tbe_status tbe_adamw_step(const tbe_adamw_desc* desc, const tbe_adamw_tensor* tensors,
                          int64_t count, const int64_t* step, const float* lr,
                          const float* scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_LM_H */
