/*
 * conv_train.h -- C ABI of the operators a training step runs around the conv layers of
 * conv.h: group normalisation with an activation, the embedding lookup with its gradient, layer
 * normalisation of a residual sum, the gated scan over time, the loss against a teacher's top
 * logits, and the global gradient norm with clipping.
 *
 * The conventions are conv.h's: device pointers owned by the caller, no allocation inside the
 * library (workspaces are sized by a query and passed in), calls that are asynchronous on
 * `stream`, outputs overwritten whole, bit-identical results run to run (fixed reduction
 * orders, no floating-point atomics), argument errors found on the host before anything is
 * enqueued and returned as a conv_status_t.  Sums, means and norms are held in fp32; a bf16
 * result is rounded once, to nearest even.  A call runs on the current device.  A workspace is
 * scratch: its contents on entry are ignored, and two calls may share one only if they cannot
 * overlap on the GPU.
 * Offsets are 64-bit: unlike in conv.h a tensor may hold more than 2^31 elements where the
 * limits stated below allow it.
 */
#ifndef IGCONV_CONV_TRAIN_H
#define IGCONV_CONV_TRAIN_H

#include "conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- group normalisation with an activation ------------------------------------------------
 * x holds B samples of C channels at P positions (P = H*W of an image, OH*OW of a conv's
 * output); the C channels form G groups of C/G consecutive channels, M = (C/G)*P values a
 * sample and group:
 *
 *   mean = sum x / M      rstd = 1 / sqrt(sum (x - mean)^2 / M + eps)
 *   xhat = (x - mean) * rstd      z = xhat * gamma[c] + beta[c]      y = act(z)
 *   dz = dy * act'(z)     dbeta[c] = sum_{b,p} dz     dgamma[c] = sum_{b,p} dz * xhat
 *   dx = rstd * (dz*gamma[c] - m1 - xhat * m2)
 *        m1 = sum over the group of dz*gamma / M,  m2 = sum over the group of dz*gamma*xhat / M
 *
 * act: none, max(z, 0) (with act'(0) = 0), z / (1 + exp(-z)), or z * Phi(z) with Phi the normal
 * distribution function (by erf).
 * Layouts (dense): CONV_LAYOUT_NCHW is (B, C, P), the conv layers' own; CONV_LAYOUT_NHWC is
 * (B, P, C), channels last.  x, y, dy, dx, gamma, beta, dgamma, dbeta have the descriptor's
 * dtype; mean and rstd are fp32, (B, G).
 * With CONV_ACT_RELU, xhat and z are computed by separate, individually rounded fp32 operations
 * in both directions: with the forward's mean and rstd the backward's z has the forward's bits
 * and its ReLU mask is exactly y > 0 of the fp32 forward.  For the other activations, whose
 * derivatives have no jump, only z's value is fixed: how its operations are joined and rounded
 * depends on the sizes.  GELU's Phi is within 3.1e-7 (fp32).
 * A value that is infinite or NaN makes its whole group NaN and leaves the others alone. */
typedef enum { CONV_LAYOUT_NCHW = 0, CONV_LAYOUT_NHWC = 1 } conv_layout_t;
typedef enum { CONV_ACT_NONE = 0, CONV_ACT_RELU = 1, CONV_ACT_SILU = 2, CONV_ACT_GELU = 3 } conv_act_t;

typedef struct {
    int32_t B, C, P, G;     /* B >= 0; C, P, G >= 1, C a multiple of G                    */
    int32_t act;            /* conv_act_t                                                 */
    int32_t layout;         /* conv_layout_t                                              */
    int32_t dtype;          /* conv_dtype_t                                               */
    float eps;              /* finite, >= 0                                               */
} conv_gn_desc_t;

/* Forward.  gamma, beta: (C), or NULL (then 1 and 0).  mean, rstd: written, or both NULL (an
 * inference call).  y may be x (in place).
 * Limits: C*P < 2^31 - 2^20, B < 2^31 - 2^25, B*G < 2^31 (CONV_ERR_UNSUPPORTED beyond).  B = 0 does
 * nothing. */
size_t conv_gn_fwd_workspace_size(const conv_gn_desc_t* desc);
int conv_gn_fwd(const conv_gn_desc_t* desc, const void* x, const void* gamma, const void* beta, void* y, float* mean,
                float* rstd, void* workspace, size_t workspace_bytes, conv_stream_t stream);

/* Backward, with the forward's x, gamma, beta, mean and rstd.  dx: written; may be dy (in
 * place).  dgamma, dbeta: written, or both NULL (frozen parameters).  B = 0 writes zeros to
 * dgamma and dbeta. */
size_t conv_gn_bwd_workspace_size(const conv_gn_desc_t* desc);
int conv_gn_bwd(const conv_gn_desc_t* desc, const void* x, const void* dy, const void* gamma, const void* beta,
                const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta, void* workspace,
                size_t workspace_bytes, conv_stream_t stream);

/* ---- embedding lookup with scaling, and its gradient ---------------------------------------
 *   y[t,:] = scale * table[idx[t],:]
 *   dtable[v,:] = scale * (sum of dy[t,:] over the t with idx[t] = v, in fp32)
 * idx: (T), int32 or int64; table, dtable: (V, D); y, dy: (T, D).
 * A token equal to padding_idx, or outside [0, V), names no row: its y is zero and it adds to
 * no gradient (no row is read for it).  padding_idx < 0: no padding row.
 * The gradient adds a row's tokens in an order that the sizes and idx fix (by parts of consecutive
 * tokens, then the parts), and rows that no token names are zeros. */
typedef enum { CONV_INDEX_I32 = 0, CONV_INDEX_I64 = 1 } conv_index_t;

typedef struct {
    int64_t T;              /* tokens, >= 0                                               */
    int32_t V, D;           /* rows of the table, values a row; >= 1                      */
    int32_t padding_idx;    /* row that stands for no token, or negative                  */
    int32_t index_dtype;    /* conv_index_t                                               */
    int32_t dtype;          /* conv_dtype_t of table, y, dy, dtable                       */
    float scale;            /* finite                                                     */
} conv_embed_desc_t;

/* Limits: T < 2^31 - 2^20, D <= 2^24 (CONV_ERR_UNSUPPORTED beyond); T*D and V*D may pass 2^31. */
int conv_embed_fwd(const conv_embed_desc_t* desc, const void* idx, const void* table, void* y, conv_stream_t stream);

size_t conv_embed_bwd_workspace_size(const conv_embed_desc_t* desc);
int conv_embed_bwd(const conv_embed_desc_t* desc, const void* idx, const void* dy, void* dtable, void* workspace,
                   size_t workspace_bytes, conv_stream_t stream);

/* ---- layer norm of a residual sum -----------------------------------------------------------
 * For each of N rows of D values:
 *
 *   total = x + residual (rounded to the dtype; without a residual total is x)
 *   mean = sum total / D      rstd = 1 / sqrt(sum (total - mean)^2 / D + eps)
 *   xhat = (total - mean) * rstd      y = xhat * gamma + beta
 *   dx = rstd * (e - m1 - xhat * m2) + dtotal      e = dy * gamma, m1 = sum e / D, m2 = sum e * xhat / D
 *   dgamma = sum over the rows of dy * xhat        dbeta = sum over the rows of dy
 *
 * dx is the gradient of x and of residual; dtotal is the gradient that reaches total by another way (a
 * residual stream goes on beside its norm), or NULL (0).  rms: the form without a mean: mean, m1
 * and beta are 0, and mean, beta and dbeta NULL.
 * All arrays dense, (N, D) or (D), of the descriptor's dtype; mean and rstd fp32, (N).
 * What is not finite stays in its row, but for the parameters' gradients.  A row of total with a NaN in it, or with
 * a mean an infinity, has NaN for rstd and for all of y and dx, and makes all of dgamma NaN (not dbeta).  Without
 * a mean, a row with an infinity has rstd 0, y NaN there and 0 elsewhere, and dx NaN; dgamma is NaN in that
 * column alone.  A NaN in dy makes its row of dx, and its column of dgamma and dbeta, NaN.
 * Sums and squares are fp32: deviations from 1.8e19 on make rstd 0, a sum of the row's values from 3.4e38 on makes the
 * row NaN, and a row whose values differ by less than some 2^-22 of their mean is normed to the mean's own rounding. */
typedef struct {
    int64_t N;              /* rows, >= 0                                                 */
    int32_t D;              /* values a row, >= 1                                         */
    int32_t rms;            /* 0 or 1                                                     */
    int32_t dtype;          /* conv_dtype_t                                               */
    float eps;              /* finite, >= 0                                               */
} conv_ln_desc_t;

/* gamma, beta: NULL counts as 1 and 0.  total: written, if and only if there is a residual.  mean and
 * rstd: written, or NULL (an inference call; with rms: rstd).  y may be x or residual, total the other;
 * y is not total.
 * Limits: N < 2^31, D < 2^30 (CONV_ERR_UNSUPPORTED beyond).  N = 0 does nothing. */
int conv_ln_fwd(const conv_ln_desc_t* desc, const void* x, const void* residual, const void* gamma, const void* beta,
                void* y, void* total, float* mean, float* rstd, conv_stream_t stream);

/* x: the forward's total.  dx may be dy or dtotal, not x.  dgamma, dbeta: written, or both NULL (rms: dgamma, or
 * NULL).  N = 0 writes zeros to them. */
size_t conv_ln_bwd_workspace_size(const conv_ln_desc_t* desc);
int conv_ln_bwd(const conv_ln_desc_t* desc, const void* x, const void* dy, const void* gamma, const float* mean,
                const float* rstd, const void* dtotal, void* dx, void* dgamma, void* dbeta, void* workspace,
                size_t workspace_bytes, conv_stream_t stream);

/* ---- gated scan over time --------------------------------------------------------------------
 * For each row b of a batch and each channel, over the steps t = 0 .. T-1:
 *
 *   z = 1 / (1 + exp(-gate[b,t]))      h[b,t] = h[b,t-1] + z * (x[b,t] - h[b,t-1])
 *
 * with h[b,-1] = h0[b] (fp32; NULL: 0).  last[b] is the state behind the row's last step, in
 * fp32: one call with T = 1 is one step of a rollout, and `last` may be h0.
 * reset (B, T), bytes: where it is not 0, h[b,t-1] counts as 0: a new sequence begins at t, and
 * nothing of the old one, not even a NaN, goes beyond.
 * lengths (B), int32: row b has its first lengths[b] steps only (0 .. T; less counts as 0, more as
 * T).  Behind them nothing is read and h is 0.
 *
 * Backward, from dh (the gradient that reaches h from outside the scan) and dlast (that reaches
 * last, fp32; NULL: 0):
 *
 *   s[t] = dh[t] + (1 - z[t+1]) * s[t+1]     (no second term across a reset; dlast enters
 *                                             at the row's last step)
 *   dx = s * z     dgate = s * (x - h[t-1]) * z * (1 - z)     dh0 = (1 - z[0]) * s[0]
 *
 * (dh0 = 0 where step 0 is a reset; dh0 = dlast for a row without steps.)  dx and dgate are 0 behind
 * a row's length.  h is the forward's output as it is kept: rounded, where it is bf16.
 *
 * The states, and every product along the time axis, are fp32; 1 - z is taken from z, so what an open gate
 * (above 16 or so) leaves of the state may be 0 instead of less than 2^-23 of it.  Time is cut into parts that
 * are joined in an order that the sizes, and what the addresses and distances are multiples of (2 to 16 bytes), fix:
 * a call gives the same bits each time, another layout of the same values may give others.  A state that
 * is infinite or NaN makes what follows it in its row and channel, up to the next reset, infinite or NaN.
 *
 * x, gate, h, dh, dx and dgate have the descriptor's dtype and lie anywhere: an array's element
 * (b, t, d) is batch * b + step * t + d elements behind its address, which is a multiple of the
 * element's size.  So x and gate may be halves of one array, and time may be the outer dimension.
 * Distances are >= 0; an output's rows do not overlap one another, nor another output's or an input's
 * (CONV_ERR_DESC where the first elements coincide; the rest is the caller's to see to).  h0, last, dlast,
 * dh0: fp32, (B, D) dense. */
typedef struct { int64_t batch, step; } conv_rows_t;

typedef struct {
    int32_t B, T, D;        /* B, T >= 0; D >= 1                                           */
    int32_t dtype;          /* conv_dtype_t                                                */
    conv_rows_t x, gate, h; /* the backward's h too                                        */
    conv_rows_t dh, dx, dgate;  /* backward only                                           */
} conv_scan_desc_t;

/* Limits: B, T, D < 2^31 - 2^20, B * D < 2^37.  B = 0 does nothing.  h0, reset, lengths and last may be NULL. */
size_t conv_scan_fwd_workspace_size(const conv_scan_desc_t* desc);
int conv_scan_fwd(const conv_scan_desc_t* desc, const void* x, const void* gate, const float* h0, const uint8_t* reset,
                  const int32_t* lengths, void* h, float* last, void* workspace, size_t workspace_bytes,
                  conv_stream_t stream);
/* dh0: written, or NULL. */
size_t conv_scan_bwd_workspace_size(const conv_scan_desc_t* desc);
int conv_scan_bwd(const conv_scan_desc_t* desc, const void* x, const void* gate, const void* h, const void* dh,
                  const float* h0, const float* dlast, const uint8_t* reset, const int32_t* lengths, void* dx,
                  void* dgate, float* dh0, void* workspace, size_t workspace_bytes, conv_stream_t stream);

/* ---- loss against a teacher's top logits ----------------------------------------------------
 * Row n has V logits z and a teacher's K entries: ids and the teacher's logits at them.  With the
 * temperature tau, P = softmax(z / tau) over all V and p = softmax(teacher / tau) over the row's
 * entries:
 *
 *   loss[n] = tau^2 * sum_k p_k * (log p_k - log P[id_k])
 *   dz[n,v] = scale * weight[n] * tau * (P[v] - sum of p_k over the k with id_k = v)
 *
 * (the factors tau^2 and tau keep the gradients' size over temperatures).  K = 1 is the cross entropy
 * with the label id_0 at tau = 1.  An entry whose id is outside [0, V), or whose teacher's logit is
 * -infinity, counts for nothing; a row without entries that count has loss 0 and dz 0, and one of weight 0
 * has dz 0, whatever z holds there.  An id may occur more than once in a row.  z may hold -infinity
 * (P is 0 there); a row that holds nothing else, +infinity or NaN gives NaN and leaves the other rows alone,
 * and so does a teacher's logit of +infinity or NaN, in the loss and in dz at the row's ids.
 *
 * z, dz: (N, V), a row's logits one behind the other, rows ld elements apart (ld >= V; dz is
 * written at the row's V elements only), of the descriptor's dtype.  ids, teacher: (N, K) dense,
 * teacher of teacher_dtype.  loss, zmax, zlog, weight: fp32, (N).  zmax[n] is the largest z of the
 * row, zlog[n] = log sum_v exp((z[v] - zmax[n]) / tau): what the backward takes.  Rows begin anywhere, but
 * every array, as everywhere but in the scan, begins at a multiple of 16 bytes (CONV_ERR_ALIGN). */
typedef struct {
    int64_t N;              /* rows, >= 0                                                  */
    int64_t ld;             /* elements from one row of z (and dz) to the next             */
    int32_t V, K;           /* logits and teacher's entries a row, >= 1                    */
    int32_t dtype;          /* conv_dtype_t of z and dz                                    */
    int32_t index_dtype;    /* conv_index_t of ids                                         */
    int32_t teacher_dtype;  /* conv_dtype_t of teacher                                     */
    float temperature;      /* 2^-60 to 2^60                                               */
} conv_distill_desc_t;

/* Limits: N < 2^27, V < 2^30, K <= 1024 (CONV_ERR_UNSUPPORTED beyond); N * ld may pass 2^31.  N = 0 does
 * nothing. */
int conv_distill_fwd(const conv_distill_desc_t* desc, const void* z, const void* ids, const void* teacher, float* loss,
                     float* zmax, float* zlog, conv_stream_t stream);

/* weight: the gradient of each loss, or NULL (1).  scale: finite.  dz may be z (in place). */
int conv_distill_bwd(const conv_distill_desc_t* desc, const void* z, const void* ids, const void* teacher,
                     const float* zmax, const float* zlog, const float* weight, float scale, void* dz,
                     conv_stream_t stream);

/* The losses and the gradient at once, for weights known before the losses: z is read once where a row's
 * part fits the chip (about 800 000 bf16 values).  dz may be z (in place). */
int conv_distill_grad(const conv_distill_desc_t* desc, const void* z, const void* ids, const void* teacher,
                      const float* weight, float scale, float* loss, void* dz, conv_stream_t stream);

/* ---- global gradient norm and clipping ------------------------------------------------------
 *   norm = sqrt(sum over every tensor and element of g^2)
 *   out  = g * min(1, max_norm / (norm + 1e-6))
 * over a list of tensors that live anywhere and may mix dtypes.  The coefficient is formed and
 * applied on the device: nothing waits for the host.  A NaN gradient makes the norm and every
 * output NaN; an infinite one makes the norm infinite and the coefficient 0 (so the infinite
 * values become NaN, the finite ones 0).  Squares are summed in fp32: a gradient above 1.8e19
 * in magnitude makes the norm infinite. */
typedef struct {
    const void* grad;       /* n elements, aligned to the element (any view's start)      */
    void* out;              /* where conv_grad_clip writes; may be grad (in place)        */
    int64_t n;              /* >= 0                                                       */
    int64_t dtype;          /* conv_dtype_t of both                                       */
} conv_grad_t;

/* `grads` is a host array of `count` entries, read before the call returns.  norm: one float,
 * written.  out is used by conv_grad_clip only.  max_norm: finite, >= 0.  Outputs must not
 * overlap other entries.  Limits: n < 2^40 an entry, 2^20 entries. */
size_t conv_grad_norm_workspace_size(const conv_grad_t* grads, int32_t count);
int conv_grad_norm(const conv_grad_t* grads, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                   conv_stream_t stream);
int conv_grad_clip(const conv_grad_t* grads, int32_t count, float max_norm, float* norm, void* workspace,
                   size_t workspace_bytes, conv_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* IGCONV_CONV_TRAIN_H */
