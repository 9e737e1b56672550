/*
 * conv_train.h -- C ABI of the operators a training step runs around the conv layers of
 * conv.h: group normalisation with an activation, the embedding lookup with its gradient, and
 * the global gradient norm with clipping.
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
