/*
 * semicrf_encoder.h -- C ABI of the operators around the semi-CRF head:
 * what an encoder needs to make emissions [B][T][C] over the head's lengths
 * (linear attention with a decay for each head, group norm with an
 * activation) and what training needs after the gradients (AdamW).
 *
 * Conventions are those of semicrf.h: device pointers owned by the caller,
 * work enqueued on `stream`, host-detectable errors returned before anything
 * is launched, no allocation, no synchronisation, no state between calls,
 * outputs overwritten and never aliasing inputs (the in-place states of
 * semicrf_linattn_step and semicrf_adamw_step aside).  Status codes are
 * semicrf_status_t.
 *
 * Lengths.  `lengths` [B] int32 may be NULL (every length is T).  Positions
 * t >= lengths[b] are never read into any result (they may hold NaN); their
 * rows of every output and gradient are 0.  A length of 0 is legal here.  A
 * length outside [0, T] makes the sequence's outputs NaN and its gradients
 * 0; it is left out of the parameters' gradients.
 */
#ifndef SEMICRF_ENCODER_H
#define SEMICRF_ENCODER_H

#include "semicrf.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of the encoder's tensors */
enum { SEMICRF_F32 = 0, SEMICRF_BF16 = 1, SEMICRF_F16 = 2 };

/* activations of the group norm (GELU with the error function) */
enum { SEMICRF_ACT_NONE = 0, SEMICRF_ACT_SILU = 1, SEMICRF_ACT_GELU = 2, SEMICRF_ACT_RELU = 3 };

/* ---- Linear attention with a decay for each head -----------------------
 *   S_t = exp(g_h) S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t
 * for each sequence b and head h, S [Dk][Dv] float32, S_{-1} = state_in (or
 * 0).  Written out, o_i = scale (sum_{j <= i} exp(g (i - j)) (q_i . k_j) v_j
 * + exp(g (i + 1)) state_in^T q_i); state_out is S after lengths[b]
 * positions (state_in itself for length 0).  g = log_decay [H] float32, at
 * most 0 in use (larger values grow as the formula says); -inf forgets
 * everything before the position itself.  g is a constant of the model: it
 * gets no gradient.
 *
 * Non-finite inputs are not checked: one at a valid position may reach any
 * row of its sequence and head (positions are worked on in blocks, whose
 * masked products are zeros times what they multiply).
 *
 * Layout.  q, k [B][T][Hq or Hk][Dk], v [B][T][Hv][Dv] of one type (F32,
 * BF16 or F16) with the element strides given for B, T and heads; the last
 * dimension is contiguous.  H is a multiple of Hq, Hk and Hv: head h reads
 * q head h / (H / Hq), and so on (shared heads).  o and grad_o
 * [B][T][H][Dv], grad_q, grad_k, grad_v [B][T][Hx][D] contiguous; the
 * gradient of a shared head is the sum over the heads that read it.  States
 * [B][H][Dk][Dv] float32 contiguous.
 *
 * 1 <= Dk, Dv <= 256 (SEMICRF_ERR_UNSUPPORTED past that); T <= 2^30; B*H <
 * 2^24 where Dk and Dv are at most 64, 2^23 at most 128, 2^22 above
 * (SEMICRF_ERR_SHAPE: a launch has at most 2^32 - 1 threads).  Offsets of
 * elements are 64 bits.
 */
typedef struct {
    int B, T, H;
    int Hq, Hk, Hv;
    int Dk, Dv;
    int dtype;
    float scale;
    int64_t q_stride[3], k_stride[3], v_stride[3]; /* B, T, head; in elements */
} semicrf_linattn_shape_t;

/* Bytes of workspace of semicrf_linattn_fwd (backward = 0) or _bwd (1).  The
 * forward call leaves the states before its segments there (none for short
 * sequences: 0 bytes). */
semicrf_status_t semicrf_linattn_workspace_size(const semicrf_linattn_shape_t *shape, int backward,
                                                size_t *bytes);

/* lengths, state_in and state_out may be NULL. */
semicrf_status_t semicrf_linattn_fwd(const semicrf_linattn_shape_t *shape, const void *q,
                                     const void *k, const void *v, const float *log_decay,
                                     const int32_t *lengths, const float *state_in, void *o,
                                     float *state_out, void *workspace, size_t workspace_bytes,
                                     void *stream);

/* Gradients of L given grad_o = dL/do and grad_state = dL/dstate_out:
 *   G_t = exp(g) G_{t+1} + scale q_t grad_o_t^T,   G after the last position
 *   = grad_state (or 0), dL/dstate_in = exp(g) G_0,
 *   grad_q_t = scale S_t grad_o_t,  grad_k_t = G_t v_t,  grad_v_t = G_t^T k_t.
 * lengths, state_in, grad_state and each output may be NULL (skipped).
 * states: the forward call's workspace as that call left it (same shape, k,
 * v, log_decay, lengths and state_in), or NULL to compute it again. */
semicrf_status_t semicrf_linattn_bwd(const semicrf_linattn_shape_t *shape, const void *q,
                                     const void *k, const void *v, const float *log_decay,
                                     const int32_t *lengths, const float *state_in,
                                     const void *states, const void *grad_o,
                                     const float *grad_state, void *grad_q, void *grad_k,
                                     void *grad_v, float *grad_state_in, void *workspace, size_t workspace_bytes, void *stream);

/* One position of B streams (shape.T = 1; the T strides are not used):
 * stream b's state, state[slots[b]] [H][Dk][Dv] of a pool of `nslots`, is
 * moved by one position in place and o [B][H][Dv] read from it.  slots NULL:
 * stream b uses slot b.  A slot outside [0, nslots) is an idle stream: its
 * row of o is 0 and no state moves.  The slots of one call are distinct. */
semicrf_status_t semicrf_linattn_step(const semicrf_linattn_shape_t *shape, const void *q,
                                      const void *k, const void *v, const float *log_decay,
                                      const int32_t *slots, int nslots, float *state, void *o,
                                      void *stream);

/* ---- Group norm with an activation, channels last ----------------------
 * x [B][T][C] contiguous (F32, BF16 or F16), G groups of C/G neighbouring
 * channels; over the lengths[b] positions and C/G channels of a group
 *   mean, var (biased),  h = (x - mean) / sqrt(var + eps),
 *   y = act(h * weight[c] + bias[c])      (weight, bias [C] float32 or NULL)
 * y [B][T][C] in x's type.  stats [B][G][2] float32 (mean, 1/sqrt(var+eps))
 * is written by the forward pass and read by the backward pass; 0, 0 for an
 * empty sequence.
 *
 * B, T, C <= 2^30, and a launch has at most 2^32 - 1 threads, 256 of them for
 * each sequence and each 256 vectors of its channels (16 bytes, or what the
 * alignment allows), up to 64 for a sequence and group; where a sequence is
 * short (T * C <= 4096), 256 for 4096 elements.  SEMICRF_ERR_SHAPE past that. */
typedef struct {
    int B, T, C, G;
    int dtype;
    int act;
    float eps;
} semicrf_groupnorm_shape_t;

semicrf_status_t semicrf_groupnorm_workspace_size(const semicrf_groupnorm_shape_t *shape,
                                                  int backward, size_t *bytes);

semicrf_status_t semicrf_groupnorm_fwd(const semicrf_groupnorm_shape_t *shape, const void *x,
                                       const float *weight, const float *bias,
                                       const int32_t *lengths, void *y, float *stats,
                                       void *workspace, size_t workspace_bytes, void *stream);

/* grad_x [B][T][C] in x's type, grad_weight, grad_bias [C] float32 (summed
 * over the batch in a fixed order); the last two may be NULL. */
semicrf_status_t semicrf_groupnorm_bwd(const semicrf_groupnorm_shape_t *shape, const void *x,
                                       const float *weight, const float *bias,
                                       const int32_t *lengths, const void *grad_y,
                                       const float *stats, void *grad_x, float *grad_weight,
                                       float *grad_bias, void *workspace, size_t workspace_bytes,
                                       void *stream);

/* ---- AdamW over many tensors -------------------------------------------
 * For every element, with g the gradient (times *grad_scale if given), every
 * operation rounded to float32 by itself in this order:
 *   m <- beta1 m + (1 - beta1) g
 *   v <- beta2 v + ((1 - beta2) g) g
 *   p <- p (1 - lr wd) - (lr / (1 - beta1^step)) (m / (sqrt(v) c + eps)),
 *        c = 1 / sqrt(1 - beta2^step)
 * and p rounded to its type.  With a float32 master copy, p is read from and
 * written to the master and the tensor gets its rounding.
 *
 * States in 8 bits: the elements of a tensor in blocks of 256, each with a
 * float32 scale.  m: float8 e4m3 (OCP, 448 the largest), code = m * ((1 /
 * max|m|) * 448), scale = max|m| * (1/448).  v is held by its root r =
 * sqrt(v): unsigned, 4 bits of exponent (bias 7) and 4 of mantissa,
 * subnormals below 2^-6, 496 the largest; code = r * ((1 / max r) * 496),
 * scale = max r * (1/496), v = (code * scale)^2.  Codes round to the
 * nearest, ties to even; a block with no magnitude over 2^-100 holds codes of
 * 0.  The update uses m and v before they are rounded to codes.
 * Non-finite gradients are not checked: they reach their element (32 bits)
 * or their block of 256 (8 bits).
 *
 * The table says where each tensor and its states lie.  The caller fills the
 * entries' fields but `first`; semicrf_adamw_table completes them in a host
 * buffer of semicrf_adamw_table_size bytes, which the caller copies to
 * device memory once and keeps, both copies, as long as the pointers hold. */
enum { SEMICRF_ADAMW_BLOCK = 4096 }; /* elements one workgroup steps */
typedef struct {
    void *p;        /* parameter, `dtype` */
    float *master;  /* float32 copy or NULL */
    void *m;        /* float32 [n], or e4m3 codes [n] */
    void *v;        /* float32 [n], or root codes [n] */
    float *m_scale; /* 8 bits: [ceil(n / 256)]; else NULL */
    float *v_scale;
    int64_t n;      /* elements; 0 is legal */
    int64_t first;  /* set by semicrf_adamw_table: workgroup of the first element */
    int32_t dtype;
    int32_t reserved;
} semicrf_adamw_tensor_t;

/* Bytes of the table of `count` tensors: the entries, then the tensor of each
 * workgroup.  SEMICRF_ERR_SHAPE for a negative n or more than 2^31 - 1
 * workgroups, SEMICRF_ERR_NULL for a missing pointer. */
semicrf_status_t semicrf_adamw_table_size(const semicrf_adamw_tensor_t *tensors, int count,
                                          int bits, size_t *bytes);
semicrf_status_t semicrf_adamw_table(const semicrf_adamw_tensor_t *tensors, int count, int bits,
                                     void *host_table, size_t bytes);

/* grads, grad_dtypes: HOST arrays of `count` device pointers and their types,
 * in the table's order; a NULL gradient leaves its tensor and states as they
 * are.  bits: 32 or 8, as the
 * table was made.  grad_scale: device float or NULL.  step >= 1, counted
 * from 1. */
semicrf_status_t semicrf_adamw_step(const void *host_table, const void *device_table,
                                    const void *const *grads, const uint8_t *grad_dtypes, int count,
                                    int bits, int64_t step,
                                    double lr, double beta1, double beta2, double eps,
                                    double weight_decay, const float *grad_scale, void *stream);

/* The values that 8-bit codes stand for: root = 0 for m, 1 for v. */
semicrf_status_t semicrf_adamw_values(const void *codes, const float *scale, int64_t n, int root,
                                      float *values, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SEMICRF_ENCODER_H */
