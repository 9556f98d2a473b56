/*
 * semicrf_layer.h -- C ABI of the operators of an encoder's layer whose memory
 * is driven by the data: the gated delta rule, rotary positions, and the
 * global norm of many gradients with clipping.
 *
 * Conventions, element types, lengths and layouts are those of
 * semicrf_encoder.h.
 */
#ifndef SEMICRF_LAYER_H
#define SEMICRF_LAYER_H

#include "semicrf_encoder.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Gated delta rule ---------------------------------------------------
 *   S_t = e^{g_t} (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T
 *   o_t = scale * S_t^T q_t
 * for each sequence and head, S [Dk][Dv] float32, S_{-1} = state_in (or 0):
 * linear attention whose decay comes with the position and whose write first
 * takes out what the decayed state says of its key.  state_out is S after
 * lengths[b] positions.  log_decay g, beta b [B][T][H] float32 contiguous; g
 * at most 0 in use (-inf forgets everything before the position; larger
 * values grow as the formula says), b in [0, 1], up to 2, for keys of length
 * at most 1: the rule is then a contraction.  Longer keys with b |k|^2 > 2
 * make S grow as the formula says.  |b| below 2^-64 counts as 2^-64.
 *
 * The shape, the layout of q, k, v, o and their gradients, shared heads and
 * states are linear attention's.  1 <= Dk, Dv <= 128 (SEMICRF_ERR_UNSUPPORTED
 * past that); T <= 2^30; B * H * ceil(T / 32) < 2^23 (SEMICRF_ERR_SHAPE: a
 * launch has at most 2^32 - 1 threads).
 *
 * Non-finite inputs are not checked: one at a valid position may reach any
 * row of its sequence and head.
 */

/* Bytes of workspace of semicrf_delta_fwd (FORWARD; KEEP with its keep), or of
 * semicrf_delta_bwd (BACKWARD). */
enum { SEMICRF_DELTA_FORWARD = 0, SEMICRF_DELTA_KEEP = 1, SEMICRF_DELTA_BACKWARD = 2 };
semicrf_status_t semicrf_delta_workspace_size(const semicrf_linattn_shape_t *shape, int pass,
                                              size_t *bytes);

/* keep != 0: what the backward pass reads again is left in the workspace.
 * lengths, state_in and state_out may be NULL. */
semicrf_status_t semicrf_delta_fwd(const semicrf_linattn_shape_t *shape, int keep, const void *q,
                                   const void *k, const void *v, const float *log_decay,
                                   const float *beta, const int32_t *lengths,
                                   const float *state_in, void *o, float *state_out,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* Gradients given grad_o and grad_state = dL/dstate_out (or NULL: 0).
 * `saved` is the workspace of a forward call with keep as that call left it
 * (same shape, k, v, log_decay, beta, lengths and state_in).  grad_log_decay and
 * grad_beta [B][T][H] float32; a log_decay's gradient is as small as e^g and keeps its
 * digits down to float32's range, below -104 (e^g is 0 in float32) it is 0.  lengths,
 * grad_state and each output may be NULL (skipped). */
semicrf_status_t semicrf_delta_bwd(const semicrf_linattn_shape_t *shape, const void *q,
                                   const void *k, const void *v, const float *log_decay,
                                   const float *beta, const int32_t *lengths, const void *saved,
                                   const void *grad_o, const float *grad_state, void *grad_q,
                                   void *grad_k, void *grad_v, float *grad_log_decay,
                                   float *grad_beta, float *grad_state_in, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* One position of B streams (shape.T = 1; the T strides are not used):
 * log_decay, beta [B][H]; slots, the pool and idle streams are those of
 * semicrf_linattn_step. */
semicrf_status_t semicrf_delta_step(const semicrf_linattn_shape_t *shape, const void *q,
                                    const void *k, const void *v, const float *log_decay,
                                    const float *beta, const int32_t *slots, int nslots,
                                    float *state, void *o, void *stream);

/* ---- Rotary positions ---------------------------------------------------
 * Each row of x [B][T][heads][D] at position p is turned in `turn` / 2 planes,
 * plane i by the angle p * frequency[i]:
 *   (a, b) <- scale * (a cos - b sin, a sin + b cos)
 * SEMICRF_ROTARY_HALF: (a, b) are elements i and i + turn / 2 of a row;
 * SEMICRF_ROTARY_INTERLEAVED: elements 2 i and 2 i + 1.  Elements from `turn`
 * on are copied.  frequency [turn / 2] float64, radians a position; angles are
 * formed and reduced in float64.  position: NULL (row t is at t), [B] int32
 * (row t of sequence b at position[b] + t) or [B][T] int32 (each row's).
 * inverse: turned the other way (with scale, the gradient).
 *
 * x [B][T][heads][D] with strides given in elements, the last dimension
 * contiguous; y the same shape, contiguous.  Two tensors of one call (queries
 * and keys) share the angles; the second may be absent (x2 NULL, heads2 0).
 * 2 <= turn <= D, even; D <= 8192 (SEMICRF_ERR_UNSUPPORTED past that); B, T <=
 * 2^30, (heads + heads2) * D < 2^28.  Rows are turned as they are, whatever a
 * sequence's length. */
enum { SEMICRF_ROTARY_HALF = 0, SEMICRF_ROTARY_INTERLEAVED = 1 };
enum { SEMICRF_POSITION_ROW = 0, SEMICRF_POSITION_SEQUENCE = 1, SEMICRF_POSITION_EACH = 2 };
typedef struct {
    int B, T;
    int heads, heads2;
    int D, turn;
    int dtype;
    int layout;
    int positions; /* SEMICRF_POSITION_... */
    int inverse;
    float scale;
    int64_t stride[3], stride2[3]; /* B, T, head; in elements */
} semicrf_rotary_shape_t;

semicrf_status_t semicrf_rotary(const semicrf_rotary_shape_t *shape, const void *x, const void *x2,
                                const double *frequency, const int32_t *position, void *y,
                                void *y2, void *stream);

/* ---- Norm of many gradients, clipping ------------------------------------
 * norm = the norm of all elements of `count` tensors together: the largest
 * magnitude (SEMICRF_NORM_MAX), the sum of magnitudes (SEMICRF_NORM_1) or the
 * root of the sum of squares (SEMICRF_NORM_2), summed in float64 in a fixed
 * order and rounded once; coefficient = min(1, max_norm / (norm + 1e-6)).  A
 * NaN anywhere makes both NaN.  No tensors, or empty ones: norm 0.
 *
 * grads, sizes, dtypes: HOST arrays of `count` device pointers, numbers of
 * elements and types.  norm, coefficient: device floats, each may be NULL.
 * clip != 0: every element is then multiplied by the coefficient in float32
 * and rounded to its type, in place (tensors are left as they are where the
 * coefficient is 1).  Tensors that share memory are then refused
 * (SEMICRF_ERR_ARG): their addresses are sorted in host memory allocated for the
 * call (SEMICRF_ERR_WORKSPACE where there is none). */
enum { SEMICRF_NORM_MAX = 0, SEMICRF_NORM_1 = 1, SEMICRF_NORM_2 = 2 };

semicrf_status_t semicrf_grad_norm_workspace_size(const int64_t *sizes, int count, size_t *bytes);
semicrf_status_t semicrf_grad_norm(void *const *grads, const int64_t *sizes,
                                   const uint8_t *dtypes, int count, int order, double max_norm,
                                   int clip, float *norm, float *coefficient, void *workspace,
                                   size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SEMICRF_LAYER_H */
