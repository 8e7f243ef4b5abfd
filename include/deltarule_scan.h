/*
 * deltarule_scan.h — C ABI of the selective scan, the short causal convolution and the norm of a layer (MI355X, gfx950).
 *
 * What a layer runs around a recurrence of this library, and the recurrence whose decay is an own one for every
 * channel and state:
 *
 *   norm         h = x + r,  y = h w / sqrt(mean(h^2) + eps)
 *   convolution  y_t[c] = act(bias[c] + sum_{j < width} w[c, j] e_{t + j}[c]),  e = the width - 1 inputs before x, then x
 *   scan         h_t[c, n] = exp(d_t[c] A[c, n]) h_{t-1}[c, n] + d_t[c] x_t[c] B_t[g, n],
 *                y_t[c] = (sum_n C_t[g, n] h_t[c, n] + D[c] x_t[c]) silu(z_t[c]),
 *                d_t[c] = softplus(dt_t[c] + dt_bias[c]),  g the group of channel c
 *
 * Memory, streams, errors, workspaces, cu_seqlens and stored states are those of deltarule.h and deltarule_decay.h:
 * device pointers on the current device, work enqueued on `stream`, argument errors found on the host before anything
 * is launched, no pointer kept. Activations (x, dt, B, C, z, residuals, the convolution's states, outputs and the gradients of
 * all of these) have the call's in_dtype, rounded once from float32; parameters (weights, biases, A, D) and their
 * gradients, the scan's states and scales are float32. Everything in between is float32; results agree with a float64
 * evaluation to about 1e-6 of the output's size (2-norm) before that rounding.
 * Pointers need the alignment of their elements; parameters, scan states, cu_seqlens, state_idx, workspaces, B and C
 * 16 bytes. A tensor with strides may be a view whose channels are dense: "token" and "batch" strides are counted in elements,
 * not negative, at most 2^24 (token) and 2^40 (batch, rows), and for B and C multiples of 16 bytes. All other tensors are
 * dense.
 * The offsets of packed sequences are not read on the host; rows that no sequence holds are neither read nor written.
 * At most 2^31 - 1024 tokens and sequences per call, at most 2^20 channels (norm: 32768); a call whose launches would pass
 * 2^32 - 1 work items is refused (DR_ERR_UNSUPPORTED).
 * A NaN or an infinity stays in its channel and sequence (gradients: also in what is summed over them), except that the gradients of B and C sum over
 * channels and a norm's row is one. Outputs of the tokens before it are not touched. In the scan's forward pass a d x that is not finite
 * makes its channel's states NaN from its token on.
 */
#ifndef DELTARULE_SCAN_H
#define DELTARULE_SCAN_H

#include "deltarule.h"
#include "deltarule_decay.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------------ convolution */
typedef enum dr_conv_act { DR_CONV_NONE = 0, DR_CONV_SILU = 1 } dr_conv_act;

/* batch, seqlen, num_seqs, in_dtype as in dr_dims; width 2, 3 or 4. */
typedef struct dr_conv_dims {
  int64_t batch;
  int64_t seqlen;
  int64_t channels;
  int64_t width;
  int64_t num_seqs;
  int64_t x_token_stride, x_batch_stride; /* of x (a step: the batch stride, between sequences) */
  int32_t in_dtype;
  int32_t activation; /* dr_conv_act */
} dr_conv_dims;

/*
 * x [B, T, C], weight [C, width], bias [C] or NULL, y [B, T, C].
 * state    [N, width - 1, C] in_dtype: the inputs in front of each sequence, oldest first; NULL: zeros
 * state_T  the last width - 1 inputs of each sequence (older ones from its state where it is shorter), or NULL; may be `state`
 * opts     NULL, or state_idx / num_slots: the states are pools of num_slots rows (see dr_opts); the rest must be zero
 */
int dr_conv_fwd(const void* x, const float* weight, const float* bias, const void* state, const int32_t* cu_seqlens,
                void* y, void* state_T, const dr_conv_dims* dims, const dr_opts* opts, hipStream_t stream);

/* One token for each of N sequences: x, y [N, C], the states [N, width - 1, C] (or the pool) updated in place.
 * A slot outside the pool gives y = 0 and touches no state. dims: batch = num_seqs = N, seqlen = 1. */
int dr_conv_step(const void* x, const float* weight, const float* bias, void* state, void* y, const dr_conv_dims* dims,
                 const dr_opts* opts, hipStream_t stream);

/* Bytes of workspace of a call of dr_conv_bwd with these dims (packed: whether it has cu_seqlens). */
int dr_conv_workspace(const dr_conv_dims* dims, int packed, int64_t* bytes);

/*
 * Gradients for dy [B, T, C] and dstate_T [N, width - 1, C] (NULL: zero): dx [B, T, C] in_dtype, dweight
 * [C, width], dbias [C] (or NULL), dstate [N, width - 1, C] in_dtype (or NULL). No atomics: the same call gives the same bits.
 */
int dr_conv_bwd(const void* x, const float* weight, const float* bias, const void* state, const int32_t* cu_seqlens,
                const void* dy, const void* dstate_T, void* dx, float* dweight, float* dbias, void* dstate,
                const dr_conv_dims* dims, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------------------------------ selective scan */
/* batch, seqlen, num_seqs, in_dtype as in dr_dims; channels a multiple of groups (at most 65536); channel c reads the B and C of group
 * c / (channels / groups); state_dim 16, 32 or 64. softplus 0: d = dt + dt_bias, 1: softplus of it. */
typedef struct dr_scan_dims {
  int64_t batch;
  int64_t seqlen;
  int64_t channels;
  int64_t groups;
  int64_t state_dim;
  int64_t num_seqs;
  int64_t x_token_stride, x_batch_stride;
  int64_t dt_token_stride, dt_batch_stride;
  int64_t b_token_stride, b_batch_stride;
  int64_t c_token_stride, c_batch_stride;
  int64_t z_token_stride, z_batch_stride;
  int32_t in_dtype;
  int32_t softplus;
} dr_scan_dims;

/* Bytes of workspace of a call of dr_scan_fwd (backward == 0) or dr_scan_bwd (backward != 0); may be 0. */
int dr_scan_workspace(const dr_scan_dims* dims, int packed, int backward, int64_t* bytes);

/*
 * x, dt, z [B, T, C] (z NULL: no gate), B, C [B, T, G, state_dim], y [B, T, C]; A [C, state_dim], D [C] or NULL, dt_bias [C] or NULL.
 * S0, S_T  states [N, C, state_dim] float32 or NULL, may be the same; opts as for dr_conv_fwd.
 * The accuracy statement covers d A <= 0.
 */
int dr_scan_fwd(const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
                const void* z, const float* dt_bias, const float* S0, const int32_t* cu_seqlens, void* y, float* S_T,
                const dr_scan_dims* dims, const dr_opts* opts, void* workspace, int64_t workspace_bytes,
                hipStream_t stream);

/* One token for each of N sequences: x, dt, z, y [N, C], B, C [N, G, state_dim], S [N, C, state_dim] (or the pool) in place. A slot
 * outside the pool gives y = 0 and touches no state. dims: batch = num_seqs = N, seqlen = 1. */
int dr_scan_step(const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
                 const void* z, const float* dt_bias, float* S, void* y, const dr_scan_dims* dims, const dr_opts* opts,
                 hipStream_t stream);

/*
 * Gradients for dy [B, T, C] in_dtype and dS_T [N, C, state_dim] float32 (NULL: zero): dx, ddt, dz [B, T, C] (dz with z),
 * dB, dC [B, T, G, state_dim] in_dtype; dA [C, state_dim], dD [C] (with D), ddt_bias [C] (with dt_bias), dS0 [N, C, state_dim] or
 * NULL. The states and their gradients are formed by the call itself. No atomics: the same call gives the same bits.
 */
int dr_scan_bwd(const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
                const void* z, const float* dt_bias, const float* S0, const int32_t* cu_seqlens, const void* dy,
                const float* dS_T, void* dx, void* ddt, float* dA, void* dB, void* dC, float* dD, void* dz,
                float* ddt_bias, float* dS0, const dr_scan_dims* dims, void* workspace, int64_t workspace_bytes,
                hipStream_t stream);

/* ------------------------------------------------------------------------------------------------ norm */
/* What y holds: values of in_dtype, or codes of the state cache's formats. */
typedef enum dr_norm_out { DR_NORM_VALUES = 0, DR_NORM_INT8 = 1, DR_NORM_E4M3 = 2 } dr_norm_out;

typedef struct dr_norm_dims {
  int64_t rows;
  int64_t channels;
  int64_t x_row_stride, residual_row_stride; /* elements */
  int32_t in_dtype;
  int32_t out; /* dr_norm_out */
  float eps;   /* finite, not negative */
  int32_t reserved; /* 0 */
} dr_norm_dims;

/*
 * x, residual [rows, C] (residual NULL: h is x), weight [C], y [rows, C].
 * h        [rows, C]: the sum as it was normalised, rounded to in_dtype; NULL if it is not wanted, and without residual. May be
 *          x or residual where that is dense.
 * 8 bits   p = h w (float32) is held as a row of the state cache is (dr_cache_format: int8, or e4m3 with a power of two), and
 *          scales[row] is that scale times 1 / sqrt(mean(h^2) + eps): y is code * scale, and the codes do not depend on the
 *          mean. A row whose p has a NaN or an infinity gets a NaN scale and zero codes. scales NULL for values.
 * The sum of squares is a float32 sum: rows whose squares overflow give zeros.
 */
int dr_norm_fwd(const void* x, const void* residual, const float* weight, void* y, float* scales, void* h,
                const dr_norm_dims* dims, hipStream_t stream);

/* Bytes of workspace of a call of dr_norm_bwd with these dims. */
int dr_norm_workspace(const dr_norm_dims* dims, int64_t* bytes);

/*
 * Gradients of the values: h [rows, C] (x_row_stride), weight, dy [rows, C], dh [rows, C] (what reaches h itself; or NULL):
 * dx [rows, C] in_dtype, the gradient of x and of residual alike; dweight [C]. dx may be dh. dims->out 0, residual_row_stride unused.
 * No atomics: the same call gives the same bits.
 */
int dr_norm_bwd(const void* h, const float* weight, const void* dy, const void* dh, void* dx, float* dweight,
                const dr_norm_dims* dims, void* workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DELTARULE_SCAN_H */
