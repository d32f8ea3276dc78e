/*
 * moe_train.h -- C ABI of the operators that train the block's experts, projections and norm, and
 * of their serving forms. The router (scores, top-k and its normalisation, the blend's coefficients)
 * has no backward pass here beyond dtopk_w, and there is none of the whole block: the caller
 * chains these calls.
 *
 * Same library (libmoe_b200.so), status codes and conventions as moe.h: device pointers,
 * caller-owned buffers, no allocation, every call asynchronous on `stream`, every host check
 * before the first launch, T == 0 returns MOE_OK and launches nothing that reads a row (the
 * backward calls then only clear the weight gradients). Three operators, each forward and
 * backward:
 *
 *   linear   z = x W^T + b,  y = act(z) + r
 *   ffn      g = u Wg^T + bg, v = u Wu^T + bu, h = act(g, v), o = h Wd^T + bd, dense
 *            (y = o + r) or over routed slots (y[t] = sum_j w[t, j] o[slot] + r[t])
 *   norm     layer norm y = (x - mean) rstd w + b,  RMS norm y = x rstd w
 *
 * Types: MOE_DTYPE_BF16 or MOE_DTYPE_F32 for every tensor of a call unless it is named f32
 * below. Sums, statistics and routing weights are f32; a bf16 result is rounded once, and so
 * are the intermediates that the comments of each call name.
 *
 * Rows may be strided (ld*, in elements, at least the row length and a multiple of 16
 * bytes); everything else is contiguous. Pointers are 16-byte aligned, row lengths multiples
 * of 16 bytes. Row indices and offsets are 64-bit throughout.
 *
 * Outputs overlap no input of the call and no other output, except that y may be the residual's
 * tensor (linear, ffn), u (ffn) or x (norm) with its stride. Rows against rows are checked
 * (MOE_ERR_INVALID_ARGUMENT); side by side in wider rows is fine. Widths above 2^28, more than
 * 2^30 rows or slots, tensors above 2^46 elements, and matrix products of 2^29 or more tiles of
 * 64 x 64 results (bf16: 128 x 256) are refused (MOE_ERR_SHAPE_OVERFLOW), by the size calls too.
 *
 * Workspace: ws of at least the matching *_workspace_size bytes for that T, any contents. Calls that may
 * overlap on the GPU (two streams, two graphs) each need their own. NULL is accepted where the
 * size is 0.
 *
 * device_status (optional, caller-owned int32 on the device, zeroed by the caller) receives
 * MOE_ERR_DEVICE_CHECK (a slot id or an offset out of range: such rows are dropped; or a slot
 * that stands twice, seen where y or du is computed: the results are not valid) or
 * MOE_ERR_DEVICE_TIMEOUT (a bounded wait gave up; the results are not valid). The first
 * error stays. The norm calls take none: they check nothing on the device and hold no wait that
 * can give up.
 *
 * Results do not depend on the run: no sum uses atomics.
 */
#ifndef MOE_TRAIN_B200_H
#define MOE_TRAIN_B200_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ linear */
enum moe_linear_activation {
    MOE_LINEAR_NONE = 0,
    MOE_LINEAR_SILU = 1, /* z sigmoid(z)          */
    MOE_LINEAR_GELU = 2  /* z Phi(z), erf form    */
};

typedef struct moe_linear_desc {
    int32_t in_features;  /* K */
    int32_t out_features; /* N */
    int32_t activation;   /* enum moe_linear_activation */
    int32_t dtype;        /* MOE_DTYPE_F32 or MOE_DTYPE_BF16 */
} moe_linear_desc;

MOE_API moe_status moe_linear_workspace_size(const moe_linear_desc *d, int64_t T, int32_t backward, size_t *bytes);

/* y [T, N] = act(x W^T + bias) + residual. x [T, K] with row stride ldx, w [N, K], bias [N]
 * or NULL, residual [T, N] with row stride ldr or NULL, y with row stride ldy. pre (optional,
 * [T, N] contiguous) receives z, which the backward pass of an activation needs. */
MOE_API moe_status moe_linear_forward(const moe_linear_desc *d, const void *x, int64_t ldx, const void *w,
                                      const void *bias, const void *residual, int64_t ldr, int64_t T, void *y,
                                      int64_t ldy, void *pre, void *ws, size_t ws_bytes, int32_t *device_status,
                                      moe_stream_t stream);

/* From dy [T, N] (row stride lddy): dz = dy * act'(pre), dx [T, K] = dz W, dw [N, K] = dz^T x,
 * db [N] = column sums of dz. Each of dx, dw, db may be NULL (not computed). pre [T, N] as the
 * forward pass wrote it; NULL without an activation. The residual's gradient is dy itself.
 * bf16 with an activation: dz is rounded to bf16 before the two products (the operand type of
 * the matrix instructions); db sums it unrounded. T == 0 clears dw and db. */
MOE_API moe_status moe_linear_backward(const moe_linear_desc *d, const void *dy, int64_t lddy, const void *x,
                                       int64_t ldx, const void *w, const void *pre, int64_t T, void *dx,
                                       int64_t lddx, void *dw, void *db, void *ws, size_t ws_bytes,
                                       int32_t *device_status, moe_stream_t stream);

/* --------------------------------------------------------- gated feed-forward
 * The routed experts of a moe_config (K = latent_dim or hidden, intermediate, num_experts,
 * top_k, activation, biases, interleaved planes; weight_format F32 or BF16), with the weight
 * planes of moe_weights (gate_w, up_w or gate_up_w, down_w and, with has_expert_bias, their
 * biases; the other fields are not read).
 *
 * expert_offsets [E + 1], sorted_slot [T*k], topk_w [T, k] f32 are moe_permute's and
 * moe_route's outputs. All three NULL with num_experts == 1 and top_k == 1: a dense gated
 * FFN over the T rows in order, weight 1 (a shared expert, a dense layer).
 *
 * pre [T*k, 2I]: the pre-activations in sorted order, columns in the order of the gate/up
 * plane's rows: gate then up, or alternating with gate_up_interleaved. */
typedef struct moe_ffn_grads {
    void *gate_w, *up_w, *gate_up_w, *gate_b, *up_b, *gate_up_b, *down_w, *down_b;
} moe_ffn_grads;

MOE_API moe_status moe_ffn_workspace_size(const moe_config *cfg, int64_t T, int32_t backward, size_t *bytes);

/* The same for calls without a routing (num_experts == 1, top_k == 1), which hold no second copy of
 * the rows: 101 MB in place of 580 MB for the backward pass of 8192 tokens, 7168 x 2048, bf16. */
MOE_API moe_status moe_ffn_dense_workspace_size(const moe_config *cfg, int64_t T, int32_t backward, size_t *bytes);

/* y [T, K] (row stride ldy) from u [T, K] (row stride ldu), plus residual [T, K] (row stride
 * ldr) or NULL. pre (optional) is kept for the backward pass; its rows behind the last sorted
 * position (slots that moe_permute dropped) are not written. bf16: h is rounded to bf16 before the down product (the operand type of the
 * matrix instructions); the slots' weighted output rows are summed in f32. */
MOE_API moe_status moe_ffn_forward(const moe_config *cfg, const moe_weights *w, const void *u, int64_t ldu,
                                   int64_t T, const int32_t *expert_offsets, const int32_t *sorted_slot,
                                   const float *topk_w, const void *residual, int64_t ldr, void *y, int64_t ldy,
                                   void *pre, void *ws, size_t ws_bytes, int32_t *device_status,
                                   moe_stream_t stream);

/* From dy [T, K] (row stride lddy), u and pre: du [T, K] (row stride lddu), dtopk_w [T, k] f32
 * (routed; may be NULL) and the gradients of the planes, [E, rows, cols] like the planes
 * (experts without rows get zeros). Required gradients: those of the planes that the config
 * has; du may be NULL. The activations are recomputed from pre. bf16: dg, dv and w h are
 * rounded to bf16 before their products, and the gate and up bias gradients are f32 sums of dg and
 * dv so rounded (down_b's of w dy unrounded); the slots' rows of du are summed in f32; dtopk_w keeps the
 * matrix instructions' truncated additions (low by about 1.5e-8 of its value per 16 of K: 2.6e-6 at
 * K = 2880, 7e-6 at 7168). T == 0 clears the gradients. */
MOE_API moe_status moe_ffn_backward(const moe_config *cfg, const moe_weights *w, const void *u, int64_t ldu,
                                    int64_t T, const int32_t *expert_offsets, const int32_t *sorted_slot,
                                    const float *topk_w, const void *pre, const void *dy, int64_t lddy, void *du,
                                    int64_t lddu, float *dtopk_w, const moe_ffn_grads *grads, void *ws,
                                    size_t ws_bytes, int32_t *device_status, moe_stream_t stream);

/* --------------------------------------------------------------------- norm */
enum moe_norm_kind { MOE_NORM_LAYER = 0, MOE_NORM_RMS = 1 };

typedef struct moe_norm_desc {
    int32_t width; /* H */
    int32_t kind;  /* enum moe_norm_kind */
    int32_t dtype; /* MOE_DTYPE_F32 or MOE_DTYPE_BF16 */
    float eps;     /* finite, > 0 */
} moe_norm_desc;

MOE_API moe_status moe_norm_workspace_size(const moe_norm_desc *d, int64_t T, int32_t backward, size_t *bytes);

/* y [T, H] (row stride ldy) from x [T, H] (row stride ldx), w [H], b [H] or NULL (layer norm
 * only). stats [T, 2] f32 (optional): mean (0 for RMS) and 1 / sqrt(var + eps). */
MOE_API moe_status moe_norm_forward(const moe_norm_desc *d, const void *x, int64_t ldx, const void *w,
                                    const void *b, int64_t T, void *y, int64_t ldy, float *stats,
                                    moe_stream_t stream);

/* dx [T, H] (row stride lddx; may be NULL), dw [H], db [H] (each may be NULL) from dy [T, H]
 * (row stride lddy), x, w and stats as the forward pass wrote them. T == 0 clears dw, db. */
MOE_API moe_status moe_norm_backward(const moe_norm_desc *d, const void *dy, int64_t lddy, const void *x,
                                     int64_t ldx, const void *w, const float *stats, int64_t T, void *dx,
                                     int64_t lddx, void *dw, void *db, void *ws, size_t ws_bytes,
                                     moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_TRAIN_B200_H */
