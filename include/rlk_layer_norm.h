/*
 * rlk_layer_norm.h - the layer norm (or RMS norm) in front of the LM head and
 * its backward pass on gfx950 (MI355X): it makes the BF16 hidden states that
 * rlk_linear and rlk_linear_logp read, takes the gradient that
 * rlk_linear_logp_backward gives of them, and leaves the norm weight's gradient
 * in float32, as rlk_l2norm reads it.
 *
 * For each row x of d values, in float32:
 *   m    = mean(x) for RLK_NORM_LAYER, 0 for RLK_NORM_RMS
 *   r    = 1 / sqrt(mean((x - m)^2) + eps)
 *   y    = bf16((x - m) * r * weight + bias)
 * and with g = dy * weight, xhat = (x - m) * r, m and r as the forward left them:
 *   dx      = r * (g - c1 - xhat * mean(g * xhat)), c1 = mean(g) for
 *             RLK_NORM_LAYER, 0 for RLK_NORM_RMS
 *   dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy
 * A row whose dy holds only zeros has dx = 0, whatever x, m, r and weight hold,
 * and a dy of 0 adds nothing to dweight, whatever x, m and r hold there (padding).
 *
 * Order: y, the statistics and dx of a row depend on the row and d alone:
 * identical rows give identical bytes in any batch. dweight and dbias are
 * summed in an order that depends on n_rows, d and whether dx takes the place of
 * x or dy (no atomics).
 *
 * Types: x (and dx) BF16 or float32, weight and bias BF16 or float32 (both the
 * same), y and dy BF16, statistics, dweight and dbias float32.
 *
 * Shapes: d a multiple of 8 in [8, 16384], row strides multiples of 8, >= d and
 * at most 2^21; matrices, weight and bias 16-byte aligned.
 *
 * Memory: every pointer is caller-owned DEVICE memory; nothing is allocated,
 * freed or synchronised, and calls can be captured into a hipGraph. But for what
 * is said of y and dx below, outputs must not overlap each other, the inputs
 * (weight and statistics among them) or the workspace. Argument
 * errors detectable on the host return a negative status (codes of rlk_logp.h)
 * before any HIP call; n_rows is at most 2^22.
 */
#ifndef RLK_LAYER_NORM_H
#define RLK_LAYER_NORM_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "rlk_logp.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { RLK_NORM_LAYER = 0, RLK_NORM_RMS = 1 };
enum { RLK_TYPE_BF16 = 0, RLK_TYPE_F32 = 1 };

/* Forward pass.
 *   x         [n_rows x d] of x_type, row stride x_stride
 *   weight    [d] of weight_type; bias [d] of weight_type, or NULL
 *   eps       finite, >= 0
 *   y         BF16 [n_rows x d], row stride y_stride; it may be x itself (BF16,
 *             the same stride; else RLK_ERR_SHAPE) and must not overlap it otherwise
 *   mean_out  [n_rows] float32, or NULL (RLK_NORM_RMS writes zeros)
 *   rstd_out  [n_rows] float32, or NULL
 * n_rows == 0 enqueues nothing. */
int32_t rlk_layer_norm(const void* x, int32_t x_type, int64_t n_rows, int64_t d, int64_t x_stride,
                       const void* weight, const void* bias, int32_t weight_type, int32_t kind, float eps,
                       uint16_t* y, int64_t y_stride, float* mean_out, float* rstd_out, hipStream_t stream);

/* Backward pass.
 *   dy        BF16 [n_rows x d], row stride dy_stride
 *   x, weight as for the forward call
 *   mean      [n_rows] float32, the forward's (RLK_NORM_RMS: not read, may be NULL)
 *   rstd      [n_rows] float32, the forward's
 *   dx        [n_rows x d] of x_type, row stride dx_stride, or NULL; it may be x
 *             itself (the same stride), or dy itself (BF16, the same stride; else
 *             RLK_ERR_SHAPE), and must not overlap them otherwise
 *   dweight, dbias
 *             [d] float32, 16-byte aligned, or NULL; at least one of the three
 *             outputs must be given (else RLK_ERR_NULL)
 *   accumulate  0: dweight and dbias are written; 1: added to (gradients of
 *             several micro-batches; replaying a captured call adds again)
 *   workspace rlk_layer_norm_backward_workspace_bytes(n_rows, d) bytes, 16-byte
 *             aligned, when dweight or dbias is given (may be NULL otherwise);
 *             calls that overlap need one each
 * n_rows == 0 sets dweight and dbias to zeros (with accumulate: leaves them). */
int32_t rlk_layer_norm_backward(const uint16_t* dy, int64_t dy_stride, const void* x, int32_t x_type,
                                int64_t n_rows, int64_t d, int64_t x_stride, const void* weight,
                                int32_t weight_type, int32_t kind, const float* mean, const float* rstd,
                                void* dx, int64_t dx_stride, float* dweight, float* dbias, int32_t accumulate,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Float32 partial sums of dweight and dbias; 0 for sizes that the call refuses. */
size_t rlk_layer_norm_backward_workspace_bytes(int64_t n_rows, int64_t d);

#ifdef __cplusplus
}
#endif

#endif /* RLK_LAYER_NORM_H */
