/*
 * rlk_linear_grad.h - gradient of the fused "linear-logp" on gfx950 (MI355X):
 * from the per-row statistics that the forward calls left, the gradients of
 * the hidden states and of the vocabulary projection, with the logits formed
 * again in pieces of the vocabulary instead of being kept.
 *
 * Defining passages (RL-Kernel documentation pages): "H100 canonical CP
 * backward validation", Change section (the training step back-propagates
 * through the logprobs); [LINEAR-LOGP], [CFG-KL], [REPRO-CANON] as in
 * rlk_linear.h.
 *
 * What is computed, for row i (a token position) and vocabulary entry j, with
 * x_ij = bf16(sum_k h_ik * w_jk) the BF16 logits of rlk_linear (bit for bit):
 *   G_ij  = d/dx_ij of sum_i (grad_ref[i] * ref_i + grad_policy[i] * policy_i)
 *           as rlk_logp_backward defines it (both terms, the target column,
 *           the row rules), rounded to BF16 as there, whatever the outputs' types
 *   grad_hidden[i][k] = sum_j G_ij * w_jk
 *   grad_weight[j][k] = sum_i G_ij * h_ik
 * with float32 sums on the matrix cores, rounded once where the output is BF16.
 * (The gradient of the rounding of x is taken as 1.)
 *
 * Rows without a gradient - both upstream gradients 0, or T == 0 - get zeros
 * in grad_hidden and add nothing to grad_weight, whatever their hidden states
 * hold; they are left out of the products. An invalid row with a nonzero
 * upstream gradient (rlk_logp_backward's rules) has NaN in its row of
 * grad_hidden and makes all of grad_weight NaN.
 *
 * Order: a row of grad_hidden is the sum of 8 partial sums, one for each
 * canonical vocabulary shard (in increasing j inside the shard), added as
 * ((s0+s1)+(s2+s3))+((s4+s5)+(s6+s7)). It depends on the row and the column
 * geometry alone: identical rows give identical bytes in any batch, and the
 * vocabulary-parallel form below gives the bytes of the whole. grad_weight is
 * summed over the rows that have a gradient, in row order, 32 rows a matrix
 * instruction: rows without one do not change its bytes.
 *
 * Shapes: as rlk_linear.h, and vocab_padded at most 2^22.
 *
 * Memory: every pointer is caller-owned DEVICE memory except `layout` (host);
 * nothing is allocated, freed or synchronised, and calls can be captured into
 * a hipGraph. Outputs must not overlap each other, the inputs or the
 * workspace. Argument errors detectable on the host return a negative status
 * (codes of rlk_logp.h) before any HIP call.
 */
#ifndef RLK_LINEAR_GRAD_H
#define RLK_LINEAR_GRAD_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "rlk_logp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a gradient is stored. */
enum {
  RLK_GRAD_BF16 = 0,   /* BF16 bits, rounded once to nearest even */
  RLK_GRAD_F32 = 1,    /* float32, the sums as they are */
  RLK_GRAD_F32_ADD = 2 /* float32, added to what is there (grad_weight only: gradients of
                          several micro-batches; replaying a captured call adds again) */
};

/* Gradients of the hidden states and of the projection (the formulas above).
 *   hidden, weight, layout
 *                 as for rlk_linear_logp; layout->row_stride is only validated
 *   rank          0 with layout->groups == 1. With groups == G > 1 the call is
 *                 rank `rank`'s part: `weight` holds the projection rows of
 *                 columns [rank*C, (rank+1)*C) below vocab_real, C =
 *                 vocab_padded / G (none when rank*C >= vocab_real; the pointer
 *                 must still be valid and aligned), the row arguments are the
 *                 whole vocabulary's, and grad_weight is the rank's rows
 *   temperature, target, ref_logp, lse, grad_ref, policy_logp, support, grad_policy
 *                 as for rlk_logp_backward (ref_logp and lse from
 *                 rlk_linear_logp or rlk_logp_*; NULL grad_ref: no reference
 *                 term; NULL grad_policy: no policy term; not both)
 *   grad_hidden   [n_rows x d_model], row stride grad_hidden_stride elements
 *                 (>= d_model, a multiple of 8, at most 2^21), 16-byte aligned, of
 *                 type RLK_GRAD_BF16 or RLK_GRAD_F32; NULL: not wanted
 *   grad_weight   [the rank's projection rows x d_model], row stride
 *                 grad_weight_stride (the same bounds), 16-byte aligned, of any
 *                 of the three types; NULL: not wanted. At least one of the
 *                 two must be given (else RLK_ERR_NULL)
 *   workspace     rlk_linear_logp_backward_workspace_bytes(...) bytes, 16-byte
 *                 aligned; calls that overlap need one each
 * n_rows == 0 sets grad_weight to zeros (RLK_GRAD_F32_ADD: leaves it). */
int32_t rlk_linear_logp_backward(const uint16_t* hidden, int64_t n_rows, int64_t d_model, int64_t hidden_stride,
                                 const uint16_t* weight, int64_t weight_stride, const rlk_vocab_layout* layout,
                                 int32_t rank, const float* temperature, const int64_t* target,
                                 const float* ref_logp, const float* lse, const float* grad_ref,
                                 const float* policy_logp, const rlk_support_state* support,
                                 const float* grad_policy, void* grad_hidden, int64_t grad_hidden_stride,
                                 int32_t grad_hidden_type, void* grad_weight, int64_t grad_weight_stride,
                                 int32_t grad_weight_type, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* Bytes of workspace for any types and either output: the rows' hidden states, the
 * BF16 gradients of 1, 2, 4 or 8 canonical shards of logits (the most that take no
 * more than 640 MiB together; one takes what it needs), and float32 partial sums of
 * grad_hidden. Never less for more rows. 0 for arguments that the call refuses. */
size_t rlk_linear_logp_backward_workspace_bytes(int64_t n_rows, int64_t d_model, const rlk_vocab_layout* layout);

/* grad_hidden of the whole vocabulary from the ranks' float32 parts, rank r's
 * [n_rows x d_model] part at parts + r * part_stride elements (rows are
 * contiguous; part_stride >= n_rows * d_model and a multiple of 4): what an
 * all-gather of the RLK_GRAD_F32 outputs yields. The same bytes for every
 * groups in {1, 2, 4, 8}.
 *   grad_hidden   as above */
int32_t rlk_linear_logp_backward_merge(const float* parts, int64_t part_stride, int32_t groups, int64_t n_rows,
                                       int64_t d_model, void* grad_hidden, int64_t grad_hidden_stride,
                                       int32_t grad_hidden_type, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RLK_LINEAR_GRAD_H */
