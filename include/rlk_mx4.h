/*
 * rlk_mx4.h - microscaled 4-bit floating point on gfx950 (MI355X): quantisation
 * of BF16 matrices into blocks of 32 values that share a power of two, and the
 * LM-head linear layer with both operands in that form, on the matrix cores'
 * block-scaled instructions. For rollout and for drafting tokens: the BF16
 * logits are those that rlk_logp_nucleus reads, and rlk_draft.h verifies what
 * was drafted from them against the BF16 head.
 *
 * Format (OCP Microscaling Formats specification v1.0, MXFP4: E2M1 elements,
 * E8M0 scales): a block is 32 consecutive values of a row,
 *   a    = max |x| over the block
 *   e    = floor(log2(a)) - 2, clamped to [-127, 127]; -127 when a = 0
 *   q_k  = the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} to x_k / 2^e, ties to
 *          the even code, magnitudes above 6 to 6; the sign of x_k is kept
 *   scale byte e + 127, code = sign * 8 + index of the magnitude
 * and the block stands for the values q_k * 2^e, each exact in BF16. A block
 * that holds NaN or an infinity has scale byte 255 and codes 0: all of its
 * values stand for NaN.
 *
 * Layout: what one matrix instruction takes from a lane lies together. The
 * matrix is cut into tiles of 32 rows; missing rows (n_rows to the next
 * multiple of 32) and missing values (d to the next multiple of 256) are
 * zeros. With R = ceil(n_rows / 32), S = 4 * ceil(d / 256):
 *   codes  [R][S][2][32][16] bytes: block b = 2s + h of row 32R' + r is the 16
 *          bytes at ((R' * S + s) * 2 + h) * 512 + r * 16; byte j holds value
 *          2j in its low four bits and value 2j + 1 in its high four bits
 *   scales [R][S/4][2][32][4] bytes: the scale byte of that block is at
 *          ((R' * S/4 + s/4) * 2 + h) * 128 + r * 4 + s % 4
 * So a tile of 32 rows can be taken out by address alone.
 *
 * Memory: every pointer is caller-owned DEVICE memory except `layout` (host);
 * nothing is allocated, freed or synchronised, and calls can be captured into
 * a hipGraph. Argument errors detectable on the host return a negative status
 * (codes of rlk_logp.h) before any HIP call; n_rows == 0 enqueues nothing.
 */
#ifndef RLK_MX4_H
#define RLK_MX4_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "rlk_logp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the codes and of the scales of an n_rows x d matrix (0 for n_rows
 * outside [0, 2^22] or d not a multiple of 32 in [32, 65536]). */
size_t rlk_mx4_codes_bytes(int64_t n_rows, int64_t d);
size_t rlk_mx4_scales_bytes(int64_t n_rows, int64_t d);

/* Quantises the BF16 matrix x [n_rows x d], row stride row_stride elements.
 *   x          16-byte aligned; row_stride >= d and a multiple of 8
 *   codes      rlk_mx4_codes_bytes(n_rows, d) bytes, 16-byte aligned
 *   scales     rlk_mx4_scales_bytes(n_rows, d) bytes, 16-byte aligned
 *   values_out the BF16 values that the blocks stand for (NaN as 0x7FC0),
 *              [n_rows x d] with row stride values_stride (>= d, a multiple of
 *              8), 16-byte aligned, or NULL; it may be x itself, with x's stride,
 *              and must not overlap it otherwise
 * codes and scales are written whole, their zeros included. */
int32_t rlk_mx4_quantize(const uint16_t* x, int64_t n_rows, int64_t d, int64_t row_stride,
                         uint8_t* codes, size_t codes_bytes, uint8_t* scales, size_t scales_bytes,
                         uint16_t* values_out, int64_t values_stride, hipStream_t stream);

/* Logits of the LM head with both operands in 4 bits:
 *   x_ij = bf16(sum_k hq_ik * wq_jk)
 * hq: the values of the quantised hidden states, wq: those of the quantised
 * projection, float32 accumulation on the matrix cores in increasing k (64
 * values a step), rounded once to nearest even. The order over k depends on k
 * alone: identical rows give identical bytes in any batch.
 *   hidden        BF16 [n_rows x d_model], row stride hidden_stride (a
 *                 multiple of 8, at most 2^21), 16-byte aligned; quantised by
 *                 this call into the workspace
 *   weight_codes, weight_scales
 *                 rlk_mx4_quantize's output for the projection [vocab_real x
 *                 d_model], 16-byte aligned
 *   layout        as for rlk_linear, vocab_real at most 2^22; row_stride is the
 *                 row stride of logits_out
 *   logits_out    BF16 [n_rows x row_stride], 16-byte aligned: columns [0,
 *                 vocab_real) hold x, [vocab_real, vocab_padded) -inf, the rest
 *                 of each row is not written. It must not overlap the
 *                 inputs or the workspace (a kernel may read hidden states
 *                 while another part of it stores logits)
 *   workspace     rlk_mx4_linear_workspace_bytes(n_rows, d_model) bytes,
 *                 16-byte aligned; calls that overlap need one each
 * d_model: a multiple of 32 in [32, 65536]. A hidden row with NaN or an
 * infinity has NaN logits. */
int32_t rlk_mx4_linear(const uint16_t* hidden, int64_t n_rows, int64_t d_model, int64_t hidden_stride,
                       const uint8_t* weight_codes, const uint8_t* weight_scales, const rlk_vocab_layout* layout,
                       uint16_t* logits_out, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Codes and scales of the hidden states; 0 for sizes that rlk_mx4_codes_bytes
 * answers with 0. */
size_t rlk_mx4_linear_workspace_bytes(int64_t n_rows, int64_t d_model);

#ifdef __cplusplus
}
#endif

#endif /* RLK_MX4_H */
