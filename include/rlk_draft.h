/*
 * rlk_draft.h - verification of drafted tokens against the target's policy on
 * gfx950 (MI355X), from given random numbers, and with no drafted tokens the
 * sampler of a rollout. Works on what rlk_logp_nucleus leaves of every row
 * (policy and reference logprob, lse, support record) and reads again only the
 * rows that a token is drawn from.
 *
 * What is computed (speculative sampling: the emitted tokens follow the
 * target's policy whatever the drafter proposed), for sequence s with K
 * drafted tokens d_0 .. d_{K-1} and K + 1 rows of target logits:
 *   p_k  the policy of the sequence's target row k: exp(z_j - lse_support) for
 *        columns j < vocab_real with x_j >= threshold, else 0; z_j = fl32(x_j /
 *        T); a point mass on the lowest-index maximum when T = 0 (greedy)
 *   q_k  the drafter's policy at the same place, from its own logits and
 *        records in the same way; a point mass on d_k when the drafter has no
 *        logits (a lookup, a copy) or its row is greedy
 *   token k is accepted while  accept_u_k < exp(log p_k(d_k) - log q_k(d_k));
 *   at the first k that is not, one token is drawn from max(p_k - q_k, 0); when
 *   all K are accepted, one is drawn from p_K:
 *   token = the lowest j with C_j > sample_u * C, C_j the sum of the columns
 *           0 .. j, C their whole sum, in float64
 * (When p_k is nowhere above q_k, which rounded statistics of equal rows can
 * give, the drafted token itself is emitted.) The logarithms are the given
 * float32 policy logprobs; sums and exponentials are in float64, in an order
 * that depends on the columns alone: a sequence's outputs do not depend on the
 * batch.
 *
 * Memory: every pointer inside the structs and every array argument is
 * caller-owned DEVICE memory; the structs and `layout` are host memory, read
 * during the call. Nothing is allocated, freed or synchronised, and calls can
 * be captured into a hipGraph; the lengths of the drafts are device data, so a
 * captured call serves other lengths. Argument errors detectable on the host
 * return a negative status (codes of rlk_logp.h) before any HIP call.
 */
#ifndef RLK_DRAFT_H
#define RLK_DRAFT_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "rlk_logp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of logits and what rlk_logp_nucleus left of them. */
typedef struct rlk_scored_rows {
  const uint16_t* logits;           /* BF16 bits [n_rows * row_stride], 16-byte aligned */
  int64_t n_rows;
  int64_t row_stride;               /* >= vocab_padded, a multiple of 8 */
  const float* temperature;         /* [n_rows] as in that call */
  const float* policy_logp;         /* [n_rows] policy_out of the row's drafted token */
  const float* ref_logp;            /* [n_rows] ref_out (target side only) */
  const float* lse;                 /* [n_rows] lse_out (target side only) */
  const rlk_support_state* support; /* [n_rows] support_out */
} rlk_scored_rows;

/* Verifies n_seq sequences.
 *   target      the target's rows, sequence after sequence: row draft_start[s]
 *               + s + k is row k of sequence s. Score row k < K with target
 *               column d_k, row K with any real column (0). n_rows >= n_draft +
 *               n_seq
 *   draft       the drafter's rows: row draft_start[s] + k, scored with column
 *               d_k; n_rows >= n_draft; ref_logp and lse are not read. NULL:
 *               every drafted token is a point mass
 *   layout      vocab_padded, vocab_real, n_shards, groups as in rlk_logp.h
 *               (groups and row_stride are validated, not used)
 *   n_draft     capacity of the arrays of drafted tokens (0 .. 2^22)
 *   draft_start [n_seq + 1] int64, non-decreasing from 0 or more to n_draft or
 *               less: sequence s has the drafted tokens [draft_start[s],
 *               draft_start[s + 1])
 *   draft_token [n_draft] int64;  accept_u [n_draft] float64 in [0, 1)
 *   sample_u    [n_seq] float64 in [0, 1)
 *   token_out   [target->n_rows] int64: in the sequence's rows its accepted
 *               tokens, the drawn token, then -1
 *   accepted_out [n_seq] int32: number of accepted drafted tokens
 *   policy_out, ref_out  [target->n_rows] float32: the emitted tokens' policy
 *               and reference logprobs: those given for accepted tokens, z -
 *               lse_support and z - lse for the drawn one (0 when greedy), 0
 *               behind it
 *   workspace   rlk_draft_workspace_bytes(n_seq, layout) bytes, 16-byte
 *               aligned; calls that overlap need one each
 * Outputs and workspace must not overlap the inputs.
 * Rows of no sequence are left as they were in the outputs. draft_token,
 * accept_u and draft may be NULL when n_draft is 0.
 * Device data that cannot be served: a sequence whose draft_start is out of
 * order or range has accepted_out = -1 and nothing else written (of two other
 * sequences that then share rows, either may have written them). Where the row
 * reached has no policy (status < 0, a temperature that is NaN, infinite or
 * below 0, a threshold that is NaN or an lse_support that is NaN or infinite,
 * on either side; greedy rows' records are read for their status alone), a
 * drafted token's policy logprob is NaN, on either side, the drafted token is
 * outside [0, vocab_real), a random number is outside [0, 1) or there is
 * nothing to draw from (the weights' sum is 0 and there is no drafted token, or
 * one whose policy logprob is -inf; or the sum is not finite: where |z| passes
 * 1e10, lse_support is too coarse), token_out is -1 and both logprobs are NaN
 * at that place, and the sequence ends there. */
int32_t rlk_draft_verify(const rlk_scored_rows* target, const rlk_scored_rows* draft,
                         const rlk_vocab_layout* layout, int64_t n_seq, int64_t n_draft,
                         const int64_t* draft_start, const int64_t* draft_token, const double* accept_u,
                         const double* sample_u, int64_t* token_out, int32_t* accepted_out, float* policy_out,
                         float* ref_out, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace: one float64 per sequence and 512 columns; 0 for an
 * invalid layout or n_seq outside [0, 2^22]. */
size_t rlk_draft_workspace_bytes(int64_t n_seq, const rlk_vocab_layout* layout);

#ifdef __cplusplus
}
#endif

#endif /* RLK_DRAFT_H */
