/*
 * fa_packed.h - C ABI of attention over packed sequences and of the norms and
 * rotation of its queries and keys (GB300, sm_103a).  Statuses, streams, the
 * device error word and the profile are those of fa.h.
 *
 * Packed sequences: sequences of different lengths lie one behind the other in
 * arrays [T, heads, d]; tokens cu[b] .. cu[b + 1] - 1 are sequence b, and a query
 * sees keys of its own sequence only.  kv head h / (H / Hkv) serves head h.
 * Arrays are bf16 device memory, 16-byte aligned, with dense channels; the
 * strides of a token and of a head are given in elements, positive multiples of 8
 * (of a dimension of one element any), below 2^34.  d: 64, 96, 128, 192, 256 or 384.
 *
 * cu (int32 [B + 1], device memory) must not decrease.  Its contents are checked
 * on the device: a sequence whose tokens do not lie in [0, T) has none.  Sequences
 * of no token are allowed.  Whatever cu holds, no call reads or writes
 * outside its arrays; rows that two sequences share hold either's results.
 */
#ifndef TILED_ATTENTION_TMEM_GB300_FA_PACKED_H_
#define TILED_ATTENTION_TMEM_GB300_FA_PACKED_H_

#include "fa_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Forward.  For query i and keys j of one sequence (causal: j <= i):
 *   s_ij = scale * q_i . k_j,  lse_i = ln sum_j exp(s_ij),  o_i = sum_j exp(s_ij - lse_i) v_j
 * q [T, H, d], k and v [T, Hkv, d] (read); o [T, H, d], lse fp32 [T, H] dense
 * (written).  Scores, maxima and sums are fp32; the probabilities that weigh v are
 * rounded to bf16, o to bf16 once.  Rows of o and lse of no sequence are left as
 * they were, and what q, k and v hold there, or in another sequence, never reaches a
 * result; a NaN or infinity in k or v of a token may reach any query of its own sequence.
 * A query whose scores are all -inf gets o = 0 and lse = -inf.  o must not
 * overlap the inputs.
 * H a multiple of Hkv, H / Hkv at most 32 (else FA_ERR_UNSUPPORTED), (T + B) * Hkv at
 * most 2^28, scale finite and > 0.  workspace: fa_packed_fwd_workspace_size bytes,
 * 256-byte aligned, not shared with a concurrent call.
 */
fa_status fa_packed_fwd(const void* q, long long q_token, long long q_head, const void* k, long long k_token,
                        long long k_head, const void* v, long long v_token, long long v_head, void* o,
                        long long o_token, long long o_head, float* lse, const int* cu, int B, int T, int H, int Hkv,
                        int d, float scale, int causal, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace fa_packed_fwd needs; 0 for shapes without work and invalid ones. */
size_t fa_packed_fwd_workspace_size(int B, int T, int H, int Hkv, int d);

/*
 * Backward.  With D_i = sum_c dO_ic o_ic, dP_ij = dO_i . v_j, P_ij = exp(s_ij - lse_i) and
 * dS_ij = P_ij (dP_ij - D_i), sums over the queries and the heads of a kv head that see key j:
 *   dv_j = sum P_ij dO_i,  dk_j = scale sum dS_ij q_i,  dq_i = scale sum_j dS_ij k_j
 * o and lse as fa_packed_fwd wrote them for the same arguments.  P and dS are rounded to bf16
 * where they enter the products, the gradients once.  Rows of no sequence (before cu[0] and
 * behind cu[B]) get gradients of zero; with B = 0 every row is one.  A NaN or
 * infinity in a row of one sequence never reaches another.  The gradients must not overlap
 * one another or the inputs.
 * variant: FA_BWD_5GEMM (d <= 128; dq is summed by reductions in fp32 whose order is not fixed),
 * FA_BWD_7GEMM (the same arguments give the same bits) or FA_BWD_AUTO (the 5-GEMM form where it
 * exists).  workspace: fa_packed_bwd_workspace_size bytes of the same shape and variant,
 * 256-byte aligned, not shared with a concurrent call.
 */
fa_status fa_packed_bwd(const void* q, long long q_token, long long q_head, const void* k, long long k_token,
                        long long k_head, const void* v, long long v_token, long long v_head, const void* o,
                        long long o_token, long long o_head, const void* dO, long long do_token, long long do_head,
                        const float* lse, void* dq, long long dq_token, long long dq_head, void* dk, long long dk_token,
                        long long dk_head, void* dv, long long dv_token, long long dv_head, const int* cu, int B, int T,
                        int H, int Hkv, int d, float scale, int causal, int variant, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace fa_packed_bwd needs (row statistics, for the 5-GEMM form an fp32 dq, tensor
 * maps); 0 for shapes without work and invalid ones.
 */
size_t fa_packed_bwd_workspace_size(int B, int T, int H, int Hkv, int d, int variant);

#ifdef __cplusplus
}
#endif

#endif /* TILED_ATTENTION_TMEM_GB300_FA_PACKED_H_ */
