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
 * outside its arrays, or does more work than T tokens are: where sequences overlap
 * so that they hold more than T tokens together, none is attended to.  The results of a call whose cu decreases are
 * unspecified otherwise.
 *
 * The calls take their arguments as a structure in host memory, which is read during
 * the call only; every call enqueues its work on `stream`.
 */
#ifndef TILED_ATTENTION_TMEM_GB300_FA_PACKED_H_
#define TILED_ATTENTION_TMEM_GB300_FA_PACKED_H_

#include "fa_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A [T, heads, d] array: its address and the strides of a token and a head in elements. */
typedef struct {
  const void* data; /* (written through where the call says so) */
  long long token;
  long long head;
} fa_rows;

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
 * 256-byte aligned, not shared with a concurrent call (may be NULL where that is 0: few sequences).
 */
typedef struct {
  fa_rows q, k, v, o;
  float* lse;
  const int* cu;
  int B, T, H, Hkv, d;
  float scale;
  int causal; /* 0 or 1 */
  void* workspace;
  size_t workspace_bytes;
  void* stream;
} fa_packed_fwd_args;
fa_status fa_packed_fwd(const fa_packed_fwd_args* a);

/* Bytes of workspace fa_packed_fwd needs on the current device; 0 for few sequences, and for shapes without
 * work and invalid ones. */
size_t fa_packed_fwd_workspace_size(int B, int T, int H, int Hkv, int d);

/*
 * Backward.  With D_i = sum_c dO_ic o_ic, dP_ij = dO_i . v_j, P_ij = exp(s_ij - lse_i) and
 * dS_ij = P_ij (dP_ij - D_i), sums over the queries and the heads of a kv head that see key j:
 *   dv_j = sum P_ij dO_i,  dk_j = scale sum dS_ij q_i,  dq_i = scale sum_j dS_ij k_j
 * o and lse as fa_packed_fwd wrote them for the same arguments.  P and dS are rounded to bf16
 * where they enter the products, the gradients once.  Rows of no sequence (before the first
 * and behind the last that lies in [0, T)) get gradients of zero; with B = 0 every row is one.
 * With H = 0 nothing is read or written (dk and dv, sums over no heads, are the caller's to clear).  A NaN or
 * infinity in a row of one sequence never reaches another.  The gradients must not overlap
 * one another or the inputs.
 * variant: FA_BWD_5GEMM (d <= 128; dq is summed by reductions in fp32 whose order is not fixed),
 * FA_BWD_7GEMM (the same arguments give the same bits) or FA_BWD_AUTO (the 5-GEMM form where it
 * exists).  workspace: fa_packed_bwd_workspace_size bytes of the same shape and variant,
 * 256-byte aligned, not shared with a concurrent call.
 */
typedef struct {
  fa_rows q, k, v, o, dO;
  const float* lse;
  fa_rows dq, dk, dv;
  const int* cu;
  int B, T, H, Hkv, d;
  float scale;
  int causal; /* 0 or 1 */
  int variant;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
} fa_packed_bwd_args;
fa_status fa_packed_bwd(const fa_packed_bwd_args* a);

/*
 * Bytes of workspace fa_packed_bwd needs on the current device (row statistics, for the 5-GEMM form an fp32 dq, tensor
 * maps); 0 for shapes without work and invalid ones.
 */
size_t fa_packed_bwd_workspace_size(int B, int T, int H, int Hkv, int d, int variant);

/*
 * Norms of queries and keys for each head, and their rotation by the token's position.  For each
 * head x of q [T, H, d] and k [T, Hkv, d], in fp32 and rounded to bf16 once:
 *   n_c = x_c r w_c,  r = (sum_c x_c^2 / d + eps)^-1/2   (n = x where the weight is NULL)
 *   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin      for pair i < rot/2: channels
 *   (a, b) = (i, i + rot/2), or (2i, 2i + 1) if `interleaved`;  y_c = n_c for c >= rot
 * with cos = rotary[position[t]][i] and sin = rotary[position[t]][rot/2 + i].  The products and the
 * sum of a rotation are rounded to fp32 one by one.
 *   rotary    fp32 [positions, rot] dense, 16-byte aligned; rot a multiple of 32, at most d (0: no rotation)
 *   position  int32 [T].  A token whose position is not in [0, positions) is left out: its
 *             rows of q_out and k_out stay as they were.
 *   q_weight, k_weight  bf16 [d], 16-byte aligned, or NULL;  eps finite and >= 0
 * q and k with strides (elements, multiples of 8; 0 is allowed); q_out may be q itself with q's strides, k_out
 * likewise, but no output may overlap another array in another way.  H + 2 Hkv at most 65535,
 * T at most 2^30.
 */
typedef struct {
  fa_rows q, k, q_out, k_out;
  const float* rotary;
  const int* position;
  const void* q_weight;
  const void* k_weight;
  int positions, rot;
  float eps;
  int interleaved; /* 0 or 1 */
  int T, H, Hkv, d;
  void* stream;
} fa_qk_norm_rope_args;
fa_status fa_qk_norm_rope(const fa_qk_norm_rope_args* a);

/*
 * Its gradients.  dq_out and dk_out: of the results; q and k: what went in (needed, and read, only where
 * there is the weight).  With g the rotation's transpose of dy, xhat = x r and z = w g:
 *   dx = r (z - xhat sum_c(xhat_c z_c) / d)  (dx = g where the weight is NULL),  dw = sum g xhat
 * dq, dk bf16, rounded once (dq may be dq_out, or q, with the same strides; dk likewise); dq_weight, dk_weight fp32 [d],
 * written where there is the weight: sums in fp32 over all tokens and heads, in a fixed order.  A token
 * without a position has gradients of zero and is not in the sums.
 * workspace: fa_qk_norm_rope_bwd_workspace_size bytes, 256-byte aligned, not shared with a
 * concurrent call (NULL where both weights are).
 */
typedef struct {
  fa_rows dq_out, dk_out, q, k, dq, dk;
  const float* rotary;
  const int* position;
  const void* q_weight;
  const void* k_weight;
  float* dq_weight;
  float* dk_weight;
  int positions, rot;
  float eps;
  int interleaved; /* 0 or 1 */
  int T, H, Hkv, d;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
} fa_qk_norm_rope_bwd_args;
fa_status fa_qk_norm_rope_bwd(const fa_qk_norm_rope_bwd_args* a);
size_t fa_qk_norm_rope_bwd_workspace_size(int T, int H, int Hkv, int d);

/*
 * New tokens on their way into the 4-bit cache (fa_paged.h) in one pass: q [T, H, d] and k
 * [T, Hkv, d] normed and rotated as by fa_qk_norm_rope (Hkv and d those of the cache), q to q_out, k
 * (rounded to bf16) and v stored as by fa_kv4_store in slots int64 [T].  k_out: the rotated keys too,
 * or NULL.  A token without a position is left out altogether; one whose slot is not in
 * [0, pages*page) is rotated but not stored.  The valid slots must be distinct.  H may be 0.
 */
typedef struct {
  const fa_kv4_cache* cache;
  fa_rows q, k, v, q_out, k_out; /* k_out.data may be NULL */
  const float* rotary;
  const int* position;
  const void* q_weight;
  const void* k_weight;
  const long long* slots;
  int positions, rot;
  float eps;
  int interleaved; /* 0 or 1 */
  int T, H;
  void* stream;
} fa_kv4_append_args;
fa_status fa_kv4_append(const fa_kv4_append_args* a);

#ifdef __cplusplus
}
#endif

#endif /* TILED_ATTENTION_TMEM_GB300_FA_PACKED_H_ */
