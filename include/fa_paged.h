/*
 * fa_paged.h - C ABI of the serving operators of the GB300 (sm_103a) attention
 * library: page tables built on the GPU, a paged key/value cache held in 4
 * bits, and attention of a few query tokens per request over that cache.
 * Statuses, streams, the device error word and the profile are those of fa.h.
 *
 * The cache.  A pool of `pages` pages of `page` tokens each (16, 32, 64 or 128),
 * for keys and for values, one block per (page, kv head):
 *   codes  uint8 [pages, Hkv, page, d/2]   two e2m1 codes a byte, channel 2c in
 *                                          the low half, 2c + 1 in the high half
 *   scales uint8 [pages, Hkv, page, d/16]  one e4m3 scale per 16 channels
 * and one fp32 gain per tensor, from 2^-100 to 2^100:
 *   value = gain * scale * code,  code in +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}.
 * A scale byte's sign bit is ignored and 0x7f reads as 480: every byte pattern
 * stands for a finite value, so slots that were never written cannot put an
 * infinity or NaN into a result.  Arrays are dense, 16-byte aligned, and may hold more than
 * 2^32 bytes.
 *
 * A slot is page * (tokens per page) + token in page.  table[b][c] (int32, row
 * stride `width`) is the page that holds tokens c*page .. c*page + page - 1 of
 * request b.  d: 64, 96, 128, 192, 256 or 384.
 *
 * Every array argument is device memory owned by the caller, index arrays and lse
 * aligned to their elements (else FA_ERR_MISALIGNED).  The contents of
 * index arrays are checked on the device where they are used: an index that is
 * out of range is skipped as each call states, and never read or written through.
 */
#ifndef TILED_ATTENTION_TMEM_GB300_FA_PAGED_H_
#define TILED_ATTENTION_TMEM_GB300_FA_PAGED_H_

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Kernel kinds of these calls and of those of fa_packed.h, for fa_profile_stop_kinds and fa_kernel_name. */
enum {
  FA_KERNEL_PAGE = 9,       /* page tables and slots */
  FA_KERNEL_KV4_STORE = 10, /* 4-bit cache: store */
  FA_KERNEL_KV4_LOAD = 11,  /* 4-bit cache: load */
  FA_KERNEL_KV4_ATTN = 12,  /* attention over the 4-bit cache */
  FA_KERNEL_KV4_MERGE = 13, /* merge of its warps' parts */
  /* fa_packed.h (attention over packed sequences counts as the dense kernels it shares) */
  FA_KERNEL_PACKED_PLAN = 14, /* packed sequences: order of work, tensor maps */
  FA_KERNEL_ROTATE = 15,      /* norms and rotation of queries and keys */
  FA_KERNEL_ROTATE_BWD = 16,  /* their gradients */
  FA_KERNEL_ROTATE_SUM = 17,  /* the weights' gradients, summed over the blocks */
  FA_KERNEL_KV4_APPEND = 18,  /* 4-bit cache: rotated append */
  FA_KERNEL_ALL_KINDS = 19
};

/* The cache as the calls take it (host memory; read during the call only). */
typedef struct {
  void* k_codes;
  void* k_scales;
  void* v_codes;
  void* v_scales;
  int pages; /* pages in the pool */
  int page;  /* tokens per page: 16, 32, 64 or 128 */
  int Hkv;
  int d;
  float k_gain;
  float v_gain;
} fa_kv4_cache;

/*
 * Page tables and slots for the next tokens of B requests.
 *   lengths     int32 [B]         tokens each request holds (negative: 0)
 *   new_tokens  int32 [B]         tokens each request gets now (negative: 0)
 *   table       int32 [B, width]  read; entries of pages taken now are written
 *   free_pages  int32 [free_size] stack of free pages, read only (NULL where free_size is 0)
 *   free_count  int32 [1]         pages on the stack (above free_size: free_size)
 *   T           capacity of `slots`
 *   slots       int64 [T]         slot of new token t, requests in order; -1 for a
 *                                 token that has none and past the last new token
 *   cu          int32 [B + 1]     first new token of each request in `slots`
 *   lengths_out int32 [B]         lengths plus the new tokens that got a slot (or whose page
 *                                 id is below 0, in the table or on the stack: slot -1)
 *   count_out   int32 [1]         pages left: the stack is free_pages[0 .. count_out)
 * Request b owns ceil(lengths/page) pages; the pages it needs beyond those (at
 * most up to `width`) are taken from the top of the stack in request order.
 * When the stack runs out, its entries become -1, and tokens on them, past
 * `width` or past T get no slot: then lengths_out[b] < lengths[b] + new_tokens[b].
 * B at most 2^21, width * page below 2^31.  With B = 0 nothing is written.
 * Inputs are not changed except `table`, so a repeated call gives the same
 * result; the outputs must not overlap the inputs.
 */
fa_status fa_page_grow(const int* lengths, const int* new_tokens, int* table, int B, int width, int page,
                       const int* free_pages, int free_size, const int* free_count, int T, long long* slots,
                       int* cu, int* lengths_out, int* count_out, void* stream);

/*
 * Slots of the tokens first[b] .. first[b] + count[b] - 1 of each request, from a
 * table that holds their pages.  Outputs as fa_page_grow; nothing is taken.
 */
fa_status fa_page_slots(const int* first, const int* count, const int* table, int B, int width, int page, int T,
                        long long* slots, int* cu, void* stream);

/*
 * Writes T tokens of k and v (bf16 [T, Hkv, d], element strides of the token
 * and the head given, multiples of 8; the channels dense) into the cache.  Per
 * group of 16 channels, in fp32: scale = e4m3(max|x| / (6 gain)), code =
 * e2m1(x / (gain scale)), each rounded to nearest even and saturating (scale 0:
 * codes of 0 with the signs of x).  The
 * quotients are good to 12 bits: exact in effect where the gain is a power of
 * two, else a quotient within 2^-12 of a border may go either way.  A NaN
 * becomes code 6 under the scale of the others.
 * slots[t] < 0 or >= pages*page: token t is skipped.  The valid slots must be
 * distinct: a slot given twice ends up with bytes of either token.
 */
fa_status fa_kv4_store(const fa_kv4_cache* cache, const void* k, const void* v, long long k_token,
                       long long k_head, long long v_token, long long v_head, const long long* slots, int T,
                       void* stream);

/*
 * Reads T tokens back as bf16 (dense [T, Hkv, d]), each value rounded once.
 * slots[t] < 0 or >= pages*page gives zeros.
 */
fa_status fa_kv4_load(const fa_kv4_cache* cache, const long long* slots, int T, void* k, void* v, void* stream);

/*
 * Attention of the newest tokens of B requests over the cache.
 *   q    bf16 [T, H, d], strides q_token and q_head (elements, multiples of 8)
 *   cu   int32 [B + 1]: request b's queries are tokens cu[b] .. cu[b+1] - 1 of q;
 *        NULL: one query a request, token b
 *   lengths int32 [B]: tokens of request b in the cache, its queries' own included
 *   o    bf16 [T, H, d], strides o_token and o_head; lse fp32 [T, H] dense
 * Query i of the n_q of request b sees the keys j <= lengths[b] - n_q + i; kv head
 * h / (H/Hkv) serves head h:
 *   s_j = scale * k_gain * q . k_j,  lse = ln sum_j exp(s_j),  o = sum_j exp(s_j - lse) v_j.
 * Scores, maxima and sums are fp32 (a score past its range is an infinity).  q is taken exactly, but for channels below 2^-17 of
 * their row's largest magnitude, which are off by 2^-25 of it at most; exp by 2^-21 of
 * itself; the probabilities that weigh v are rounded to f16, o to bf16 once.
 * A query that sees no key, or whose scores are all -inf, gets o = 0 and lse = -inf;
 * other infinities, as from one in q, and NaN make their row NaN.  Rows of o and lse that no
 * query of a request owns are left as they were.  The first max_q queries of a
 * request are computed (max_q times H/Hkv below 2^31).  A request whose queries do
 * not lie in [0, T) has none; requests that share a query leave either's result in
 * its row.  o may be q itself where the strides are the same and no two requests share
 * a query, but must not overlap it in another way.  A token whose table entry is not in
 * [0, pages), or lies past `width`, is no key.
 * H a multiple of Hkv; scale finite and > 0.  workspace: fa_kv4_attn_workspace_size
 * bytes, 256-byte aligned, not shared with a concurrent call.
 */
fa_status fa_kv4_attn(const fa_kv4_cache* cache, const void* q, long long q_token, long long q_head, int T,
                      const int* cu, int max_q, const int* table, int width, const int* lengths, int B, int H,
                      float scale, void* o, long long o_token, long long o_head, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace fa_kv4_attn needs on the current device (fp32 partial results
 * of requests that several SMs share); 0 where it needs none (few tokens: `workspace`
 * may be NULL) and for invalid shapes.  max_q: 1 where `cu` is NULL.
 */
size_t fa_kv4_attn_workspace_size(int B, int H, int Hkv, int d, int max_q, int page, int width);

#ifdef __cplusplus
}
#endif

#endif /* TILED_ATTENTION_TMEM_GB300_FA_PAGED_H_ */
