/*
 * pulsar_serving.h -- C ABI of the serving operators of libpulsar_b200.so:
 * many requests of different lengths over one paged KV cache.
 *
 * Phase 1 and Phase 2 (pulsar.h) work on one sequence, or on a batch of
 * caches of equal length.  These calls serve requests of any lengths
 * together: the page tables and slot map of a step, the rotation of its new
 * tokens with their append to the cache, causal attention over packed
 * prompts, and attention of new tokens over the pages.
 *
 * The conventions of pulsar.h hold (device pointers, the caller's workspace
 * with its status block, stream order, pa_status, PA_F32 / PA_BF16), and:
 *  - A packed batch of B requests has cu_q [B + 1] int32, cu_q[0] = 0: rows
 *    cu_q[b] .. cu_q[b + 1] - 1 of its tensors are request b's new tokens.
 *    The tensors have N rows, N >= cu_q[B]; rows from cu_q[B] on are padding
 *    and are left as they were (outputs) or not read (inputs).
 *  - q, k, v rows are [heads][d], dense, with a stride of ld* ELEMENTS from
 *    one token to the next (a slice of a fused projection is fine); base
 *    addresses and strides are multiples of 16 bytes.
 *  - The cache is k_pages, v_pages [n_pages][page_size][hkv][d] of dtype, K
 *    rotated; page_size is a power of two, 16 .. 32768.  Its slots are
 *    numbered page * page_size + offset, below 2^31.  This is also the
 *    memory order of Phase 1's retained cache [N][block][hkv][d].
 *  - block_table [B][max_pages] int32, a stride of table_stride entries from
 *    one request to the next: entry i of request b is the page of its keys
 *    i * page_size ..; entries past its last key are not read.
 *  - d is 64 or 128; hq % hkv == 0, hq / hkv <= 64; query head h reads kv head
 *    h / (hq / hkv).  B <= 8192, N < 2^31.
 *  - Lengths and tables are read on the device only, so a captured call may
 *    be replayed with other lengths that fit the same arguments.  Calls that
 *    share a workspace, captured or not, must not overlap on the GPU.  Lengths
 *    out of range (a cu_q that falls or passes N, a negative kv_len or one
 *    above max_pages * page_size) set PA_ERR_INVALID in the workspace status
 *    and that request is skipped; a page outside [0, n_pages) sets it and
 *    its keys read as zeros.  Where a cu_q falls, requests may share rows:
 *    which of them such a row is answered for is not defined.
 */
#ifndef PULSAR_B200_SERVING_H
#define PULSAR_B200_SERVING_H

#include "pulsar.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of scratch pa_paged_schedule needs (the status block). */
size_t pa_paged_schedule_workspace_size(int32_t B);

/*
 * The page tables and slot map of one step, from the requests' lengths.
 *  q_len          [B] int32, new tokens of each request (0 allowed).
 *  kv_len         [B] int32, tokens each request has in the cache.
 *  block_table    in/out: the first ceil(kv_len / page_size) entries of a
 *                 request are its pages; the pages it needs for its new
 *                 tokens are written behind them.  Must not overlap the
 *                 lengths or free_pages.
 *  free_pages     [n_free] int32: new pages are taken from its front, in
 *                 the order of the requests.
 *  cu_q           out [B + 1] int32: exclusive prefix sum of q_len.
 *  kv_len_out     out [B] int32: kv_len + q_len (kv_len if refused).  Must
 *                 not overlap kv_len.
 *  positions      out [n_tokens] int32: the position of every new token,
 *                 kv_len + its index; 0 in padding rows.
 *  slots          out [n_tokens] int32: its cache slot; -1 in padding rows
 *                 and for a refused request's tokens.
 *  n_used         out [1] int32: pages taken from free_pages.
 * A request whose pages do not fit its table row, or the free pages left by
 * the requests before it, is refused as a whole: it takes no page, its slots
 * are -1, and the status reads PA_ERR_CAPACITY.  (A request counts its pages
 * against the pool even when it is refused for the pool, so those after it
 * that need pages are refused too.)  A negative length counts as 0 and sets
 * PA_ERR_INVALID, as does sum(q_len) > n_tokens (the tokens past n_tokens
 * get no position or slot) and a page whose slots would pass 2^31 - 1 (its
 * slots are -1).  Integer work: the results are exact and deterministic.
 */
int pa_paged_schedule(const int32_t* q_len, const int32_t* kv_len, int32_t B, int32_t* block_table,
                      int64_t table_stride, int32_t max_pages, const int32_t* free_pages,
                      int32_t n_free, int32_t page_size, int64_t n_tokens, int32_t* cu_q,
                      int32_t* kv_len_out, int32_t* positions, int32_t* slots, int32_t* n_used,
                      void* ws, size_t ws_bytes, void* stream);

/* Bytes of scratch pa_paged_append needs (the status block). */
size_t pa_paged_append_workspace_size(int64_t N);

/*
 * Rotation of N new tokens and their append to the paged cache.
 *  q, k, v        [N][hq | hkv | hkv][d] dtype, unrotated, strides ldq, ldk,
 *                 ldv.  q may be NULL (then q_out is not written).
 *  positions      [N] int32 (not read when rope_theta == 0).
 *  slots          [N] int32, distinct where >= 0; a token with a negative
 *                 slot is not written to the cache.  A slot of n_slots or
 *                 more sets PA_ERR_INVALID and is skipped.
 *  k_pages, v_pages  in/out [n_slots][hkv][d]: rows slots[i] receive token
 *                 i's rotated K and its V.  slots, k_pages and v_pages may be
 *                 NULL together: nothing is appended (v is then not read).
 *                 They must not overlap one another or what the call reads.
 *  q_out          out [N][hq][d] dense: the rotated q.  May equal q when ldq
 *                 is hq * d.
 *  k_out_opt      out [N][hkv][d] dense: the rotated k, or NULL.  May equal k
 *                 when ldk is hkv * d.
 * q_out and k_out_opt are written for all N tokens, those without a slot
 * included.
 * RoPE is rotate-half, omega_m = rope_theta^(-2m/d), the angle reduced in
 * fp64, the rotation in fp32, one rounding to dtype; rope_theta == 0: no
 * rotation.
 */
int pa_paged_append(const void* q, const void* k, const void* v, int dtype, int64_t N, int64_t ldq,
                    int64_t ldk, int64_t ldv, int32_t hq, int32_t hkv, int32_t d, double rope_theta,
                    const int32_t* positions, const int32_t* slots, void* k_pages, void* v_pages,
                    int64_t n_slots, void* q_out, void* k_out_opt, void* ws, size_t ws_bytes,
                    void* stream);

/* Bytes of scratch pa_prompt_attend needs; 0 for invalid arguments. */
size_t pa_prompt_attend_workspace_size(int32_t B, int64_t N, int32_t hq, int32_t hkv, int32_t d,
                                       int dtype);

/*
 * Causal attention over B packed prompts of different lengths:
 * o_i = sum_{j <= i} p_ij v_j with p_i the softmax over j <= i of
 * q_i . k_j / sqrt(d), inside each prompt.
 *  q, k, v        [N][hq | hkv | hkv][d] dtype, K and Q rotated, strides ldq,
 *                 ldk, ldv.
 *  o              out [N][hq][d] dtype, dense; must not overlap the inputs.
 *  lse_opt        out [N][hq] float: natural-log sum of exp of the row's
 *                 scaled scores, or NULL.
 * Precision (bf16): the products q . k are exact and summed in fp32; the
 * softmax and all sums are fp32 (the tensor cores' drop what an addition cannot
 * hold: at most 2^-9 of sum p |v|, however many keys; 3e-4 measured); the
 * probabilities may be rounded to bf16
 * for the product with V (one rounding, half a step of 2^-7 relative; the
 * row sum is taken before it); one rounding of o.
 * A masked key adds nothing whatever its K and V hold (infinities and NaN
 * included); a visible non-finite V makes that column of o non-finite (the
 * infinity, or NaN).  A visible key whose score is -inf weighs nothing, and a
 * row all of whose keys are such counts as one that sees no key: lse = -inf and,
 * where V is finite, o = 0.
 */
int pa_prompt_attend(const void* q, const void* k, const void* v, int dtype, int64_t N, int64_t ldq,
                     int64_t ldk, int64_t ldv, const int32_t* cu_q, int32_t B, int32_t hq,
                     int32_t hkv, int32_t d, void* o, float* lse_opt, void* ws, size_t ws_bytes,
                     void* stream);

/* Bytes of scratch pa_paged_attend needs; 0 for invalid arguments. */
size_t pa_paged_attend_workspace_size(int32_t B, int64_t N, int32_t max_q, int32_t max_pages,
                                      int32_t page_size, int32_t hq, int32_t hkv, int32_t d,
                                      int dtype);

/*
 * Attention of each request's new tokens over its paged cache, which already
 * holds them (pa_paged_append): row i of request b, at position
 * kv_len[b] - q_len[b] + i, sees the keys up to its own position.  A
 * generated token is a request with one new token; a prompt's chunk is one
 * with many; both may be in one call.
 *  q              [N][hq][d] dtype, rotated, stride ldq.
 *  cu_q           [B + 1] int32; kv_len [B] int32, keys in the cache, new
 *                 tokens included.
 *  max_q          an upper bound of the requests' new tokens, 1 <= max_q; a
 *                 longer request sets PA_ERR_INVALID and is skipped.
 *  o, lse_opt     out as in pa_prompt_attend.
 * A row that sees no key (kv_len below its request's new tokens) gives o = 0
 * and lse = -inf.  Precision and non-finite values as in pa_prompt_attend.
 */
int pa_paged_attend(const void* q, int dtype, int64_t N, int64_t ldq, const int32_t* cu_q,
                    const int32_t* kv_len, int32_t B, int32_t max_q, const int32_t* block_table,
                    int64_t table_stride, int32_t max_pages, int32_t page_size, const void* k_pages,
                    const void* v_pages, int32_t n_pages, int32_t hq, int32_t hkv, int32_t d, void* o,
                    float* lse_opt, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PULSAR_B200_SERVING_H */
