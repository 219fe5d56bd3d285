/*
 * kda_kv4.h -- C ABI of the paged 4-bit key/value cache for the
 * softmax-attention layers that a hybrid decoder keeps between its recurrent
 * layers (page "Kimi K3：架构、训练与百万 Token Agentic RL 技术解读" §2: three KDA layers
 * to one attention layer; §9: the physical blocks of the prefix cache): block
 * tables and slot maps, the cache's write and read-back, and attention over it.
 *
 * The conventions of kda.h hold: device pointers owned by the caller, nothing
 * allocated, asynchronous on `stream`, argument errors found on the host before
 * anything is launched, conditions that only the device sees (a page, slot,
 * length or prefix-sum array out of range) reported through kda_device_error()
 * as KDA_ERR_INVALID_ARG after the work, never by an access out of range.
 *
 * The cache is uint8 [num_pages][Hkv][page_size / 16][17 D], 16-byte aligned: for
 * each page and key/value head, units of 16 tokens of 17 D bytes.  A unit holds
 *   keys    [16 rows][D / 2]: row r's 32-bit word at place t (D / 32) + j holds channels
 *           32 j + 8 t .. + 7, four bits each, the lowest channel in the lowest bits;
 *   values  [2 blocks of 8 tokens][8 g][8 tokens][D / 32 j] 16-bit words: channels
 *           32 j + 4 g .. + 3, in the same order;
 *   key scales [16][D / 32] and value scales [16][D / 32], one byte for 32 channels.
 * A stored value is the E2M1 code (sign bit over 0, 0.5, 1, 1.5, 2, 3, 4, 6) times
 * 2^(scale byte - 127).  The scale is the smallest power of two, 2^-126 at least,
 * that leaves no channel of the 32 above 6; codes are rounded to nearest, ties to
 * the even code.  32 channels with an inf or NaN among them are stored as scale
 * byte 255, which reads back as NaN.  (This is the block format that the OCP
 * microscaling specification calls MXFP4, with a scale rule that never saturates;
 * the order inside a unit is the order in which the attention kernel's matrix
 * instructions take their operands.)
 * Token p of a sequence lies in page block_table[p / page_size], place p % page_size;
 * its slot is page * page_size + place.
 * page_size is a multiple of 16, at most 4096; D is 64 or 128;
 * num_pages * page_size is at most 2^31 - 1.
 */
#ifndef KDA_GB300_KDA_KV4_H
#define KDA_GB300_KDA_KV4_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of a cache of num_pages pages, or SIZE_MAX when the sizes are invalid. */
KDA_API size_t kda_kv4_cache_bytes(int64_t num_pages, int32_t Hkv, int32_t page_size, int32_t D);

/*
 * Block tables and slot maps of one step from request lengths.
 *
 *  cached_lens, new_lens  int32[N]: tokens of each request in the cache, and tokens that
 *               this step adds (either may be 0)
 *  block_table  int32[N][max_pages], row stride max_pages: the first
 *               ceil(cached / page_size) entries of a row are read (only the last, partly
 *               filled one is); the entries of the pages that the new tokens begin are
 *               written, request by request, with the next entries of free_pages
 *  free_pages   int32[num_free], free_start int32[1]: the pages that are free are
 *               free_pages[free_start ..]
 *  cu_seqlens   int32[N + 1]: prefix sums of new_lens (what kda_chunk_fwd takes)
 *  seq_lens     int32[N]: cached + new (what kda_kv4_attention takes)
 *  slot_map, positions  int32[num_tokens], 16-byte aligned: each new token's slot, and its
 *               position in its request; -1 behind the last new token
 *  free_next    int32[1]: the first entry of free_pages that is still free afterwards
 * num_tokens is the room in slot_map and positions.  Not every request may get what it
 * asks for: tokens whose page is not there (the free pages used up, the row too short, a
 * partly filled page with a negative entry) get slot -1, table entries without a free page
 * get -1; negative lengths count as 0; of more than num_tokens new tokens the first are
 * mapped, and pages that begin behind them get the entry -1.  Each of these is reported
 * (kda_device_error).  seq_lens and free_next count every new token and its pages, those
 * without a slot among them: after a report a caller goes on from its own lengths, table and
 * free_start of before the call.  The same inputs give the same outputs, whatever the table's
 * entries behind the cached pages hold.
 * N is at most 28672 (its prefix sums are held in shared memory), else KDA_ERR_UNSUPPORTED.
 * No output may overlap an input or another output.
 */
KDA_API kda_status kda_page_map(const int32_t* cached_lens, const int32_t* new_lens, int32_t N,
                                int32_t* block_table, int32_t max_pages, const int32_t* free_pages,
                                int64_t num_free, const int32_t* free_start, int32_t page_size,
                                int64_t num_tokens, int32_t* cu_seqlens, int32_t* seq_lens, int32_t* slot_map,
                                int32_t* positions, int32_t* free_next, cudaStream_t stream);

/*
 * Writes T tokens' keys and values into the cache.
 *  k, v      [T][Hkv][D] dtype dt, 16-byte aligned; the strides from token to token and from
 *            head to head are given in elements, multiples of 16 bytes, channels contiguous
 *  slot_map  int32[T]: slots; a negative one leaves its token out; one beyond the cache is
 *            reported and left out.  No two tokens may have the same slot.
 */
KDA_API kda_status kda_kv4_append(const void* k, const void* v, const int32_t* slot_map, int64_t T, int32_t Hkv,
                                  int32_t D, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                  int64_t v_head_stride, kda_dtype dt, void* cache, int64_t num_pages,
                                  int32_t page_size, cudaStream_t stream);

/*
 * Reads tokens back: k, v [T][Hkv][D] dtype dt, dense, get the values that the cache holds at
 * the slots; zeros for a negative slot, and for one beyond the cache, which is reported.  They
 * are exact in either type, but for 4 * 2^126 = 2^128, to which |x| from 3.5 * 2^126 on is rounded
 * and which reads back as inf.  k, v 16-byte aligned.
 */
KDA_API kda_status kda_kv4_gather(const void* cache, int64_t num_pages, int32_t page_size, const int32_t* slot_map,
                                  int64_t T, int32_t Hkv, int32_t D, kda_dtype dt, void* k, void* v,
                                  cudaStream_t stream);

/*
 * Bytes of device scratch memory for kda_kv4_attention with these sizes, or SIZE_MAX when
 * they are invalid.
 */
KDA_API size_t kda_kv4_attention_workspace_size(int64_t T, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                                int32_t max_q_len, kda_dtype dt);

/*
 * Softmax attention of each sequence's newest tokens over its cached keys and values:
 *   o = sum_p softmax_p(sm_scale q . k_p) v_p,   lse = ln sum_p exp(sm_scale q . k_p)
 * over p <= L - n + i for the i-th of the sequence's n query tokens, L cached tokens
 * (kda_kv4_append writes the new tokens' keys and values first).  A decode step has n = 1,
 * the verification of draft tokens a few, a chunk of a prompt many.  Query head h reads
 * key/value head h / (Hq / Hkv).
 *
 *  q    [T][Hq][D] dtype dt, strides in elements as for kda_kv4_append
 *  o    [T][Hq][D] dtype dt, dense, 16-byte aligned;  lse fp32 [T][Hq] or NULL
 *  block_table int32[N][max_pages], seq_lens int32[N] (L)
 *  cu_seqlens  int32[N + 1]: sequence s has the query tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1;
 *              NULL for one token each (then T = N)
 *  max_q_len   the most query tokens of a sequence (>= 1)
 *  workspace   kda_kv4_attention_workspace_size bytes, 256-byte aligned, contents do not matter
 * A query that sees no token (L = 0, or n > L and i < n - L) gets o = 0 and lse = -inf.  What
 * lies in the cache behind L, or at positions that a query does not see, never reaches its
 * result; a key or value group stored as not finite makes the results of the queries that
 * see it NaN (of a value group: its 32 channels).
 * Scores, softmax statistics and sums are fp32.  bf16 inputs multiply exactly (a row of q is
 * scaled by a power of two into fp16's range), the softmax weights enter the second product
 * as fp16, relative to the largest and to the largest scale of their 32 value channels so far;
 * fp32 inputs take both products in two fp16 parts.  bf16 calls with many query rows per
 * key/value head (max_q_len Hq / Hkv) run a kernel that also holds keys and values in fp16,
 * keys relative to the largest scale of 128 tokens, values to that of their 32 channels so far:
 * exact for groups down to 2^-21 of it.
 * One kernel runs the whole call, chosen by the numbers of tokens, heads and sequences; a step with
 * long chunks beside many single tokens may be faster as a call for each kind.
 * A length beyond the table, a page beyond the cache, a cu_seqlens that decreases, does not
 * begin at 0 or passes T, and a sequence of more than max_q_len tokens are reported; the
 * outputs of such a sequence are unspecified, no access leaves the arrays.
 * Query tokens of no sequence keep their o and lse.  Calls in flight at once need a workspace
 * each.
 * KDA_ERR_UNSUPPORTED: D not 64 or 128; N beyond 65535; Hq / Hkv beyond 128.
 */
KDA_API kda_status kda_kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* cache,
                                     int64_t num_pages, int32_t page_size, const int32_t* block_table,
                                     int32_t max_pages, const int32_t* seq_lens, const int32_t* cu_seqlens,
                                     int64_t T, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q_len,
                                     float sm_scale, kda_dtype dt, void* o, float* lse, void* workspace,
                                     size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_KDA_KV4_H */
