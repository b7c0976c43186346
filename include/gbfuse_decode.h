/*
 * gbfuse_decode -- the operators of a decode step around the paged K/V cache
 * that gbf_qkv_split_norm_rope writes: block tables and slot maps from request
 * lengths, attention of one new token per request, sampling of the next token.
 * Part of libgbfuse.so; C ABI, GB300 (sm_103a).
 *
 * The conventions are gbfuse.h's: caller-owned buffers, work enqueued on
 * `stream` without synchronising, gbf_status return values with gbf_last_error()
 * for the message, data-dependent faults caught on the device, skipped and
 * reported by gbf_device_status() (GBF_EDEVICE).  No call keeps state between
 * calls; every call may be captured into a CUDA graph, allows programmatic
 * dependent launch, and gives the same bits whenever it is given the same
 * inputs.  Index tensors are int32.
 *
 * The paged cache: k_cache, v_cache are [cache_rows, n_kv_heads, head_dim]; block
 * i is rows i * block_size ... (i + 1) * block_size - 1; position p of request b
 * lives in row block_table[b, p / block_size] * block_size + p % block_size.
 */
#ifndef GBFUSE_DECODE_H
#define GBFUSE_DECODE_H

#include "gbfuse.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gbfd_paged_slots -- the block tables, slot maps and positions of one step.
 *
 * Request b holds ctx_lens[b] cached tokens and brings new_lens[b] more (1 for
 * a decode row, a prompt's length, 0 for none; negative: it has ended).  In
 * request order:
 *   - the blocks it lacks, ceil((ctx + new) / bs) - ceil(ctx / bs), are taken
 *     from the front of a ring of free block ids and entered in its row of
 *     block_table;
 *   - an ended request's ceil(ctx / bs) blocks go back behind the ring's end;
 *   - token i of request b, the packed token start[b] + i, gets
 *     pos = ctx + i and slot = block_table[b, pos / bs] * bs + pos % bs.
 * seq_lens[b] = ctx + new (0 when it has ended); start[b] = tokens of the
 * requests before b (start[batch] = all; sums past 2^31 - 1 stay there).  The slots and positions are what
 * gbf_qkv_split_norm_rope takes, seq_lens and block_table what
 * gbfd_paged_attention takes.
 *
 * ctx_lens, new_lens: device int32 [batch]; block_table: device int32, batch
 * rows of max_blocks entries, table_stride entries apart, updated in place;
 * free_ring: device int32 [num_blocks], a ring buffer, updated in place; ring:
 * device int32 [2], the ring's first entry and how many are free; ring_out:
 * the same after the call; slots, pos: device int32 [tokens]; start: device
 * int32 [batch + 1] or NULL.  Entries of slots and pos behind the last token,
 * and table entries no new block goes to, keep their values.  seq_lens may
 * equal ctx_lens and ring_out may equal ring (in place); with separate ones a
 * repeated call writes the same values again.
 *
 * A request is refused -- its slots are -1, its seq_lens entry stays ctx, it
 * takes no block, the device error word is set -- when its length is negative
 * or does not fit its table row (or int32), or when the free blocks run out before it
 * (all later requests that need a block are then refused too).  A ctx that is itself
 * out of range gives the nearest length that is not: 0, or max_blocks * block_size.  A block id
 * outside [0, num_blocks) sets the error word and gives slot -1; an ended request's goes
 * back into the ring as it is, and sets the error word again, with slot -1, for whoever
 * takes it from there (ids are looked at where they are used, not sought out).  A ring state
 * out of range sets it, is passed on to ring_out as it is, and has no free block;
 * with one, or where the ring would come to hold more than num_blocks, nothing is
 * given back: ended requests that hold blocks are refused.  More packed tokens than `tokens`
 * set the error word too; the excess is not written.
 * Requires batch <= 8192, block_size >= 1, num_blocks * block_size < 2^31.
 * batch == 0 enqueues nothing and writes nothing.
 */
GBF_API int gbfd_paged_slots(const int32_t* ctx_lens, const int32_t* new_lens, int64_t batch, int32_t* block_table,
                             int64_t table_stride, int64_t max_blocks, int block_size, int32_t* free_ring,
                             const int32_t* ring, int64_t num_blocks, int32_t* seq_lens, int32_t* ring_out,
                             int32_t* slots, int32_t* pos, int64_t tokens, int32_t* start, void* stream);

/*
 * gbfd_paged_attention -- attention of one new token per request over its
 * cached positions:  s_j = scale * q . k_j,  out = sum_j softmax(s)_j v_j,
 * lse = ln sum_j exp(s_j), for j in [0, len) or, with window > 0, the last
 * `window` of them (len counts the new token, whose K and V are in the cache).
 * Query head h reads KV head h / (n_q_heads / n_kv_heads).  A request of
 * length 0 gives out = 0 and lse = -inf, and so does one with no score above -inf; a
 * score that is NaN or +inf gives out = lse = NaN, an infinite value in V an out that is
 * not finite.  Float32 scores, sums and outputs.
 *
 * q: device bf16 [batch, n_q_heads, head_dim]; k_cache, v_cache: device bf16
 * [cache_rows, n_kv_heads, head_dim]; block_table: device int32, batch rows of
 * max_blocks entries, table_stride entries apart; seq_lens: device int32
 * [batch]; out: device bf16 [batch, n_q_heads, head_dim], or with out_scale > 0
 * device uint8 E4M3 codes of out / out_scale (saturated to +-448), as
 * gbf_linear_fp8_act takes them with x_scale = out_scale; out_scale = 0: bf16.
 * lse: device float32 [batch, n_q_heads] or NULL.  workspace: device memory of
 * gbfd_paged_attention_workspace() bytes, whose contents need not be set and do
 * not outlive the call; calls that may run at the same time need their own.
 * A length outside [0, max_blocks * block_size] (or above 2^31 - 17) is clamped, and a position
 * whose block id lies outside the cache is left out; both set the device error
 * word.  Rows of the cache no position refers to are not read.
 * Requires head_dim % 16 == 0, head_dim <= 256, n_q_heads % n_kv_heads == 0,
 * cache_rows < 2^31, batch <= 2^30, 16-byte aligned q, k_cache, v_cache, out, workspace; scale
 * > 0 and finite.  batch == 0 enqueues nothing.  out and lse may not overlap each other or an input.
 * How the work is split follows from batch, heads, window and max_blocks * block_size, not from the lengths, which only
 * the device knows: for few or short requests, a max_blocks (or a window) no wider than they need saves 2 to 8 us.
 */
GBF_API int gbfd_paged_attention(const void* q, const void* k_cache, const void* v_cache, int64_t cache_rows,
                                 const int32_t* block_table, int64_t table_stride, int64_t max_blocks,
                                 int block_size, const int32_t* seq_lens, int64_t batch, int n_q_heads,
                                 int n_kv_heads, int head_dim, float scale, int64_t window, void* out,
                                 float out_scale, float* lse, void* workspace, int64_t workspace_bytes,
                                 void* stream);

/* Bytes of workspace gbfd_paged_attention needs for any batch, lengths and
 * block size with these heads (0 for heads it does not support). */
GBF_API int64_t gbfd_paged_attention_workspace(int n_q_heads, int n_kv_heads, int head_dim);

/*
 * gbfd_sample_tokens -- the next token of each request.
 *
 * With w_i = exp((l_i - max l) / T), and candidates ordered by logit (larger
 * first; equal logits by index, lower first):
 *   top-k keeps the first k (k <= 0: all);
 *   top-p keeps, of those, each candidate before which less than top_p of
 *     their mass lies (>= 1: all; the first is always kept);
 *   min-p keeps, of those, the ones with w_i >= min_p (<= 0: all);
 *   the token is, in index order, the first at which the running kept mass
 *     passes u times the kept mass.
 * Temperatures below 1e-30 count as 1e-30.  T = 0 takes the largest logit (the lowest index of equals) whatever else is
 * set.  Weights are 43-bit fixed-point numbers and their sums exact, so the
 * token does not depend on the order of summation.  logprob = ln(w / kept mass)
 * of the token, 0 for T = 0.  -inf and NaN logits are no candidates.
 *
 * logits: device bf16 (f32 = 0) or float32 (f32 = 1) [batch, vocab], rows
 * logits_stride elements apart (>= vocab, any alignment of a row; the first
 * 16-byte aligned); uniform: device float32 [batch] in [0, 1); temperature, top_p,
 * min_p: device float32 [batch] or NULL (1, off, off); top_k: device int32
 * [batch] or NULL (off); tokens: device int32 [batch]; logprob: device float32
 * [batch] or NULL.
 * A temperature that is negative or not finite, a NaN top_p, a min_p that is
 * NaN or above 1, a uniform outside [0, 1) and a row without a candidate give
 * token -1 and logprob NaN and set the device error word.
 * Requires 1 <= vocab <= 2^20.
 */
GBF_API int gbfd_sample_tokens(const void* logits, int f32, int64_t batch, int64_t vocab, int64_t logits_stride,
                               const float* uniform, const float* temperature, const int32_t* top_k,
                               const float* top_p, const float* min_p, int32_t* tokens, float* logprob,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBFUSE_DECODE_H */
