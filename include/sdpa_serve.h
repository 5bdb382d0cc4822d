/*
 * sdpa_serve — attention for serving on AMD Instinct MI355X (gfx950): packed
 * prompts without the probability map, the attention weight that each key
 * received, and a paged 8-bit key/value cache with the attention that reads
 * it and the eviction that cuts it.
 *
 * A server's path: sdpa_prompt_fwd over the new prompts, sdpa_key_weights for
 * the weights an eviction goes by, sdpa_cache_append of their keys and values,
 * sdpa_cache_evict where a sequence is over its budget, then for every step
 * sdpa_cache_append of the new tokens and sdpa_cache_attention over the cache,
 * which also adds to the weights.
 *
 * Conventions of every call are those of sdpa_math.h: descriptors with sizes
 * and strides in elements, device pointers, a HIP stream, validation before
 * any launch (on error nothing is enqueued and sdpa_math_last_error() tells
 * why). The library allocates nothing, never synchronises, reads device data
 * only on the device and keeps nothing between calls; no launch is a memset
 * and no result depends on an order of atomics, so calls can be recorded into
 * HIP graphs and repeat bit for bit. A workspace is scratch for its call:
 * calls that share one must be ordered (two graphs with one workspace must
 * not run at once). Lengths, page tables and rows of weights go up to 2^30
 * tokens.
 */
#ifndef SDPA_SERVE_H
#define SDPA_SERVE_H

#include "sdpa_math.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * sdpa_prompt_fwd — attention over packed sequences, output and row
 * log-sum-exp only: sdpa_math_fwd_varlen without its probability map (whose
 * Tq * Hq * max_seqlen_kv elements a long prompt cannot afford), in one sweep
 * over the keys.
 * q [Tq, Hq, D]; k [Tkv, Hkv, D]; v [Tkv, Hkv, D]: f32, f16 or bf16; D 32, 64
 *      or 128
 * cu_seqlens_q, cu_seqlens_kv, n_seqs, max_seqlen_q, max_seqlen_kv,
 * is_causal (0, 1 top-left, 2 bottom-right, per sequence), scale, enable_gqa
 *      as sdpa_math_fwd_varlen
 * out  [Tq, Hq, D] q dtype; lse [Tq, Hq] f32 (natural logarithm); a row that
 *      keeps no key gives 0 and -inf; tokens of no sequence are not written
 * O is accumulated in float32 from probabilities rounded to q's 16-bit type
 * (relative to a running row reference) and rounded once more to q's type;
 * float32 calls round nothing. A key or value that a row does not keep has no
 * effect on it, whatever it holds.
 * Layout as sdpa_math_fwd_varlen.
 */
sdpa_status_t sdpa_prompt_fwd(const sdpa_tensor_t* q, const sdpa_tensor_t* k, const sdpa_tensor_t* v,
                              const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv, int64_t n_seqs,
                              int64_t max_seqlen_q, int64_t max_seqlen_kv, int is_causal, float scale,
                              int enable_gqa, sdpa_tensor_t* out, sdpa_tensor_t* lse, void* hip_stream);

/*
 * sdpa_key_weights — the attention weight every key received:
 *   weights[b, h', j] = sum over the query heads h of key head h' and the
 *                       rows i of sequence b that keep key j of
 *                       exp(scale * q_i . k_j - lse_i)
 * (the column sums of the probabilities that sdpa_math_fwd_varlen writes,
 * without writing them).
 * lse     [Tq, Hq] f32: of sdpa_prompt_fwd or sdpa_math_fwd_varlen on the same
 *         q, k, is_causal and scale; rows whose lse is -inf or +inf add nothing
 * weights [n_seqs, Hkv, max_seqlen_kv] f32, last dim contiguous: zeros past
 *         each sequence's keys
 * workspace  at least sdpa_key_weights_workspace_bytes bytes, 16-byte aligned
 * Other arguments as sdpa_prompt_fwd. The sum's order is fixed.
 */
sdpa_status_t sdpa_key_weights(const sdpa_tensor_t* q, const sdpa_tensor_t* k, const sdpa_tensor_t* lse,
                               const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv, int64_t n_seqs,
                               int64_t max_seqlen_q, int64_t max_seqlen_kv, int is_causal, float scale,
                               int enable_gqa, sdpa_tensor_t* weights, void* workspace, size_t workspace_bytes,
                               void* hip_stream);

/* Bytes of workspace for sdpa_key_weights (float32 partial sums of every key
 * for each query head and range of rows). *bytes is 0 on error. */
sdpa_status_t sdpa_key_weights_workspace_bytes(const sdpa_tensor_t* q, const sdpa_tensor_t* k, int64_t n_seqs,
                                               int64_t max_seqlen_q, int64_t max_seqlen_kv, int enable_gqa,
                                               size_t* bytes);

/*
 * The paged 8-bit cache: pages of P tokens (P 16, 32, 64 or 128).
 *   k        [n_pages, Hkv, P, D] e4m3 codes
 *   v        [n_pages, Hkv, D, P] e4m3 codes, the tokens of a page innermost
 *   k_scale, v_scale [n_pages, Hkv] f32: a code stands for its e4m3 value times
 *            its page's and head's scale, a power of two
 * All contiguous; D 32, 64 or 128; n_pages at least 1. A page belongs to one
 * sequence while it is written; sequences may share pages that are only read.
 *
 * A page table is a device int32 array [n_seqs, max_pages] (row stride
 * table_stride elements, max_pages at least): entry p of a row is the page of
 * tokens p P .. p P + P - 1. kv_lens is a device int32 array [n_seqs] of
 * lengths, cut to [0, max_pages P]. Only entries that hold tokens are read. A
 * token whose entry is outside [0, n_pages) is not written, and not seen.
 */
typedef struct {
    sdpa_tensor_t k, v, k_scale, v_scale;
} sdpa_cache_t;

/*
 * sdpa_cache_append — write new tokens behind those a sequence holds.
 * k, v  [T, Hkv, D] f16 or bf16, 16-byte aligned rows; tokens cu_seqlens[b] ..
 *       cu_seqlens[b + 1] (at most max_new of them) go to positions
 *       kv_lens[b] .. of sequence b; tokens past its pages are not written.
 *       kv_lens is not changed.
 * For every page, head and k or v: a page that starts with a new token takes
 * the smallest power of two s >= 2^-126 with max |x| <= 448 s over its new
 * finite elements; a page that already holds tokens takes the larger of that
 * and its scale, and its held codes are rounded to the new scale. Codes are
 * x / s rounded to nearest even; infinities and NaN become NaN and do not
 * count for the scale. Slots that receive no token keep their codes.
 */
sdpa_status_t sdpa_cache_append(const sdpa_cache_t* cache, const sdpa_tensor_t* k, const sdpa_tensor_t* v,
                                const int32_t* page_table, int64_t n_seqs, int64_t max_pages,
                                int64_t table_stride, const int32_t* kv_lens, const int32_t* cu_seqlens,
                                int64_t max_new, void* hip_stream);

/*
 * sdpa_cache_attention — attention of each sequence's last tokens over its
 * cached keys and values.
 * q     [T, Hq, D] f16 or bf16 (16-byte aligned rows): tokens cu_seqlens_q[b]
 *       .. cu_seqlens_q[b + 1] (at most max_seqlen_q) of sequence b, which are
 *       the last of its kv_lens[b] cached tokens (append them first)
 * max_kv  bound of the lengths (the launch covers max_kv keys; longer
 *       sequences are cut to it, the table's capacity at most)
 * is_causal  nonzero: new token i of n keeps keys j <= kv_lens[b] - n + i
 *       (bottom-right); 0: every key
 * weights, weights_out  NULL, or f32 [n_seqs, Hkv, W], last dim contiguous:
 *       weights_out = weights + the sum over the key head's query heads and
 *       the new tokens of each key's probability (keys at and past W are not
 *       counted). They may be the same tensor; otherwise they do not overlap.
 * out   [T, Hq, D] q dtype; lse [T, Hq] f32; a row that keeps no key gives 0
 *       and -inf; tokens of no sequence are not written
 * workspace  at least sdpa_cache_attention_workspace_bytes bytes, 16-byte
 *       aligned (NULL when that is 0)
 * O is accumulated in float32 from probabilities carried with 16 bits, and
 * rounded once. A token that a row does not keep has no effect on it.
 */
sdpa_status_t sdpa_cache_attention(const sdpa_tensor_t* q, const sdpa_cache_t* cache, const int32_t* page_table,
                                   int64_t n_seqs, int64_t max_pages, int64_t table_stride,
                                   const int32_t* kv_lens, const int32_t* cu_seqlens_q, int64_t max_seqlen_q,
                                   int64_t max_kv, int is_causal, float scale, int enable_gqa,
                                   const sdpa_tensor_t* weights, sdpa_tensor_t* weights_out, sdpa_tensor_t* out,
                                   sdpa_tensor_t* lse, void* workspace, size_t workspace_bytes, void* hip_stream);

/* Bytes of workspace for sdpa_cache_attention: row statistics and float32
 * partial outputs of every key range, and, when weights are gathered, the
 * float32 scores. `gather` is nonzero when weights are passed. */
sdpa_status_t sdpa_cache_attention_workspace_bytes(const sdpa_tensor_t* q, const sdpa_cache_t* cache,
                                                   int64_t n_seqs, int64_t max_pages, int64_t max_seqlen_q,
                                                   int64_t max_kv, int enable_gqa, int gather, size_t* bytes);

/*
 * sdpa_cache_evict — keep at most `budget` tokens of every sequence and key
 * head: its last `recent` tokens (0 <= recent <= budget) and, of the others,
 * those with the largest weights, the lowest position among equals (NaN counts
 * as larger than +inf). The kept tokens move, in order, to the pages of
 * to_table (int32 [n_seqs, to_pages], at least budget tokens; distinct pages
 * that hold no token of a sequence in this call); the present pages are left
 * as they are. A sequence within the budget moves whole. Every page moved to
 * takes the largest scale of its tokens, codes are rounded to it, and its
 * slots past the kept tokens hold zeros.
 * weights, weights_out  f32 [n_seqs, Hkv, W] as in sdpa_cache_attention (the
 *       lengths are cut to W): weights_out holds the kept tokens' weights in
 *       order and zeros behind them
 * kept      int32 [n_seqs, Hkv, budget], contiguous: positions kept, -1 behind
 * new_lens  int32 [n_seqs]: min(length, budget); not kv_lens itself, which every head reads
 */
sdpa_status_t sdpa_cache_evict(const sdpa_cache_t* cache, const int32_t* page_table, int64_t n_seqs,
                               int64_t max_pages, int64_t table_stride, const int32_t* kv_lens,
                               const sdpa_tensor_t* weights, sdpa_tensor_t* weights_out, int64_t budget,
                               int64_t recent, const int32_t* to_table, int64_t to_pages, int64_t to_stride,
                               int32_t* kept, int32_t* new_lens, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SDPA_SERVE_H */
