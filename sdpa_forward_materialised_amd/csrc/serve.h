// Internal interface of the serving operators (attention over packed prompts
// without the probability map, the attention weight each key received, the
// paged 8-bit cache). Not installed; see include/sdpa_math.h.
#pragma once

#include <cstddef>
#include <cstdint>

namespace sdpa {

// Packed sequences: token-major tensors, strides in elements ordered
// (head, token). B sequences whose token ranges are cu_q[b] .. cu_q[b+1] and
// cu_k[b] .. cu_k[b+1]; max_q and max_k bound their lengths.
struct PackArgs {
    const void* q;
    const void* k;
    const void* v;
    void* o;
    float* lse;       // written by the prompt kernel, read by the key-weight kernel
    float* w;         // key weights [B, Hkv, w_cols]
    float* ws;        // key weights: partial sums [split][B][Hkv][max_k]
    int64_t q_s[2], k_s[2], v_s[2], o_s[2], l_s[2], w_s[2];  // w_s: (batch, head)
    const int* cu_q;
    const int* cu_k;
    int Tq, Tkv;
    int B, Hq, Hkv, group;
    int max_q, max_k;
    int causal;           // 0 none, 1 top-left, 2 bottom-right (per sequence)
    int o_vec;            // rows of O take aligned 16-byte stores
    int q_mul;            // 1, or the factor -1 or 0 that the queries are taken with
    float scale_log2;     // |scale| * log2(e) (1 when the scale is 0)
    int groups;           // prompt: key groups (1, 2 or 4)
    int n_blk;            // blocks per (sequence, head)
    int n_split;          // key weights: query ranges per key block and query head
    int split_rows;       // key weights: queries of a range
    int w_cols;           // key weights: row length (zeros past a sequence's keys)
    uint32_t q_ext, k_ext, v_ext, o_ext, l_ext;  // byte extents of one (sequence, head) slice
};

constexpr int PROMPT_ROWS = 128;  // query rows of a prompt kernel's workgroup of one or two key groups; of four, a quarter
int launch_prompt(int dtype, int D, const PackArgs& a, void* stream);
constexpr int KEY_WEIGHT_KEYS = 128;  // keys of one workgroup of the key-weight kernel
int launch_key_weights(int dtype, int D, const PackArgs& a, void* stream);

// The paged 8-bit cache. k [n_pages, Hkv, page, D] and v [n_pages, Hkv, D, page]
// hold e4m3 codes, ks and vs [n_pages, Hkv] their scales (powers of two); all
// contiguous. A row of the page table lists a sequence's pages in order.
struct CacheArgs {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int n_pages, page, page_log2, Hkv, D;
    const int* table;
    int64_t table_s;      // elements between table rows
    int max_pages;        // pages a row lists
    const int* lens;      // tokens held (append: before the call)
    int B;
    const int* cu;        // new tokens of sequence b: cu[b] .. cu[b+1]
    int T;                // packed new tokens
    int max_new;          // bound of a sequence's new tokens
    // append: the new keys and values, strides (head, token)
    const void* nk;
    const void* nv;
    int64_t nk_s[2], nv_s[2];
    int slots;            // pages a sequence's new tokens may touch
    // attention
    const void* q;
    void* o;
    float* lse;
    int64_t q_s[2], o_s[2], l_s[2];
    int Hq, group;
    int max_kv;           // bound of the lengths
    int causal;
    int q_mul;            // as PackArgs
    float scale_log2;
    int row_blocks;       // blocks of query rows per (sequence, key head)
    int rows;             // query rows per (sequence, key head), at most: group * max_new
    int n_ranges;         // key ranges
    int range_keys;       // keys of a range (a multiple of 256)
    float2* ws_ml;        // [B][Hkv][rows][n_ranges] row reference and sum
    float* ws_o;          // [B][Hkv][rows][n_ranges][D] partial sums
    float* ws_t;          // [B][Hkv][rows][t_cols] base-2 scores, when weights are gathered
    int t_cols;
    const float* w_in;    // weights [B, Hkv, w_cols], strides (batch, head)
    float* w_out;
    int64_t wi_s[2], wo_s[2];
    int w_cols;
    // eviction
    const int* to;        // pages the kept tokens move to
    int64_t to_s;
    int to_pages;
    int budget, recent;
    int* kept;            // [B, Hkv, budget]
    int* new_lens;        // [B]
};

int launch_cache_append(int dtype, const CacheArgs& a, void* stream);
int launch_cache_attention(int dtype, const CacheArgs& a, void* stream);
int launch_cache_evict(const CacheArgs& a, void* stream);
constexpr int CACHE_MAX_RANGES = 512;  // key ranges of a call, at most
// query rows of one workgroup of the attention kernel, given the rows of a call
inline int cache_block_rows(int rows) { return rows <= 16 ? 16 : 32; }

}  // namespace sdpa
