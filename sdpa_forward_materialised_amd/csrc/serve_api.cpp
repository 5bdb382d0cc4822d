// Host side of the serving operators' C ABI (include/sdpa_serve.h): argument
// validation, launch planning and the launches. No device memory is allocated
// here, nothing is synchronised and no device data is read.

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <initializer_list>

#include "api_checks.h"
#include "sdpa_internal.h"
#include "sdpa_serve.h"
#include "serve.h"

using namespace sdpa_api;

namespace {

#define TRY(expr)                              \
    do {                                       \
        const sdpa_status_t st_ = (expr);      \
        if (st_ != SDPA_OK) return st_;        \
    } while (0)

sdpa_status_t launched(int err) {
    if (err != 0)
        return fail(SDPA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(static_cast<hipError_t>(err)));
    return SDPA_OK;
}

bool head_dim_ok(int64_t D) { return D == 32 || D == 64 || D == 128; }

sdpa_status_t check_f32(const sdpa_tensor_t* t, const char* name, int ndim, const int64_t* want) {
    TRY(check_tensor(t, name, ndim));
    if (t->dtype != SDPA_F32) return fail(SDPA_ERR_INVALID_ARG, "%s must be f32", name);
    return check_dims(t, name, want, ndim);
}

// |scale| in base 2 and the factor (1, -1, 0) that the queries are taken with:
// the kernels then take maxima before they scale.
sdpa_status_t split_scale(float scale, float* scale_log2, int* mul) {
    if (!std::isfinite(scale)) return fail(SDPA_ERR_INVALID_ARG, "scale must be finite");
    *mul = scale > 0.0f ? 1 : scale < 0.0f ? -1 : 0;
    *scale_log2 = scale == 0.0f ? 1.0f : std::fabs(scale) * 1.4426950408889634f;
    return SDPA_OK;
}

sdpa_status_t check_heads(int64_t Hq, int64_t Hkv, int enable_gqa) {
    if (Hkv <= 0 || Hq % Hkv != 0)
        return fail(SDPA_ERR_INVALID_ARG, "query heads (%lld) are not a multiple of key/value heads (%lld)",
                    (long long)Hq, (long long)Hkv);
    if (Hq != Hkv && !enable_gqa)
        return fail(SDPA_ERR_INVALID_ARG, "Hq (%lld) != Hkv (%lld) needs enable_gqa", (long long)Hq, (long long)Hkv);
    return SDPA_OK;
}

// (head, token) strides of a token-major tensor
void pack_strides(const sdpa_tensor_t* t, int64_t* s) {
    s[0] = eff_stride(t, 1);
    s[1] = eff_stride(t, 0);
}

// byte extent of one (sequence, head) slice of at most `rows` tokens
sdpa_status_t pack_extent(const sdpa_tensor_t* t, const char* name, int64_t rows, int64_t cols, uint32_t* ext) {
    const int64_t pitch = eff_stride(t, 0);
    const int64_t e = rows > 0 ? ((rows - 1) * pitch + cols) * elt_size(t->dtype) : 0;
    if (pitch < 0 || e >= (int64_t(1) << 30))
        return fail(SDPA_ERR_UNSUPPORTED, "one (sequence, head) slice of %s spans 1 GiB or more", name);
    *ext = (uint32_t)e;
    return SDPA_OK;
}

// Workgroups of a launch, a product of factors >= 0.
sdpa_status_t grid_ok(std::initializer_list<int64_t> factors) {
    int64_t n = 1;
    for (int64_t f : factors)
        if (__builtin_mul_overflow(n, f, &n) || n > INT32_MAX) return fail(SDPA_ERR_UNSUPPORTED, "grid too large");
    return SDPA_OK;
}

// Lengths that the kernels' 32-bit positions, rounded up to tiles and ranges, can hold.
constexpr int64_t kMaxTokens = int64_t(1) << 30;

// Checks q, k and the sequence bounds; fills what both packed operators share.
sdpa_status_t pack_args(const sdpa_tensor_t* q, const sdpa_tensor_t* k, int64_t n_seqs, int64_t max_q, int64_t max_k,
                        int enable_gqa, sdpa::PackArgs* a) {
    TRY(check_tensor(q, "q", 3));
    TRY(check_tensor(k, "k", 3));
    if (q->dtype != SDPA_F32 && q->dtype != SDPA_F16 && q->dtype != SDPA_BF16)
        return fail(SDPA_ERR_INVALID_ARG, "q dtype %s is not f32, f16 or bf16", dtype_name(q->dtype));
    if (k->dtype != q->dtype) return fail(SDPA_ERR_INVALID_ARG, "q, k, v dtypes differ");
    if (n_seqs < 0 || max_q < 0 || max_k < 0)
        return fail(SDPA_ERR_INVALID_ARG, "sequence count and maximum lengths must be non-negative");
    if (k->sizes[2] != q->sizes[2]) return fail(SDPA_ERR_INVALID_ARG, "q and k head dims differ");
    TRY(check_heads(q->sizes[1], k->sizes[1], enable_gqa));
    if (q->sizes[0] > INT32_MAX || k->sizes[0] > INT32_MAX || max_q > INT32_MAX || max_k > INT32_MAX ||
        n_seqs > INT32_MAX || q->sizes[1] > INT32_MAX)
        return fail(SDPA_ERR_UNSUPPORTED, "sizes beyond 2^31 are not supported");
    if (!head_dim_ok(q->sizes[2]))
        return fail(SDPA_ERR_UNSUPPORTED, "head dim %lld is not implemented (32, 64, 128)", (long long)q->sizes[2]);
    for (const sdpa_tensor_t* t : {q, k})
        if (numel(t) > 0 && !rows_aligned(t, 16))
            return fail(SDPA_ERR_UNSUPPORTED, "q, k, v need 16-byte aligned bases and 16-byte multiple strides");
    std::memset(a, 0, sizeof *a);
    a->q = q->data;
    a->k = k->data;
    pack_strides(q, a->q_s);
    pack_strides(k, a->k_s);
    a->Tq = (int)q->sizes[0];
    a->Tkv = (int)k->sizes[0];
    a->B = (int)n_seqs;
    a->Hq = (int)q->sizes[1];
    a->Hkv = (int)k->sizes[1];
    a->group = a->Hq / a->Hkv;
    a->max_q = (int)std::min<int64_t>(max_q, a->Tq);
    a->max_k = (int)std::min<int64_t>(max_k, a->Tkv);
    if (a->max_q > kMaxTokens || a->max_k > kMaxTokens)
        return fail(SDPA_ERR_UNSUPPORTED, "sequences of more than 2^30 tokens are not supported");
    TRY(pack_extent(q, "q", a->max_q, q->sizes[2], &a->q_ext));
    return pack_extent(k, "k", a->max_k, k->sizes[2], &a->k_ext);
}

sdpa_status_t check_cu(int64_t n_seqs, const void* cu_q, const void* cu_k, int is_causal) {
    if (n_seqs > 0 && (!cu_q || !cu_k)) return fail(SDPA_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_kv are required");
    if (is_causal < 0 || is_causal > 2) return fail(SDPA_ERR_INVALID_ARG, "is_causal must be 0, 1 or 2");
    return SDPA_OK;
}

// Prompt attention: key groups (a wave's chain of tiles is shorter by as
// much), where blocks of 128 rows leave wave slots empty.
// float32: always four (rows in blocks of 32).
// 16 bits, four: up to 256 blocks of 128 rows and D below 128. Measured, four
// groups and two: 1024 + 700 tokens x 8 heads of 64 (128 blocks) 10.7 and 15.3
// us, 6000 x 4 of 64 (188) 40.9 and 55.9, 2048 and less ragged ones x 4 of 64
// (256) 24.8 and 24.5, of 32 14.9 and 20.2, 1024 and less ragged ones x 8 of 64
// (320) 17.3 and 16.2; 1024 x 4 x 16 of 64 (512) 31 and 23. At D = 128 a CU
// holds one such workgroup: 20.1 and 21.9, 50 and 35 for 128 and 256 blocks.
// Two: where one group a block leaves slots empty (512 workgroups of four waves
// fill two slots of every SIMD) and the chain is long enough to pay for the
// join. Measured, one group and two: 4096 tokens x 16 heads of 128 (512 blocks)
// 91 and 86 us, the 320 blocks above 18.5 and 16.2; 2048 x 4 x 16 heads of 64
// (1024 blocks) 50 and 61, 512 + 300 tokens x 16 heads of 128 13.7 and 14.3.
int prompt_groups(const sdpa::PackArgs& a, int dtype, int64_t D) {
    if (dtype == SDPA_F32) return 4;
    const int64_t blocks = (int64_t)a.B * a.Hq * cdiv(a.max_q, sdpa::PROMPT_ROWS);
    if (D < 128 && blocks <= 256) return 4;
    return blocks <= 512 && a.max_k >= 768 ? 2 : 1;
}

// Key weights: ranges of one query head's rows, enough for 2048 workgroups
// (two rounds of the 1024 resident ones: the triangle of a causal call needs
// them to balance), of 256 rows at least; of fewer, down to 64, only for the
// first 512 workgroups. Measured with 1024, 2048 and 4096 workgroups:
// 2048 + 1531 tokens x 16 heads of 128 38.7, 32.1 and 36.7 us, 8191 tokens x 16
// heads of 64 136, 120 and 128 us; with at least 256, 128 and 64 rows: 1000
// tokens x 2 heads of 128 13.1, 11.7 and 11.5 (float32: 45, 30 and 26), but
// 1024 + 700 x 8 heads of 128 14.5, 17.6 and 21.8.
void plan_key_weights(sdpa::PackArgs* a) {
    a->n_blk = (int)cdiv(a->max_k, sdpa::KEY_WEIGHT_KEYS);
    const int64_t blocks = std::max<int64_t>(1, (int64_t)a->B * a->Hq * a->n_blk);
    const int64_t want = std::max<int64_t>({1, std::min<int64_t>(cdiv(2048, blocks), a->max_q / 256),
                                            std::min<int64_t>(cdiv(512, blocks), a->max_q / 64)});
    a->split_rows = (int)std::max<int64_t>(64, cdiv(cdiv(a->max_q, want), 64) * 64);
    a->n_split = (int)std::max<int64_t>(1, cdiv(a->max_q, a->split_rows));
}

int64_t key_weight_ws(const sdpa::PackArgs& a) { return (int64_t)a.group * a.n_split * a.B * a.Hkv * a.max_k * 4; }

// ---------------------------------------------------------------- the cache

sdpa_status_t cache_args(const sdpa_cache_t* c, int64_t n_seqs, int64_t max_pages, sdpa::CacheArgs* a) {
    if (!c) return fail(SDPA_ERR_INVALID_ARG, "cache is NULL");
    const sdpa_tensor_t* t[4] = {&c->k, &c->v, &c->k_scale, &c->v_scale};
    const char* names[4] = {"cache k", "cache v", "cache k_scale", "cache v_scale"};
    for (int i = 0; i < 4; ++i) {
        TRY(check_tensor(t[i], names[i], i < 2 ? 4 : 2));
        if (t[i]->dtype != (i < 2 ? SDPA_E4M3 : SDPA_F32))
            return fail(SDPA_ERR_INVALID_ARG, "%s has dtype %s, expected %s", names[i], dtype_name(t[i]->dtype),
                        i < 2 ? "e4m3" : "f32");
        int64_t run = 1;
        for (int d = t[i]->ndim - 1; d >= 0; --d) {
            if (t[i]->sizes[d] != 1 && t[i]->strides[d] != run)
                return fail(SDPA_ERR_UNSUPPORTED, "%s must be contiguous", names[i]);
            run *= t[i]->sizes[d];
        }
    }
    const int64_t n = c->k.sizes[0], H = c->k.sizes[1], P = c->k.sizes[2], D = c->k.sizes[3];
    const int64_t wv[4] = {n, H, D, P}, wsc[2] = {n, H};
    TRY(check_dims(&c->v, "cache v", wv, 4));
    TRY(check_dims(&c->k_scale, "cache k_scale", wsc, 2));
    TRY(check_dims(&c->v_scale, "cache v_scale", wsc, 2));
    if (P != 16 && P != 32 && P != 64 && P != 128)
        return fail(SDPA_ERR_UNSUPPORTED, "pages of %lld tokens are not implemented (16, 32, 64, 128)", (long long)P);
    if (!head_dim_ok(D)) return fail(SDPA_ERR_UNSUPPORTED, "head dim %lld is not implemented (32, 64, 128)", (long long)D);
    if (n < 1 || H < 1) return fail(SDPA_ERR_INVALID_ARG, "the cache holds no pages or no heads");
    if (n > INT32_MAX || H > INT32_MAX || n_seqs > INT32_MAX || max_pages > INT32_MAX / P)
        return fail(SDPA_ERR_UNSUPPORTED, "sizes beyond 2^31 are not supported");
    if (max_pages > kMaxTokens / P)
        return fail(SDPA_ERR_UNSUPPORTED, "page tables of more than 2^30 tokens are not supported");
    if (n_seqs < 0 || max_pages < 0) return fail(SDPA_ERR_INVALID_ARG, "sequence and page counts must be non-negative");
    if (reinterpret_cast<uintptr_t>(c->k.data) % 16 || reinterpret_cast<uintptr_t>(c->v.data) % 16)
        return fail(SDPA_ERR_UNSUPPORTED, "cache k and v need 16-byte aligned bases");
    std::memset(a, 0, sizeof *a);
    a->k = static_cast<uint8_t*>(c->k.data);
    a->v = static_cast<uint8_t*>(c->v.data);
    a->ks = static_cast<float*>(c->k_scale.data);
    a->vs = static_cast<float*>(c->v_scale.data);
    a->n_pages = (int)n;
    a->Hkv = (int)H;
    a->page = (int)P;
    a->page_log2 = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    a->D = (int)D;
    a->B = (int)n_seqs;
    a->max_pages = (int)max_pages;
    return SDPA_OK;
}

sdpa_status_t set_table(const int32_t* table, int64_t stride, const int32_t* lens, sdpa::CacheArgs* a) {
    if (a->B > 0 && !lens) return fail(SDPA_ERR_INVALID_ARG, "kv_lens is required");
    if (a->B > 0 && a->max_pages > 0 && !table) return fail(SDPA_ERR_INVALID_ARG, "page_table is required");
    if (a->B > 1 && stride < a->max_pages)
        return fail(SDPA_ERR_INVALID_ARG, "page table rows overlap (stride %lld, %d pages)", (long long)stride, a->max_pages);
    a->table = table;
    a->table_s = a->B > 1 ? stride : 0;
    a->lens = lens;
    return SDPA_OK;
}

sdpa_status_t check_tokens(const sdpa_tensor_t* t, const char* name, int64_t D) {
    TRY(check_tensor(t, name, 3));
    if (t->dtype != SDPA_F16 && t->dtype != SDPA_BF16)
        return fail(SDPA_ERR_INVALID_ARG, "%s dtype %s is not f16 or bf16", name, dtype_name(t->dtype));
    if (t->sizes[2] != D)
        return fail(SDPA_ERR_INVALID_ARG, "%s has head dim %lld, the cache %lld", name, (long long)t->sizes[2], (long long)D);
    if (t->sizes[0] > INT32_MAX || t->sizes[1] > INT32_MAX)
        return fail(SDPA_ERR_UNSUPPORTED, "sizes beyond 2^31 are not supported");
    if (numel(t) > 0 && !rows_aligned(t, 16))
        return fail(SDPA_ERR_UNSUPPORTED, "%s needs a 16-byte aligned base and 16-byte multiple strides", name);
    return SDPA_OK;
}

// weights [n_seqs, Hkv, W] and where they go
sdpa_status_t set_weights(const sdpa_tensor_t* in, sdpa_tensor_t* out, sdpa::CacheArgs* a) {
    TRY(check_tensor(in, "weights", 3));
    TRY(check_tensor(out, "weights_out", 3));
    const int64_t want[3] = {a->B, a->Hkv, in->sizes[2]};
    TRY(check_f32(in, "weights", 3, want));
    TRY(check_f32(out, "weights_out", 3, want));
    if (in->sizes[2] > kMaxTokens) return fail(SDPA_ERR_UNSUPPORTED, "weights of more than 2^30 keys are not supported");
    if (in->data == out->data && (eff_stride(in, 0) != eff_stride(out, 0) || eff_stride(in, 1) != eff_stride(out, 1)))
        return fail(SDPA_ERR_INVALID_ARG, "weights and weights_out overlap: one tensor, or two");
    a->w_in = static_cast<const float*>(in->data);
    a->w_out = static_cast<float*>(out->data);
    for (int i = 0; i < 2; ++i) {
        a->wi_s[i] = eff_stride(in, i);
        a->wo_s[i] = eff_stride(out, i);
    }
    a->w_cols = (int)in->sizes[2];
    return SDPA_OK;
}

// Key ranges: enough workgroups, of 256 keys or more, for two on each of the
// 256 CUs, which is how many are resident. Measured with 256, 512, 768 and 1024
// workgroups: 4 sequences of up to 32768 keys, 8 new tokens, 8 key heads of 128
// 84, 65, 78 and 75 us; 32 sequences of 1000 to 4096 keys, 8 key heads of 128
// 60, 43, 50 and 50 us; one of 32768 keys 24, 22, 22 and 27 us.
constexpr int64_t kCacheGroups = 512;

void plan_cache(sdpa::CacheArgs* a, bool gather) {
    a->rows = a->group * a->max_new;
    const int block = sdpa::cache_block_rows(a->rows);
    a->row_blocks = (int)cdiv(a->rows, block);
    const int64_t base = std::max<int64_t>(1, (int64_t)a->B * a->Hkv * a->row_blocks);
    const int64_t most = std::max<int64_t>(1, cdiv(a->max_kv, 256));
    const int64_t n = std::min<int64_t>(sdpa::CACHE_MAX_RANGES, std::min(most, cdiv(kCacheGroups, base)));
    a->range_keys = (int)std::max<int64_t>(256, cdiv(cdiv(a->max_kv, n), 256) * 256);
    a->n_ranges = (int)std::max<int64_t>(1, cdiv(a->max_kv, a->range_keys));
    a->t_cols = gather ? (int)cdiv(a->max_kv, 64) * 64 : 0;
}

struct CacheWs {
    int64_t ml, o, t, total;  // byte offsets, and the whole
};
CacheWs cache_ws(const sdpa::CacheArgs& a, bool gather) {
    CacheWs w{0, 0, 0, 0};
    if (a.n_ranges == 1 && !gather) return w;
    const int64_t rows = (int64_t)a.B * a.Hkv * a.rows;
    w.o = cdiv(rows * a.n_ranges * 8, 256) * 256;
    w.t = w.o + rows * a.n_ranges * a.D * 4;
    w.total = w.t + rows * a.t_cols * 4;
    return w;
}

sdpa_status_t attention_args(const sdpa_tensor_t* q, const sdpa_cache_t* cache, int64_t n_seqs, int64_t max_pages,
                             int64_t max_q, int64_t max_kv, int enable_gqa, bool gather, sdpa::CacheArgs* a) {
    TRY(cache_args(cache, n_seqs, max_pages, a));
    TRY(check_tokens(q, "q", a->D));
    TRY(check_heads(q->sizes[1], a->Hkv, enable_gqa));
    if (max_q < 0 || max_kv < 0) return fail(SDPA_ERR_INVALID_ARG, "maximum lengths must be non-negative");
    a->q = q->data;
    pack_strides(q, a->q_s);
    a->T = (int)q->sizes[0];
    a->Hq = (int)q->sizes[1];
    a->group = a->Hq / a->Hkv;
    a->max_new = (int)std::min<int64_t>(max_q, a->T);
    a->max_kv = (int)std::min<int64_t>(max_kv, max_pages * a->page);
    if ((int64_t)a->group * a->max_new > INT32_MAX / 2) return fail(SDPA_ERR_UNSUPPORTED, "too many query rows");
    plan_cache(a, gather);
    return SDPA_OK;
}

}  // namespace

extern "C" {

sdpa_status_t sdpa_prompt_fwd(const sdpa_tensor_t* q, const sdpa_tensor_t* k, const sdpa_tensor_t* v,
                              const int32_t* cu_q, const int32_t* cu_k, int64_t n_seqs, int64_t max_q, int64_t max_k,
                              int is_causal, float scale, int enable_gqa, sdpa_tensor_t* out, sdpa_tensor_t* lse,
                              void* hip_stream) {
    g_last_error.clear();
    sdpa::PackArgs a;
    TRY(pack_args(q, k, n_seqs, max_q, max_k, enable_gqa, &a));
    TRY(check_tensor(v, "v", 3));
    if (v->dtype != q->dtype) return fail(SDPA_ERR_INVALID_ARG, "q, k, v dtypes differ");
    if (v->sizes[0] != k->sizes[0] || v->sizes[1] != k->sizes[1])
        return fail(SDPA_ERR_INVALID_ARG, "k and v disagree on tokens or heads");
    if (v->sizes[2] != q->sizes[2])
        return fail(SDPA_ERR_UNSUPPORTED, "value head dim != query head dim is not implemented");
    if (numel(v) > 0 && !rows_aligned(v, 16))
        return fail(SDPA_ERR_UNSUPPORTED, "q, k, v need 16-byte aligned bases and 16-byte multiple strides");
    TRY(check_cu(n_seqs, cu_q, cu_k, is_causal));
    TRY(check_tensor(out, "out", 3));
    if (out->dtype != q->dtype) return fail(SDPA_ERR_INVALID_ARG, "out must have the query dtype");
    TRY(check_dims(out, "out", q->sizes, 3));
    TRY(check_f32(lse, "lse", 2, q->sizes));
    TRY(split_scale(scale, &a.scale_log2, &a.q_mul));
    if (n_seqs == 0 || a.Hq == 0 || a.max_q == 0) return SDPA_OK;
    a.v = v->data;
    a.o = out->data;
    a.lse = static_cast<float*>(lse->data);
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.causal = is_causal;
    pack_strides(v, a.v_s);
    pack_strides(out, a.o_s);
    pack_strides(lse, a.l_s);
    a.o_vec = rows_aligned(out, 16);
    TRY(pack_extent(v, "v", a.max_k, v->sizes[2], &a.v_ext));
    TRY(pack_extent(out, "out", a.max_q, out->sizes[2], &a.o_ext));
    TRY(pack_extent(lse, "lse", a.max_q, 1, &a.l_ext));
    const int D = (int)q->sizes[2];
    a.groups = prompt_groups(a, q->dtype, D);
    a.n_blk = (int)cdiv(a.max_q, a.groups == 4 ? sdpa::PROMPT_ROWS / 4 : sdpa::PROMPT_ROWS);
    TRY(grid_ok({n_seqs, a.Hq, a.n_blk}));
    return launched(sdpa::launch_prompt(q->dtype, D, a, hip_stream));
}

sdpa_status_t sdpa_key_weights_workspace_bytes(const sdpa_tensor_t* q, const sdpa_tensor_t* k, int64_t n_seqs,
                                               int64_t max_q, int64_t max_k, int enable_gqa, size_t* bytes) {
    g_last_error.clear();
    if (!bytes) return fail(SDPA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    sdpa::PackArgs a;
    TRY(pack_args(q, k, n_seqs, max_q, max_k, enable_gqa, &a));
    plan_key_weights(&a);
    *bytes = (size_t)key_weight_ws(a);
    return SDPA_OK;
}

sdpa_status_t sdpa_key_weights(const sdpa_tensor_t* q, const sdpa_tensor_t* k, const sdpa_tensor_t* lse,
                               const int32_t* cu_q, const int32_t* cu_k, int64_t n_seqs, int64_t max_q, int64_t max_k,
                               int is_causal, float scale, int enable_gqa, sdpa_tensor_t* weights, void* workspace,
                               size_t workspace_bytes, void* hip_stream) {
    g_last_error.clear();
    sdpa::PackArgs a;
    TRY(pack_args(q, k, n_seqs, max_q, max_k, enable_gqa, &a));
    TRY(check_f32(lse, "lse", 2, q->sizes));
    TRY(check_cu(n_seqs, cu_q, cu_k, is_causal));
    if (max_k > kMaxTokens) return fail(SDPA_ERR_UNSUPPORTED, "weights of more than 2^30 keys are not supported");
    const int64_t want[3] = {n_seqs, a.Hkv, max_k};
    TRY(check_f32(weights, "weights", 3, want));
    TRY(split_scale(scale, &a.scale_log2, &a.q_mul));
    plan_key_weights(&a);
    if (n_seqs == 0 || max_k == 0) return SDPA_OK;
    const int64_t need = key_weight_ws(a);
    if (need > 0 && (!workspace || workspace_bytes < (size_t)need || reinterpret_cast<uintptr_t>(workspace) % 16))
        return fail(SDPA_ERR_INVALID_ARG, "the workspace needs %lld bytes, 16-byte aligned", (long long)need);
    a.lse = static_cast<float*>(lse->data);
    a.w = static_cast<float*>(weights->data);
    a.ws = static_cast<float*>(workspace);
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.causal = is_causal;
    a.w_cols = (int)max_k;
    pack_strides(lse, a.l_s);
    a.w_s[0] = eff_stride(weights, 0);
    a.w_s[1] = eff_stride(weights, 1);
    TRY(pack_extent(lse, "lse", a.max_q, 1, &a.l_ext));
    TRY(grid_ok({n_seqs, a.Hq, a.n_split, a.n_blk}));
    TRY(grid_ok({n_seqs, a.Hkv, 65536}));  // rows of the sum's grid
    return launched(sdpa::launch_key_weights(q->dtype, (int)q->sizes[2], a, hip_stream));
}

sdpa_status_t sdpa_cache_append(const sdpa_cache_t* cache, const sdpa_tensor_t* k, const sdpa_tensor_t* v,
                                const int32_t* page_table, int64_t n_seqs, int64_t max_pages, int64_t table_stride,
                                const int32_t* kv_lens, const int32_t* cu_seqlens, int64_t max_new, void* hip_stream) {
    g_last_error.clear();
    sdpa::CacheArgs a;
    TRY(cache_args(cache, n_seqs, max_pages, &a));
    TRY(set_table(page_table, table_stride, kv_lens, &a));
    TRY(check_tokens(k, "k", a.D));
    TRY(check_tokens(v, "v", a.D));
    if (v->dtype != k->dtype) return fail(SDPA_ERR_INVALID_ARG, "k and v dtypes differ");
    TRY(check_dims(v, "v", k->sizes, 3));
    if (k->sizes[1] != a.Hkv)
        return fail(SDPA_ERR_INVALID_ARG, "k has %lld heads, the cache %d", (long long)k->sizes[1], a.Hkv);
    if (max_new < 0) return fail(SDPA_ERR_INVALID_ARG, "max_new must be non-negative");
    if (n_seqs > 0 && !cu_seqlens) return fail(SDPA_ERR_INVALID_ARG, "cu_seqlens is required");
    a.cu = cu_seqlens;
    a.T = (int)k->sizes[0];
    a.max_new = (int)std::min<int64_t>(std::min<int64_t>(max_new, a.T), max_pages * a.page);
    if (n_seqs == 0 || a.max_new == 0) return SDPA_OK;
    a.nk = k->data;
    a.nv = v->data;
    pack_strides(k, a.nk_s);
    pack_strides(v, a.nv_s);
    // n tokens that start anywhere touch at most 1 + (n - 1 + P - 1) / P pages
    a.slots = 1 + (a.max_new + a.page - 2) / a.page;
    TRY(grid_ok({2, n_seqs, a.Hkv, a.slots}));
    return launched(sdpa::launch_cache_append(k->dtype, a, hip_stream));
}

sdpa_status_t sdpa_cache_attention_workspace_bytes(const sdpa_tensor_t* q, const sdpa_cache_t* cache, int64_t n_seqs,
                                                   int64_t max_pages, int64_t max_q, int64_t max_kv, int enable_gqa,
                                                   int gather, size_t* bytes) {
    g_last_error.clear();
    if (!bytes) return fail(SDPA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    sdpa::CacheArgs a;
    TRY(attention_args(q, cache, n_seqs, max_pages, max_q, max_kv, enable_gqa, gather != 0, &a));
    *bytes = (size_t)cache_ws(a, gather != 0).total;
    return SDPA_OK;
}

sdpa_status_t sdpa_cache_attention(const sdpa_tensor_t* q, const sdpa_cache_t* cache, const int32_t* page_table,
                                   int64_t n_seqs, int64_t max_pages, int64_t table_stride, const int32_t* kv_lens,
                                   const int32_t* cu_q, int64_t max_q, int64_t max_kv, int is_causal, float scale,
                                   int enable_gqa, const sdpa_tensor_t* weights, sdpa_tensor_t* weights_out,
                                   sdpa_tensor_t* out, sdpa_tensor_t* lse, void* workspace, size_t workspace_bytes,
                                   void* hip_stream) {
    g_last_error.clear();
    const bool gather = weights != nullptr;
    if (gather != (weights_out != nullptr)) return fail(SDPA_ERR_INVALID_ARG, "weights and weights_out go together");
    sdpa::CacheArgs a;
    TRY(attention_args(q, cache, n_seqs, max_pages, max_q, max_kv, enable_gqa, gather, &a));
    TRY(set_table(page_table, table_stride, kv_lens, &a));
    if (gather) TRY(set_weights(weights, weights_out, &a));
    if (n_seqs > 0 && !cu_q) return fail(SDPA_ERR_INVALID_ARG, "cu_seqlens_q is required");
    if (is_causal != 0 && is_causal != 1) return fail(SDPA_ERR_INVALID_ARG, "is_causal must be 0 or 1 (bottom-right)");
    TRY(check_tensor(out, "out", 3));
    if (out->dtype != q->dtype) return fail(SDPA_ERR_INVALID_ARG, "out must have the query dtype");
    TRY(check_dims(out, "out", q->sizes, 3));
    TRY(check_f32(lse, "lse", 2, q->sizes));
    TRY(split_scale(scale, &a.scale_log2, &a.q_mul));
    if (n_seqs == 0 || (a.rows == 0 && !gather)) return SDPA_OK;
    const CacheWs w = cache_ws(a, gather);
    if (w.total > 0 && (!workspace || workspace_bytes < (size_t)w.total || reinterpret_cast<uintptr_t>(workspace) % 16))
        return fail(SDPA_ERR_INVALID_ARG, "the workspace needs %lld bytes, 16-byte aligned", (long long)w.total);
    a.cu = cu_q;
    a.o = out->data;
    a.lse = static_cast<float*>(lse->data);
    a.causal = is_causal;
    pack_strides(out, a.o_s);
    pack_strides(lse, a.l_s);
    if (w.total > 0) {
        uint8_t* p = static_cast<uint8_t*>(workspace);
        a.ws_ml = reinterpret_cast<float2*>(p + w.ml);
        a.ws_o = reinterpret_cast<float*>(p + w.o);
        if (gather) a.ws_t = reinterpret_cast<float*>(p + w.t);
    }
    TRY(grid_ok({a.row_blocks, a.Hkv, n_seqs, a.n_ranges}));
    TRY(grid_ok({n_seqs, a.Hkv, a.rows + cdiv(a.w_cols, 256)}));
    return launched(sdpa::launch_cache_attention(q->dtype, a, hip_stream));
}

sdpa_status_t sdpa_cache_evict(const sdpa_cache_t* cache, const int32_t* page_table, int64_t n_seqs, int64_t max_pages,
                               int64_t table_stride, const int32_t* kv_lens, const sdpa_tensor_t* weights,
                               sdpa_tensor_t* weights_out, int64_t budget, int64_t recent, const int32_t* to_table,
                               int64_t to_pages, int64_t to_stride, int32_t* kept, int32_t* new_lens,
                               void* hip_stream) {
    g_last_error.clear();
    sdpa::CacheArgs a;
    TRY(cache_args(cache, n_seqs, max_pages, &a));
    TRY(set_table(page_table, table_stride, kv_lens, &a));
    TRY(set_weights(weights, weights_out, &a));
    if (budget < 1 || budget > INT32_MAX) return fail(SDPA_ERR_INVALID_ARG, "budget must be at least 1");
    if (budget > kMaxTokens) return fail(SDPA_ERR_UNSUPPORTED, "a budget of more than 2^30 tokens is not supported");
    if (recent < 0 || recent > budget) return fail(SDPA_ERR_INVALID_ARG, "recent must lie between 0 and budget");
    const int64_t most = std::min<int64_t>(budget, std::min<int64_t>(max_pages * a.page, a.w_cols));
    if (to_pages < cdiv(most, a.page))
        return fail(SDPA_ERR_INVALID_ARG, "to_table lists %lld pages, %lld tokens need %lld", (long long)to_pages,
                    (long long)most, (long long)cdiv(most, a.page));
    if (n_seqs > 1 && to_stride < to_pages) return fail(SDPA_ERR_INVALID_ARG, "to_table rows overlap");
    if (n_seqs == 0) return SDPA_OK;
    if ((!to_table && most > 0) || !kept || !new_lens)
        return fail(SDPA_ERR_INVALID_ARG, "to_table, kept and new_lens are required");
    if (std::less<const int32_t*>()(new_lens, kv_lens + n_seqs) && std::less<const int32_t*>()(kv_lens, new_lens + n_seqs))
        return fail(SDPA_ERR_INVALID_ARG, "new_lens overlaps kv_lens");
    a.to = to_table;
    a.to_s = n_seqs > 1 ? to_stride : 0;
    a.to_pages = (int)cdiv(most, a.page);
    a.budget = (int)budget;
    a.recent = (int)recent;
    a.kept = kept;
    a.new_lens = new_lens;
    TRY(grid_ok({2, n_seqs, a.Hkv, std::max(1, a.to_pages)}));  // the selection is launched without pages too
    return launched(sdpa::launch_cache_evict(a, hip_stream));
}

}  // extern "C"
