// The paged 8-bit cache: writing keys and values into it, attention over it,
// and moving the tokens that are kept when it is cut.
//
// A page holds `page` tokens of every key head. k codes lie token-major
// [page, D]; v codes lie transposed [D, page], so that the tokens of one
// head-dim column are contiguous: that is the order the O^T += V^T P^T
// product takes them in, and the attention kernel loads both operands straight
// from memory into matrix registers, without a pass through LDS. A scale is a
// power of two: e4m3 is a floating format, so a finer scale would gain no
// precision, and a code moves to a larger scale exactly unless it becomes
// subnormal there.
#include "sdpa_device.h"
#include "serve.h"

#define SDPA_INLINE __attribute__((always_inline))

namespace sdpa {

constexpr float E4M3_MAX = 448.0f;
constexpr float SCALE_MIN = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ bool finite(float x) {
    return (__builtin_bit_cast(uint32_t, x) & 0x7f800000u) != 0x7f800000u;
}
// The smallest power of two (2^-126 at least) under which amax is at most
// 448 = 1.75 * 2^8: with amax = f 2^x, 1 <= f < 2, that is 2^(x - 8), or the
// next one when f > 1.75.
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent
    return __builtin_bit_cast(float, (uint32_t)max(e, 1) << 23);
}
// 1 / s for a power of two s >= 2^-126 (2^126 at most)
__device__ __forceinline__ float inverse(float s) {
    return __builtin_bit_cast(float, (254u << 23) - __builtin_bit_cast(uint32_t, s));
}
// Two e4m3 codes of x0, x1 (round to nearest even, |x| <= 448); what is not
// finite becomes the NaN code.
__device__ __forceinline__ uint32_t encode2(float x0, float x1) {
    uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x0, x1, 0, false) & 0xffffu;
    if (!finite(x0)) c = (c & 0xff00u) | 0x7fu;
    if (!finite(x1)) c = (c & 0x00ffu) | 0x7f00u;
    return c;
}
__device__ __forceinline__ void decode4(uint32_t c, float* x) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    x[0] = lo[0];
    x[1] = lo[1];
    x[2] = hi[0];
    x[3] = hi[1];
}
// four codes under scale old_s to the same values under new_s (ratio = old_s / new_s <= 1)
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
    float x[4];
    decode4(c, x);
    return encode2(x[0] * ratio, x[1] * ratio) | encode2(x[2] * ratio, x[3] * ratio) << 16;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = Tr<T>::to_f((v[e >> 1] >> (16 * (e & 1))) & 0xffffu);
}

__device__ __forceinline__ int held_tokens(const CacheArgs& a, int b) {
    return (int)min((int64_t)max(a.lens[b], 0), (int64_t)a.max_pages * a.page);
}

// ----------------------------------------------------------------------- append
//
// One workgroup per (page, key head) and per k or v: the new tokens' largest
// magnitude gives the scale they need; a page that already holds tokens keeps
// the larger of that and its own scale, its codes re-rounded when it grows.
// Reads 2 bytes and writes 1 per element: bound by HBM, and by latency for
// single tokens.
template <typename T>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256)))
void sdpa_cache_append_kernel(const CacheArgs a) {
    __shared__ float red[4];
    __shared__ __attribute__((aligned(16))) uint8_t tr[128 * (128 + 4)];  // v codes [D][page + 4]
    const int tid = threadIdx.x;
    int id = blockIdx.x;
    const int is_v = id & 1;
    id >>= 1;
    const int h = id % a.Hkv;
    id /= a.Hkv;
    const int slot = id % a.slots, b = id / a.slots;
    const int c0 = min(max(a.cu[b], 0), a.T);
    const int held = held_tokens(a, b);
    const int count = (int)min((int64_t)min(min(max(a.cu[b + 1], c0), a.T) - c0, a.max_new),
                               (int64_t)a.max_pages * a.page - held);
    const int pi = (held >> a.page_log2) + slot;
    const int lo = max(held, pi * a.page), hi = min(held + count, (pi + 1) * a.page);
    if (lo >= hi) return;
    const int page = a.table[b * a.table_s + pi];
    if (page < 0 || page >= a.n_pages) return;
    const int off = lo - pi * a.page, n = hi - lo;
    const int ch = a.D / 8;  // 8-element chunks of a token
    const int64_t* st = is_v ? a.nv_s : a.nk_s;
    const T* src = static_cast<const T*>(is_v ? a.nv : a.nk) + h * st[0] + (int64_t)(c0 + lo - held) * st[1];
    float* const scale = (is_v ? a.vs : a.ks) + (int64_t)page * a.Hkv + h;
    uint8_t* const dst = (is_v ? a.v : a.k) + ((int64_t)page * a.Hkv + h) * a.page * a.D;

    float amax = 0.0f;
    for (int i = tid; i < n * ch; i += 256) {
        float x[8];
        load8(src + (i / ch) * st[1] + (i % ch) * 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite(x[e]) ? fabsf(x[e]) : 0.0f);
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2) amax = fmaxf(amax, __shfl_xor(amax, k));
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    const float was = off > 0 ? *scale : 0.0f;
    __syncthreads();  // every thread has read the old scale
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float now = fmaxf(scale_for(amax), was);
    const float inv = inverse(now);
    if (tid == 0) *scale = now;
    if (off > 0 && now > was) {  // the held codes move to the larger scale
        const float ratio = was * inv;
        if (!is_v) {
            for (int i = tid; i < off * a.D / 4; i += 256) {
                uint32_t* p = reinterpret_cast<uint32_t*>(dst) + i;
                *p = rescale4(*p, ratio);
            }
        } else {
            for (int i = tid; i < off * a.D; i += 256) {
                uint8_t* p = dst + (i / off) * a.page + i % off;
                *p = (uint8_t)rescale4(*p, ratio);
            }
        }
    }
    const int pitch = a.page + 4;
    for (int i = tid; i < n * ch; i += 256) {
        const int t = i / ch, c = i % ch;
        float x[8];
        load8(src + t * st[1] + c * 8, x);
        u32x2 code;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            code[e] = encode2(x[4 * e] * inv, x[4 * e + 1] * inv) | encode2(x[4 * e + 2] * inv, x[4 * e + 3] * inv) << 16;
        if (!is_v) {
            *reinterpret_cast<u32x2*>(dst + (off + t) * a.D + c * 8) = code;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) tr[(c * 8 + e) * pitch + t] = (uint8_t)(code[e >> 2] >> (8 * (e & 3)));
        }
    }
    if (!is_v) return;
    __syncthreads();
    if (off == 0 && n == a.page) {  // a whole page: 4 tokens a store
        const int per = a.page / 4;
        for (int i = tid; i < a.D * per; i += 256) {
            const int d = i / per, t = 4 * (i % per);
            *reinterpret_cast<uint32_t*>(dst + d * a.page + t) = *reinterpret_cast<const uint32_t*>(tr + d * pitch + t);
        }
    } else {
        for (int i = tid; i < a.D * n; i += 256) {
            const int d = i / n, t = i % n;
            dst[d * a.page + off + t] = tr[d * pitch + t];
        }
    }
}

int launch_cache_append(int dtype, const CacheArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(2u * a.B * a.Hkv * a.slots), block(256);
    if (dtype == DT_F16) sdpa_cache_append_kernel<_Float16><<<grid, block, 0, s>>>(a);
    else sdpa_cache_append_kernel<__bf16><<<grid, block, 0, s>>>(a);
    return (int)hipGetLastError();
}

// -------------------------------------------------------------------- attention
//
// One workgroup of four waves per (sequence, key head, block of query rows,
// key range); the rows are the range's new tokens times the query heads of
// the key head. A wave takes 64 keys at a time. S^T = K Q^T and
// O^T += V^T P^T run on 16x16x32 products with the keys of a tile numbered so
// that the scores leave the first product as the operand of the second and
// every load is 16 contiguous bytes: row m of score block c is token
// 16 (m / 4) + 4 c + m % 4, so lane (row, g) holds the scores of tokens
// 16 g .. 16 g + 15, and takes v codes of exactly these tokens. Any 16 tokens
// that start at a multiple of 16 lie in one page, so one scale of k and one of
// v serve a lane's tile. Codes become bf16 (k: the type of q) exactly; the
// probabilities, times the scale of v, go in as their bf16 rounding plus its
// rounded residual (16 bits), so that O is rounded once, to its own type.
// Bytes of K and V bound it: 2 D per token and key head.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <typename T> struct Ops8;
template <> struct Ops8<__bf16> {
    static __device__ __forceinline__ bf16x8 widen(uint32_t a, uint32_t b) {
        const bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
        const bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
        const bf16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
        const bf16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
        return __builtin_bit_cast(bf16x8, u32x4{__builtin_bit_cast(uint32_t, x0), __builtin_bit_cast(uint32_t, x1),
                                                __builtin_bit_cast(uint32_t, x2), __builtin_bit_cast(uint32_t, x3)});
    }
    static __device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Ops8<_Float16> {
    static __device__ __forceinline__ f16x8 widen(uint32_t a, uint32_t b) {
        const f16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
        const f16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
        const f16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
        const f16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
        return __builtin_bit_cast(f16x8, u32x4{__builtin_bit_cast(uint32_t, x0), __builtin_bit_cast(uint32_t, x1),
                                               __builtin_bit_cast(uint32_t, x2), __builtin_bit_cast(uint32_t, x3)});
    }
    static __device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// the tokens of sequence b that a call sees, and its new tokens
struct CacheSeq {
    int len, q0, n;
};
__device__ __forceinline__ CacheSeq cache_sequence(const CacheArgs& a, int b) {
    CacheSeq s;
    s.len = min(held_tokens(a, b), a.max_kv);
    s.q0 = min(max(a.cu[b], 0), a.T);
    s.n = min(min(max(a.cu[b + 1], s.q0), a.T) - s.q0, a.max_new);
    return s;
}

template <typename T, int D, int RT>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2)))
void sdpa_cache_attention_kernel(const CacheArgs a) {
    using O = Ops8<T>;
    using OB = Ops8<__bf16>;
    using vec = typename Tr<T>::vec;
    constexpr int NW = 4, ROWS = 16 * RT, ND = D / 16, NKS = D / 32;
    constexpr int KB = D / 4;                      // bytes of a key row one lane holds
    constexpr int OP = D + 4;                      // partial output pitch
    __shared__ __attribute__((aligned(16))) float part[NW * ROWS * OP];
    __shared__ float2 ml[NW][ROWS];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    int id = blockIdx.x;
    const int rblk = id % a.row_blocks;
    id /= a.row_blocks;
    const int h = id % a.Hkv;
    id /= a.Hkv;
    const int b = id % a.B, range = id / a.B;
    const CacheSeq s = cache_sequence(a, b);
    const int rows = s.n * a.group;
    if (rblk * ROWS >= rows) return;
    const int j0 = range * a.range_keys, j1 = min(s.len, j0 + a.range_keys);
    if (range > 0 && j0 >= s.len) return;

    // Q: lane (row, g) holds head-dim g KB + 8 c .. + 7 of product step c
    vec qf[RT][NKS];
    int limit[RT];  // the last key the row keeps
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = rblk * ROWS + 16 * rt + n;
        const bool ok = r < rows;
        const int tok = ok ? r / a.group : 0, head = h * a.group + (ok ? r - tok * a.group : 0);
        limit[rt] = a.causal ? s.len - s.n + tok : s.len - 1;
        const T* qp = static_cast<const T*>(a.q) + head * a.q_s[0] + (int64_t)(s.q0 + tok) * a.q_s[1] + g * KB;
#pragma unroll
        for (int c = 0; c < NKS; ++c) {
            u32x4 x = *reinterpret_cast<const u32x4*>(qp + 8 * c);
            if (a.q_mul != 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = a.q_mul == 0 ? 0u : x[e] ^ 0x80008000u;
            qf[rt][c] = __builtin_bit_cast(vec, x);
        }
    }
    f32x4 oacc[RT][ND];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -INFINITY;
        l[rt] = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) oacc[rt][d] = f32x4{};
    }
    const int* const trow = a.table + b * a.table_s;
    const int first_cut = a.causal ? s.len - s.n + 1 : s.len;  // every row keeps the keys before it

    for (int t0 = j0 + 64 * wave; t0 < j1; t0 += 64 * NW) {
        // pages of this lane's key rows (16 (n / 4) ..) and of its values (16 g ..)
        const int jk = t0 + 16 * (n >> 2), jv = t0 + 16 * g;
        const int pk_raw = jk < s.len ? trow[jk >> a.page_log2] : -1;
        const int pv_raw = jv < s.len ? trow[jv >> a.page_log2] : -1;
        const bool okk = pk_raw >= 0 && pk_raw < a.n_pages, okv = pv_raw >= 0 && pv_raw < a.n_pages;
        const int64_t pk = okk ? pk_raw : 0, pv = okv ? pv_raw : 0;
        const int live = okv ? min(s.len - jv, 16) : 0;  // tokens of this lane that exist
        const uint8_t* kp = a.k + ((pk * a.Hkv + h) * a.page + (jk & (a.page - 1)) + (n & 3)) * D + g * KB;
        const uint8_t* vp = a.v + ((pv * a.Hkv + h) * D + n) * a.page + (jv & (a.page - 1));
        uint32_t kc[4][KB / 4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if constexpr (KB >= 16) {
#pragma unroll
                for (int e = 0; e < KB / 16; ++e) {
                    const u32x4 x = *reinterpret_cast<const u32x4*>(kp + 4 * c * D + 16 * e);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kc[c][4 * e + i] = x[i];
                }
            } else {
                const u32x2 x = *reinterpret_cast<const u32x2*>(kp + 4 * c * D);
                kc[c][0] = x[0];
                kc[c][1] = x[1];
            }
        }
        u32x4 vc[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d) vc[d] = *reinterpret_cast<const u32x4*>(vp + (int64_t)16 * d * a.page);
        const float ks = a.ks[pv * a.Hkv + h] * a.scale_log2, vs = a.vs[pv * a.Hkv + h];

        const bool ragged = __builtin_amdgcn_ballot_w64(live < 16) != 0;
        const bool cut = ragged || t0 + 64 > first_cut;
        if (ragged) {  // codes past the end may be anything, NaN among them
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = min(max(live - 4 * i, 0), 4);
                const uint32_t mask = k == 4 ? 0xffffffffu : (1u << (8 * k)) - 1u;
#pragma unroll
                for (int d = 0; d < ND; ++d) vc[d][i] &= mask;
            }
        }
        f32x4 acc[RT][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[rt][c] = f32x4{};
#pragma unroll
            for (int e = 0; e < NKS; ++e) {
                const vec ka = O::widen(kc[c][2 * e], kc[c][2 * e + 1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) acc[rt][c] = O::mfma(ka, qf[rt][e], acc[rt][c]);
            }
        }
        float top[RT];
        bool grow = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            top[rt] = -INFINITY;
            const int lim = min(limit[rt] - jv, live - 1);  // among this lane's 16 tokens
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x = acc[rt][i >> 2][i & 3] * ks;
                if (cut) x = i > lim ? -INFINITY : x;
                acc[rt][i >> 2][i & 3] = x;
                top[rt] = fmaxf(top[rt], x);
            }
            grow = grow || top[rt] > m[rt] + 8.0f;
            if (a.ws_t) {
                const int r = rblk * ROWS + 16 * rt + n;
                if (r < rows && jv < a.t_cols) {
                    float* tp = a.ws_t + (((int64_t)b * a.Hkv + h) * a.rows + r) * a.t_cols + jv;
#pragma unroll
                    for (int c = 0; c < 4; ++c) *reinterpret_cast<f32x4*>(tp + 4 * c) = acc[rt][c];
                }
            }
        }
        if (__builtin_amdgcn_ballot_w64(grow) != 0) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float up = fmaxf(top[rt], __shfl_xor(top[rt], 16));
                up = fmaxf(m[rt], fmaxf(up, __shfl_xor(up, 32)));
                const float f = up == -INFINITY ? 1.0f : fast_exp2(m[rt] - up);
                m[rt] = up;
                l[rt] *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) oacc[rt][d][r] *= f;
            }
        }
        bf16x8 ph[RT][2], pl[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float mu = m[rt] == -INFINITY ? 0.0f : m[rt];
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = fast_exp2(acc[rt][i >> 2][i & 3] - mu);
                l[rt] += p[i];
                p[i] *= vs;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                ph[rt][c] = Tr<__bf16>::cvt8(p + 8 * c);
                pl[rt][c] = Tr<__bf16>::lo8(p + 8 * c, ph[rt][c]);
            }
        }
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bf16x8 va = OB::widen(vc[d][2 * c], vc[d][2 * c + 1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    oacc[rt][d] = OB::mfma(va, ph[rt][c], oacc[rt][d]);
                    oacc[rt][d] = OB::mfma(va, pl[rt][c], oacc[rt][d]);
                }
            }
    }

    // the four waves' rows joined
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        float x = l[rt] + __shfl_xor(l[rt], 16);
        x += __shfl_xor(x, 32);
        if (g == 0) ml[wave][16 * rt + n] = make_float2(m[rt], x);
        float* op = part + (wave * ROWS + 16 * rt + n) * OP + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(op + 16 * d) = oacc[rt][d];
    }
    __syncthreads();
    const bool whole = a.ws_ml == nullptr;  // one range, no weights: this is the result
    for (int i = tid; i < ROWS * (D / 4); i += 256) {
        const int row = i / (D / 4), d = 4 * (i % (D / 4)), r = rblk * ROWS + row;
        if (r >= rows) continue;
        float top = ml[0][row].x;
#pragma unroll
        for (int w = 1; w < NW; ++w) top = fmaxf(top, ml[w][row].x);
        f32x4 x = {};
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = ml[w][row].x == -INFINITY ? 0.0f : fast_exp2(ml[w][row].x - top);
            sum += f * ml[w][row].y;
            const f32x4 y = *reinterpret_cast<const f32x4*>(part + (w * ROWS + row) * OP + d);
            if (f != 0.0f) x += f * y;
        }
        const int tok = r / a.group, head = h * a.group + r - tok * a.group;
        if (whole) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            typedef T t4 __attribute__((ext_vector_type(4)));
            x *= inv;
            T* op = static_cast<T*>(a.o) + head * a.o_s[0] + (int64_t)(s.q0 + tok) * a.o_s[1] + d;
            const t4 y = __builtin_convertvector(x, t4);
#pragma unroll
            for (int e = 0; e < 4; ++e) op[e] = y[e];
            if (d == 0)
                a.lse[head * a.l_s[0] + (int64_t)(s.q0 + tok) * a.l_s[1]] =
                    sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * LN2;
        } else {
            const int64_t at = (((int64_t)b * a.Hkv + h) * a.rows + r) * a.n_ranges + range;
            *reinterpret_cast<f32x4*>(a.ws_o + at * D + d) = x;
            if (d == 0) a.ws_ml[at] = make_float2(top, sum);
        }
    }
}

// The ranges joined: O and LSE of every row, and the weights plus each key's
// sum of probabilities over the rows. Workgroups below n_rows take one row
// each, the rest 256 keys each of one (sequence, key head).
template <typename T>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256)))
void sdpa_cache_join_kernel(const CacheArgs a, int n_rows) {
    __shared__ float part[256];
    const int tid = threadIdx.x;
    if ((int)blockIdx.x < n_rows) {
        int id = blockIdx.x;
        const int r = id % a.rows;
        id /= a.rows;
        const int h = id % a.Hkv, b = id / a.Hkv;
        const CacheSeq s = cache_sequence(a, b);
        if (r >= s.n * a.group) return;
        const int nr = max(1, (s.len + a.range_keys - 1) / a.range_keys);
        const int64_t at = (((int64_t)b * a.Hkv + h) * a.rows + r) * a.n_ranges;
        float top = -INFINITY;
        for (int i = 0; i < nr; ++i) top = fmaxf(top, a.ws_ml[at + i].x);
        const int per = 256 / a.D, d = tid % a.D, k = tid / a.D;
        float sum = 0.0f, x = 0.0f;
        for (int i = 0; i < nr; ++i) {
            const float2 e = a.ws_ml[at + i];
            const float f = e.x == -INFINITY ? 0.0f : fast_exp2(e.x - top);
            sum += f * e.y;
            if (f != 0.0f && i % per == k) x += f * a.ws_o[(at + i) * a.D + d];
        }
        part[tid] = x;
        __syncthreads();
        if (k != 0) return;
        for (int i = 1; i < per; ++i) x += part[i * a.D + d];
        const int tok = r / a.group, head = h * a.group + r - tok * a.group;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        static_cast<T*>(a.o)[head * a.o_s[0] + (int64_t)(s.q0 + tok) * a.o_s[1] + d] = (T)(x * inv);
        if (d == 0)
            a.lse[head * a.l_s[0] + (int64_t)(s.q0 + tok) * a.l_s[1]] =
                sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * LN2;
        return;
    }
    int id = blockIdx.x - n_rows;
    const int nj = (a.w_cols + 255) / 256;
    const int j = (id % nj) * 256 + tid;
    id /= nj;
    const int h = id % a.Hkv, b = id / a.Hkv;
    const CacheSeq s = cache_sequence(a, b);
    const int nr = max(1, (s.len + a.range_keys - 1) / a.range_keys);
    const int rows = s.n * a.group;
    const int64_t row0 = ((int64_t)b * a.Hkv + h) * a.rows;
    const float w = j < a.w_cols ? a.w_in[b * a.wi_s[0] + h * a.wi_s[1] + j] : 0.0f;
    float x = 0.0f;  // the rows' sum first, so that adding it to the weight rounds once
    for (int r0 = 0; r0 < rows; r0 += 256) {  // LSE of up to 256 rows at a time
        __syncthreads();
        float lse2 = INFINITY;  // a row without keys adds nothing
        if (r0 + tid < rows) {
            const int64_t at = (row0 + r0 + tid) * a.n_ranges;
            float top = -INFINITY, sum = 0.0f;
            for (int i = 0; i < nr; ++i) top = fmaxf(top, a.ws_ml[at + i].x);
            for (int i = 0; i < nr; ++i) {
                const float2 e = a.ws_ml[at + i];
                sum += e.x == -INFINITY ? 0.0f : e.y * fast_exp2(e.x - top);
            }
            if (sum != 0.0f) lse2 = top + __builtin_amdgcn_logf(sum);
        }
        part[tid] = lse2;
        __syncthreads();
        if (j < s.len)
            for (int r = r0; r < min(rows, r0 + 256); ++r)
                x += fast_exp2(a.ws_t[(row0 + r) * a.t_cols + j] - part[r - r0]);
    }
    if (j < a.w_cols) a.w_out[b * a.wo_s[0] + h * a.wo_s[1] + j] = w + x;
}

template <typename T, int RT>
static int launch_cache_attention_rt(const CacheArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)a.row_blocks * a.Hkv * a.B * a.n_ranges), block(256);
    if (a.row_blocks > 0) switch (a.D) {
        case 32: sdpa_cache_attention_kernel<T, 32, RT><<<grid, block, 0, s>>>(a); break;
        case 64: sdpa_cache_attention_kernel<T, 64, RT><<<grid, block, 0, s>>>(a); break;
        case 128: sdpa_cache_attention_kernel<T, 128, RT><<<grid, block, 0, s>>>(a); break;
        default: return (int)hipErrorInvalidValue;
    }
    int e = (int)hipGetLastError();
    if (e || (!a.ws_ml && !a.w_out)) return e;
    const int n_rows = a.B * a.Hkv * a.rows;
    const int n_w = a.w_out ? a.B * a.Hkv * ((a.w_cols + 255) / 256) : 0;
    if (n_rows + n_w > 0) sdpa_cache_join_kernel<T><<<dim3(n_rows + n_w), block, 0, s>>>(a, n_rows);
    return (int)hipGetLastError();
}

int launch_cache_attention(int dtype, const CacheArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool one = cache_block_rows(a.rows) == 16;
    if (dtype == DT_F16) return one ? launch_cache_attention_rt<_Float16, 1>(a, s) : launch_cache_attention_rt<_Float16, 2>(a, s);
    return one ? launch_cache_attention_rt<__bf16, 1>(a, s) : launch_cache_attention_rt<__bf16, 2>(a, s);
}

// --------------------------------------------------------------------- eviction
//
// sdpa_cache_select_kernel: one workgroup per (sequence, key head) finds the
// tokens to keep. Weights become integers of the same order (NaN highest);
// three passes of a radix histogram (11, 11 and 10 bits) find the value of
// the last token kept; then each wave counts, and after a scan over the waves
// emits, the kept tokens of its stretch of the sequence in order, of the tied
// ones the first.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    if (x != x) return 0xffffffffu;
    if (x == 0.0f) return 0x80000000u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int SELECT_THREADS = 1024;

__global__ __attribute__((amdgpu_flat_work_group_size(SELECT_THREADS, SELECT_THREADS)))
void sdpa_cache_select_kernel(const CacheArgs a) {
    constexpr int NT = SELECT_THREADS, NWV = NT / 64;
    __shared__ int hist[2048];
    __shared__ int wsum[NWV], wtie[NWV];
    __shared__ int pick_s, above_s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv;
    const int len = (int)min((int64_t)held_tokens(a, b), (int64_t)a.w_cols);
    const int n = min(len, a.budget);
    const int late = len - min(a.recent, n);  // tokens from here on are kept
    int need = n - (len - late);              // of the tokens before
    const float* w = a.w_in + b * a.wi_s[0] + h * a.wi_s[1];
    int* kept = a.kept + ((int64_t)b * a.Hkv + h) * a.budget;

    uint32_t pick = 0;   // the order key of the last token kept, found from the high bits down
    const bool all = need == late;
    if (!all && need > 0) {
        uint32_t mask = 0;
        const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int nb = 1 << bits[pass];
            for (int i = tid; i < nb; i += NT) hist[i] = 0;
            __syncthreads();
            for (int j = tid; j < late; j += NT) {
                const uint32_t u = order_key(w[j]);
                if ((u & mask) == pick) atomicAdd(&hist[(u >> shifts[pass]) & (nb - 1)], 1);
            }
            __syncthreads();
            // the highest bin that, with all above it, holds `need` tokens
            if (wave == 0) {
                int run = 0;
                for (int base = nb - 64; base >= 0; base -= 64) {
                    const int c = hist[base + 63 - lane];
                    int x = c;  // sums over the lanes up to this one: bins from the top down
#pragma unroll
                    for (int k = 1; k < 64; k *= 2) {
                        const int y = __shfl_up(x, k);
                        if (lane >= k) x += y;
                    }
                    const uint64_t hit = __builtin_amdgcn_ballot_w64(run + x >= need);
                    if (hit) {
                        const int f = __builtin_ctzll(hit);
                        if (lane == f) {
                            pick_s = base + 63 - lane;
                            above_s = run + x - c;
                        }
                        break;
                    }
                    run += __shfl(x, 63);
                }
            }
            __syncthreads();
            pick |= (uint32_t)pick_s << shifts[pass];
            mask |= (uint32_t)(nb - 1) << shifts[pass];
            need -= above_s;
            __syncthreads();
        }
    }
    // need: how many tokens equal to `pick` are kept
    const int per = ((len + NT - 1) / NT) * 64;  // a wave's stretch
    const int w0 = min(len, wave * per), w1 = min(len, w0 + per);
    const bool none = n - (len - late) == 0;
    auto above = [&](int j, uint32_t u) SDPA_INLINE { return j >= late || (!none && (all || u > pick)); };
    auto tied = [&](int j, uint32_t u) SDPA_INLINE { return j < late && !none && !all && u == pick; };
    int cnt = 0, tie = 0;
    for (int j0 = w0; j0 < w1; j0 += 64) {
        const int j = j0 + lane;
        const uint32_t u = j < w1 ? order_key(w[j]) : 0u;
        cnt += __popcll(__builtin_amdgcn_ballot_w64(j < w1 && above(j, u)));
        tie += __popcll(__builtin_amdgcn_ballot_w64(j < w1 && tied(j, u)));
    }
    if (lane == 0) {
        wsum[wave] = cnt;
        wtie[wave] = tie;
    }
    __syncthreads();
    int at = 0, ties = 0;
    for (int i = 0; i < wave; ++i) {
        const int before = min(ties + wtie[i], need) - min(ties, need);
        at += wsum[i] + before;
        ties += wtie[i];
    }
    const uint64_t below = (uint64_t(1) << lane) - 1;
    for (int j0 = w0; j0 < w1; j0 += 64) {
        const int j = j0 + lane;
        const uint32_t u = j < w1 ? order_key(w[j]) : 0u;
        const bool is_tie = j < w1 && tied(j, u);
        const uint64_t tb = __builtin_amdgcn_ballot_w64(is_tie);
        const bool keep = j < w1 && (above(j, u) || (is_tie && ties + __popcll(tb & below) < need));
        const uint64_t kb = __builtin_amdgcn_ballot_w64(keep);
        if (keep) kept[at + __popcll(kb & below)] = j;
        at += __popcll(kb);
        ties += __popcll(tb);
    }
    for (int i = n + tid; i < a.budget; i += NT) kept[i] = -1;
    __syncthreads();
    // weights of the kept tokens, in place too: a token never moves up, and
    // each round's reads end before its writes begin
    float* wo = a.w_out + b * a.wo_s[0] + h * a.wo_s[1];
    for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + tid;
        const float x = i < n ? w[kept[i]] : 0.0f;
        __syncthreads();
        if (i < n) wo[i] = x;
    }
    __syncthreads();
    for (int i = n + tid; i < a.w_cols; i += NT) wo[i] = 0.0f;
    if (h == 0 && tid == 0) a.new_lens[b] = n;
}

// sdpa_cache_move_kernel: one workgroup per page moved to, and k or v. The
// page's scale is the largest of its tokens' scales; slots past the kept
// tokens hold zeros.
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256)))
void sdpa_cache_move_kernel(const CacheArgs a) {
    __shared__ int src_page[128], src_off[128];
    __shared__ float ratio[128];
    __shared__ float red[4];
    const int tid = threadIdx.x;
    int id = blockIdx.x;
    const int is_v = id & 1;
    id >>= 1;
    const int h = id % a.Hkv;
    id /= a.Hkv;
    const int b = id % a.B, i0 = (id / a.B) * a.page;
    const int len = (int)min((int64_t)held_tokens(a, b), (int64_t)a.w_cols);
    const int n = min(min(len, a.budget) - i0, a.page);
    if (n <= 0) return;
    const int to = a.to[b * a.to_s + i0 / a.page];
    if (to < 0 || to >= a.n_pages) return;
    const float* const scales = is_v ? a.vs : a.ks;
    float top = 0.0f;
    if (tid < a.page) {
        int page = -1, off = 0;
        float sc = 0.0f;
        if (tid < n) {
            const int j = a.kept[((int64_t)b * a.Hkv + h) * a.budget + i0 + tid];
            page = a.table[b * a.table_s + (j >> a.page_log2)];
            off = j & (a.page - 1);
            if (page < 0 || page >= a.n_pages) page = -1;
            else sc = scales[(int64_t)page * a.Hkv + h];
        }
        src_page[tid] = page;
        src_off[tid] = off;
        ratio[tid] = sc;
        top = sc;
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2) top = fmaxf(top, __shfl_xor(top, k));
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    top = fmaxf(top, SCALE_MIN);
    const float inv = inverse(top);
    const uint8_t* const src = is_v ? a.v : a.k;
    uint8_t* const dst = (is_v ? a.v : a.k) + ((int64_t)to * a.Hkv + h) * a.page * a.D;
    if (!is_v) {
        const int per = a.D / 4;
        for (int i = tid; i < a.page * per; i += 256) {
            const int t = i / per, c = i - t * per;
            uint32_t x = 0;
            if (src_page[t] >= 0) {
                x = *reinterpret_cast<const uint32_t*>(src + (((int64_t)src_page[t] * a.Hkv + h) * a.page + src_off[t]) * a.D + 4 * c);
                x = rescale4(x, ratio[t] * inv);
            }
            *reinterpret_cast<uint32_t*>(dst + t * a.D + 4 * c) = x;
        }
    } else {
        for (int i = tid; i < a.page * a.D; i += 256) {
            const int d = i / a.page, t = i - d * a.page;
            uint32_t x = 0;
            if (src_page[t] >= 0) {
                x = src[(((int64_t)src_page[t] * a.Hkv + h) * a.D + d) * a.page + src_off[t]];
                x = rescale4(x, ratio[t] * inv) & 0xffu;
            }
            dst[d * a.page + t] = (uint8_t)x;
        }
    }
    if (tid == 0) (is_v ? a.vs : a.ks)[(int64_t)to * a.Hkv + h] = top;
}

int launch_cache_evict(const CacheArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    sdpa_cache_select_kernel<<<dim3(a.B * a.Hkv), dim3(SELECT_THREADS), 0, s>>>(a);
    int e = (int)hipGetLastError();
    if (e || a.to_pages == 0) return e;
    sdpa_cache_move_kernel<<<dim3(2u * a.B * a.Hkv * a.to_pages), dim3(256), 0, s>>>(a);
    return (int)hipGetLastError();
}

}  // namespace sdpa
