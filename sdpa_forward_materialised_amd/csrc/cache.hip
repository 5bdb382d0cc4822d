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

__device__ __forceinline__ int held_tokens(const CacheArgs& a, int b) {
    return (int)min((int64_t)max(a.lens[b], 0), (int64_t)a.max_pages * a.page);
}

// ----------------------------------------------------------------------- append
//
// One wave per (page, key head), the page's new keys and values in its
// registers: for each of the two, the largest magnitude gives the scale they
// need; a page that already holds tokens keeps the larger of that and its own
// scale, its codes re-rounded when it grows. A lane takes 8 head-dim columns of
// 4 consecutive tokens, so that both layouts are written without a pass through
// LDS: k as 8 codes of a token, v as 4 tokens of a column. Reads 2 bytes and
// writes 1 per element; the chain lengths -> table -> elements -> scale of
// dependent loads bounds it, which k and v go through together.
template <int D, int P, bool V>
__device__ __forceinline__ void rescale_held(uint8_t* dst, int off, float ratio, int lane) {
    // words of 4 codes: k, those of the tokens before `off`; v, of their 4
    // slots those before `off`
    constexpr int ROW = V ? P / 4 : D / 4;
    const int n = V ? D * ROW : off * ROW;
    for (int i0 = lane; i0 < n; i0 += 8 * 64) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + 64 * k;
            w[k] = i < n && (!V || 4 * (i % ROW) < off) ? reinterpret_cast<const uint32_t*>(dst)[i] : 0u;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + 64 * k, t = V ? 4 * (i % ROW) : 0;
            if (i >= n || (V && t >= off)) continue;
            const int m = V ? min(off - t, 4) : 4;
            const uint32_t mask = m == 4 ? 0xffffffffu : (1u << (8 * m)) - 1u;
            reinterpret_cast<uint32_t*>(dst)[i] = (rescale4(w[k], ratio) & mask) | (w[k] & ~mask);
        }
    }
}

template <typename T, int D, int P>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256)))
void sdpa_cache_append_kernel(const CacheArgs a) {
    constexpr int LOG = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    constexpr int CH = D / 8, NU = (P / 4 * CH + 63) / 64;  // units of 4 tokens, units of a lane at most
    // up to 4 units of a lane stay in registers; of more, the second half is
    // read again (from cache) when its codes are made
    constexpr int KEEP = NU < 4 ? NU : 4;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int id = blockIdx.x * 4 + wave;
    const int h = id % a.Hkv;
    id /= a.Hkv;
    const int slot = id % a.slots, b = id / a.slots;
    if (b >= a.B) return;
    const int c0 = min(max(a.cu[b], 0), a.T);
    const int held = held_tokens(a, b);
    const int count = (int)min((int64_t)min(min(max(a.cu[b + 1], c0), a.T) - c0, a.max_new),
                               (int64_t)a.max_pages * P - held);
    const int pi = (held >> LOG) + slot;
    const int lo = max(held, pi * P), hi = min(held + count, (pi + 1) * P);
    if (lo >= hi) return;
    const int page = a.table[b * a.table_s + pi];
    if (page < 0 || page >= a.n_pages) return;
    const int off = lo - pi * P, end = hi - pi * P;  // the page's new slots
    const int t_first = off & ~3, units = ((end - t_first + 3) >> 2) * CH;
    const int64_t at = (int64_t)page * a.Hkv + h, tok0 = c0 + pi * P - held;
    // element [slot][column] of the page's new tokens
    const T* const src[2] = {static_cast<const T*>(a.nk) + h * a.nk_s[0] + tok0 * a.nk_s[1],
                             static_cast<const T*>(a.nv) + h * a.nv_s[0] + tok0 * a.nv_s[1]};
    const int64_t row[2] = {a.nk_s[1], a.nv_s[1]};
    float* const scale[2] = {a.ks + at, a.vs + at};
    uint8_t* const dst[2] = {a.k + at * P * D, a.v + at * P * D};

    u32x4 x[2][KEEP][4];
    auto load_unit = [&](int kv, int u, u32x4* y) SDPA_INLINE {
        const int unit = lane + 64 * u, t = t_first + 4 * (unit / CH), c = unit % CH;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[k] = u32x4{};
            if (t + k >= off && t + k < end) y[k] = *reinterpret_cast<const u32x4*>(src[kv] + (t + k) * row[kv] + 8 * c);
        }
    };
    float amax[2] = {0.0f, 0.0f};
    // whether token k of any lane's unit u is new: single tokens skip the rest
    auto any_new = [&](int u, int k) SDPA_INLINE {
        const int t = t_first + 4 * ((lane + 64 * u) / CH) + k;
        return __builtin_amdgcn_ballot_w64(t >= off && t < end) != 0;
    };
    auto take_max = [&](int kv, int u, const u32x4* y) SDPA_INLINE {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!any_new(u, k)) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = Tr<T>::to_f((y[k][e >> 1] >> (16 * (e & 1))) & 0xffffu);
                amax[kv] = fmaxf(amax[kv], finite(f) ? fabsf(f) : 0.0f);
            }
        }
    };
#pragma unroll
    for (int u = KEEP; u < NU; ++u) {
        if (64 * u >= units) break;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) load_unit(kv, u, x[kv][u % KEEP]);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) take_max(kv, u, x[kv][u % KEEP]);
    }
#pragma unroll
    for (int u = 0; u < KEEP; ++u)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) load_unit(kv, u, x[kv][u]);
    float was[2], inv[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) was[kv] = off > 0 ? *scale[kv] : 0.0f;
#pragma unroll
    for (int u = 0; u < KEEP; ++u) {
        if (64 * u >= units) break;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) take_max(kv, u, x[kv][u]);
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) amax[kv] = fmaxf(amax[kv], __shfl_xor(amax[kv], k));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float now = fmaxf(scale_for(amax[kv]), was[kv]);
        inv[kv] = inverse(now);
        if (lane == 0) *scale[kv] = now;
        if (off > 0 && now > was[kv]) {  // the held codes move to the larger scale
            if (kv == 0) rescale_held<D, P, false>(dst[0], off, was[0] * inv[0], lane);
            else rescale_held<D, P, true>(dst[1], off, was[1] * inv[1], lane);
        }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        if (64 * u >= units) break;
        const int unit = lane + 64 * u, t = t_first + 4 * (unit / CH), c = unit % CH;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            if (u >= KEEP) load_unit(kv, u, x[kv][u % KEEP]);
            if (t >= end) continue;
            uint32_t code[4][2];  // [token][4 columns]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                code[k][0] = code[k][1] = 0u;
                if (!any_new(u, k)) continue;
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = Tr<T>::to_f((x[kv][u % KEEP][k][e >> 1] >> (16 * (e & 1))) & 0xffffu) * inv[kv];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    code[k][e] = encode2(f[4 * e], f[4 * e + 1]) | encode2(f[4 * e + 2], f[4 * e + 3]) << 16;
            }
            if (kv == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (t + k >= off && t + k < end) *reinterpret_cast<u32x2*>(dst[0] + (t + k) * D + 8 * c) = u32x2{code[k][0], code[k][1]};
                continue;
            }
            const bool whole = t >= off && t + 4 <= end;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t w = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) w |= ((code[k][e >> 2] >> (8 * (e & 3))) & 0xffu) << (8 * k);
                uint8_t* p = dst[1] + (8 * c + e) * P + t;
                if (whole) {
                    *reinterpret_cast<uint32_t*>(p) = w;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (t + k >= off && t + k < end) p[k] = (uint8_t)(w >> (8 * k));
                }
            }
        }
    }
}

template <typename T, int D>
static int launch_append(const CacheArgs& a, hipStream_t s) {
    const int64_t waves = (int64_t)a.B * a.Hkv * a.slots;
    const dim3 grid((uint32_t)((waves + 3) / 4)), block(256);
    switch (a.page) {
        case 16: sdpa_cache_append_kernel<T, D, 16><<<grid, block, 0, s>>>(a); break;
        case 32: sdpa_cache_append_kernel<T, D, 32><<<grid, block, 0, s>>>(a); break;
        case 64: sdpa_cache_append_kernel<T, D, 64><<<grid, block, 0, s>>>(a); break;
        default: sdpa_cache_append_kernel<T, D, 128><<<grid, block, 0, s>>>(a); break;
    }
    return (int)hipGetLastError();
}

template <typename T>
static int launch_append_t(const CacheArgs& a, hipStream_t s) {
    return a.D == 32 ? launch_append<T, 32>(a, s) : a.D == 64 ? launch_append<T, 64>(a, s) : launch_append<T, 128>(a, s);
}

int launch_cache_append(int dtype, const CacheArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == DT_F16 ? launch_append_t<_Float16>(a, s) : launch_append_t<__bf16>(a, s);
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
    // the order of the sequences moves on by one with every range: the ids of
    // an XCD go to its shader engines in turn, and the ranges past a short
    // sequence's end should not always fall to the same ones
    const int range = id / a.B, b = (id + range) % a.B;
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

    uint32_t odd = 0;
    // The page of 16 tokens from j on (-1: none), of this lane's key rows
    // (tokens 16 (n / 4) .. of a tile) and of its values (16 g ..). A tile's
    // loads are spread over the loop: its pages a tile ahead, its keys behind
    // the products of the tile before, its values ahead of its own products.
    auto page_of = [&](int j) SDPA_INLINE -> int { return j < s.len ? trow[j >> a.page_log2] : -1; };
    uint32_t kc[4][KB / 4];
    auto load_keys = [&](int t0, int page) SDPA_INLINE {
        const int64_t p = page >= 0 && page < a.n_pages ? page : 0;
        const int j = t0 + 16 * (n >> 2);
        const uint8_t* kp = a.k + ((p * a.Hkv + h) * a.page + (j & (a.page - 1)) + (n & 3)) * D + g * KB;
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
    };
    int t0 = j0 + 64 * wave;
    int pk = -1, pv_raw = -1;
    if (t0 < j1) {
        pk = page_of(t0 + 16 * (n >> 2));
        pv_raw = page_of(t0 + 16 * g);
        load_keys(t0, pk);
    }
    for (; t0 < j1; t0 += 64 * NW) {
        const int jv = t0 + 16 * g;
        const bool okv = pv_raw >= 0 && pv_raw < a.n_pages;
        const int64_t pv = okv ? pv_raw : 0;
        const int live = okv ? min(s.len - jv, 16) : 0;  // tokens of this lane that exist
        const uint8_t* vp = a.v + ((pv * a.Hkv + h) * D + n) * a.page + (jv & (a.page - 1));
        u32x4 vc[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d) vc[d] = *reinterpret_cast<const u32x4*>(vp + (int64_t)16 * d * a.page);
        const float ks = a.ks[pv * a.Hkv + h] * a.scale_log2, vs = a.vs[pv * a.Hkv + h];
        const int next = t0 + 64 * NW;
        if (next < j1) {
            pk = page_of(next + 16 * (n >> 2));
            pv_raw = page_of(next + 16 * g);
        }

        const bool ragged = __builtin_amdgcn_ballot_w64(live < 16) != 0;
        const bool cut = ragged || t0 + 64 > first_cut;
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
        if (next < j1) load_keys(next, pk);
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
        if (ragged) {  // codes past the end may be anything, NaN among them
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = min(max(live - 4 * i, 0), 4);
                const uint32_t mask = k == 4 ? 0xffffffffu : (1u << (8 * k)) - 1u;
#pragma unroll
                for (int d = 0; d < ND; ++d) vc[d][i] &= mask;
            }
        }
        if (cut) {
            // NaN among the values, where a row may not keep it (0 times NaN
            // would take it in): read as 0 here, added to its rows at the end
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t nan = (((vc[d][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                    odd |= nan;
                    vc[d][i] &= ~(nan * 0xffu);
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

    // NaN values of this wave's tiles that not every row keeps, one token at a time
    if (__builtin_amdgcn_ballot_w64(odd != 0) != 0) {
        for (int t = j0 + 64 * wave; t < j1; t += 64 * NW) {
            if (t + 64 <= first_cut) continue;
            for (int j = t; j < min(t + 64, s.len); ++j) {
                const int page = trow[j >> a.page_log2];
                if (page < 0 || page >= a.n_pages) continue;
                const uint8_t* vp = a.v + (((int64_t)page * a.Hkv + h) * D + 4 * g) * a.page + (j & (a.page - 1));
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool nan = (vp[(16 * d + r) * a.page] & 0x7f) == 0x7f;
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            if (nan && j <= limit[rt]) oacc[rt][d][r] = NAN;
                    }
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

// reference and sum of a row from its ranges' statistics, read by `n` lanes (a
// power of two) of which this is `lane`
__device__ __forceinline__ float2 join_stats(const float2* ml, int nr, int lane, int n) {
    float top = -INFINITY, sum = 0.0f;
    for (int i0 = lane; i0 < nr; i0 += 4 * n) {
        float2 e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = i0 + k * n < nr ? ml[i0 + k * n] : make_float2(-INFINITY, 0.0f);
        float up = top;
#pragma unroll
        for (int k = 0; k < 4; ++k) up = fmaxf(up, e[k].x);
        if (up == -INFINITY) continue;
        sum *= fast_exp2(top - up);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += e[k].y * fast_exp2(e[k].x - up);
        top = up;
    }
    for (int k = 1; k < n; k *= 2) {
        const float t2 = __shfl_xor(top, k), s2 = __shfl_xor(sum, k), up = fmaxf(top, t2);
        if (up != -INFINITY) sum = sum * fast_exp2(top - up) + s2 * fast_exp2(t2 - up);
        top = up;
    }
    return make_float2(top, sum);
}

// The ranges joined: O and LSE of every row, and the weights plus each key's
// sum of probabilities over the rows. Workgroups below n_rows take one row
// each, the rest 256 keys each of one (sequence, key head). Latency bounds it:
// a row's statistics are read by all threads at once.
template <typename T>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256)))
void sdpa_cache_join_kernel(const CacheArgs a, int n_rows) {
    __shared__ float part[256];
    __shared__ float factor[CACHE_MAX_RANGES];
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
        const int per = 256 / a.D, d = tid % a.D, k = tid / a.D;
        const float* const ws = a.ws_o + at * a.D + d;
        const float2 st = join_stats(a.ws_ml + at, nr, tid & 63, 64);
        for (int i = tid; i < nr; i += 256) {
            const float t = a.ws_ml[at + i].x;
            factor[i] = t == -INFINITY ? 0.0f : fast_exp2(t - st.x);
        }
        __syncthreads();
        float x = 0.0f;
        for (int i0 = k; i0 < nr; i0 += 8 * per) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = i0 + e * per < nr ? ws[(int64_t)(i0 + e * per) * a.D] : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = factor[min(i0 + e * per, nr - 1)];
                if (f != 0.0f) x += f * y[e];
            }
        }
        part[tid] = x;
        __syncthreads();
        if (k != 0) return;
        for (int i = 1; i < per; ++i) x += part[i * a.D + d];
        const int tok = r / a.group, head = h * a.group + r - tok * a.group;
        const float inv = st.y == 0.0f ? 0.0f : 1.0f / st.y;
        static_cast<T*>(a.o)[head * a.o_s[0] + (int64_t)(s.q0 + tok) * a.o_s[1] + d] = (T)(x * inv);
        if (d == 0)
            a.lse[head * a.l_s[0] + (int64_t)(s.q0 + tok) * a.l_s[1]] =
                st.y == 0.0f ? -INFINITY : (st.x + __builtin_amdgcn_logf(st.y)) * LN2;
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
    const bool live = j < min(s.len, a.w_cols);
    float x = 0.0f;  // the rows' sum first, so that adding it to the weight rounds once
    for (int r0 = 0; r0 < rows && j - tid < s.len; r0 += 32) {  // LSE of 32 rows at a time, eight lanes each
        const int r = r0 + (tid >> 3);
        float2 st = make_float2(-INFINITY, 0.0f);
        if (r < rows) st = join_stats(a.ws_ml + (row0 + r) * a.n_ranges, nr, tid & 7, 8);
        __syncthreads();
        if ((tid & 7) == 0) part[tid >> 3] = st.y == 0.0f ? INFINITY : st.x + __builtin_amdgcn_logf(st.y);
        __syncthreads();
        if (live) {
            const float* const tp = a.ws_t + (row0 + r0) * a.t_cols + j;
            const int n = min(32, rows - r0);
            for (int i0 = 0; i0 < n; i0 += 4) {
                float t[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = i0 + e < n ? tp[(int64_t)(i0 + e) * a.t_cols] : -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) x += fast_exp2(t[e] - part[min(i0 + e, n - 1)]);
            }
        }
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
// tokens to keep. The weights of the candidates (the tokens before the recent
// ones) become integers of the same order (NaN highest), counted from the
// smallest of them, so that the highest 11 bits of their range tell many of
// them apart: a histogram of those gives the bin that holds the last candidate
// kept. A bin of at most SELECT_LIST tokens is listed and one wave finds the
// value bit by bit with ballots; a longer one (many weights nearly equal) is
// taken apart by further histograms. After a scan over the waves' counts each
// wave emits its kept tokens in order, of those tied with the last the first.
// Counts are integers and the list's order has no effect, so the atomics leave
// nothing to chance. The integers stay in registers, 64 a thread, which is
// enough for 65536 candidates; beyond that every pass reads the weights again
// (an eviction of 8 heads of 65536 tokens takes 127 us so, 70 with registers).
// One CU bounds it, its loads (28 % of 32768 tokens' time), LDS atomics (23 %)
// and the ordered stores: 32768 tokens 25 us, 4096 9.8 (MI355X).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);  // negative: all bits turn, else the sign
    const uint32_t mag = u << 1;
    return mag > 0xff000000u ? 0xffffffffu : mag == 0u ? 0x80000000u : k;  // NaN; -0 as 0
}
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xffffffffu) return __builtin_bit_cast(float, 0x7fc00000u);
    return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

constexpr int SELECT_THREADS = 1024;
constexpr int SELECT_LIST = 256;
constexpr int SELECT_WORDS = 64;

// all lanes of a row of 16 get the row's smallest / largest
template <bool MAX>
__device__ __forceinline__ uint32_t row_extreme(uint32_t x) {
    auto with = [&](uint32_t y) SDPA_INLINE { x = MAX ? max(x, y) : min(x, y); };
    with(__builtin_amdgcn_update_dpp(x, x, 0x128, 0xf, 0xf, false));  // rotated by 8, 4, 2, 1
    with(__builtin_amdgcn_update_dpp(x, x, 0x124, 0xf, 0xf, false));
    with(__builtin_amdgcn_update_dpp(x, x, 0x122, 0xf, 0xf, false));
    with(__builtin_amdgcn_update_dpp(x, x, 0x121, 0xf, 0xf, false));
    return x;
}
template <bool MAX>
__device__ __forceinline__ uint32_t wave_extreme(uint32_t x) {
    const int y = (int)row_extreme<MAX>(x);
    uint32_t z = (uint32_t)__builtin_amdgcn_readlane(y, 0);
#pragma unroll
    for (int r = 16; r < 64; r += 16) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_readlane(y, r);
        z = MAX ? max(z, o) : min(z, o);
    }
    return z;
}

// f(4 i) for every i below words / 4 (N at most), unrolled
template <int... I, typename F>
__device__ __forceinline__ void by_four(std::integer_sequence<int, I...>, int words, F f) {
    (void)((4 * I < words && (f(std::integral_constant<int, 4 * I>{}), true)) && ...);
}

// WORDS: 64-token words whose integers a wave keeps in registers, a multiple of
// 4 (0: any number, read again from memory).
template <int WORDS>
__global__ __attribute__((amdgpu_flat_work_group_size(SELECT_THREADS, SELECT_THREADS)))
void sdpa_cache_select_kernel(const CacheArgs a) {
    constexpr int NT = SELECT_THREADS, NWV = NT / 64, NB = 2048;
    static_assert(NWV == 16, "the waves' extremes fit one row of lanes");
    __shared__ int hist[NB];
    __shared__ uint32_t list[SELECT_LIST];
    __shared__ uint32_t lo_s[NWV], hi_s[NWV];
    __shared__ int wsum[NWV], wtie[NWV];
    __shared__ int pick_s, above_s, bin_s, list_n;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv;
    const int len = (int)min((int64_t)held_tokens(a, b), (int64_t)a.w_cols);
    const int n = min(len, a.budget);
    const int late = len - min(a.recent, n);  // tokens from here on are kept, those before are candidates
    const int take = n - (len - late);        // candidates kept
    const float* w = a.w_in + b * a.wi_s[0] + h * a.wi_s[1];
    float* wo = a.w_out + b * a.wo_s[0] + h * a.wo_s[1];
    int* kept = a.kept + ((int64_t)b * a.Hkv + h) * a.budget;
    // a wave's stretch: `words` words of 64 tokens, a multiple of 4
    const int words = ((late + 4 * NT - 1) / (4 * NT)) * 4;
    const int t0 = wave * words * 64 + lane;

    float recent[4];  // the first recent weights, in flight behind all that follows
    if constexpr (WORDS > 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) recent[e] = e * NT + tid < len - late ? w[late + e * NT + tid] : 0.0f;
    }
    constexpr std::make_integer_sequence<int, WORDS / 4> quads{};
    uint32_t key[WORDS > 0 ? WORDS : 1] = {};
    uint32_t base = 0;  // what `each` takes from the integers
    // f(word, integer) for this wave's words in order; no candidate has integer 0, all else has
    auto each = [&](auto f) SDPA_INLINE {
        if constexpr (WORDS > 0) {
            by_four(quads, words, [&](auto i) SDPA_INLINE {
#pragma unroll
                for (int e = 0; e < 4; ++e) f(i + e, key[i + e]);
            });
        } else {
            for (int i = 0; i < words; i += 4) {
                uint32_t k[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = t0 + 64 * (i + e);
                    k[e] = j < late ? order_key(w[j]) - base : 0u;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) f(i + e, k[e]);
            }
        }
    };
    if constexpr (WORDS > 0) {
        const rsrc_t wr = make_rsrc(w, (uint32_t)late * 4);
        by_four(quads, words, [&](auto i) SDPA_INLINE {
#pragma unroll
            for (int e = 0; e < 4; ++e) key[i + e] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(wr, 4 * (t0 + 64 * (i + e)), 0, 0);
        });
        int end = late;  // opaque: the comparisons are made again, rather than kept for every word
        asm volatile("" : "+s"(end));
        by_four(quads, words, [&](auto i) SDPA_INLINE {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                key[i + e] = t0 + 64 * (i + e) < end ? order_key(__builtin_bit_cast(float, key[i + e])) : 0u;
        });
    }
    // the largest `pick` that `take` candidates reach, and how many of those equal to it are kept
    uint32_t pick = take == 0 ? 0xffffffffu : 0u;  // none, or every candidate
    int need = 0;
    if (take > 0 && take < late) {
        auto clear = [&]() SDPA_INLINE {
            for (int i = tid; i < NB; i += NT) hist[i] = 0;
        };
        // one more token in bin `bin` for every lane with `in` (all lanes call)
        auto add = [&](int bin, bool in) SDPA_INLINE {
            const uint64_t who = __builtin_amdgcn_ballot_w64(in);
            if (who == 0) return;
            const int first = __builtin_amdgcn_readlane(bin, __builtin_ctzll(who));
            if (__builtin_amdgcn_ballot_w64(in && bin != first) == 0) {  // one bin (equal weights): one addition
                if (lane == 0) atomicAdd(&hist[first], __popcll(who));
            } else if (in) {
                atomicAdd(&hist[bin], 1);
            }
        };
        clear();
        if (tid == 0) list_n = 0;
        uint32_t lo = 0xffffffffu, hi = 0;
        each([&](int, uint32_t k) SDPA_INLINE {
            lo = min(lo, k - 1);  // 0 counts as the largest
            hi = max(hi, k);
        });
        lo = wave_extreme<false>(lo);
        hi = wave_extreme<true>(hi);
        if (lane == 0) {
            lo_s[wave] = lo;
            hi_s[wave] = hi;
        }
        __syncthreads();
        base = __builtin_amdgcn_readfirstlane((int)row_extreme<false>(lo_s[lane & 15]));
        // integers are 1 .. hi - base now, of `rem` bits that `pick` lacks
        int rem = 32 - __builtin_clz(__builtin_amdgcn_readfirstlane((int)row_extreme<true>(hi_s[lane & 15])) - base);
        if constexpr (WORDS > 0) {
            by_four(quads, words, [&](auto i) SDPA_INLINE {
#pragma unroll
                for (int e = 0; e < 4; ++e) key[i + e] -= key[i + e] != 0 ? base : 0u;
            });
        }
        need = take;
        bool first = true;
        while (rem > 0) {
            if (!first && bin_s <= SELECT_LIST) {  // bin_s: tokens that share the bits found
                uint32_t none = 0;  // opaque, as below
                asm volatile("" : "+s"(none));
                each([&](int, uint32_t k) SDPA_INLINE {
                    if (k != none && k >> rem == pick >> rem) list[atomicAdd(&list_n, 1)] = k & ((1u << rem) - 1);
                });
                __syncthreads();
                if (wave == 0) {
                    uint32_t x[SELECT_LIST / 64], v = 0;
#pragma unroll
                    for (int e = 0; e < SELECT_LIST / 64; ++e) x[e] = lane + 64 * e < list_n ? list[lane + 64 * e] : 0u;
                    auto reach = [&](uint32_t t) SDPA_INLINE {  // tokens of at least t > 0
                        int c = 0;
#pragma unroll
                        for (int e = 0; e < SELECT_LIST / 64; ++e) c += __popcll(__builtin_amdgcn_ballot_w64(x[e] >= t));
                        return c;
                    };
                    for (int bit = rem - 1; bit >= 0; --bit)
                        if (reach(v | 1u << bit) >= need) v |= 1u << bit;
                    if (lane == 0) {
                        pick_s = (int)v;
                        above_s = reach(v + 1);
                    }
                }
                __syncthreads();
                pick |= (uint32_t)pick_s;
                need -= above_s;
                break;
            }
            const int shift = max(rem - 11, 0);
            if (!first) {
                clear();
                __syncthreads();
            }
            uint32_t none = 0;  // opaque: compared in every pass, rather than a mask kept for every word
            asm volatile("" : "+s"(none));
            each([&](int, uint32_t k) SDPA_INLINE {
                add((int)(k >> shift) & (NB - 1), k != none && (first || k >> rem == pick >> rem));
            });
            __syncthreads();
            // the highest bin that, with all above it, holds `need` tokens:
            // a wave sums 128 bins, from the top down over lanes and waves
            const int top = NB - 1 - wave * 128 - 2 * lane;
            const int c0 = hist[top], c1 = hist[top - 1];
            int x = c0 + c1;
#pragma unroll
            for (int k = 1; k < 64; k *= 2) {
                const int y = __shfl_up(x, k);
                if (lane >= k) x += y;
            }
            if (lane == 63) wsum[wave] = x;
            __syncthreads();
            int before = 0;
            for (int i = 0; i < wave; ++i) before += wsum[i];
            const int upto = before + x;  // tokens in the bins down to this lane's second
            if (upto >= need && upto - c0 - c1 < need) {
                const bool one = upto - c1 >= need;
                pick_s = one ? top : top - 1;
                above_s = one ? upto - c1 - c0 : upto - c1;
                bin_s = one ? c0 : c1;
            }
            __syncthreads();
            pick |= (uint32_t)pick_s << shift;
            need -= above_s;
            rem = shift;
            first = false;
        }
    }
    // count, over the waves
    pick = (uint32_t)__builtin_amdgcn_readfirstlane((int)pick);
    need = __builtin_amdgcn_readfirstlane(need);
    int cnt = 0, tie = 0;
    each([&](int, uint32_t k) SDPA_INLINE {
        cnt += __popcll(__builtin_amdgcn_ballot_w64(k > pick));
        tie += __popcll(__builtin_amdgcn_ballot_w64(k == pick));
    });
    __syncthreads();
    if (lane == 0) {
        wsum[wave] = cnt;
        wtie[wave] = tie;
    }
    __syncthreads();
    int at = 0, ties = 0;
    for (int i = 0; i < wave; ++i) {
        at += wsum[i] + min(ties + wtie[i], need) - min(ties, need);
        ties += wtie[i];
    }
    asm volatile("" : "+s"(pick));  // opaque: compared again, rather than every word's two masks kept
    const uint64_t below = (uint64_t(1) << lane) - 1;
    const rsrc_t kr = make_rsrc(kept, 4 * (uint32_t)max(take, 0)), wor = make_rsrc(wo, 4 * (uint32_t)max(take, 0));
    each([&](int i, uint32_t k) SDPA_INLINE {
        uint64_t kb = __builtin_amdgcn_ballot_w64(k > pick);
        const uint64_t tb = __builtin_amdgcn_ballot_w64(k == pick);
        if (tb != 0) {
            const bool tied = (tb >> lane & 1) && ties + __popcll(tb & below) < need;
            kb |= __builtin_amdgcn_ballot_w64(tied);
            ties += __popcll(tb);
        }
        if (kb >> lane & 1) {
            const int to = at + __popcll(kb & below);
            if constexpr (WORDS > 0) {
                __builtin_amdgcn_raw_buffer_store_b32(t0 + 64 * i, kr, 4 * to, 0, 0);
                // in place too: every candidate is in registers
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, key_value(k + base)), wor, 4 * to, 0, 0);
            } else {
                kept[to] = t0 + 64 * i;
            }
        }
        at += __popcll(kb);
    });
    for (int i = tid; i < len - late; i += NT) kept[take + i] = late + i;
    for (int i = n + tid; i < a.budget; i += NT) kept[i] = -1;
    // the recent tokens' weights (or, without integers in registers, all): a
    // token never moves up, and every round's reads end before its writes
    // begin, so that they may move in place. The first recent ones were read
    // before the barriers above.
    int i0 = 0;
    if constexpr (WORDS > 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e * NT + tid < len - late) wo[take + e * NT + tid] = recent[e];
        i0 = take + 4 * NT;
    } else {
        __syncthreads();
    }
    for (; i0 < n; i0 += 4 * NT) {
        float x[4] = {};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e * NT + tid;
            if (i < n) x[e] = w[WORDS > 0 ? late + i - take : kept[i]];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i0 + e * NT + tid < n) wo[i0 + e * NT + tid] = x[e];
        __syncthreads();
    }
    for (int i = n + tid; i < a.w_cols; i += NT) wo[i] = 0.0f;
    if (h == 0 && tid == 0) a.new_lens[b] = n;
}

// sdpa_cache_move_kernel: one workgroup per (page moved to, key head). The
// page's scales are the largest of its tokens' scales; slots past the kept
// tokens hold zeros. k rows move as 16-byte pieces. The bytes of a v token lie
// `page` apart, so that every cache line of a v page that keeps a token is
// read whatever the access: these pages are staged in LDS whole (kept tokens
// are ordered, so few pages hold them), in batches of MOVE_STAGE bytes, and
// the tokens' columns picked there. 16 KB a batch leave room for eight
// workgroups a CU, which hide the loads (16 sequences of up to 4096 tokens, 8
// heads, to 1024: 27 us, 3.6 TB/s of what it has to move; 32 KB 32 us, 64 KB
// 45). The chain kept -> table -> scale -> page
// of dependent loads is gone through once for k and v together, and the loads
// of k and of the first batch of v are in flight at once.
template <int BYTES>
constexpr int MOVE_STAGE = BYTES > 16 * 1024 ? BYTES : 16 * 1024;

template <int D, int P>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256)))
void sdpa_cache_move_kernel(const CacheArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t stage[MOVE_STAGE<D * P>];
    __shared__ int src_slot[P], src_off[P], page_list[P];
    __shared__ float rk[P], rv[P];
    __shared__ float redk[2], redv[2];
    __shared__ int firsts[2];
    constexpr int LOG = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    const int tid = threadIdx.x, lane = tid & 63;
    int id = blockIdx.x;
    const int h = id % a.Hkv;
    id /= a.Hkv;
    const int b = (id + id / a.B) % a.B, i0 = (id / a.B) * P;  // rotated, as the attention's ranges
    const int len = (int)min((int64_t)held_tokens(a, b), (int64_t)a.w_cols);
    const int n = min(min(len, a.budget) - i0, P);
    if (n <= 0) return;
    const int to = a.to[b * a.to_s + i0 / P];
    if (to < 0 || to >= a.n_pages) return;
    if (tid < 128) {  // the first two waves: the page's tokens
        float sk = 0.0f, sv = 0.0f;
        int page = -1;
        bool first = false;  // this token is the first of its source page
        if (tid < n) {
            const int* const kp = a.kept + ((int64_t)b * a.Hkv + h) * a.budget + i0;
            const int j = kp[tid], before = tid > 0 ? kp[tid - 1] : -1;
            first = tid == 0 || (j >> LOG) != (before >> LOG);
            page = a.table[b * a.table_s + (j >> LOG)];
            if (page < 0 || page >= a.n_pages) {
                page = -1;
            } else {
                sk = a.ks[(int64_t)page * a.Hkv + h];
                sv = a.vs[(int64_t)page * a.Hkv + h];
            }
            src_off[tid] = j & (P - 1);
        }
        if (tid < P) {
            rk[tid] = sk;
            rv[tid] = sv;
        }
        // number the source pages in order
        const uint64_t fb = __builtin_amdgcn_ballot_w64(first);
        const int slot = __popcll(fb & ((uint64_t(2) << lane) - 1)) - 1;
        if (lane == 0) firsts[tid >> 6] = __popcll(fb);
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
            sk = fmaxf(sk, __shfl_xor(sk, k));
            sv = fmaxf(sv, __shfl_xor(sv, k));
        }
        if (lane == 0) {
            redk[tid >> 6] = sk;
            redv[tid >> 6] = sv;
        }
        // the second wave numbers from 64 on for now (its pages follow the first's 64 at most)
        if (tid < P) src_slot[tid] = tid < n ? slot : -1;
        if (first) page_list[P > 64 && tid >= 64 ? 64 + slot : slot] = page;
    }
    __syncthreads();
    const int n_lo = firsts[0];
    const float top_k = fmaxf(fmaxf(redk[0], redk[1]), SCALE_MIN), top_v = fmaxf(fmaxf(redv[0], redv[1]), SCALE_MIN);
    const float inv_k = inverse(top_k), inv_v = inverse(top_v);
    // source page number p: page_list[p], or past n_lo the second wave's (a
    // token whose page began in the first wave has slot -1 there: page n_lo - 1)
    auto page_of = [&](int p) SDPA_INLINE -> int { return P > 64 && p >= n_lo ? page_list[64 + p - n_lo] : page_list[p]; };
    auto slot_of = [&](int t) SDPA_INLINE -> int {
        return t >= n ? -1 : P > 64 && t >= 64 ? n_lo + src_slot[t] : src_slot[t];
    };
    const int n_src = n_lo + (P > 64 ? firsts[1] : 0);
    if (tid == 0) {
        a.ks[(int64_t)to * a.Hkv + h] = top_k;
        a.vs[(int64_t)to * a.Hkv + h] = top_v;
    }
    constexpr int BYTES = D * P, CHUNKS = BYTES / 16;
    constexpr int BATCH = MOVE_STAGE<BYTES> / BYTES < P ? MOVE_STAGE<BYTES> / BYTES : P;  // v pages staged at a time
    constexpr int NL = (BATCH * CHUNKS + 255) / 256;                         // 16-byte loads of a thread
    constexpr int PER = D / 16, NK = (CHUNKS + 255) / 256;                   // pieces of a k row, pieces of a thread
    u32x4 kx[NK];
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        const int i = tid + 256 * k, t = i / PER, sl = i < CHUNKS ? slot_of(t) : -1;
        const int pg = sl < 0 ? -1 : page_of(sl);
        kx[k] = u32x4{};
        if (pg >= 0)
            kx[k] = *reinterpret_cast<const u32x4*>(a.k + (((int64_t)pg * a.Hkv + h) * P + src_off[t]) * D + 16 * (i % PER));
    }
    // thread: token t of the page, v columns d0, d0 + STEP, ...
    constexpr int STEP = 256 / P, NC = D / STEP, G = NC < 4 ? NC : 4;
    const int t = tid % P, d0 = tid / P;
    const int mine = slot_of(t);
    const bool exists = mine >= 0 && page_of(max(mine, 0)) >= 0;
    const float f = rv[t] * inv_v;
    uint32_t col[(NC + 3) / 4];
#pragma unroll
    for (int k = 0; k < (NC + 3) / 4; ++k) col[k] = 0u;
    for (int s0 = 0; s0 < n_src; s0 += BATCH) {
        const int m = min(BATCH, n_src - s0);
        u32x4 x[NL];
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const int i = tid + 256 * k;
            const int64_t pg = max(page_of(s0 + min(i / CHUNKS, m - 1)), 0);
            if (i < m * CHUNKS) x[k] = reinterpret_cast<const u32x4*>(a.v + (pg * a.Hkv + h) * BYTES)[i % CHUNKS];
        }
#pragma unroll
        for (int k = 0; k < NL; ++k)
            if (tid + 256 * k < m * CHUNKS) reinterpret_cast<u32x4*>(stage)[tid + 256 * k] = x[k];
        __syncthreads();
        if (exists && mine >= s0 && mine < s0 + m) {
            const uint8_t* const p = stage + (mine - s0) * BYTES + src_off[t];
#pragma unroll
            for (int k = 0; k < NC; k += G) {
                uint32_t c = 0;
#pragma unroll
                for (int e = 0; e < G; ++e) c |= (uint32_t)p[(d0 + (k + e) * STEP) * P] << (8 * e);
                col[k / 4] = f != 1.0f ? rescale4(c, f) : c;
            }
        }
        __syncthreads();
    }
    uint8_t* const kd = a.k + ((int64_t)to * a.Hkv + h) * BYTES;
    uint8_t* const vd = a.v + ((int64_t)to * a.Hkv + h) * BYTES;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        const int i = tid + 256 * k;
        if (i >= CHUNKS) break;
        const float fk = rk[i / PER] * inv_k;
        if (fk != 1.0f)
#pragma unroll
            for (int e = 0; e < 4; ++e) kx[k][e] = rescale4(kx[k][e], fk);
        reinterpret_cast<u32x4*>(kd)[i] = kx[k];
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) stage[(d0 + k * STEP) * P + t] = (uint8_t)(col[k / 4] >> (8 * (k % 4)));
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        const int i = tid + 256 * k;
        if (i < CHUNKS) reinterpret_cast<u32x4*>(vd)[i] = reinterpret_cast<const u32x4*>(stage)[i];
    }
}

template <int D>
static int launch_move(const CacheArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)a.B * a.Hkv * a.to_pages), block(256);
    switch (a.page) {
        case 16: sdpa_cache_move_kernel<D, 16><<<grid, block, 0, s>>>(a); break;
        case 32: sdpa_cache_move_kernel<D, 32><<<grid, block, 0, s>>>(a); break;
        case 64: sdpa_cache_move_kernel<D, 64><<<grid, block, 0, s>>>(a); break;
        default: sdpa_cache_move_kernel<D, 128><<<grid, block, 0, s>>>(a); break;
    }
    return (int)hipGetLastError();
}

int launch_cache_evict(const CacheArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    // lengths are at most the weights' row and the table's pages
    const int64_t pages = (int64_t)a.max_pages * a.page, most = a.w_cols < pages ? a.w_cols : pages;
    const dim3 grid(a.B * a.Hkv), block(SELECT_THREADS);
    if (most <= 1024 * SELECT_WORDS) sdpa_cache_select_kernel<SELECT_WORDS><<<grid, block, 0, s>>>(a);
    else sdpa_cache_select_kernel<0><<<grid, block, 0, s>>>(a);
    int e = (int)hipGetLastError();
    if (e || a.to_pages == 0) return e;
    return a.D == 32 ? launch_move<32>(a, s) : a.D == 64 ? launch_move<64>(a, s) : launch_move<128>(a, s);
}

}  // namespace sdpa
