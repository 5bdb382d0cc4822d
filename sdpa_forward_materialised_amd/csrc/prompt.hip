// Attention over packed prompts without the probability map, and the weight
// that every key of those prompts received.
//
// sdpa_prompt_kernel: O = softmax(scale Q K^T) V and the row log-sum-exp, in
// one sweep over the keys. With a running reference m_i >= max_j s_ij - 8 (in
// base 2) of every row, l_i = sum_j 2^(s_ij - m_i) and
// A_i = sum_j 2^(s_ij - m_i) v_j are updated tile by tile; a tile whose row
// maximum passes m_i + 8 raises m_i and scales l_i and A_i by 2^(old - new).
// O_i = A_i / l_i, LSE_i = (m_i + log2 l_i) ln 2. A reference up to 2^8 below
// the maximum loses nothing (float32 sums, 16-bit floating weights keep their
// relative precision) and most tiles then skip the scaling of A.
#include "twopass.h"
#include "serve.h"

namespace sdpa {

// sequence b of packed tensors, clamped to them
struct Seq {
    int q0, k0, nq, nk, coff;
};
__device__ __forceinline__ Seq sequence(const PackArgs& a, int b) {
    Seq s;
    s.q0 = min(max(a.cu_q[b], 0), a.Tq);
    s.k0 = min(max(a.cu_k[b], 0), a.Tkv);
    s.nq = min(min(max(a.cu_q[b + 1], s.q0), a.Tq) - s.q0, a.max_q);
    s.nk = min(min(max(a.cu_k[b + 1], s.k0), a.Tkv) - s.k0, a.max_k);
    s.coff = a.causal == 2 ? s.nk - s.nq : 0;
    return s;
}

template <typename T>
__device__ __forceinline__ typename Tr<T>::vec load_operand(rsrc_t r, uint32_t off, int mul) {
    if constexpr (sizeof(T) == 2) {
        u32x4 x = ld128(r, off);
        if (mul != 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = mul == 0 ? 0u : x[e] ^ 0x80008000u;
        }
        return as_vec<T>(x);
    } else {
        const float x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
        return mul == 1 ? x : mul == 0 ? 0.0f : -x;
    }
}

// Workgroup id -> (block counted from the heaviest, sequence, head): blocks
// of the same index are neighbours (heaviest first over the whole grid), and
// the ids that land on one XCD (id % 8) share key heads. Within an XCD ids go
// to its shader engines in turn, so the order of a row's (sequence, head)
// pairs moves on by one with every block: without that, the empty workgroups
// of a short sequence in a ragged batch always fall to the same engines, whose
// CUs then stay idle (two sequences of 12289 and 5003 tokens, 16 heads of 128:
// PROMPT_ROT).
struct PackWork {
    int b, h, blk;
};
__device__ __forceinline__ PackWork pack_work(int id, int B, int H, int n_blk) {
    const int n = B * H;
    PackWork w;
    w.blk = id / n;
    int r = id % n;
    if (n % 8 == 0) {
        const int per = n >> 3;
        r = (r & 7) * per + ((r >> 3) + w.blk) % per;
    } else {
        r = (r + w.blk) % n;
    }
    w.h = r / B;
    w.b = r - w.h * B;
    return w;
}

template <typename T, int D>
struct PromptCfg {
    static constexpr int NW = 4;
    static constexpr int RB = 1;                         // 32-row blocks per wave
    static constexpr int TN = sizeof(T) == 2 ? 64 : 32;  // keys per tile
    using C = TwoPassCfg<T, D, NW, MASK_NONE, true, TN, true>;
    static constexpr int QB = 32 * RB * NW;
    static constexpr int LDS_BYTES = 4 * C::TILEB;
};

template <typename T, int D>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(PromptCfg<T, D>::RB == 2 ? 1 : 2)))
void sdpa_prompt_kernel(const PackArgs a) {
    using P = PromptCfg<T, D>;
    using C = typename P::C;
    using TR = Tr<T>;
    using vec = typename TR::vec;
    constexpr int SZ = (int)sizeof(T), RB = P::RB, NW = P::NW, TN = P::TN, NKB = TN / 32, ND = D / 32;
    constexpr int KSTEP = 2 * TR::KH, NKS = D / KSTEP;
    __shared__ __attribute__((aligned(16))) uint8_t smem[P::LDS_BYTES];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const PackWork w = pack_work(blockIdx.x, a.B, a.Hq, a.n_blk);
    const Seq s = sequence(a, w.b);
    const int q0 = (a.n_blk - 1 - w.blk) * P::QB;
    if (q0 >= s.nq) return;
    const int kend = a.causal ? min(s.nk, max(0, min(q0 + P::QB, s.nq) + s.coff)) : s.nk;
    const int ntiles = (kend + TN - 1) / TN;
    const int hk = w.h / a.group;

    const rsrc_t qr = make_rsrc(static_cast<const T*>(a.q) + s.q0 * a.q_s[1] + w.h * a.q_s[0], a.q_ext);
    const rsrc_t kr = make_rsrc(static_cast<const T*>(a.k) + s.k0 * a.k_s[1] + hk * a.k_s[0], a.k_ext);
    const rsrc_t vr = make_rsrc(static_cast<const T*>(a.v) + s.k0 * a.v_s[1] + hk * a.v_s[0], a.v_ext);
    const rsrc_t orr = make_rsrc(static_cast<T*>(a.o) + s.q0 * a.o_s[1] + w.h * a.o_s[0], a.o_ext);
    const rsrc_t lr = make_rsrc(a.lse + s.q0 * a.l_s[1] + w.h * a.l_s[0], a.l_ext);
    const uint32_t krow = (uint32_t)(a.k_s[1] * SZ), vrow = (uint32_t)(a.v_s[1] * SZ);

    auto load_tile = [&](int t) SDPA_INLINE {
        uint8_t* const kd = smem + (t & 1) * 2 * C::TILEB;
        uint8_t* const vd = kd + C::TILEB;
#pragma unroll
        for (int jj = 0; jj < C::NI / NW; ++jj) {
            const int j = jj * NW + wave;
            const int row = j * C::RPI + lane / C::CPR;
            const bool ok = t * TN + row < s.nk;
            const int ck = (lane % C::CPR) ^ C::fk(row), cv = (lane % C::CPR) ^ C::fv(row);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(kr, (lds_void*)(kd + j * 1024), 16, pred(ok, row * krow + ck * 16),
                                                     (uint32_t)(t * TN) * krow, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (lds_void*)(vd + j * 1024), 16, pred(ok, row * vrow + cv * 16),
                                                     (uint32_t)(t * TN) * vrow, 0, 0);
        }
    };
    static_assert(C::NI % NW == 0, "tile loads split evenly over the waves");

    const int qw = q0 + wave * 32 * RB;  // this wave's first row
    int qi[RB];
    vec qf[RB][NKS];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        qi[rb] = qw + 32 * rb + n;
        const bool ok = qi[rb] < s.nq;
        const uint32_t qoff = (uint32_t)((ok ? qi[rb] : 0) * a.q_s[1] * SZ);
#pragma unroll
        for (int c = 0; c < NKS; ++c)
            qf[rb][c] = load_operand<T>(qr, pred(ok, qoff + (c * KSTEP + hf * TR::KH) * SZ), a.q_mul);
    }
    f32x16 oacc[RB][ND];
    float m[RB], l[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        m[rb] = -INFINITY;
        l[rb] = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) oacc[rb][d] = f32x16{};
    }
    const int kr0 = swap23(n);
    const int trg = lane >> 4, trs = lane & 15;
    const int tr_row = 8 * (trg >> 1) + (trs >> 2);
    const int tr_col = 16 * (trg & 1) + 4 * (((trs & 1) << 1) | ((trs >> 1) & 1));

    auto tile = [&](int t, auto edge_c) SDPA_INLINE {
        constexpr bool edge = decltype(edge_c)::value;
        const uint8_t* const kt = smem + (t & 1) * 2 * C::TILEB;
        const uint8_t* const vt = kt + C::TILEB;
        f32x16 acc[RB][NKB];
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) acc[rb][kb] = f32x16{};
#pragma unroll
            for (int c = 0; c < NKS; ++c) {
                const int row = 32 * kb + kr0, elem = c * KSTEP + hf * TR::KH;
                const uint8_t* p = kt + C::pos_k(row, elem * SZ / 16) * 16 + ((elem * SZ) & 15);
                const vec ka = *reinterpret_cast<const vec*>(p);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) acc[rb][kb] = TR::mfma(ka, qf[rb][c], acc[rb][kb]);
            }
        }
        float top[RB];
        bool grow = false;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            if constexpr (edge) {
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    const int jb = t * TN + 32 * kb;
                    const int lim = min(s.nk - 1 - jb, a.causal ? qi[rb] + s.coff - jb : 0x7fffffff) - 8 * hf;
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[rb][kb][r] = kk(0, r) > lim ? -INFINITY : acc[rb][kb][r];
                }
            }
            float x = acc[rb][0][0];
#pragma unroll
            for (int i = 1; i < 16 * NKB; ++i) x = fmaxf(x, acc[rb][i >> 4][i & 15]);
            top[rb] = x * a.scale_log2;
            grow = grow || top[rb] > m[rb] + 8.0f;
        }
        if (__builtin_amdgcn_ballot_w64(grow) != 0) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const float up = fmaxf(m[rb], fmaxf(top[rb], __shfl_xor(top[rb], 32)));
                const float f = up == -INFINITY ? 1.0f : fast_exp2(m[rb] - up);
                m[rb] = up;
                l[rb] *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) oacc[rb][d][r] *= f;
            }
        }
        float p[RB][16 * NKB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            const float mu = m[rb] == -INFINITY ? 0.0f : m[rb];
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 16 * NKB; ++i) {
                p[rb][i] = fast_exp2(__builtin_fmaf(acc[rb][i >> 4][i & 15], a.scale_log2, -mu));
                sum += p[rb][i];
            }
            l[rb] += sum;
        }
        // A^T += V^T P^T
        if constexpr (SZ == 2) {
#pragma unroll
            for (int kc = 0; kc < 2 * NKB; ++kc) {  // 16 keys each
                vec pv[RB];
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) pv[rb] = TR::cvt8(p[rb] + 8 * kc);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    u32x2 half[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = 16 * kc + tr_row + 4 * r, col = 32 * d + tr_col;
                        half[r] = lds_read_tr16(vt + C::pos_v(row, col * SZ / 16) * 16 + ((col * SZ) & 15));
                    }
                    const vec va = __builtin_bit_cast(vec, u32x4{half[0][0], half[0][1], half[1][0], half[1][1]});
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) oacc[rb][d] = TR::mfma(va, pv[rb], oacc[rb][d]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16 * NKB; ++i) {
                const int row = 32 * (i >> 4) + kk(hf, i & 15);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int col = 32 * d + swap23(n);
                    const float va = *reinterpret_cast<const float*>(vt + C::pos_v(row, col * SZ / 16) * 16 + ((col * SZ) & 15));
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) oacc[rb][d] = TR::mfma(va, p[rb][i], oacc[rb][d]);
                }
            }
        }
    };

    // tiles before t_full hold kept keys only, for every row of the wave;
    // tiles from t_end on none
    const int last_row = min(qw + 32 * RB, s.nq) - 1;
    const bool live = qw < s.nq;
    const int t_end = !live ? 0 : a.causal ? max(0, min(ntiles, (last_row + s.coff + TN) / TN)) : ntiles;
    const int t_full = min(t_end, (a.causal ? max(0, min(s.nk, qw + s.coff + 1)) : s.nk) / TN);
    if (ntiles > 0) load_tile(0);
    wait_vmem();
    __syncthreads();
    for (int t = 0; t < ntiles; ++t) {
        if (t + 1 < ntiles) load_tile(t + 1);
        if (t < t_full) tile(t, std::false_type{});
        else if (t < t_end) tile(t, std::true_type{});
        wait_vmem();
        __syncthreads();
    }

#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const bool ok = qi[rb] < s.nq;
        const float sum = l[rb] + __shfl_xor(l[rb], 32);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const uint32_t ooff = (uint32_t)((ok ? qi[rb] : 0) * a.o_s[1] * SZ);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = oacc[rb][d][r] * inv;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (a.o_vec) store8<T, true>(orr, ooff, ok, 32 * d + 16 * c + 8 * hf, D, x + 8 * c);
                else store8<T, false>(orr, ooff, ok, 32 * d + 16 * c + 8 * hf, D, x + 8 * c);
            }
        }
        const float lse = sum == 0.0f ? -INFINITY : (m[rb] + __builtin_amdgcn_logf(sum)) * LN2;
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, lse), lr,
                                              pred(ok && hf == 0, (uint32_t)((ok ? qi[rb] : 0) * a.l_s[1] * 4)), 0, 0);
    }
}

// The same for 16-bit types and many rows: 64 rows a wave (two 32-row blocks
// that share every K and V operand read from LDS: with one block a wave the
// operand reads alone take the LDS as long as the products take the matrix
// units), 256 rows a workgroup, and the three parts of neighbouring 32-key
// blocks run interleaved, one wave keeping matrix and vector units busy at
// once: step j does the exponentials of block j between the products
// S(j + 1) = K Q^T and A += V P(j - 1)^T. Row references are whole numbers, so
// that the weights P(j - 1), rounded already, scale exactly when a reference
// rises in step j.
#ifndef AHD
#define AHD 2
#endif
#ifndef WIDE_RB
#define WIDE_RB 1
#endif
template <typename T, int D>
struct WideCfg {
    static constexpr int NW = 4, RB = WIDE_RB, TN = 64;
    using C = TwoPassCfg<T, D, NW, MASK_NONE, true, TN, true>;
    static constexpr int QB = 32 * RB * NW;
    static constexpr int LDS_BYTES = 4 * C::TILEB;
};

template <typename T, int D>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(WIDE_RB == 2 ? 1 : 2)))
void sdpa_prompt_wide_kernel(const PackArgs a) {
    using P = WideCfg<T, D>;
    using C = typename P::C;
    using TR = Tr<T>;
    using vec = typename TR::vec;
    constexpr int SZ = 2, RB = P::RB, NW = P::NW, TN = P::TN, ND = D / 32, NKS = D / 16;
    constexpr int SLOTS = RB * NKS, EPS = 16 * RB / SLOTS;  // products of each kind in a step; exponentials per slot
    __shared__ __attribute__((aligned(16))) uint8_t smem[P::LDS_BYTES];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const PackWork w = pack_work(blockIdx.x, a.B, a.Hq, a.n_blk);
    const Seq s = sequence(a, w.b);
    const int q0 = (a.n_blk - 1 - w.blk) * P::QB;
    if (q0 >= s.nq) return;
    const int kend = a.causal ? min(s.nk, max(0, min(q0 + P::QB, s.nq) + s.coff)) : s.nk;
    const int ntiles = (kend + TN - 1) / TN;
    const int hk = w.h / a.group;

    const rsrc_t qr = make_rsrc(static_cast<const T*>(a.q) + s.q0 * a.q_s[1] + w.h * a.q_s[0], a.q_ext);
    const rsrc_t kr = make_rsrc(static_cast<const T*>(a.k) + s.k0 * a.k_s[1] + hk * a.k_s[0], a.k_ext);
    const rsrc_t vr = make_rsrc(static_cast<const T*>(a.v) + s.k0 * a.v_s[1] + hk * a.v_s[0], a.v_ext);
    const rsrc_t orr = make_rsrc(static_cast<T*>(a.o) + s.q0 * a.o_s[1] + w.h * a.o_s[0], a.o_ext);
    const rsrc_t lr = make_rsrc(a.lse + s.q0 * a.l_s[1] + w.h * a.l_s[0], a.l_ext);
    const uint32_t krow = (uint32_t)(a.k_s[1] * SZ), vrow = (uint32_t)(a.v_s[1] * SZ);

    // K tiles in buffers 0 and 1, V tiles in 2 and 3. A wave's loads of a tile
    // lie NW * RPI rows apart, where the layouts' chunk order repeats: one
    // lane offset each for K and V, the rest is uniform.
    constexpr int LROWS = NW * C::RPI;
    static_assert(C::fk(LROWS) == 0 && C::fv(LROWS) == 0, "the chunk order repeats from one load to the next");
    const int lrow = wave * C::RPI + lane / C::CPR;
    const uint32_t kvo = lrow * krow + ((lane % C::CPR) ^ C::fk(lrow)) * 16;
    const uint32_t vvo = lrow * vrow + ((lane % C::CPR) ^ C::fv(lrow)) * 16;
    auto load_tile = [&](rsrc_t r, uint8_t* dst, int t, uint32_t vo, uint32_t row) SDPA_INLINE {
        const int limit = s.nk - t * TN;
#pragma unroll
        for (int jj = 0; jj < C::NI / NW; ++jj)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + (jj * NW + wave) * 1024), 16,
                                                     pred(lrow + jj * LROWS < limit, vo + (uint32_t)(t * TN + jj * LROWS) * row),
                                                     0, 0, 0);
    };
    auto load_k = [&](int t) SDPA_INLINE { load_tile(kr, smem + (t & 1) * C::TILEB, t, kvo, krow); };
    auto load_v = [&](int t) SDPA_INLINE { load_tile(vr, smem + (2 + (t & 1)) * C::TILEB, t, vvo, vrow); };

    const int qw = q0 + wave * 32 * RB;  // this wave's first row
    vec qf[RB][NKS];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int qi = qw + 32 * rb + n;
        const bool ok = qi < s.nq;
        const uint32_t qoff = (uint32_t)((ok ? qi : 0) * a.q_s[1] * SZ);
#pragma unroll
        for (int c = 0; c < NKS; ++c) qf[rb][c] = load_operand<T>(qr, pred(ok, qoff + (c * 16 + hf * 8) * SZ), a.q_mul);
    }
    f32x16 oacc[RB][ND], sc[2][RB];  // sc[j & 1]: scores of block j
    vec pv[2][RB][2];                // pv[j & 1]: weights of block j
    float m[RB], l[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        m[rb] = -INFINITY;
        l[rb] = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) oacc[rb][d] = f32x16{};
    }
    const int kr0 = swap23(n);
    const int trg = lane >> 4, trs = lane & 15;
    const int tr_row = 8 * (trg >> 1) + (trs >> 2);
    const int tr_col = 16 * (trg & 1) + 4 * (((trs & 1) << 1) | ((trs >> 1) & 1));
    auto k_op = [&](const uint8_t* kt, int half, int c) SDPA_INLINE -> vec {
        return *reinterpret_cast<const vec*>(kt + C::pos_k(32 * half + kr0, 2 * c + hf) * 16);
    };
    auto v_op = [&](const uint8_t* vt, int half, int kc, int d) SDPA_INLINE -> vec {
        u32x2 x[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 32 * half + 16 * kc + tr_row + 4 * r, col = 32 * d + tr_col;
            x[r] = lds_read_tr16(vt + C::pos_v(row, col * SZ / 16) * 16 + ((col * SZ) & 15));
        }
        return __builtin_bit_cast(vec, u32x4{x[0][0], x[0][1], x[1][0], x[1][1]});
    };

    // Step j (its parity PAR): exponentials of block j, with QK the scores of
    // block j + 1 from K half KH of kt, with PV the sum of block j - 1 from V
    // half VH of vt. edge: block j holds keys that some row does not keep.
    auto step = [&](auto par_c, auto exp_c, auto qk_c, auto pv_c, bool edge, int j, const uint8_t* kt, const uint8_t* vt)
        SDPA_INLINE {
        constexpr int PAR = decltype(par_c)::value;
        constexpr bool EXP = decltype(exp_c)::value, QK = decltype(qk_c)::value, PV = decltype(pv_c)::value;
        // K half of block j + 1 and V half of block j - 1
        constexpr int KH = (PAR + 1) & 1, VH = (PAR + 1) & 1;
        constexpr int AHEAD = AHD;  // operands read ahead of their product
        vec ka[NKS], va[2 * ND];
        if constexpr (QK)
#pragma unroll
            for (int c = 0; c < (AHEAD < NKS ? AHEAD : NKS); ++c) ka[c] = k_op(kt, KH, c);
        if constexpr (PV)
#pragma unroll
            for (int c = 0; c < (AHEAD < 2 * ND ? AHEAD : 2 * ND); ++c) va[c] = v_op(vt, VH, c / ND, c % ND);
        float mu[RB], sum[RB] = {};
        if constexpr (EXP) {
            float top[RB];
            bool grow = false;
            if (edge)
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    const int qi = qw + 32 * rb + n;
                    const int lim = min(s.nk - 1 - 32 * j, a.causal ? qi + s.coff - 32 * j : 0x7fffffff) - 8 * hf;
#pragma unroll
                    for (int r = 0; r < 16; ++r) sc[PAR][rb][r] = kk(0, r) > lim ? -INFINITY : sc[PAR][rb][r];
                }
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const f32x16& x = sc[PAR][rb];
                float y = fmaxf(fmaxf(x[0], x[1]), x[2]);
#pragma unroll
                for (int r = 3; r < 15; r += 2) y = fmaxf(fmaxf(y, x[r]), x[r + 1]);
                top[rb] = fmaxf(y, x[15]) * a.scale_log2;
                grow = grow || top[rb] > m[rb] + 8.0f;
            }
            if (__builtin_amdgcn_ballot_w64(grow) != 0) {
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    const float up = fmaxf(m[rb], __builtin_ceilf(fmaxf(top[rb], __shfl_xor(top[rb], 32))));
                    const float f = up == -INFINITY ? 1.0f : fast_exp2(m[rb] - up);
                    m[rb] = up;
                    l[rb] *= f;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) oacc[rb][d][r] *= f;
                    if constexpr (PV) {
#pragma unroll
                        for (int kc = 0; kc < 2; ++kc) {
                            const u32x4 b = __builtin_bit_cast(u32x4, pv[1 - PAR][rb][kc]);
                            float x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = TR::to_f((b[e >> 1] >> (16 * (e & 1))) & 0xffffu) * f;
                            pv[1 - PAR][rb][kc] = TR::cvt8(x);
                        }
                    }
                }
            }
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) mu[rb] = m[rb] == -INFINITY ? 0.0f : -m[rb];
        }
        if constexpr (QK)
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) sc[1 - PAR][rb] = f32x16{};
        __builtin_amdgcn_sched_barrier(0);
        float p[16 * RB];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int rb = i % RB, c = i / RB;
            if constexpr (QK) {
                sc[1 - PAR][rb] = TR::mfma(ka[c], qf[rb][c], sc[1 - PAR][rb]);
                if (rb == 0 && c + AHEAD < NKS) ka[c + AHEAD] = k_op(kt, KH, c + AHEAD);
            }
            if constexpr (PV) {
                oacc[rb][c % ND] = TR::mfma(va[c], pv[1 - PAR][rb][c / ND], oacc[rb][c % ND]);
                if (rb == RB - 1 && c + AHEAD < 2 * ND) va[c + AHEAD] = v_op(vt, VH, (c + AHEAD) / ND, (c + AHEAD) % ND);
            }
            if constexpr (EXP) {
#pragma unroll
                for (int e = i * EPS; e < (i + 1) * EPS; ++e) {
                    p[e] = fast_exp2(__builtin_fmaf(sc[PAR][e >> 4][e & 15], a.scale_log2, mu[e >> 4]));
                    sum[e >> 4] += p[e];
                    if (e % 8 == 7) {
                        // opaque: the compiler would carry the eight floats into the next step and round them there
                        u32x4 b = __builtin_bit_cast(u32x4, TR::cvt8(p + (e & ~7)));
                        asm volatile("" : "+v"(b));
                        pv[PAR][e >> 4][(e >> 3) & 1] = as_vec<T>(b);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (EXP)
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) l[rb] += sum[rb];
    };
    static_assert(2 * ND == NKS, "as many V as K operands in a step");

    // tiles before t_full hold kept keys only, for every row of the wave;
    // tiles from t_end on none
    const int last_row = min(qw + 32 * RB, s.nq) - 1;
    const bool live = qw < s.nq;
    const int t_end = !live ? 0 : a.causal ? max(0, min(ntiles, (last_row + s.coff + TN) / TN)) : ntiles;
    const int t_full = min(t_end, (a.causal ? max(0, min(s.nk, qw + s.coff + 1)) : s.nk) / TN);
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    constexpr std::true_type on{};
    constexpr std::false_type off{};
    // iteration t: K tile t and V tile t - 1 are staged; steps 2 t - 1 and 2 t
    auto stage = [&](int t) SDPA_INLINE {
        wait_vmem();
        __syncthreads();
        if (t + 1 < ntiles) load_k(t + 1);
        if (t < ntiles) load_v(t);
    };
    auto kt = [&](int t) SDPA_INLINE -> const uint8_t* { return smem + (t & 1) * C::TILEB; };
    auto vt = [&](int t) SDPA_INLINE -> const uint8_t* { return smem + (2 + ((t - 1) & 1)) * C::TILEB; };
    if (ntiles > 0) load_k(0);
    int t = 0;
    if (t_end > 0) {
        stage(0);
        step(odd, off, on, off, false, -1, kt(0), vt(0));
        step(even, on, on, off, t_full == 0, 0, kt(0), vt(0));
        for (t = 1; t < t_end; ++t) {
            stage(t);
            step(odd, on, on, on, t > t_full, 2 * t - 1, kt(t), vt(t));
            step(even, on, on, on, t >= t_full, 2 * t, kt(t), vt(t));
        }
        stage(t);
        step(odd, on, off, on, t > t_full, 2 * t - 1, kt(t), vt(t));
        step(even, off, off, on, false, 2 * t, kt(t), vt(t));
        ++t;
    }
    for (; t <= ntiles; ++t) stage(t);

#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int qi = qw + 32 * rb + n;
        const bool ok = qi < s.nq;
        const float sum = l[rb] + __shfl_xor(l[rb], 32);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const uint32_t ooff = (uint32_t)((ok ? qi : 0) * a.o_s[1] * SZ);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = oacc[rb][d][r] * inv;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (a.o_vec) store8<T, true>(orr, ooff, ok, 32 * d + 16 * c + 8 * hf, D, x + 8 * c);
                else store8<T, false>(orr, ooff, ok, 32 * d + 16 * c + 8 * hf, D, x + 8 * c);
            }
        }
        const float lse = sum == 0.0f ? -INFINITY : (m[rb] + __builtin_amdgcn_logf(sum)) * LN2;
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, lse), lr,
                                              pred(ok && hf == 0, (uint32_t)((ok ? qi : 0) * a.l_s[1] * 4)), 0, 0);
    }
}

template <typename T>
static int launch_prompt_t(int D, const PackArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)a.B * a.Hq * a.n_blk), block(256);
    if constexpr (sizeof(T) == 2) {
        if (a.wide) {
            switch (D) {
                case 32: sdpa_prompt_wide_kernel<T, 32><<<grid, block, 0, s>>>(a); break;
                case 64: sdpa_prompt_wide_kernel<T, 64><<<grid, block, 0, s>>>(a); break;
                case 128: sdpa_prompt_wide_kernel<T, 128><<<grid, block, 0, s>>>(a); break;
                default: return (int)hipErrorInvalidValue;
            }
            return (int)hipGetLastError();
        }
    }
    switch (D) {
        case 32: sdpa_prompt_kernel<T, 32><<<grid, block, 0, s>>>(a); break;
        case 64: sdpa_prompt_kernel<T, 64><<<grid, block, 0, s>>>(a); break;
        case 128: sdpa_prompt_kernel<T, 128><<<grid, block, 0, s>>>(a); break;
        default: return (int)hipErrorInvalidValue;
    }
    return (int)hipGetLastError();
}

int launch_prompt(int dtype, int D, const PackArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case DT_F32: return launch_prompt_t<float>(D, a, s);
        case DT_F16: return launch_prompt_t<_Float16>(D, a, s);
        default: return launch_prompt_t<__bf16>(D, a, s);
    }
}

// ------------------------------------------------------------------ key weights
//
// W[b, h', j] = sum over the query heads h of key head h' and the rows i that
// keep key j of exp(s_hij - LSE_hi). A workgroup holds 256 keys in registers
// (64 per wave) and runs over a range of one query head's rows, 64 at a time
// through LDS: S = Q K^T puts one key in each lane's column, so the sum over
// rows is lane-local. Rows whose LSE is -inf keep no key and add nothing.
template <typename T, int D>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2)))
void sdpa_key_weight_kernel(const PackArgs a) {
    constexpr int NW = 4, TN = sizeof(T) == 2 ? 64 : 32, KB = sizeof(T) == 2 ? 2 : 1;
    using C = TwoPassCfg<T, D, NW, MASK_NONE, true, TN, true>;
    using TR = Tr<T>;
    using vec = typename TR::vec;
    constexpr int SZ = (int)sizeof(T), NQB = TN / 32, KSTEP = 2 * TR::KH, NKS = D / KSTEP;
    constexpr int BLK = 32 * KB * NW;
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * C::TILEB];
    __shared__ float lse_s[2][TN];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int per = a.Hq * a.n_split;
    const PackWork w = pack_work(blockIdx.x, a.B, per, a.n_blk);
    const int h = w.h / a.n_split, split = w.h - h * a.n_split;
    const Seq s = sequence(a, w.b);
    const int k0 = w.blk * BLK;  // causal: low keys are the heaviest
    if (k0 >= s.nk) return;
    const int hk = h / a.group;
    // rows of this range; the first row that keeps a key of the block
    int r0 = split * a.split_rows;
    const int r1 = min(s.nq, r0 + a.split_rows);
    if (a.causal) r0 = max(r0, (k0 - s.coff) / TN * TN);
    const int ntiles = r1 > r0 ? (r1 - r0 + TN - 1) / TN : 0;

    const rsrc_t qr = make_rsrc(static_cast<const T*>(a.q) + s.q0 * a.q_s[1] + h * a.q_s[0], a.q_ext);
    const rsrc_t kr = make_rsrc(static_cast<const T*>(a.k) + s.k0 * a.k_s[1] + hk * a.k_s[0], a.k_ext);
    const rsrc_t lr = make_rsrc(a.lse + s.q0 * a.l_s[1] + h * a.l_s[0], a.l_ext);
    const uint32_t qrow = (uint32_t)(a.q_s[1] * SZ);

    const int kw = k0 + wave * 32 * KB;
    vec kf[KB][NKS];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int key = kw + 32 * kb + n;
        const bool ok = key < s.nk;
        const uint32_t off = (uint32_t)((ok ? key : 0) * a.k_s[1] * SZ);
#pragma unroll
        for (int c = 0; c < NKS; ++c) kf[kb][c] = load_operand<T>(kr, pred(ok, off + (c * KSTEP + hf * TR::KH) * SZ), a.q_mul);
    }
    auto load_tile = [&](int t) SDPA_INLINE {
        uint8_t* const qd = smem + (t & 1) * C::TILEB;
        const int base = r0 + t * TN;
#pragma unroll
        for (int jj = 0; jj < C::NI / NW; ++jj) {
            const int j = jj * NW + wave;
            const int row = j * C::RPI + lane / C::CPR;
            const int cq = (lane % C::CPR) ^ C::fk(row);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(qr, (lds_void*)(qd + j * 1024), 16,
                                                     pred(base + row < r1, row * qrow + cq * 16), (uint32_t)base * qrow, 0, 0);
        }
    };
    // -LSE in base 2 of a tile's rows; rows past the range and dead rows -inf
    auto load_lse = [&](int t) SDPA_INLINE -> float {
        const int row = r0 + t * TN + (int)threadIdx.x;
        const bool ok = (int)threadIdx.x < TN && row < r1;
        const float x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                      lr, pred(ok, (uint32_t)((ok ? row : 0) * a.l_s[1] * 4)), 0, 0));
        return ok && x != -INFINITY ? -x * LOG2E : -INFINITY;
    };
    float sum[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) sum[kb] = 0.0f;
    auto tile = [&](int t, auto edge_c) SDPA_INLINE {
        constexpr bool edge = decltype(edge_c)::value;
        const uint8_t* const qt = smem + (t & 1) * C::TILEB;
#pragma unroll
        for (int qb = 0; qb < NQB; ++qb) {
            f32x16 acc[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) acc[kb] = f32x16{};
#pragma unroll
            for (int c = 0; c < NKS; ++c) {
                const int row = 32 * qb + swap23(n), elem = c * KSTEP + hf * TR::KH;
                const vec qa = *reinterpret_cast<const vec*>(qt + C::pos_k(row, elem * SZ / 16) * 16 + ((elem * SZ) & 15));
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) acc[kb] = TR::mfma(qa, kf[kb][c], acc[kb]);
            }
            float nl[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) nl[r] = lse_s[t & 1][32 * qb + kk(hf, r)];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                // row i keeps key j when j <= i + coff
                const int lim = a.causal ? kw + 32 * kb + n - s.coff - (r0 + t * TN + 32 * qb) - 8 * hf : -64;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float p = fast_exp2(__builtin_fmaf(acc[kb][r], a.scale_log2, nl[r]));
                    if constexpr (edge) p = kk(0, r) < lim || nl[r] == -INFINITY ? 0.0f : p;
                    sum[kb] += p;
                }
            }
        }
    };
    if (ntiles > 0) {
        load_tile(0);
        const float x = load_lse(0);
        if (threadIdx.x < TN) lse_s[0][threadIdx.x] = x;
        wait_vmem();
    }
    __syncthreads();
    for (int t = 0; t < ntiles; ++t) {
        float x = 0.0f;
        if (t + 1 < ntiles) {
            load_tile(t + 1);
            x = load_lse(t + 1);
        }
        tile(t, std::true_type{});
        wait_vmem();
        if (t + 1 < ntiles && threadIdx.x < TN) lse_s[(t + 1) & 1][threadIdx.x] = x;
        __syncthreads();
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int key = kw + 32 * kb + n;
        const float x = sum[kb] + __shfl_xor(sum[kb], 32);
        if (hf == 0 && key < s.nk)
            a.ws[(((int64_t)(h % a.group * a.n_split + split) * a.B + w.b) * a.Hkv + hk) * a.max_k + key] = x;
    }
}

// W = the ranges' sums in order; zeros past a sequence's keys
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256)))
void sdpa_key_weight_sum_kernel(const PackArgs a) {
    const int cols = a.w_cols, j = blockIdx.x * 256 + threadIdx.x;
    const int b = blockIdx.y / a.Hkv, hk = blockIdx.y - b * a.Hkv;
    if (j >= cols) return;
    const Seq s = sequence(a, b);
    float x = 0.0f;
    if (j < s.nk)
        for (int i = 0; i < a.group * a.n_split; ++i)
            x += a.ws[(((int64_t)i * a.B + b) * a.Hkv + hk) * a.max_k + j];
    a.w[b * a.w_s[0] + hk * a.w_s[1] + j] = x;
}

template <typename T>
static int launch_key_weights_t(int D, const PackArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)a.B * a.Hq * a.n_split * a.n_blk), block(256);
    if (a.n_blk > 0 && a.n_split > 0) {
        switch (D) {
            case 32: sdpa_key_weight_kernel<T, 32><<<grid, block, 0, s>>>(a); break;
            case 64: sdpa_key_weight_kernel<T, 64><<<grid, block, 0, s>>>(a); break;
            case 128: sdpa_key_weight_kernel<T, 128><<<grid, block, 0, s>>>(a); break;
            default: return (int)hipErrorInvalidValue;
        }
    }
    const int e = (int)hipGetLastError();
    if (e) return e;
    sdpa_key_weight_sum_kernel<<<dim3((a.w_cols + 255) / 256, a.B * a.Hkv), block, 0, s>>>(a);
    return (int)hipGetLastError();
}

int key_weight_block(int dtype) { return dtype == DT_F32 ? 128 : 256; }

int launch_key_weights(int dtype, int D, const PackArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case DT_F32: return launch_key_weights_t<float>(D, a, s);
        case DT_F16: return launch_key_weights_t<_Float16>(D, a, s);
        default: return launch_key_weights_t<__bf16>(D, a, s);
    }
}

}  // namespace sdpa
