// Attention over packed prompts without the probability map, and the weight
// that every key of those prompts received.
//
// sdpa_prompt_kernel (16-bit types) and sdpa_prompt_f32_kernel:
// O = softmax(scale Q K^T) V and the row log-sum-exp, in one sweep over the
// keys. With a running reference m_i of every row, l_i = sum_j 2^(s_ij - m_i)
// and A_i = sum_j 2^(s_ij - m_i) v_j are updated block by block (s in base 2);
// a block whose weights pass a limit raises m_i to the row's maximum and scales
// l_i and A_i by 2^(old - new). O_i = A_i / l_i, LSE_i = (m_i + log2 l_i) ln 2.
// m_i is the maximum of some block, so l_i >= 1, and weights above 1, up to the
// limit (2^8 in float32, 2^12 in the 16-bit types), lose nothing: the sums are
// float32 and 16-bit floating weights keep their relative precision. Most
// blocks then skip the scaling of A.
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

// Buffer-to-LDS copy of 16 bytes a lane, to lds + 16 lane. Written as assembly
// (it has no register output), because the compiler, which cannot tell the
// tile being filled from the tile being read, waits for the builtin's copies
// before the next LDS read: every tile's loads were waited for as soon as they
// were issued. Copies are counted in order with the other vector memory
// operations; wait_copies(n) waits until at most n of them are under way, and
// stands, with the barrier, between a copy and the first read of its bytes.
typedef uint32_t desc_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ desc_t make_desc(const void* base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return desc_t{(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, bytes, (uint32_t)RSRC_WORD3};
}
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(lds_void*)p; }
__device__ __forceinline__ void copy_to_lds(desc_t d, uint32_t lds, uint32_t off) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is named, though the compiler reserves it
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(d)
                 : "m0", "memory");
#pragma clang diagnostic pop
}
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N < 64, "the counter's six bits");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | N >> 4 << 14);
}

// For a wave that copies its own tiles, without barriers: all but the last N
// copies have landed; its LDS reads are done, so that a copy may take their
// place. Neither reads nor products move across.
template <int N>
__device__ __forceinline__ void landed() {
    __builtin_amdgcn_sched_barrier(0);
    wait_copies<N>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void reads_done() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_sched_barrier(0);
}

// An operand of the products from memory: all loads are in flight before the
// first is touched.
template <typename T, int N>
__device__ __forceinline__ void load_operands(rsrc_t r, const uint32_t* off, int mul, typename Tr<T>::vec* out) {
    if constexpr (sizeof(T) == 2) {
        u32x4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = ld128(r, off[i]);
        if (mul != 1) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] = mul == 0 ? 0u : x[i][e] ^ 0x80008000u;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = as_vec<T>(x[i]);
    } else {
        const float f = (float)mul;
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off[i], 0, 0));
        if (mul != 1)
#pragma unroll
            for (int i = 0; i < N; ++i) out[i] = mul == 0 ? 0.0f : f * out[i];
    }
}

// Workgroup id -> (block counted from the heaviest, sequence, head): blocks
// of the same index are neighbours (heaviest first over the whole grid), and
// the ids that land on one XCD (id % 8) share key heads. Within an XCD ids go
// to its shader engines in turn, so the order of a row's (sequence, head)
// pairs moves on by one with every block: without that, the empty workgroups
// of a short sequence in a ragged batch always fall to the same engines, whose
// CUs then stay idle (two sequences of 12289 and 5003 tokens, 16 heads of 128:
// 1011 us without the step, 727 with it).
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

// Values that are not finite, in tiles that hold keys which some row does not
// keep: a product takes them into every row of its block, kept or not (0 times
// NaN). Where a block's sums come out not finite, the workgroup takes the block
// again with such values read as 0 in these tiles (clean_tile), and adds them
// to the rows that keep their keys at the end (add_kept).
template <typename T>
__device__ __forceinline__ uint32_t clean_word(uint32_t w) {
    if constexpr (sizeof(T) == 4) {
        return (w & 0x7f800000u) == 0x7f800000u ? 0u : w;
    } else {
        constexpr uint32_t E = std::is_same<T, __bf16>::value ? 0x7f80u : 0x7c00u;
        const uint32_t lo = (w & E) == E ? 0u : w & 0xffffu, hi = ((w >> 16) & E) == E ? 0u : w & 0xffff0000u;
        return lo | hi;
    }
}
template <typename T, int BYTES, int THREADS = 256>
__device__ __forceinline__ void clean_tile(uint8_t* tile, int thread) {
    for (int i = thread; i < BYTES / 16; i += THREADS) {
        u32x4 x = reinterpret_cast<u32x4*>(tile)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = clean_word<T>(x[e]);
        reinterpret_cast<u32x4*>(tile)[i] = x;
    }
}
template <int ND>
__device__ __forceinline__ bool all_finite(const f32x16* x) {
    float z = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) z = __builtin_fmaf(x[d][r], 0.0f, z);
    return z == 0.0f;
}
// keys [j0, j1) of v; the row keeps j <= last
template <typename T, int ND>
__device__ __forceinline__ void add_kept(rsrc_t v, uint32_t row_bytes, int j0, int j1, int last, int hf, f32x16* x) {
    constexpr int SZ = (int)sizeof(T), W = SZ == 2 ? 4 : 8;
    for (int j = j0; j < j1; ++j)
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t w[W];
#pragma unroll
                for (int i = 0; i < W / 4; ++i) {
                    const u32x4 y = ld128(v, (uint32_t)j * row_bytes + (32 * d + 16 * c + 8 * hf) * SZ + 16 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[4 * i + e] = y[e];
                }
                bool any = false;
#pragma unroll
                for (int i = 0; i < W; ++i) any = any || clean_word<T>(w[i]) != w[i];
                if (__builtin_amdgcn_ballot_w64(any) == 0) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f;
                    if constexpr (SZ == 2) f = Tr<T>::to_f((w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
                    else f = __builtin_bit_cast(float, w[e]);
                    const bool odd = (__builtin_bit_cast(uint32_t, f) & 0x7f800000u) == 0x7f800000u;
                    if (odd && j <= last) x[d][8 * c + e] += f;
                }
            }
}

// O (32-column blocks d0 .. d0 + N - 1 of it) and LSE of the lane's row: x the
// sum of its half's columns relative to m, l its half of the weights
template <typename T, int N>
__device__ __forceinline__ void store_rows(rsrc_t o, rsrc_t lse, const PackArgs& a, int row, bool ok, int hf, const f32x16* x, float m,
                                           float l, int d0 = 0) {
    const float sum = l + __shfl_xor(l, 32);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const uint32_t ooff = (uint32_t)((ok ? row : 0) * a.o_s[1] * (int)sizeof(T));
#pragma unroll
    for (int d = 0; d < N; ++d) {
        float y[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) y[r] = x[d][r] * inv;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int col = 32 * (d0 + d) + 16 * c + 8 * hf;
            if (a.o_vec) store8<T, true>(o, ooff, ok, col, col + 8, y + 8 * c);
            else store8<T, false>(o, ooff, ok, col, col + 8, y + 8 * c);
        }
    }
    if (d0 > 0) return;
    const float z = sum == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(sum)) * LN2;
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, z), lse,
                                          pred(ok && hf == 0, (uint32_t)((ok ? row : 0) * a.l_s[1] * 4)), 0, 0);
}

// The sums of four waves that took every fourth key block of the same rows,
// joined and stored, 32 columns a wave. x: `pitch` floats of LDS for each wave,
// its own until here.
template <typename T, int ND>
__device__ __forceinline__ void join_waves(rsrc_t o, rsrc_t lse, const PackArgs& a, int row, bool ok, int hf, int lane, int wave,
                                           const f32x16* sums, float m, float l, float* x, int pitch, float2 (*ml)[64]) {
    constexpr int NW = 4;
    float* const js = x + lane;
    ml[wave][lane] = make_float2(m, l);
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) js[wave * pitch + (d * 16 + r) * 64] = sums[d][r];
    __syncthreads();
    if (wave >= ND) return;
    float2 e[NW];
    float up = -INFINITY, total = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        e[i] = ml[i][lane];
        up = fmaxf(up, e[i].x);
    }
    f32x16 y = {};
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const float f = e[i].x == -INFINITY ? 0.0f : fast_exp2(e[i].x - up);
        total += e[i].y * f;
#pragma unroll
        for (int r = 0; r < 16; ++r) y[r] += js[i * pitch + (wave * 16 + r) * 64] * f;
    }
    store_rows<T, 1>(o, lse, a, row, ok, hf, &y, up, total, wave);
}

// float32: the matrix instructions (32x32x2, D / 2 of them for the scores and
// as many for the sums of 32 rows by 32 keys) bound it. A workgroup takes 32
// rows, and its four waves, one on each SIMD, every fourth key tile each, so
// that the chain of a call of few rows is a quarter as long as with 32 rows a
// wave (1024 + 700 tokens, 2 heads of 128: 49 us against 169; 16 heads of 4096
// tokens: 64 wide 308 against 424, 111 TFLOP/s, 128 wide 689 against 697; only
// a full chip of short chains loses, 1024 + 1000 tokens, 32 heads of 128: 253
// against 206). A wave's tiles are its own: it copies them, waits for its own
// copies (no barrier), and copies the next K behind the score products and the
// next V behind the sums. At D = 128 Q and the sums take 128 registers and the
// operands read ahead the rest of 512, so one wave a SIMD; below, two.
template <int D>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(D == 128 ? 1 : 2)))
void sdpa_prompt_f32_kernel(const PackArgs a) {
    constexpr int SZ = 4, NW = 4, TN = 32, ND = D / 32;
    using C = TwoPassCfg<float, D, NW, MASK_NONE, true, TN, true>;
    using TR = Tr<float>;
    constexpr int KSTEP = 2 * TR::KH, NKS = D / KSTEP;
    static_assert(ND * 16 * 64 * 4 <= 2 * C::TILEB, "a wave's sums fit its tiles");
    __shared__ __attribute__((aligned(16))) uint8_t smem[NW * 2 * C::TILEB];
    __shared__ float2 ml_s[NW][64];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const PackWork w = pack_work(blockIdx.x, a.B, a.Hq, a.n_blk);
    const Seq s = sequence(a, w.b);
    const int q0 = (a.n_blk - 1 - w.blk) * 32;
    if (q0 >= s.nq) return;
    const int kend = a.causal ? min(s.nk, max(0, min(q0 + 32, s.nq) + s.coff)) : s.nk;
    const int ntiles = (kend + TN - 1) / TN;
    const int hk = w.h / a.group;

    const rsrc_t qr = make_rsrc(static_cast<const float*>(a.q) + s.q0 * a.q_s[1] + w.h * a.q_s[0], a.q_ext);
    const desc_t kd = make_desc(static_cast<const float*>(a.k) + s.k0 * a.k_s[1] + hk * a.k_s[0], a.k_ext);
    const desc_t vd = make_desc(static_cast<const float*>(a.v) + s.k0 * a.v_s[1] + hk * a.v_s[0], a.v_ext);
    const rsrc_t orr = make_rsrc(static_cast<float*>(a.o) + s.q0 * a.o_s[1] + w.h * a.o_s[0], a.o_ext);
    const rsrc_t lr = make_rsrc(a.lse + s.q0 * a.l_s[1] + w.h * a.l_s[0], a.l_ext);
    const uint32_t krow = (uint32_t)(a.k_s[1] * SZ), vrow = (uint32_t)(a.v_s[1] * SZ);

    uint8_t* const kt = smem + wave * 2 * C::TILEB;
    uint8_t* const vt = kt + C::TILEB;
    const uint32_t kl = lds_address(kt), vl = kl + C::TILEB;
    auto load_k = [&](int t) SDPA_INLINE {
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int row = j * C::RPI + lane / C::CPR;
            copy_to_lds(kd, kl + j * 1024, pred(t * TN + row < s.nk, (uint32_t)(t * TN + row) * krow +
                                                                         ((lane % C::CPR) ^ C::fk(row)) * 16));
        }
    };
    auto load_v = [&](int t) SDPA_INLINE {
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int row = j * C::RPI + lane / C::CPR;
            copy_to_lds(vd, vl + j * 1024, pred(t * TN + row < s.nk, (uint32_t)(t * TN + row) * vrow +
                                                                         ((lane % C::CPR) ^ C::fv(row)) * 16));
        }
    };

    const int qi = q0 + n;  // this lane's row
    const bool ok = qi < s.nq;
    const uint32_t qoff = (uint32_t)((ok ? qi : 0) * a.q_s[1] * SZ);
    float qf[NKS];
    uint32_t qo[NKS];
#pragma unroll
    for (int c = 0; c < NKS; ++c) qo[c] = pred(ok, qoff + (c * KSTEP + hf * TR::KH) * SZ);
    load_operands<float, NKS>(qr, qo, a.q_mul, qf);
    // the first tile with a key that some row does not keep
    const int t_cut = (a.causal ? max(0, min(s.nk, q0 + s.coff + 1)) : s.nk) / TN;
    const int kr0 = swap23(n);
    f32x16 oacc[ND];
    float m, l;
    bool again = false;
    for (;;) {
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) oacc[d] = f32x16{};
        if (wave < ntiles) {
            load_k(wave);
            load_v(wave);
        }
        for (int t = wave; t < ntiles; t += NW) {
            const bool more = t + NW < ntiles;
            landed<C::NI>();
            f32x16 acc = {};
#pragma unroll
            for (int c = 0; c < NKS; ++c) {
                const int elem = c * KSTEP + hf * TR::KH;
                const float ka = *reinterpret_cast<const float*>(kt + C::pos_k(kr0, elem * SZ / 16) * 16 + ((elem * SZ) & 15));
                acc = TR::mfma(ka, qf[c], acc);
            }
            reads_done();
            if (more) load_k(t + NW);
            if (t >= t_cut) {
                const int lim = min(s.nk - 1 - t * TN, a.causal ? qi + s.coff - t * TN : 0x7fffffff) - 8 * hf;
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[r] = kk(0, r) > lim ? -INFINITY : acc[r];
            }
            float top = acc[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) top = fmaxf(top, acc[r]);
            top *= a.scale_log2;
            if (__builtin_amdgcn_ballot_w64(top > m + 8.0f) != 0) {
                const float up = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
                const float f = up == -INFINITY ? 1.0f : fast_exp2(m - up);
                m = up;
                l *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) oacc[d][r] *= f;
            }
            float p[16];
            const float mu = m == -INFINITY ? 0.0f : m;
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                p[r] = fast_exp2(__builtin_fmaf(acc[r], a.scale_log2, -mu));
                sum += p[r];
            }
            l += sum;
            if (more) landed<C::NI>();
            else landed<0>();
            if (again && t >= t_cut) {
                clean_tile<float, C::TILEB, 64>(vt, lane);
                reads_done();
            }
            // A^T += V^T P^T
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = kk(hf, r);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int col = 32 * d + swap23(n);
                    const float va = *reinterpret_cast<const float*>(vt + C::pos_v(row, col * SZ / 16) * 16 + ((col * SZ) & 15));
                    oacc[d] = TR::mfma(va, p[r], oacc[d]);
                }
            }
            reads_done();
            if (more) load_v(t + NW);
        }
        // a wave's tiles are its own, and so is taking them again
        if (again || t_cut >= ntiles || __builtin_amdgcn_ballot_w64(!all_finite<ND>(oacc)) == 0) break;
        again = true;
    }
    if (again) {
        const rsrc_t vr = make_rsrc(static_cast<const float*>(a.v) + s.k0 * a.v_s[1] + hk * a.v_s[0], a.v_ext);
        for (int t = wave; t < ntiles; t += NW)
            if (t >= t_cut)
                add_kept<float, ND>(vr, vrow, t * TN, min(kend, t * TN + TN), a.causal ? qi + s.coff : s.nk - 1, hf, oacc);
    }

    join_waves<float, ND>(orr, lr, a, qi, ok, hf, lane, wave, oacc, m, l, reinterpret_cast<float*>(smem), 2 * C::TILEB / 4, ml_s);
}

// The same for 16-bit types, with the three parts of neighbouring 32-key
// blocks interleaved, so that one wave keeps matrix and vector units busy at
// once: step j does the exponentials of block j between the products
// S(j + 1) = K Q^T and A += V P(j - 1)^T. Nothing waits for a maximum: the
// exponentials take the reference they find, and only where a lane's sum over
// a block passes 2^12 (or a row has no reference yet, in its first block) the
// reference rises to the row's maximum, A and l are scaled and the block's
// weights taken again, while its scores are still there.
//
// NG: key groups, for calls whose blocks of 128 rows leave the chip's wave
// slots empty. With two, a workgroup is twice four waves, which take the same
// rows and every other tile each and join their sums at the end: the chain of
// tiles is half as long. With four (D of 32 and 64, whose tiles fit two
// workgroups a CU that way) it is 32 rows and four waves that take every fourth
// block of 32 keys each, from tiles of their own and so without barriers, as
// the float32 kernel.
template <typename T, int D, int NG>
struct PromptCfg {
    static constexpr int NW = 4, TN = 64;
    using C = TwoPassCfg<T, D, NW, MASK_NONE, true, TN, true>;
    static constexpr int QB = NG == 4 ? 32 : 32 * NW;
    static constexpr int THREADS = NG == 2 ? 512 : 256;
    // two K and two V tiles for a group of four waves, one of each for a wave of its own
    static constexpr int TILE_BYTES = (NG == 4 ? 2 : 4) * NG * C::TILEB;
    static constexpr int JOIN_BYTES = NG > 1 ? NW * (D / 32) * 16 * 64 * 4 : 0;  // one group's sums
    static constexpr int LDS_BYTES = TILE_BYTES > JOIN_BYTES ? TILE_BYTES : JOIN_BYTES;
};

template <typename T, int D, int NG>
__global__ __attribute__((amdgpu_flat_work_group_size(PromptCfg<T, D, NG>::THREADS, PromptCfg<T, D, NG>::THREADS), amdgpu_waves_per_eu(2)))
void sdpa_prompt_kernel(const PackArgs a) {
    using P = PromptCfg<T, D, NG>;
    using C = typename P::C;
    using TR = Tr<T>;
    using vec = typename TR::vec;
    constexpr int SZ = 2, NW = P::NW, TN = P::TN, ND = D / 32, NKS = D / 16;
    constexpr int EPS = 16 / NKS;  // exponentials beside each of a step's products
    __shared__ __attribute__((aligned(16))) uint8_t smem[P::LDS_BYTES];
    __shared__ float2 ml_s[NG > 1 ? NW : 1][64];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % NW;
    const int n = lane & 31, hf = lane >> 5;
    const PackWork w = pack_work(blockIdx.x, a.B, a.Hq, a.n_blk);
    const Seq s = sequence(a, w.b);
    const int q0 = (a.n_blk - 1 - w.blk) * P::QB;
    if (q0 >= s.nq) return;
    const int kend = a.causal ? min(s.nk, max(0, min(q0 + P::QB, s.nq) + s.coff)) : s.nk;
    const int hk = w.h / a.group;

    const rsrc_t qr = make_rsrc(static_cast<const T*>(a.q) + s.q0 * a.q_s[1] + w.h * a.q_s[0], a.q_ext);
    const desc_t kd = make_desc(static_cast<const T*>(a.k) + s.k0 * a.k_s[1] + hk * a.k_s[0], a.k_ext);
    const desc_t vd = make_desc(static_cast<const T*>(a.v) + s.k0 * a.v_s[1] + hk * a.v_s[0], a.v_ext);
    const rsrc_t orr = make_rsrc(static_cast<T*>(a.o) + s.q0 * a.o_s[1] + w.h * a.o_s[0], a.o_ext);
    const rsrc_t lr = make_rsrc(a.lse + s.q0 * a.l_s[1] + w.h * a.l_s[0], a.l_ext);
    const uint32_t krow = (uint32_t)(a.k_s[1] * SZ), vrow = (uint32_t)(a.v_s[1] * SZ);

    const int qw = NG == 4 ? q0 : q0 + wave * 32, qi = qw + n;  // this wave's first row; this lane's
    const bool ok = qi < s.nq;
    vec qf[NKS];
    const uint32_t qoff = (uint32_t)((ok ? qi : 0) * a.q_s[1] * SZ);
    uint32_t qo[NKS];
#pragma unroll
    for (int c = 0; c < NKS; ++c) qo[c] = pred(ok, qoff + (c * 16 + hf * 8) * SZ);
    load_operands<T, NKS>(qr, qo, a.q_mul, qf);
    f32x16 oacc[ND], sc[2];  // sc[j & 1]: scores of block j
    vec pv[2][2];            // pv[j & 1]: weights of block j
    float m, l;
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
        constexpr int AHEAD = 2;  // operands read ahead of their product
        vec ka[NKS], va[2 * ND];
        if constexpr (QK)
#pragma unroll
            for (int c = 0; c < (AHEAD < NKS ? AHEAD : NKS); ++c) ka[c] = k_op(kt, KH, c);
        if constexpr (PV)
#pragma unroll
            for (int c = 0; c < (AHEAD < 2 * ND ? AHEAD : 2 * ND); ++c) va[c] = v_op(vt, VH, c / ND, c % ND);
        float mu, sum = 0.0f;
        if constexpr (EXP) {
            if (edge) {
                const int lim = min(s.nk - 1 - 32 * j, a.causal ? qi + s.coff - 32 * j : 0x7fffffff) - 8 * hf;
#pragma unroll
                for (int r = 0; r < 16; ++r) sc[PAR][r] = kk(0, r) > lim ? -INFINITY : sc[PAR][r];
            }
            mu = m == -INFINITY ? 0.0f : -m;
        }
        if constexpr (QK) sc[1 - PAR] = f32x16{};
        __builtin_amdgcn_sched_barrier(0);
        // weights r8 .. r8 + 7 of the block
        auto weights8 = [&](int r8, const float* p) SDPA_INLINE {
            // opaque: the compiler would carry the eight floats into the next step and round them there
            u32x4 b = __builtin_bit_cast(u32x4, TR::cvt8(p));
            asm volatile("" : "+v"(b));
            pv[PAR][r8 >> 3] = as_vec<T>(b);
        };
        float p[16];
#pragma unroll
        for (int c = 0; c < NKS; ++c) {
            if constexpr (QK) {
                sc[1 - PAR] = TR::mfma(ka[c], qf[c], sc[1 - PAR]);
                if (c + AHEAD < NKS) ka[c + AHEAD] = k_op(kt, KH, c + AHEAD);
            }
            if constexpr (PV) {
                oacc[c % ND] = TR::mfma(va[c], pv[1 - PAR][c / ND], oacc[c % ND]);
                if (c + AHEAD < 2 * ND) va[c + AHEAD] = v_op(vt, VH, (c + AHEAD) / ND, (c + AHEAD) % ND);
            }
            if constexpr (EXP) {
#pragma unroll
                for (int e = c * EPS; e < (c + 1) * EPS; ++e) {
                    p[e] = fast_exp2(__builtin_fmaf(sc[PAR][e], a.scale_log2, mu));
                    sum += p[e];
                    if (e % 8 == 7) weights8(e & 8, p + (e & ~7));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (EXP) {
            // a sum past 2^12, or no reference yet: raise it and take block j again
            if (__builtin_amdgcn_ballot_w64(sum > 4096.0f || m == -INFINITY) != 0) {
                const f32x16& x = sc[PAR];
                float top = x[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, x[r]);
                top *= a.scale_log2;
                const float up = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
                const float f = up == -INFINITY ? 1.0f : fast_exp2(m - up);
                m = up;
                l *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) oacc[d][r] *= f;
                const float nm = up == -INFINITY ? 0.0f : -up;
                sum = 0.0f;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    p[r] = fast_exp2(__builtin_fmaf(x[r], a.scale_log2, nm));
                    sum += p[r];
                    if (r % 8 == 7) weights8(r & 8, p + (r & ~7));
                }
            }
            l += sum;
        }
    };
    static_assert(2 * ND == NKS, "as many V as K operands in a step");

    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    constexpr std::true_type on{};
    constexpr std::false_type off{};
    auto start = [&]() SDPA_INLINE {
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) oacc[d] = f32x16{};
    };
    // the first key that some row of the workgroup does not keep
    const int first_cut = a.causal ? max(0, min(s.nk, q0 + s.coff + 1)) : s.nk;
    bool again = false;

    if constexpr (NG < 4) {
        const int grp = NG > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) : 0;
        uint8_t* const buf = smem + grp * 4 * C::TILEB;  // this group's tiles
        // K tiles in buffers 0 and 1, V tiles in 2 and 3. A wave's loads of a
        // tile lie NW * RPI rows apart, where the layouts' chunk order repeats:
        // one lane offset each for K and V, the rest is uniform.
        constexpr int LROWS = NW * C::RPI;
        static_assert(C::fk(LROWS) == 0 && C::fv(LROWS) == 0, "the chunk order repeats from one load to the next");
        const int lrow = wave * C::RPI + lane / C::CPR;
        const uint32_t kvo = lrow * krow + ((lane % C::CPR) ^ C::fk(lrow)) * 16;
        const uint32_t vvo = lrow * vrow + ((lane % C::CPR) ^ C::fv(lrow)) * 16;
        auto load_tile = [&](desc_t r, uint32_t dst, int t, uint32_t vo, uint32_t row) SDPA_INLINE {
            const int limit = s.nk - t * TN;
#pragma unroll
            for (int jj = 0; jj < C::NI / NW; ++jj)
                copy_to_lds(r, dst + (jj * NW + wave) * 1024,
                            pred(lrow + jj * LROWS < limit, vo + (uint32_t)(t * TN + jj * LROWS) * row));
        };
        const uint32_t lds = lds_address(buf);
        auto tile = [&](int u) SDPA_INLINE { return u * NG + grp; };  // this group's tile u
        auto load_k = [&](int u) SDPA_INLINE { load_tile(kd, lds + (u & 1) * C::TILEB, tile(u), kvo, krow); };
        auto load_v = [&](int u) SDPA_INLINE { load_tile(vd, lds + (2 + (u & 1)) * C::TILEB, tile(u), vvo, vrow); };
        // tiles before t_full hold kept keys only, for every row of the wave;
        // tiles from t_end on none
        const int ntiles = (kend + TN - 1) / TN;
        const int last_row = min(qw + 32, s.nq) - 1;
        const bool live = qw < s.nq;
        const int t_end = !live ? 0 : a.causal ? max(0, min(ntiles, (last_row + s.coff + TN) / TN)) : ntiles;
        const int t_full = min(t_end, (a.causal ? max(0, min(s.nk, qw + s.coff + 1)) : s.nk) / TN);
        const int t_cut = first_cut / TN;
        // iteration u of the group's tiles: K tile u and V tile u - 1 are
        // staged; the second half of tile u - 1 and the first of tile u are taken
        auto stage = [&](int u) SDPA_INLINE {
            wait_copies<0>();
            __syncthreads();
            if (again) {  // V tile u - 1, wherever some row of the workgroup does not keep all of it
                if (u > 0 && tile(u - 1) >= t_cut && tile(u - 1) < ntiles)
                    clean_tile<T, C::TILEB>(buf + (2 + ((u - 1) & 1)) * C::TILEB, threadIdx.x & 255);
                __syncthreads();
            }
            if (tile(u + 1) < ntiles) load_k(u + 1);
            if (tile(u) < ntiles) load_v(u);
        };
        auto kt = [&](int u) SDPA_INLINE -> const uint8_t* { return buf + (u & 1) * C::TILEB; };
        auto vt = [&](int u) SDPA_INLINE -> const uint8_t* { return buf + (2 + ((u - 1) & 1)) * C::TILEB; };
        const int u_all = (ntiles + NG - 1) / NG;  // iterations of the longest group
        const int u_end = NG == 1 ? t_end : t_end > grp ? (t_end - grp + NG - 1) / NG : 0;  // this wave's tiles
        for (;;) {
            start();
            if (tile(0) < ntiles) load_k(0);
            int u = 0;
            if (u_end > 0) {
                stage(0);
                step(odd, off, on, off, false, -1, kt(0), vt(0));
                step(even, on, on, off, tile(0) >= t_full, 2 * tile(0), kt(0), vt(0));
                for (u = 1; u < u_end; ++u) {
                    stage(u);
                    step(odd, on, on, on, tile(u - 1) >= t_full, 2 * tile(u - 1) + 1, kt(u), vt(u));
                    step(even, on, on, on, tile(u) >= t_full, 2 * tile(u), kt(u), vt(u));
                }
                stage(u);
                step(odd, on, off, on, tile(u - 1) >= t_full, 2 * tile(u - 1) + 1, kt(u), vt(u));
                step(even, off, off, on, false, 0, kt(u), vt(u));
                ++u;
            }
            for (; u <= u_all; ++u) stage(u);
            if (again || t_cut >= ntiles) break;
            again = __syncthreads_or(!all_finite<ND>(oacc)) != 0;
            if (!again) break;
        }
        if constexpr (NG > 1) {  // the second group's sums, then the first's join them
            float* const js = reinterpret_cast<float*>(smem) + wave * ND * 16 * 64 + lane;
            __syncthreads();
            if (grp == 1) {
                ml_s[wave][lane] = make_float2(m, l);
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) js[(d * 16 + r) * 64] = oacc[d][r];
            }
            __syncthreads();
            if (grp == 1) return;
            const float2 o = ml_s[wave][lane];
            const float up = fmaxf(m, o.x);
            const float f0 = m == -INFINITY ? 0.0f : fast_exp2(m - up), f1 = o.x == -INFINITY ? 0.0f : fast_exp2(o.x - up);
            m = up;
            l = l * f0 + o.y * f1;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) oacc[d][r] = oacc[d][r] * f0 + js[(d * 16 + r) * 64] * f1;
        }
        if (again) {
            const rsrc_t vr = make_rsrc(static_cast<const T*>(a.v) + s.k0 * a.v_s[1] + hk * a.v_s[0], a.v_ext);
            add_kept<T, ND>(vr, vrow, t_cut * TN, kend, a.causal ? qi + s.coff : s.nk - 1, hf, oacc);
        }
        store_rows<T, ND>(orr, lr, a, qi, ok, hf, oacc, m, l);
    } else {
        // Blocks of 32 keys, every fourth this wave's: its j-th lies in half
        // j & 1 of its K tile, and of its V tile. An even number of them is
        // taken; what lies past kend keeps nothing.
        uint8_t* const kt = smem + wave * 2 * C::TILEB;
        uint8_t* const vt = kt + C::TILEB;
        const uint32_t kl = lds_address(kt);
        constexpr int NB = C::NI / 2;  // copies of a block
        const int blocks = (kend + 31) / 32, mine = wave < blocks ? ((blocks - wave + NG - 1) / NG + 1) & ~1 : 0;
        auto block = [&](int j) SDPA_INLINE { return j * NG + wave; };
        auto load_block = [&](desc_t r, uint32_t dst, int j, uint32_t row, auto order) SDPA_INLINE {
            const int limit = s.nk - 32 * block(j);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int x = i * C::RPI + lane / C::CPR;
                copy_to_lds(r, dst + (j & 1) * (C::TILEB / 2) + i * 1024,
                            pred(x < limit, (uint32_t)(32 * block(j) + x) * row + ((lane % C::CPR) ^ order(x)) * 16));
            }
        };
        auto load_k = [&](int j) SDPA_INLINE { load_block(kd, kl, j, krow, [](int x) { return C::fk(x); }); };
        auto load_v = [&](int j) SDPA_INLINE { load_block(vd, kl + C::TILEB, j, vrow, [](int x) { return C::fv(x); }); };
        static_assert(C::fk(32) == 0 && C::fv(32) == 0, "the chunk order of both halves of a tile is the same");
        const int full = first_cut / 32;  // blocks before hold kept keys only
        // step j: K block j + 1 and V block j - 1 have landed; behind it the
        // copies of those that take their places leave
        auto staged = [&](int j) SDPA_INLINE {
            if (j + 2 < mine) landed<2 * NB>();
            else if (j < mine) landed<NB>();
            else landed<0>();
            if (again && j > 0 && block(j - 1) >= full) {
                clean_tile<T, C::TILEB / 2, 64>(vt + ((j - 1) & 1) * (C::TILEB / 2), lane);
                reads_done();
            }
        };
        auto taken = [&](int j) SDPA_INLINE {
            reads_done();
            if (j + 3 < mine) load_k(j + 3);
            if (j >= 0 && j + 1 < mine) load_v(j + 1);
        };
        auto edge = [&](int j) SDPA_INLINE { return block(j) >= full; };
        for (;;) {
            start();
            if (mine == 0) break;
            load_k(0);
            load_k(1);
            load_v(0);
            staged(-1);
            step(odd, off, on, off, false, -1, kt, vt);
            taken(-1);
            staged(0);
            step(even, on, on, off, edge(0), block(0), kt, vt);
            taken(0);
            int j = 1;
            for (; j + 1 < mine; j += 2) {
                staged(j);
                step(odd, on, on, on, edge(j), block(j), kt, vt);
                taken(j);
                staged(j + 1);
                step(even, on, on, on, edge(j + 1), block(j + 1), kt, vt);
                taken(j + 1);
            }
            staged(j);
            step(odd, on, off, on, edge(j), block(j), kt, vt);
            taken(j);
            staged(j + 1);
            step(even, off, off, on, false, 0, kt, vt);
            reads_done();
            if (again || full >= blocks || __builtin_amdgcn_ballot_w64(!all_finite<ND>(oacc)) == 0) break;
            again = true;
        }
        if (again) {
            const rsrc_t vr = make_rsrc(static_cast<const T*>(a.v) + s.k0 * a.v_s[1] + hk * a.v_s[0], a.v_ext);
            for (int j = 0; j < mine; ++j)
                if (edge(j))
                    add_kept<T, ND>(vr, vrow, 32 * block(j), min(kend, 32 * block(j) + 32), a.causal ? qi + s.coff : s.nk - 1, hf,
                                    oacc);
        }
        join_waves<T, ND>(orr, lr, a, qi, ok, hf, lane, wave, oacc, m, l, reinterpret_cast<float*>(smem), 2 * C::TILEB / 4, ml_s);
    }
}

template <typename T, int D>
static void launch_prompt_td(const PackArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)a.B * a.Hq * a.n_blk);
    if constexpr (sizeof(T) == 4) {
        sdpa_prompt_f32_kernel<D><<<grid, 256, 0, s>>>(a);
    } else {
        if constexpr (D < 128)
            if (a.groups == 4) {
                sdpa_prompt_kernel<T, D, 4><<<grid, 256, 0, s>>>(a);
                return;
            }
        if (a.groups == 2) sdpa_prompt_kernel<T, D, 2><<<grid, 512, 0, s>>>(a);
        else sdpa_prompt_kernel<T, D, 1><<<grid, 256, 0, s>>>(a);
    }
}

template <typename T>
static int launch_prompt_t(int D, const PackArgs& a, hipStream_t s) {
    switch (D) {
        case 32: launch_prompt_td<T, 32>(a, s); break;
        case 64: launch_prompt_td<T, 64>(a, s); break;
        case 128: launch_prompt_td<T, 128>(a, s); break;
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
// keep key j of exp(s_hij - LSE_hi). A workgroup holds 128 keys in registers
// (32 per wave) and runs over a range of one query head's rows, 64 at a time
// through LDS: S = Q K^T puts one key in each lane's column, so the sum over
// rows is lane-local. Rows whose LSE is -inf keep no key and add nothing.
//
// The exponentials bound it (16 of them a lane, with a multiply-add and an
// addition each, to D / 16 products: 549 cycles of the vector unit for 32 rows
// by 64 keys, measured, to 272 of the matrix unit at D = 64), so it runs four
// waves a SIMD with little state, whose products and exponentials overlap
// between waves. 2048 + 1531 tokens, 16 heads of 128: 33 us with the sums, against 44 with 64
// keys a wave (two waves a SIMD) and 38 interleaved by hand as the prompt
// kernel.
template <typename T, int D>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(4)))
void sdpa_key_weight_kernel(const PackArgs a) {
    constexpr int NW = 4, TN = sizeof(T) == 2 ? 64 : 32;
    using C = TwoPassCfg<T, D, NW, MASK_NONE, true, TN, true>;
    using TR = Tr<T>;
    using vec = typename TR::vec;
    constexpr int SZ = (int)sizeof(T), NQB = TN / 32, KSTEP = 2 * TR::KH, NKS = D / KSTEP;
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * C::TILEB];
    __shared__ __attribute__((aligned(16))) float lse_s[2][TN];
    __shared__ int odd_s[2];  // a row of the tile has an infinite LSE

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int per = a.Hq * a.n_split;
    const PackWork w = pack_work(blockIdx.x, a.B, per, a.n_blk);
    const int h = w.h / a.n_split, split = w.h - h * a.n_split;
    const Seq s = sequence(a, w.b);
    const int k0 = w.blk * KEY_WEIGHT_KEYS;  // causal: low keys are the heaviest
    if (k0 >= s.nk) return;
    const int hk = h / a.group;
    // rows of this range; the first row that keeps a key of the block
    int r0 = split * a.split_rows;
    const int r1 = min(s.nq, r0 + a.split_rows);
    if (a.causal) r0 = max(r0, (k0 - s.coff) / TN * TN);
    const int ntiles = r1 > r0 ? (r1 - r0 + TN - 1) / TN : 0;
    const int kw = k0 + wave * 32;
    float* const ws = a.ws + (((int64_t)(h % a.group * a.n_split + split) * a.B + w.b) * a.Hkv + hk) * a.max_k;

    const desc_t qd = make_desc(static_cast<const T*>(a.q) + s.q0 * a.q_s[1] + h * a.q_s[0], a.q_ext);
    const rsrc_t kr = make_rsrc(static_cast<const T*>(a.k) + s.k0 * a.k_s[1] + hk * a.k_s[0], a.k_ext);
    const rsrc_t lr = make_rsrc(a.lse + s.q0 * a.l_s[1] + h * a.l_s[0], a.l_ext);
    const uint32_t qrow = (uint32_t)(a.q_s[1] * SZ);
    if (ntiles == 0) {  // no row of this range keeps a key of the block
        for (int key = kw + lane; key < min(kw + 32, s.nk); key += 64) ws[key] = 0.0f;
        return;
    }
    vec kf[NKS];
    {
        const int key = kw + n;
        const bool ok = key < s.nk;
        const uint32_t row = (uint32_t)((ok ? key : 0) * a.k_s[1] * SZ);
        uint32_t off[NKS];
#pragma unroll
        for (int c = 0; c < NKS; ++c) off[c] = pred(ok, row + (c * KSTEP + hf * TR::KH) * SZ);
        load_operands<T, NKS>(kr, off, a.q_mul, kf);
    }
    constexpr int LROWS = NW * C::RPI;
    const int lrow = wave * C::RPI + lane / C::CPR;
    const uint32_t qvo = lrow * qrow;
    constexpr bool SAME = C::fk(LROWS) == 0;  // the chunk order repeats from one load to the next
    const uint32_t lds = lds_address(smem);
    auto load_q = [&](int t) SDPA_INLINE {
        const uint32_t dst = lds + (t & 1) * C::TILEB;
        const int base = r0 + t * TN;
#pragma unroll
        for (int jj = 0; jj < C::NI / NW; ++jj) {
            const uint32_t c = ((lane % C::CPR) ^ C::fk(SAME ? lrow : lrow + jj * LROWS)) * 16;
            copy_to_lds(qd, dst + (jj * NW + wave) * 1024,
                        pred(base + jj * LROWS + lrow < r1, qvo + c + (uint32_t)(base + jj * LROWS) * qrow));
        }
    };
    // -LSE in base 2 of a tile's rows (the first wave); rows past the range and rows without keys: -inf
    auto load_lse = [&](int t) SDPA_INLINE -> float {
        const int row = r0 + t * TN + lane;
        const bool ok = lane < TN && row < r1;
        const float x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                      lr, pred(ok, (uint32_t)((ok ? row : 0) * a.l_s[1] * 4)), 0, 0));
        return ok ? x : -INFINITY;
    };
    auto store_lse = [&](int t, float x) SDPA_INLINE {
        const int row = r0 + t * TN + lane;
        const bool inf = fabsf(x) == INFINITY;
        if (lane < TN) lse_s[t & 1][lane] = inf ? -INFINITY : -x * LOG2E;
        const bool odd = __builtin_amdgcn_ballot_w64(lane < TN && row < r1 && inf) != 0;
        if (lane == 0) odd_s[t & 1] = odd;
    };
    const int kr0 = swap23(n);
    float sum = 0.0f;
    // the tile's rows, 32 at a time
    auto tile = [&](int t) SDPA_INLINE {
        const uint8_t* const qt = smem + (t & 1) * C::TILEB;
#pragma unroll
        for (int qb = 0; qb < NQB; ++qb) {
            const float* const lp = lse_s[t & 1] + 32 * qb;
            float nl[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) nl[r] = lp[kk(hf, r)];
            f32x16 acc = {};
#pragma unroll
            for (int c = 0; c < NKS; ++c) {
                const int row = 32 * qb + kr0, elem = c * KSTEP + hf * TR::KH;
                const vec qa = *reinterpret_cast<const vec*>(qt + C::pos_k(row, elem * SZ / 16) * 16 + ((elem * SZ) & 15));
                acc = TR::mfma(qa, kf[c], acc);
            }
            const int i0 = r0 + t * TN + 32 * qb;  // the block's first row
            if ((a.causal && i0 + s.coff < kw + 31) || odd_s[t & 1]) {
                // row i keeps key j when j <= i + coff; rows of infinite LSE count for nothing
                const int lim = a.causal ? kw + n - s.coff - i0 - 8 * hf : -64;
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[r] = kk(0, r) < lim || nl[r] == -INFINITY ? -INFINITY : acc[r];
            }
            float x[2] = {0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r & 1] += fast_exp2(__builtin_fmaf(acc[r], a.scale_log2, nl[r]));
            sum += x[0] + x[1];
        }
    };
    // iteration t: row tile t and its LSE are staged
    load_q(0);
    float x = 0.0f;
    if (wave == 0) x = load_lse(0);
    for (int t = 0; t < ntiles; ++t) {
        if (wave == 0) store_lse(t, x);
        wait_copies<0>();
        __syncthreads();
        if (t + 1 < ntiles) {
            load_q(t + 1);
            if (wave == 0) x = load_lse(t + 1);
        }
        tile(t);
    }
    const int key = kw + n;
    const float total = sum + __shfl_xor(sum, 32);
    if (hf == 0 && key < s.nk) ws[key] = total;
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

int launch_key_weights(int dtype, int D, const PackArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case DT_F32: return launch_key_weights_t<float>(D, a, s);
        case DT_F16: return launch_key_weights_t<_Float16>(D, a, s);
        default: return launch_key_weights_t<__bf16>(D, a, s);
    }
}

}  // namespace sdpa
