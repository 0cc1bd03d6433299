// Attention of one token's queries over tiles of an 8-bit cache, one warp at a time:
// the arithmetic of the block-split kernel (ckv_q8_blocks.cuh).
//
// Mathematics.  With codes k, v and scales s_k, s_v of a token's block and head:
//   x_t = (q . k_t) s_k log2(e)/sqrt(d),  o = sum_t 2^x_t s_v v_t / sum_t 2^x_t.
// The codes go to fp16, which holds them exactly (int8 and e4m3 alike), and
// stay unscaled in the products; the scales multiply the fp32 scores and the
// weights.
//
// What bounds it: HBM, if the SM keeps up.  At the copy rate an SM receives
// about 23 codes a clock, each of which meets up to 8 query heads, so the
// products go to the tensor cores (mma.sync m16n8k16: a group's heads are at
// most 8 columns; tcgen05's tiles have at least 64 rows of queries to fill), and
// the work that is left is turning codes into fp16.  The tile's tokens are the
// rows of A in Q K^T and the reduction index of P V, the heads the 8 columns of
// B, so 16 tokens cost 2 d/16 products:
//   S [token, head]  = K [token, dim]  Q^T [dim, head]
//   O [dim, head]   += V^T [dim, token] P [token, head]
// d = 128, 4 heads, all of a call's instructions counted: 380 warp instructions for 16
// tokens of int8, 277 of e4m3.  That is about half of the issue slots (the captures:
// 49 % and 37 %), the tensor pipe 17 %.
// A q row is normalised to a power of two and held as fp16 hi + lo (22 bits),
// and so is a weight; with at most 4 heads a group hi and lo are columns 0..3
// and 4..7 of one product, with 8 heads they take a product each.
//
// Fragments are loaded without rearranging bytes: the reduction index of Q K^T may
// be permuted freely when Q is permuted alike, so a lane takes 16 consecutive
// codes of its token's row (its own t-th or t+4-th 16-byte chunk); the rows of V^T
// (output dims) likewise, so a lane takes d/8 consecutive codes of 4 tokens, and
// pairs of tokens are interleaved bytewise.  Tiles are staged by cp.async with
// the 16-byte chunks of a row swizzled so that both patterns meet no bank
// conflict (q8_swz).
//
// Statistics.  m0 is the running reference of x (raised when an x passes it by
// 8), the sum uses p = 2^(x - m0).  The weights carry s_v, whose size the
// softmax does not know, so they have a reference of their own:
// w = p c s_v with c a power of two such that w is in (2^4, 2^5] at its largest
// when set and at most 2^15 at any time (fp16's range); hi + lo then keep 2^-29
// of the largest weight.  c leaves again, exactly, when a partial is written.
#pragma once

#include <type_traits>

#include "ckv_decode.cuh"
#include "ckv_q8.cuh"

namespace ckv {

constexpr int Q8_HALF = 16;  // tokens of a product's tile
constexpr float Q8_M_INIT = -1e30f;

// A staged tile of NH such halves (1 or 2).
template <int D, int NH>
struct Q8Geom {
    static constexpr int TOK = NH * Q8_HALF;
    static constexpr int HALF = Q8_HALF * D;       // bytes of 16 rows
    static constexpr int V = NH * HALF;            // K's halves, then V's
    static constexpr int CH = D / 16;              // 16-byte chunks per row
    static constexpr int SCALES = 2 * NH * HALF;   // float [NH][2]: K's and V's scale of each half (dense)
    static constexpr int SLOT = SCALES + 128;      // bytes of a ring slot (a multiple of 128)
    static constexpr int KS = D / 16;              // k-steps of Q K^T
    static constexpr int MT = D / 16;              // 16-dim tiles of V^T
};

// Byte offset of 16-byte chunk c of token row r in 16 staged rows.  Q K^T reads
// chunk t (t+4) of rows g, 8 lanes at a time: rows 2i, 2i+1 x 4 chunks; P V reads
// d/8 bytes at chunk position g of rows 2t (2t+1, 2t+8, 2t+9): 4 even or odd
// rows x the chunks of 2 (d = 128) or 4 (d = 64, 8-byte reads) values of g.
// Both cover all 32 banks once.
template <int D>
__device__ __forceinline__ int q8_swz(int r, int c) {
    if constexpr (D == 128) return r * 128 + ((c ^ ((((r ^ (r >> 2)) & 1) << 2) | (r & 2))) << 4);
    else return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1)) << 4);
}

__device__ __forceinline__ void q8_mma(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                       unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void q8_mma0(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                        unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Pairs of fp32 in one 64-bit register, for the packed add and product.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <int OFF>
__device__ __forceinline__ uint4 lds128(unsigned a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4+%5];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a), "n"(OFF) : "memory");
    return r;
}
template <int OFF>
__device__ __forceinline__ uint2 lds64(unsigned a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2+%3];" : "=r"(r.x), "=r"(r.y) : "r"(a), "n"(OFF) : "memory");
    return r;
}
__device__ __forceinline__ float lds32f(unsigned a) {
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ unsigned smem_addr32(const void* p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ unsigned q8_transpose(unsigned x) {
    unsigned y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ unsigned pack_half2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&v);
}
__device__ __forceinline__ float2 unpack_half2(unsigned w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// w m + a for a pair of fp16 (m and a their bits)
__device__ __forceinline__ unsigned half2_fma(unsigned w, unsigned short m, unsigned short a) {
    const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&w),
                              __halves2half2(__ushort_as_half(m), __ushort_as_half(m)),
                              __halves2half2(__ushort_as_half(a), __ushort_as_half(a)));
    return *reinterpret_cast<const unsigned*>(&x);
}

// the smaller of the two, NaN if either is
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A K word's four codes as two fp16 pairs, in an order of their own (K_PAIR).
// int8: bytes 0, 2 and 1, 3; flipped to 128 + c they are the fp16 subnormals (128 + c)
// 2^-24, and times 2^15 less 2^-2 that is c 2^-9, exact: five instructions for four
// codes.  The products' sums are then of the size of sum |q c|.  (With the bias left in,
// and taken off through the accumulators' start, they would be 128 sum |q| large
// whatever the codes are, and the tensor core truncates them: 12 to 50 times the error
// of the scores where most codes are small, as beside a large channel's.  Codes as
// subnormals, c 2^-24, give 5 times: it aligns them like normal numbers of the least
// exponent.  The two instructions cost 0 to 4 % of a call.)  e4m3: bytes 0, 1 and 2, 3.
template <int FMT>
__device__ __forceinline__ void q8_k_halves(unsigned w, unsigned& p0, unsigned& p1) {
    if constexpr (FMT == Q8_I8) {
        w ^= 0x80808080u;
        p0 = half2_fma(w & 0x00ff00ffu, 0x7800, 0xb400);
        p1 = half2_fma(__byte_perm(w, 0u, 0x4341), 0x7800, 0xb400);
    } else {
        p0 = e4m3x2_half2((unsigned short)(w & 0xffffu));
        p1 = e4m3x2_half2((unsigned short)(w >> 16));
    }
}
template <int FMT> constexpr float K_UNIT = FMT == Q8_I8 ? 0x1p9f : 1.f;  // a K code of 1 enters the products as 1 / K_UNIT
// Dims of a word's fp16 pairs: pair i holds dims first(i) and first(i) + step.
template <int FMT> struct KPair {
    static constexpr int step = FMT == Q8_I8 ? 2 : 1;
    static constexpr int second = FMT == Q8_I8 ? 1 : 2;  // first(0) = 0
};

// The words of two tokens (a, b), four dims each: h[i] = fp16 (a_i, b_i).  int8: a
// byte flipped to 128 + c is the low part of an fp16 in [1024, 1280), whose step is 1,
// and 1152 comes off again.
template <int FMT>
__device__ __forceinline__ void q8_v_halves(unsigned a, unsigned b, unsigned (&h)[4]) {
    if constexpr (FMT == Q8_I8) {
        const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        a ^= 0x80808080u;
        b ^= 0x80808080u;
        const unsigned lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);  // a0 b0 a1 b1, a2 b2 a3 b3
        const unsigned w[4] = {__byte_perm(lo, 0x64646464u, 0x4140), __byte_perm(lo, 0x64646464u, 0x4342),
                               __byte_perm(hi, 0x64646464u, 0x4140), __byte_perm(hi, 0x64646464u, 0x4342)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&w[i]), bias);
            h[i] = *reinterpret_cast<const unsigned*>(&x);
        }
    } else {
        const unsigned lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);  // a0 b0 a1 b1, a2 b2 a3 b3
        h[0] = e4m3x2_half2((unsigned short)(lo & 0xffffu));
        h[1] = e4m3x2_half2((unsigned short)(lo >> 16));
        h[2] = e4m3x2_half2((unsigned short)(hi & 0xffffu));
        h[3] = e4m3x2_half2((unsigned short)(hi >> 16));
    }
}

// 16 bytes to shared address s + SO from g + GO
template <int SO, int GO>
__device__ __forceinline__ void cp_async_16i(unsigned s, const void* g) {
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%3], 16;\n" ::"r"(s), "l"(g), "n"(SO), "n"(GO) : "memory");
}
__device__ __forceinline__ void cp_async_16s(unsigned s, const void* g, int size) {  // size 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(g), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_async_4s(unsigned s, const void* g, int size) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(s), "l"(g), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_async_4p(unsigned s, const void* g, bool pred) {  // nothing when !pred
    asm volatile("{\n.reg .pred p;\nsetp.ne.s32 p, %2, 0;\n@p cp.async.ca.shared.global [%0], [%1], 4;\n}\n" ::"r"(s),
                 "l"(g), "r"((int)pred)
                 : "memory");
}

// The state of one warp over one unit's tokens: lane 4 g + t.  QLO: q may have lo
// parts (with 8 heads a group they take registers and products of their own, which
// bf16 rows, exact in one fp16, do without; with fewer heads nothing).
template <int D, int GQ, int FMT, int NH, bool QLO>
struct Q8Warp {
    using QG = Q8Geom<D, NH>;
    static constexpr bool SPLIT = GQ == 8;  // hi and lo in products of their own
    unsigned qh[QG::KS][2];                 // Q^T fragments (SPLIT: hi; else hi in columns 0..3, lo or hi again in 4..7)
    unsigned ql[SPLIT && QLO ? QG::KS : 1][2];
    bool q_lo;                              // some lo is not zero (q in fp32)
    float qf[2];                            // per head of this lane: 2^e log2(e)/sqrt(d)
    float m0[2], mw[2], c[2], l[2];         // references of x and of x + log2 s_v, weight factor, sum
    f32x2 o[QG::MT][2];                     // columns 2t, 2t + 1 of rows g and g + 8 of each 16-dim tile

    __device__ __forceinline__ static int head(int t, int e) { return SPLIT ? 2 * t + e : (2 * t + e) & 3; }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m0[e] = mw[e] = Q8_M_INIT;
            c[e] = 1.f;
            l[e] = 0.f;
        }
#pragma unroll
        for (int m = 0; m < QG::MT; ++m) o[m][0] = o[m][1] = 0ull;
    }

    // q: the group's first row.  Lane (g, t) holds column g: head g (SPLIT), or
    // head g & 3, hi for g < 4 and lo otherwise; dims 16 (t + 4 j) + 4 w + 0..3
    // are k-step 4 j + w, in the order of the K word's pairs.  fetch_q only loads, so that the latency of q and of
    // what the caller loads next overlap.
    struct RawQ {
        uint4 w[QG::KS];
    };
    __device__ __forceinline__ static RawQ fetch_q(const void* q, int dtype, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int h = SPLIT ? g : g & 3;
        RawQ r;
#pragma unroll
        for (int s = 0; s < QG::KS; ++s) {
            const int dim = 16 * (t + 4 * (s >> 2)) + 4 * (s & 3);
            const size_t at = (size_t)(h < GQ ? h : 0) * D + dim;
            if (dtype == CKV_DTYPE_BF16) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(q) + at);
                r.w[s] = make_uint4(w.x << 16, w.x & 0xffff0000u, w.y << 16, w.y & 0xffff0000u);
            } else {
                r.w[s] = *reinterpret_cast<const uint4*>(static_cast<const float*>(q) + at);
            }
        }
        return r;
    }
    __device__ __forceinline__ void set_q(const RawQ& r, int dtype, float scale_log2, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const bool real = (SPLIT ? g : g & 3) < GQ;
        float x[QG::KS][4];
        unsigned amax = 0;
#pragma unroll
        for (int s = 0; s < QG::KS; ++s) {
            const unsigned w[4] = {r.w[s].x, r.w[s].y, r.w[s].z, r.w[s].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[s][i] = real ? __uint_as_float(w[i]) : 0.f;
                amax = max(amax, __float_as_uint(x[s][i]) & 0x7fffffffu);
            }
        }
        amax = max(amax, __shfl_xor_sync(FULL, amax, 1));
        amax = max(amax, __shfl_xor_sync(FULL, amax, 2));
        // the row's largest magnitude goes to [2^14, 2^15): codes and sums stay in
        // range, and 2^-29 of it is still a normal fp16.  Rows below 2^-100 count
        // as that large.
        const int e = max((int)(amax >> 23), 27) - 127 - 14;  // amax = m 2^(e + 14), e in [-114, 114]
        const float down = __uint_as_float((unsigned)(127 - e) << 23);
        const float f = __uint_as_float((unsigned)(127 + e) << 23) * scale_log2;
        using KP = KPair<FMT>;
#pragma unroll
        for (int s = 0; s < QG::KS; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[s][KP::second * i] *= down;
                x[s][KP::second * i + KP::step] *= down;
                qh[s][i] = pack_half2(x[s][KP::second * i], x[s][KP::second * i + KP::step]);
            }
        // bf16 rows are exact in one fp16; without lo parts columns 4..7 repeat 0..3,
        // and no lane has to fetch the scores of its weights' heads
        q_lo = QLO && dtype == CKV_DTYPE_F32;
        if (q_lo) {
#pragma unroll
            for (int s = 0; s < QG::KS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 h2 = unpack_half2(qh[s][i]);
                    const unsigned lo = pack_half2(x[s][KP::second * i] - h2.x, x[s][KP::second * i + KP::step] - h2.y);
                    if constexpr (SPLIT && QLO) ql[s][i] = lo;
                    else if (!SPLIT && g >= 4) qh[s][i] = lo;
                }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) qf[k] = __shfl_sync(FULL, f, head(t, k) * 4) * K_UNIT<FMT>;
    }
    __device__ __forceinline__ static const void* q_row(const void* q, int dtype, size_t row) {
        return static_cast<const char*>(q) + row * D * (dtype == CKV_DTYPE_BF16 ? 2 : 4);
    }

    // One tile staged at sm; mask: which of its tokens count.  UNIFORM: the 16
    // tokens of a half have one scale each for K and V, staged with the tile;
    // otherwise (NH = 1) lane i has the K scale of token i, lane 16 + i its V scale
    // in `scale`.  lam (NEIGHBOURS): lam(i, x) receives the largest x over the group's
    // heads of the tile's token i, from one lane per token.  Two halves at a time
    // give the products independent work and share the checks, the loads'
    // bookkeeping and the fp32 additions.
    template <bool UNIFORM, bool NEIGHBOURS, typename Lam>
    __device__ __forceinline__ void tile(unsigned sm, unsigned mask, float scale, int lane, Lam lam) {
        static_assert(UNIFORM || NH == 1, "a lane per scale");
        const int g = lane >> 2, t = lane & 3;
        if (mask == 0u) return;  // uniform over the warp
        // rows 8 apart are 8 D bytes apart; chunks t and t + 4 (d = 128) differ in bit 6,
        // and so do, a row on, rows 2t and 2t + 1
        const unsigned ks = sm + q8_swz<D>(g, t), ks2 = sm + (q8_swz<D>(g, t) ^ 64);

        // S: rows g, g + 8 of each half, columns 2t, 2t + 1; even and odd k-steps apart
        float s[NH][2][2];  // [half][token g | g + 8][head]
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            float sa[4], sb[4];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 ka = j ? lds128<QG::HALF>(i ? ks2 : ks) : lds128<0>(i ? ks2 : ks);
                const uint4 kb = j ? lds128<QG::HALF + 8 * D>(i ? ks2 : ks) : lds128<8 * D>(i ? ks2 : ks);
                const unsigned wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int k = 4 * i + w;
                    unsigned a0, a1, a2, a3;
                    q8_k_halves<FMT>(wa[w], a0, a2);
                    q8_k_halves<FMT>(wb[w], a1, a3);
                    if (k <= 1) q8_mma0(k ? sb : sa, a0, a1, a2, a3, qh[k][0], qh[k][1]);
                    else q8_mma((w & 1) ? sb : sa, a0, a1, a2, a3, qh[k][0], qh[k][1]);
                    if constexpr (SPLIT && QLO) {
                        if (q_lo) q8_mma((w & 1) ? sb : sa, a0, a1, a2, a3, ql[k][0], ql[k][1]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i >> 1][i & 1] = sa[i] + sb[i];
        }
        if (!SPLIT && q_lo) {  // uniform
#pragma unroll
            for (int i = 0; i < 4 * NH; ++i)
                s[i >> 2][i >> 1 & 1][i & 1] += __shfl_xor_sync(FULL, s[i >> 2][i >> 1 & 1][i & 1], 2);
        }
        constexpr int NS = UNIFORM ? 1 : 2;
        float vs[NH][NS], kf[NH][NS][2];
#pragma unroll
        for (int j = 0; j < NH; ++j)
#pragma unroll
            for (int r = 0; r < NS; ++r) {
                float kscale;
                if constexpr (UNIFORM) {
                    kscale = lds32f(sm + QG::SCALES + 8 * j);
                    vs[j][r] = lds32f(sm + QG::SCALES + 8 * j + 4);
                } else {
                    kscale = __shfl_sync(FULL, scale, g + 8 * r);
                    vs[j][r] = __shfl_sync(FULL, scale, 16 + g + 8 * r);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) kf[j][r][e] = kscale * qf[e];
            }
        auto on = [&](int j, int r) { return (mask >> (16 * j + 8 * r + g) & 1u) != 0u; };
        if (mask != (NH == 2 ? 0xffffffffu : 0xffffu)) {  // uniform
#pragma unroll
            for (int j = 0; j < NH; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // a scale of zero, or one that was not copied: the score is zero, and -inf stays -inf
                        const bool none = kf[j][r % NS][e] == 0.f;
                        s[j][r][e] = !on(j, r) ? -INFINITY : none ? 0.f : s[j][r][e];
                        if (r == 1 || NS == 2) kf[j][r % NS][e] = none ? 1.f : kf[j][r % NS][e];
                    }
        }

        if constexpr (NEIGHBOURS) {
#pragma unroll
            for (int j = 0; j < NH; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float v = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (head(t, e) < GQ) v = fmaxf(v, s[j][r][e] * kf[j][r % NS][e]);
                    v = fmaxf(v, __shfl_xor_sync(FULL, v, 1));
                    if constexpr (SPLIT) v = fmaxf(v, __shfl_xor_sync(FULL, v, 2));
                    if (t == 0) lam(16 * j + 8 * r + g, v);
                }
        }

        float p[NH][2][2], w[NH][2][2];
        auto weights = [&]() {
            float cv[NH][NS][2];
            bool high = false, wide = false;
#pragma unroll
            for (int j = 0; j < NH; ++j)
#pragma unroll
                for (int r = 0; r < NS; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        cv[j][r][e] = min_nan(c[e] * vs[j][r], 0x1p127f);  // not inf: a weight of zero stays one; NaN stays
                        wide = wide || cv[j][r][e] > 128.f;
                    }
#pragma unroll
            for (int j = 0; j < NH; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // one rounding for x - m0: the largest weights are the most exact
                        p[j][r][e] = exp2_approx(fmaf(s[j][r][e], kf[j][r % NS][e], -m0[e]));
                        w[j][r][e] = p[j][r][e] * cv[j][r % NS][e];
                        high = high || p[j][r][e] > 256.f;
                    }
            if (__any_sync(FULL, wide)) {  // with p <= 2^8 only these can pass 2^15
#pragma unroll
                for (int i = 0; i < 4 * NH; ++i) high = high || w[i >> 2][i >> 1 & 1][i & 1] > 32768.f;
            }
            return __any_sync(FULL, high);
        };
        if (weights()) {
            // raise the references to this tile's largest values
            float fo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = Q8_M_INIT, mv = Q8_M_INIT;
#pragma unroll
                for (int j = 0; j < NH; ++j)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float x = s[j][r][e] * kf[j][r % NS][e];
                        if (on(j, r)) {
                            mx = fmaxf(mx, x);
                            mv = fmaxf(mv, x + __log2f(vs[j][r % NS]));
                        }
                    }
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1) {
                    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, k));
                    mv = fmaxf(mv, __shfl_xor_sync(FULL, mv, k));
                }
                const float mn = fmaxf(m0[e], mx);
                mw[e] = fmaxf(mw[e], mv);
                const int k2 = (int)fminf(fmaxf(5.f - ceilf(mw[e] - mn), -120.f), 120.f);
                const int up = k2 + 127 - (int)(__float_as_uint(c[e]) >> 23);  // c grows by 2^up
                const float f = exp2_approx(m0[e] - mn);
                // the factor of what is summed so far is at most 2.  Where c grows by more
                // than 2^100 (V scales that fall while the scores jump) f may be zero and 2^up
                // infinite: in one exponent there
                fo[e] = up > 100 ? exp2_approx(m0[e] - mn + (float)up)
                                 : f * __uint_as_float((unsigned)(127 + max(up, -126)) << 23);
                m0[e] = mn;
                c[e] = __uint_as_float((unsigned)(127 + k2) << 23);
                l[e] *= f;
            }
            const f32x2 f2 = pack2(fo[0], fo[1]);
#pragma unroll
            for (int m = 0; m < QG::MT; ++m) {
                o[m][0] = mul2(o[m][0], f2);
                o[m][1] = mul2(o[m][1], f2);
            }
            weights();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = p[0][0][e] + p[0][1][e];
            if constexpr (NH == 2) x += p[1][0][e] + p[1][1][e];
            l[e] += x;
        }

        // P fragments: token pairs of column g
        unsigned b[NH][SPLIT ? 2 : 1][2];
#pragma unroll
        for (int j = 0; j < NH; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const unsigned hi = pack_half2(w[j][r][0], w[j][r][1]);
                const float2 back = unpack_half2(hi);
                const unsigned lo = pack_half2(w[j][r][0] - back.x, w[j][r][1] - back.y);
                if constexpr (SPLIT) {
                    b[j][0][r] = q8_transpose(hi);
                    b[j][1][r] = q8_transpose(lo);
                } else {
                    b[j][0][r] = q8_transpose(t < 2 ? hi : lo);
                }
            }
        // O: lane's codes are dims (d/8) g + 0..d/8-1 of tokens 2t, 2t+1, 2t+8, 2t+9 of each half
        unsigned vw[NH][4][D / 32];
        {
            constexpr int N = 8 * D;  // 8 rows on
            const int at = D == 128 ? q8_swz<D>(2 * t, g) : q8_swz<D>(2 * t, g >> 1);
            const unsigned low = sm + QG::V + (D == 128 ? 0 : 8 * (g & 1));
            const unsigned v0 = low + at, v1 = low + (at ^ 64);
#pragma unroll
            for (int j = 0; j < NH; ++j) {
                if constexpr (D == 128) {
                    const uint4 x[4] = {j ? lds128<QG::HALF>(v0) : lds128<0>(v0),
                                        j ? lds128<QG::HALF + 128>(v1) : lds128<128>(v1),
                                        j ? lds128<QG::HALF + N>(v0) : lds128<N>(v0),
                                        j ? lds128<QG::HALF + N + 128>(v1) : lds128<N + 128>(v1)};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        vw[j][k][0] = x[k].x; vw[j][k][1] = x[k].y; vw[j][k][2] = x[k].z; vw[j][k][3] = x[k].w;
                    }
                } else {
                    const uint2 x[4] = {j ? lds64<QG::HALF>(v0) : lds64<0>(v0), j ? lds64<QG::HALF>(v1) : lds64<0>(v1),
                                        j ? lds64<QG::HALF + N>(v0) : lds64<N>(v0),
                                        j ? lds64<QG::HALF + N>(v1) : lds64<N>(v1)};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        vw[j][k][0] = x[k].x; vw[j][k][1] = x[k].y;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            unsigned a[NH][2][4];  // [half][tokens 2t, 2t + 1 | 2t + 8, 2t + 9][code of the word]
#pragma unroll
            for (int j = 0; j < NH; ++j) {
                q8_v_halves<FMT>(vw[j][0][i], vw[j][1][i], a[j][0]);
                q8_v_halves<FMT>(vw[j][2][i], vw[j][3][i], a[j][1]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // a tile's products start from zero and are added in fp32: the
                // tensor core truncates its sums, which over the hundreds of
                // tiles of a long request would cost 4e-6 of the output
                float d[4];
#pragma unroll
                for (int j = 0; j < NH; ++j)
#pragma unroll
                    for (int y = 0; y < (SPLIT ? 2 : 1); ++y) {
                        if (j == 0 && y == 0)
                            q8_mma0(d, a[j][0][2 * k], a[j][0][2 * k + 1], a[j][1][2 * k], a[j][1][2 * k + 1], b[j][y][0],
                                    b[j][y][1]);
                        else
                            q8_mma(d, a[j][0][2 * k], a[j][0][2 * k + 1], a[j][1][2 * k], a[j][1][2 * k + 1], b[j][y][0],
                                   b[j][y][1]);
                    }
                o[2 * i + k][0] = add2(o[2 * i + k][0], pack2(d[0], d[1]));
                o[2 * i + k][1] = add2(o[2 * i + k][1], pack2(d[2], d[3]));
            }
        }
    }

    // The warp's partial: m and l per head, the accumulators [head][dim] at acc.
    __device__ __forceinline__ void write(float* m, float* ls, float* acc, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 4; k <= 16; k <<= 1) l[e] += __shfl_xor_sync(FULL, l[e], k);
        const float inv[2] = {1.f / c[0], 1.f / c[1]};
#pragma unroll
        for (int i = 0; i < QG::MT; ++i) {
            const float2 x = unpack2(o[i][0]), y = unpack2(o[i][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float a = (e ? x.y : x.x) * inv[e], b = (e ? y.y : y.x) * inv[e];
                if constexpr (!SPLIT) {
                    a += __shfl_xor_sync(FULL, a, 2);
                    b += __shfl_xor_sync(FULL, b, 2);
                }
                const int h = head(t, e);
                if ((SPLIT || t < 2) && h < GQ)
                    *reinterpret_cast<float2*>(acc + h * D + (D / 8) * g + 2 * i) = make_float2(a, b);
            }
        }
        if (g == 0 && (SPLIT || t < 2)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = head(t, e);
                if (h < GQ) {
                    m[h] = m0[e];
                    ls[h] = l[e];
                }
            }
        }
    }
};

}  // namespace ckv
