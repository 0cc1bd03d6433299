// Attention of one token's queries over 16-token tiles of an 8-bit cache, one
// warp at a time: shared by the dense kernel (ckv_q8_dense.cu) and the sparse one
// (ckv_q8_sparse.cu).
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
// B, so a tile of 16 tokens costs 2 d/16 products:
//   S [token, head]  = K [token, dim]  Q^T [dim, head]
//   O [dim, head]   += V^T [dim, token] P [token, head]
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
// w = p c s_v with c a power of two such that w <= 2^7 when set and <= 2^15 at
// any time (fp16's range); hi + lo then keep 2^-25 of the largest weight's size
// at worst.  c leaves again, exactly, when a partial is written.
#pragma once

#include <type_traits>

#include "ckv_decode.cuh"
#include "ckv_q8.cuh"

namespace ckv {

constexpr int Q8_TOK = 16;  // tokens of a tile
constexpr float Q8_M_INIT = -1e30f;

template <int D>
struct Q8Geom {
    static constexpr int TILE = Q8_TOK * D;        // bytes of a K or V tile
    static constexpr int CH = D / 16;              // 16-byte chunks per row
    static constexpr int SCALES = 2 * TILE;        // float [16] of K, then of V
    static constexpr int MASK = SCALES + 128;      // 16 bits: the tokens that count
    static constexpr int SLOT = SCALES + 256;      // bytes of a ring slot (a multiple of 128)
    static constexpr int KS = D / 16;              // k-steps of Q K^T
    static constexpr int MT = D / 16;              // 16-dim tiles of V^T
};

// Byte offset of 16-byte chunk c of token row r in a staged tile.  Q K^T reads
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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Codes c0..c3 of a word as two fp16 pairs (c0, c1), (c2, c3).  int8: the
// biased byte is the low part of an fp16 in [1024, 1280), whose step is 1.
template <int FMT>
__device__ __forceinline__ void q8_halves(unsigned w, unsigned& p01, unsigned& p23) {
    if constexpr (FMT == Q8_I8) {
        const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        w ^= 0x80808080u;
        const unsigned a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
        p01 = *reinterpret_cast<const unsigned*>(&x);
        p23 = *reinterpret_cast<const unsigned*>(&y);
    } else {
        p01 = e4m3x2_half2((unsigned short)(w & 0xffffu));
        p23 = e4m3x2_half2((unsigned short)(w >> 16));
    }
}

__device__ __forceinline__ void cp_async_4z(void* smem, const void* gmem, bool pred) {
    unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(smem));
    int sz = pred ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(s), "l"(gmem), "r"(sz) : "memory");
}

// The state of one warp over one unit's tokens: lane 4 g + t.
template <int D, int GQ, int FMT>
struct Q8Warp {
    using QG = Q8Geom<D>;
    static constexpr bool SPLIT = GQ == 8;  // hi and lo in products of their own
    unsigned qh[QG::KS][2];                 // Q^T fragments (SPLIT: hi; else hi in columns 0..3, lo in 4..7)
    unsigned ql[SPLIT ? QG::KS : 1][2];
    bool q_lo;                              // SPLIT: some lo is not zero (q in fp32)
    float qf[2];                            // per head of this lane: 2^e log2(e)/sqrt(d)
    float m0[2], mw[2], c[2], l[2];         // references of x and of x + log2 s_v, weight factor, sum
    float o[QG::MT][4];

    __device__ __forceinline__ static int head(int t, int e) { return SPLIT ? 2 * t + e : (2 * t + e) & 3; }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m0[e] = mw[e] = Q8_M_INIT;
            c[e] = 1.f;
            l[e] = 0.f;
        }
#pragma unroll
        for (int m = 0; m < QG::MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][i] = 0.f;
    }

    // q: the group's first row.  Lane (g, t) holds column g: head g (SPLIT), or
    // head g & 3, hi for g < 4 and lo otherwise; dims 16 (t + 4 j) + 4 w + 0..3
    // are k-step 4 j + w.
    __device__ __forceinline__ void load_q(const void* q, int dtype, float scale_log2, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int h = SPLIT ? g : g & 3;
        const bool real = h < GQ;
        float x[QG::KS][4];
        unsigned amax = 0;
#pragma unroll
        for (int s = 0; s < QG::KS; ++s) {
            const int dim = 16 * (t + 4 * (s >> 2)) + 4 * (s & 3);
            const size_t at = (size_t)(real ? h : 0) * D + dim;
            if (dtype == CKV_DTYPE_BF16) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(q) + at);
                x[s][0] = bf16_lo(w.x); x[s][1] = bf16_hi(w.x); x[s][2] = bf16_lo(w.y); x[s][3] = bf16_hi(w.y);
            } else {
                const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(q) + at);
                x[s][0] = w.x; x[s][1] = w.y; x[s][2] = w.z; x[s][3] = w.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!real) x[s][i] = 0.f;
                amax = max(amax, __float_as_uint(x[s][i]) & 0x7fffffffu);
            }
        }
        amax = max(amax, __shfl_xor_sync(FULL, amax, 1));
        amax = max(amax, __shfl_xor_sync(FULL, amax, 2));
        // the row's largest magnitude goes to [2^14, 2^15): codes and sums stay in
        // range, and 2^-29 of it is still a normal fp16.  Rows below 2^-100 count
        // as that large.
        const int e = max((int)(amax >> 23), 27) - 127 - 14;  // amax = m 2^(e + 14)
        const float down = __uint_as_float((unsigned)(127 - min(e, 126)) << 23);
        const float f = __uint_as_float((unsigned)(127 + min(max(e, -126), 126)) << 23) * scale_log2;
        bool any_lo = false;
#pragma unroll
        for (int s = 0; s < QG::KS; ++s) {
            unsigned hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = x[s][2 * i] * down, b = x[s][2 * i + 1] * down;
                hi[i] = pack_half2(a, b);
                const float2 r = unpack_half2(hi[i]);
                lo[i] = pack_half2(a - r.x, b - r.y);
                if constexpr (SPLIT) {
                    qh[s][i] = hi[i];
                    ql[s][i] = lo[i];
                    any_lo = any_lo || lo[i] != 0u;
                } else {
                    qh[s][i] = g < 4 ? hi[i] : lo[i];
                }
            }
        }
        q_lo = SPLIT && __any_sync(FULL, any_lo);
#pragma unroll
        for (int k = 0; k < 2; ++k) qf[k] = __shfl_sync(FULL, f, head(t, k) * 4);
    }

    // One staged tile.  lam (NEIGHBOURS): lam(i, x) receives the largest x over
    // the group's heads of the tile's token i, from one lane per token.
    template <bool NEIGHBOURS, typename Lam>
    __device__ __forceinline__ void tile(const unsigned char* sm, int lane, Lam lam) {
        const int g = lane >> 2, t = lane & 3;
        const unsigned mask = *reinterpret_cast<const unsigned*>(sm + QG::MASK);
        if (mask == 0u) return;  // uniform over the warp
        const float* sc = reinterpret_cast<const float*>(sm + QG::SCALES);

        // S: rows g, g + 8, columns 2t, 2t + 1; even and odd k-steps apart
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const uint4 ka = *reinterpret_cast<const uint4*>(sm + q8_swz<D>(g, t + 4 * j));
            const uint4 kb = *reinterpret_cast<const uint4*>(sm + q8_swz<D>(g + 8, t + 4 * j));
            const unsigned wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int s = 4 * j + w;
                unsigned a0, a1, a2, a3;
                q8_halves<FMT>(wa[w], a0, a2);
                q8_halves<FMT>(wb[w], a1, a3);
                q8_mma((w & 1) ? sb : sa, a0, a1, a2, a3, qh[s][0], qh[s][1]);
                if constexpr (SPLIT) {
                    if (q_lo) q8_mma((w & 1) ? sb : sa, a0, a1, a2, a3, ql[s][0], ql[s][1]);
                }
            }
        }
        float s[2][2];  // [token g | g + 8][head]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = sa[i] + sb[i];
            if constexpr (!SPLIT) x += __shfl_xor_sync(FULL, x, 2);
            s[i >> 1][i & 1] = x;
        }
        const float ks[2] = {sc[g], sc[g + 8]}, vs[2] = {sc[16 + g], sc[24 + g]};
        const bool on[2] = {(mask >> g & 1u) != 0u, (mask >> (g + 8) & 1u) != 0u};
        float kf[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) kf[r][e] = ks[r] * qf[e];

        if constexpr (NEIGHBOURS) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float v = -INFINITY;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (head(t, e) < GQ && on[r]) v = fmaxf(v, s[r][e] * kf[r][e]);
                v = fmaxf(v, __shfl_xor_sync(FULL, v, 1));
                if constexpr (SPLIT) v = fmaxf(v, __shfl_xor_sync(FULL, v, 2));
                if (t == 0) lam(g + 8 * r, v);
            }
        }

        float p[2][2], w[2][2];
        auto weights = [&]() {
            bool high = false;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // one rounding for x - m0: the largest weights are the most exact
                    const float y = on[r] ? fmaf(s[r][e], kf[r][e], -m0[e]) : -INFINITY;
                    p[r][e] = exp2_approx(y);
                    w[r][e] = p[r][e] * c[e] * vs[r];
                    high = high || y > 8.f || w[r][e] > 32768.f;
                }
            return __any_sync(FULL, high);
        };
        if (weights()) {
            // raise the references to this tile's largest values
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = Q8_M_INIT, mv = Q8_M_INIT;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float x = s[r][e] * kf[r][e];
                    if (on[r]) {
                        mx = fmaxf(mx, x);
                        mv = fmaxf(mv, x + __log2f(vs[r]));
                    }
                }
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1) {
                    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, k));
                    mv = fmaxf(mv, __shfl_xor_sync(FULL, mv, k));
                }
                const float mn = fmaxf(m0[e], mx);
                mw[e] = fmaxf(mw[e], mv);
                const int k2 = (int)fminf(fmaxf(7.f - ceilf(mw[e] - mn), -120.f), 120.f);
                const float cn = __uint_as_float((unsigned)(127 + k2) << 23);
                const float f = exp2_approx(m0[e] - mn);
                const float fo = f * (cn / c[e]);
                m0[e] = mn;
                c[e] = cn;
                l[e] *= f;
#pragma unroll
                for (int m = 0; m < QG::MT; ++m) {
                    o[m][e] *= fo;
                    o[m][2 + e] *= fo;
                }
            }
            weights();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) l[e] += p[0][e] + p[1][e];

        // P fragments: token pairs of column g
        unsigned b[SPLIT ? 2 : 1][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const unsigned hi = pack_half2(w[r][0], w[r][1]);
            const float2 back = unpack_half2(hi);
            const unsigned lo = pack_half2(w[r][0] - back.x, w[r][1] - back.y);
            if constexpr (SPLIT) {
                b[0][r] = q8_transpose(hi);
                b[1][r] = q8_transpose(lo);
            } else {
                b[0][r] = q8_transpose(t < 2 ? hi : lo);
            }
        }
        // O: lane's codes are dims (d/8) g + 0..d/8-1 of tokens 2t, 2t+1, 2t+8, 2t+9
        unsigned vw[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = 2 * t + (k & 1) + 8 * (k >> 1);
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(sm + QG::TILE + q8_swz<D>(r, g));
                vw[k][0] = x.x; vw[k][1] = x.y; vw[k][2] = x.z; vw[k][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(sm + QG::TILE + q8_swz<D>(r, g >> 1) + 8 * (g & 1));
                vw[k][0] = x.x; vw[k][1] = x.y;
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            // bytes of two tokens interleaved, then the pairs' fp16
            unsigned a[2][4];  // [tokens 2t | 2t + 8][code of the word]
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                q8_halves<FMT>(__byte_perm(vw[2 * k][i], vw[2 * k + 1][i], 0x5140), a[k][0], a[k][1]);
                q8_halves<FMT>(__byte_perm(vw[2 * k][i], vw[2 * k + 1][i], 0x7362), a[k][2], a[k][3]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                q8_mma(o[2 * i + k], a[0][2 * k], a[0][2 * k + 1], a[1][2 * k], a[1][2 * k + 1], b[0][0], b[0][1]);
                if constexpr (SPLIT)
                    q8_mma(o[2 * i + k], a[0][2 * k], a[0][2 * k + 1], a[1][2 * k], a[1][2 * k + 1], b[1][0], b[1][1]);
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
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float a = o[i][e] * inv[e], b = o[i][2 + e] * inv[e];
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
