// Indexed sparse decode attention (and the dense comparator) for sm_100a.
//
// CommunityKV runs exact softmax attention over the selected communities
// plus the sink tokens, read straight from the whole cache ("CommunityKV:
// Efficient Long-Context Decoding via Graph Partitioning", rit.work summary,
// section "A graph of tokens replaces re-clustering", paragraphs 4-5).  This
// is a matrix-vector product over gathered rows: bandwidth-bound, so it runs
// on the CUDA cores, not the tensor cores.
//
// Work split (stream-K over warps): the selected tokens of all graph units
// are laid end to end (selection.unit_prefix); warp w of W takes the slice
// [w*per, (w+1)*per) with per = ceil(total/W), whatever units it crosses, so
// every warp reads the same number of K/V rows regardless of how skewed the
// community sizes are.  A warp writes one partial (running max m, sum l,
// unnormalised accumulator) per unit segment into slot w + u, and, when
// neighbours are wanted, each list entry's graph logit;
// which is unique because slices and units are both contiguous and ordered.
// All warps of the persistent grid finish together, so the merge of each
// unit's slots is a second, small kernel launched as a programmatic
// dependent: its launch overlaps the attention kernel's tail and it waits
// (in hardware, griddepcontrol) for that kernel's results; every operand is
// fetched in one round of independent loads.
//
// Inside a warp: each half-warp owns one token row at a time, a lane owns
// D/16 consecutive elements (16 bytes for bf16, d = 128); K and V rows of
// 8 tokens per iteration are staged by cp.async into a per-warp ring of
// Stages<GQ> iterations (2 for one head per graph, where more resident warps
// matter more, 3 otherwise), so loads stay in flight while one is computed.
// Logits of the GQA group's heads are reduced with a value-exchanging
// butterfly; the softmax uses exp2 with log2(e)/sqrt(d) folded into q and a
// lazily raised running max (raised only when a logit exceeds it by more
// than 2^8), which is exact after the final division.
#include <math.h>
#include <type_traits>

#include "ckv_decode.cuh"

namespace ckv {

constexpr int DEC_WARPS = 4;
constexpr int TOK_PER_IT = 8;
constexpr float RESCALE_THRESH = 8.0f;

template <int GQ> struct Stages { static constexpr int v = GQ == 1 ? 2 : 3; };
template <int GQ> struct MinBlocks { static constexpr int v = GQ == 1 ? 6 : (GQ == 2 ? 5 : (GQ == 4 ? 4 : 2)); };

template <typename T, int D>
struct RowGeom {
    static constexpr int E = D / 16;
    static constexpr int PART = E * ElemBytes<T>::v;
    static constexpr int ROW = 16 * PART;
    static constexpr int TILE = TOK_PER_IT * ROW;
};

// bf16 caches whose graphs serve several query heads use the tensor-core
// segment loop (ckv_decode_mma.cuh); the others the scalar one below.
template <typename T, int GQ>
struct UseMma {
    static constexpr bool v = std::is_same<T, __nv_bfloat16>::value && GQ >= 2;
};
template <typename T, int GQ>
struct DecMinBlocks {
    static constexpr int v = UseMma<T, GQ>::v ? 2 : MinBlocks<GQ>::v;
};
template <int D>
struct MmaGeom;

template <typename T, int D, int GQ>
struct DecSmem {
    static constexpr int PBUF = TOK_PER_IT * GQ * 4;
    static constexpr int SCALAR = Stages<GQ>::v * 2 * RowGeom<T, D>::TILE + ((PBUF + 127) / 128) * 128;
    static constexpr int MMA = 3 * 2 * 16 * D * 2;  // MMA_STAGES x (K, V) x MMA_TOK rows of bf16
    static constexpr int WARP = UseMma<T, GQ>::v ? MMA : SCALAR;
    static constexpr int CTA_FIXED = DEC_WARPS * WARP;
};

#include "ckv_decode_mma.cuh"

// One warp, one unit, list positions [lo, hi) of the unit's selection (or
// cache positions, dense).  Full iterations (all 8 tokens valid, past the
// sinks) take a path without per-token masks; only the last, partial
// iteration and the one holding the sinks test each token.
template <typename T, int D, int GQ, bool DENSE>
__device__ __forceinline__ void process_segment(const DecodeParams& p, int u, int lo, int hi, int slot,
                                                unsigned char* wsm, int lane) {
    using RG = RowGeom<T, D>;
    constexpr int E = RG::E, PART = RG::PART, ROW = RG::ROW, TILE = RG::TILE;
    constexpr int LG = Log2<GQ>::v;
    constexpr int NS = Stages<GQ>::v;
    const int half = lane >> 4, l16 = lane & 15;
    const int hl = head_of_lane<GQ>(lane);
    const bool owner = (lane & ((16 >> LG) - 1)) == 0;
    const int64_t st = p.st;
    const bool want_nbr = !DENSE && p.want_nbr;

    int b, kvh, h0;
    unit_heads(p, u, GQ, DENSE, b, kvh, h0);
    const T* Kb = static_cast<const T*>(p.k) + b * p.sb + kvh * p.sh + l16 * E;
    const T* Vb = static_cast<const T*>(p.v) + b * p.sb + kvh * p.sh + l16 * E;
    const int32_t* toks = DENSE ? nullptr : p.sel_tok + (size_t)u * p.tok_cap;

    float qr[GQ][E];
#pragma unroll
    for (int h = 0; h < GQ; ++h) {
        load_row_part<T, E>(static_cast<const T*>(p.q) + ((size_t)b * p.Hq + h0 + h) * D + l16 * E, qr[h]);
#pragma unroll
        for (int e = 0; e < E; ++e) qr[h][e] *= p.scale_log2;
    }

    const int n = hi - lo;
    const int nit = (n + TOK_PER_IT - 1) / TOK_PER_IT;
    const int nfull = n / TOK_PER_IT;
    float* pbuf = reinterpret_cast<float*>(wsm + NS * 2 * TILE);

    int win_cur = 0, win_nxt = 0;
    if constexpr (!DENSE) {
        win_cur = (lane < n) ? __ldg(toks + lo + lane) : 0;
        win_nxt = (32 + lane < n) ? __ldg(toks + lo + 32 + lane) : 0;
    }

    int stage_in = 0;  // ring slot the next issue fills
    auto issue = [&](int it, auto full_tag) {
        constexpr bool ALL_VALID = decltype(full_tag)::value;
        unsigned char* kt = wsm + stage_in * 2 * TILE;
        stage_in = (stage_in + 1 == NS) ? 0 : stage_in + 1;
        unsigned char* vt = kt + TILE;
        if constexpr (!DENSE) {
            if (it > 0 && (it & 3) == 0) {
                win_cur = win_nxt;
                const int nx = (it + 4) * TOK_PER_IT + lane;
                win_nxt = (nx < n) ? __ldg(toks + lo + nx) : 0;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = it * TOK_PER_IT + 2 * j + half;
            const bool valid = ALL_VALID || i < n;
            int pos;
            if constexpr (DENSE) {
                pos = lo + i;
            } else {
                pos = __shfl_sync(ckv::FULL, win_cur, ((it & 3) << 3) + 2 * j + half);
                pos = checked_index(pos, 0, p.T_cap, p.dev_err, 0);
            }
            if (!ALL_VALID) pos = valid ? pos : 0;
            const int64_t off = (int64_t)pos * st;
            const int r = 2 * j + half;
            cp_async_part<PART>(kt + r * ROW + l16 * PART, Kb + off, valid);
            cp_async_part<PART>(vt + r * ROW + l16 * PART, Vb + off, valid);
        }
        cp_async_commit();
    };
    auto issue_any = [&](int it) {
        if (it < nfull) issue(it, std::true_type{});
        else if (it < nit) issue(it, std::false_type{});
        else cp_async_commit();
    };

#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue_any(s);

    float m_run = -INFINITY, l_run = 0.f;
    float acc[GQ][E];
#pragma unroll
    for (int h = 0; h < GQ; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] = 0.f;
    float* lamu = DENSE ? nullptr : p.ws.lam + (size_t)u * p.ws.lam_cap;
    int stage_out = 0;  // ring slot computed next

    auto compute = [&](int it, auto full_tag) {
        constexpr bool ALL_VALID = decltype(full_tag)::value;
        const unsigned char* kt = wsm + stage_out * 2 * TILE;
        const unsigned char* vt = kt + TILE;
        stage_out = (stage_out + 1 == NS) ? 0 : stage_out + 1;

        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float kf[E];
            load_row_part<T, E>(reinterpret_cast<const T*>(kt + (2 * j + half) * ROW + l16 * PART), kf);
            float part[GQ];
#pragma unroll
            for (int h = 0; h < GQ; ++h) {
                float a = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) a = fmaf(qr[h][e], kf[e], a);
                part[h] = a;
            }
            s[j] = halfwarp_reduce_heads<GQ>(part, lane);
            if (!ALL_VALID && it * TOK_PER_IT + 2 * j + half >= n) s[j] = -INFINITY;
        }

        float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        mx = fmaxf(mx, __shfl_xor_sync(ckv::FULL, mx, 16));
        const bool need = mx > m_run + RESCALE_THRESH;
        if (__any_sync(ckv::FULL, need)) {
            const float m_new = need ? mx : m_run;
            const float f = (m_run == -INFINITY) ? 0.f : exp2_approx(m_run - m_new);
            l_run *= f;
            m_run = m_new;
#pragma unroll
            for (int h = 0; h < GQ; ++h) {
                const float fh = __shfl_sync(ckv::FULL, f, (lane & 16) | (h << (4 - LG)));
#pragma unroll
                for (int e = 0; e < E; ++e) acc[h][e] *= fh;
            }
        }

        float pj[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) pj[j] = exp2_approx(s[j] - m_run);
        l_run += (pj[0] + pj[1]) + (pj[2] + pj[3]);

        if constexpr (GQ > 1) {
            if (owner) {
#pragma unroll
                for (int j = 0; j < 4; ++j) pbuf[(2 * j + half) * GQ + hl] = pj[j];
            }
            __syncwarp();
        }

#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float ph[GQ];
            if constexpr (GQ == 1) {
                ph[0] = pj[j];
            } else {
#pragma unroll
                for (int h = 0; h < GQ; h += 2) {
                    const float2 t2 = *reinterpret_cast<const float2*>(pbuf + (2 * j + half) * GQ + h);
                    ph[h] = t2.x;
                    ph[h + 1] = t2.y;
                }
            }
            float vf[E];
            load_row_part<T, E>(reinterpret_cast<const T*>(vt + (2 * j + half) * ROW + l16 * PART), vf);
#pragma unroll
            for (int h = 0; h < GQ; ++h)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[h][e] = fmaf(ph[h], vf[e], acc[h][e]);
        }

        if (want_nbr) {
            // graph logit of each token (max over the group's heads) for the
            // neighbour search in the merge kernel
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float lam = halfwarp_max_over_heads<GQ>(s[j]);
                const int i = it * TOK_PER_IT + 2 * j + half;
                if (l16 == 0 && (ALL_VALID || i < n)) lamu[lo + i] = lam;
            }
        }
    };

    for (int it = 0; it < nit; ++it) {
        __syncwarp();
        issue_any(it + NS - 1);
        cp_async_wait<NS - 1>();
        if (it < nfull) compute(it, std::true_type{});
        else compute(it, std::false_type{});
    }
    cp_async_wait<0>();

#pragma unroll
    for (int h = 0; h < GQ; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] += __shfl_xor_sync(FULL, acc[h][e], 16);
    l_run += __shfl_xor_sync(FULL, l_run, 16);

    const DecodeWs& ws = p.ws;
    if (lane < 16) {
#pragma unroll
        for (int h = 0; h < GQ; ++h) {
            float* dst = ws.acc + ((size_t)slot * GQ + h) * D + l16 * E;
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *reinterpret_cast<float4*>(dst + e) = make_float4(acc[h][e], acc[h][e + 1], acc[h][e + 2], acc[h][e + 3]);
        }
        if (owner) {
            ws.m[(size_t)slot * GQ + hl] = m_run;
            ws.l[(size_t)slot * GQ + hl] = l_run;
        }
    }
}

template <typename T, int D, int GQ, bool DENSE>
__global__ void __launch_bounds__(DEC_WARPS * 32, DecMinBlocks<T, GQ>::v) decode_main(const __grid_constant__ DecodeParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    pdl_wait();  // the selection comes from the kernel before
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char* wsm = smem + warp * DecSmem<T, D, GQ>::WARP;
    int* s_pre = reinterpret_cast<int*>(smem + DecSmem<T, D, GQ>::CTA_FIXED);
    const int w = blockIdx.x * DEC_WARPS + warp;

    int total;
    if constexpr (!DENSE) {
        // exclusive prefix of the units' token counts, computed by every block
        // (each thread scans a contiguous chunk); block 0 also publishes it
        __shared__ int s_warp[33];
        const int seg = (p.U + blockDim.x - 1) / blockDim.x;
        const int b0 = min(p.U, (int)threadIdx.x * seg), b1 = min(p.U, b0 + seg);
        int own = 0;
        for (int i = b0; i < b1; ++i) {
            int x = p.n_tok[i];
            if constexpr (kDebugChecks) {
                if (x < 0 || x > p.tok_cap) {
                    atomicOr(p.dev_err, CKV_DEVERR_INDEX);
                    x = max(0, min(x, p.tok_cap));
                }
            }
            s_pre[i] = x;
            own += x;
        }
        int all;
        int run = block_exclusive_scan(own, s_warp, &all);
        for (int i = b0; i < b1; ++i) {
            const int x = s_pre[i];
            s_pre[i] = run;
            run += x;
        }
        if (threadIdx.x == 0) s_pre[p.U] = all;
        __syncthreads();
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i <= p.U; i += blockDim.x) p.unit_prefix[i] = s_pre[i];
        total = s_pre[p.U];
    } else {
        total = p.U * p.T;
    }
    if (total <= 0) return;
    const DynSplit sp = dyn_split(total, p.W, DENSE);

    // tokens [start, end) of the concatenated lists; partial of unit u in
    // slot sbase + u
    auto run_range = [&](int start, int end, int sbase) {
        int u;
        if constexpr (DENSE) {
            u = start / p.T;
        } else {
            int a = 0, c = p.U;  // s_pre[a] <= start < s_pre[c]
            while (c - a > 1) {
                const int mid = (a + c) >> 1;
                if (s_pre[mid] <= start) a = mid;
                else c = mid;
            }
            u = a;
        }
        while (true) {
            const int ubeg = DENSE ? u * p.T : s_pre[u];
            const int uend = DENSE ? ubeg + p.T : s_pre[u + 1];
            const int lo = max(start, ubeg), hi = min(end, uend);
            if (lo < hi) {
                if constexpr (UseMma<T, GQ>::v)
                    process_segment_mma<D, GQ, DENSE>(p, u, lo - ubeg, hi - ubeg, sbase + u, wsm, lane);
                else
                    process_segment<T, D, GQ, DENSE>(p, u, lo - ubeg, hi - ubeg, sbase + u, wsm, lane);
            }
            if (end <= uend || u + 1 >= p.U) break;
            ++u;
        }
    };

    // static slice: slots [0, W + U)
    const int start = w * sp.per_s;
    if (start < sp.R) run_range(start, min(start + sp.per_s, sp.R), w);
    // dynamic chunks: slots [W + U, W + 2U + nch)
    while (true) {
        int c = 0;
        if (lane == 0) c = atomicAdd(p.ws.ticket, 1);
        c = __shfl_sync(FULL, c, 0);
        if (c >= sp.nch) break;
        const int c0 = sp.R + c * sp.chk;
        run_range(c0, min(c0 + sp.chk, total), p.W + p.U + c);
    }
}


// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Partial slots: W + U for the static slices, then NCH_MAX + U for the
// dynamic chunks, then MERGE_PAD spares.
static size_t decode_slots(int U) { return (size_t)MAX_DECODE_WARPS + NCH_MAX + 2 * (size_t)U + MERGE_PAD; }

size_t decode_ws_bytes(int U, int gq, int d, int lam_cap) {
    const size_t slots = decode_slots(U);
    return align256(slots * gq * 4) * 2 + align256(slots * gq * d * 4) + align256((size_t)U * lam_cap * 4);
}

// ws: the workspace base (its head holds the ticket); the parts follow the head
DecodeWs carve_decode_ws(void* ws, size_t head, int U, int gq, int d, int lam_cap) {
    const size_t slots = decode_slots(U);
    char* p = static_cast<char*>(ws);
    DecodeWs w;
    w.ticket = reinterpret_cast<int*>(p);
    p += head;
    w.m = reinterpret_cast<float*>(p);
    p += align256(slots * gq * 4);
    w.l = reinterpret_cast<float*>(p);
    p += align256(slots * gq * 4);
    w.acc = reinterpret_cast<float*>(p);
    p += align256(slots * gq * d * 4);
    w.lam = reinterpret_cast<float*>(p);
    w.lam_cap = lam_cap;
    return w;
}

namespace {

template <typename T, int D, int GQ, bool DENSE>
cudaError_t launch_decode_t(DecodeParams p, cudaStream_t st) {
    static LaunchCache lc;
    auto kern = decode_main<T, D, GQ, DENSE>;
    const size_t smem = DecSmem<T, D, GQ>::CTA_FIXED + (DENSE ? 0 : (size_t)(p.U + 1) * 4);
    int per_sm = 0, sms = 0;
    cudaError_t e = prepare_launch(kern, lc, smem, DEC_WARPS * 32, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    if (sms <= 0 || per_sm <= 0) return cudaErrorInvalidConfiguration;
    int blocks = sms * per_sm;
    if (blocks * DEC_WARPS > MAX_DECODE_WARPS) blocks = MAX_DECODE_WARPS / DEC_WARPS;
    p.W = blocks * DEC_WARPS;
    e = launch_pdl(KK_ATTENTION, kern, dim3(blocks), dim3(DEC_WARPS * 32), smem, st, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(KK_MERGE, decode_merge<T, D, GQ, DENSE>, dim3(p.U), dim3(D + (DENSE ? 0 : 32 * NBR_WARPS)),
                      0, st, p);
}

template <bool DENSE>
cudaError_t dispatch(const CacheView& c, int gq, DecodeParams p, cudaStream_t st) {
#define CKV_DEC_CASE(TT, DD, GG)                                                      \
    if (c.d == DD && gq == GG) return launch_decode_t<TT, DD, GG, DENSE>(p, st);
    if (c.dtype == CKV_DTYPE_BF16) {
        CKV_DEC_CASE(__nv_bfloat16, 128, 1) CKV_DEC_CASE(__nv_bfloat16, 128, 2)
        CKV_DEC_CASE(__nv_bfloat16, 128, 4) CKV_DEC_CASE(__nv_bfloat16, 128, 8)
        CKV_DEC_CASE(__nv_bfloat16, 64, 1) CKV_DEC_CASE(__nv_bfloat16, 64, 2)
        CKV_DEC_CASE(__nv_bfloat16, 64, 4) CKV_DEC_CASE(__nv_bfloat16, 64, 8)
    } else {
        CKV_DEC_CASE(float, 128, 1) CKV_DEC_CASE(float, 128, 2)
        CKV_DEC_CASE(float, 128, 4) CKV_DEC_CASE(float, 128, 8)
        CKV_DEC_CASE(float, 64, 1) CKV_DEC_CASE(float, 64, 2)
        CKV_DEC_CASE(float, 64, 4) CKV_DEC_CASE(float, 64, 8)
    }
#undef CKV_DEC_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_sparse_decode(const CacheView& c, const GraphView& g, const SelView& s,
                                 const void* q, float* out, int32_t* nbr8, void* ws, const AssignParams* ap,
                                 cudaStream_t st) {
    DecodeParams p{};
    p.k = c.k;
    p.v = c.v;
    p.sb = c.sb;
    p.sh = c.sh;
    p.st = c.st;
    p.q = q;
    p.Hq = c.Hq;
    p.Hkv = c.Hkv;
    p.G = g.G;
    p.U = c.B * g.G;
    p.per_head = g.mode == CKV_GRAPH_PER_HEAD;
    p.S = g.S;
    p.sel_tok = s.sel_tok;
    p.tok_cap = s.tok_cap;
    p.T_cap = c.T_cap;
    p.dev_err = g.dev_err;
    p.unit_prefix = s.unit_prefix;
    p.n_tok = s.n_tok;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d);
    p.ws = carve_decode_ws(ws, ws_head_bytes(c.B, c.Hq), p.U, g.gq, c.d, s.tok_cap);
    p.want_nbr = nbr8 != nullptr || ap != nullptr;
    p.out = out;
    p.nbr8 = nbr8;
    if (ap) {
        p.append = 1;
        p.ap = *ap;
    }
    return dispatch<false>(c, g.gq, p, st);
}

cudaError_t launch_dense_decode(const CacheView& c, const void* q, int T, float* out, void* ws,
                                cudaStream_t st) {
    DecodeParams p{};
    p.k = c.k;
    p.v = c.v;
    p.sb = c.sb;
    p.sh = c.sh;
    p.st = c.st;
    p.q = q;
    p.Hq = c.Hq;
    p.Hkv = c.Hkv;
    p.G = c.Hkv;
    p.U = c.B * c.Hkv;
    p.per_head = 0;
    p.T = T;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d);
    const int gq = c.Hq / c.Hkv;
    p.ws = carve_decode_ws(ws, ws_head_bytes(c.B, c.Hq), p.U, gq, c.d, 0);
    p.out = out;
    return dispatch<true>(c, gq, p, st);
}

}  // namespace ckv
