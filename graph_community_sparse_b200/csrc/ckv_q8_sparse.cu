// Attention over the selected positions of the paged 8-bit cache, sm_100a
// (ckv_sparse_decode_q8): CommunityKV's exact attention over the selected
// communities plus the sinks ("CommunityKV: Efficient Long-Context Decoding via
// Graph Partitioning", rit.work summary, section "A graph of tokens replaces
// re-clustering", paragraphs 4-5), read in place from a cache in 8 bits.  The
// tile arithmetic and what bounds it: ckv_q8_attend.cuh.
//
// Without neighbours to find, one launch of the block-split kernel
// (ckv_q8_blocks.cuh).  With them, two: the graph logits of the whole list have to
// be there before the search, so the split over warps (equal slices of the
// concatenated lists, then chunks by ticket) and the merge kernel with its
// neighbour search and fused update are those of the 16/32-bit cache's attention
// (ckv_decode.cuh).  What differs is the way to a row: a list entry's position goes
// through the request's block table, one window of 32 entries ahead of the copies,
// and each row brings its own two scales.
#include "ckv_q8_blocks.cuh"

namespace ckv {

constexpr int QS_WARPS = 4;
constexpr int QS_TOK = 16;    // tokens of a tile: 16 warps an SM then have room for three
constexpr int QS_STAGES = 3;
constexpr int QS_CTAS = 4;    // resident blocks per SM

struct SparseQ8Params {
    DecodeParams d;
    Q8View c;
};

template <int D, int GQ, int FMT>
__device__ __forceinline__ void sparse_q8_segment(const SparseQ8Params& p, int u, int lo, int hi, int slot,
                                                  unsigned char* ring, int lane) {
    using QG = Q8Geom<D, 1>;
    const TableView& t = p.c.t;
    int b, kvh, h0;
    unit_heads(p.d, u, GQ, false, b, kvh, h0);
    const int32_t* toks = p.d.sel_tok + (size_t)u * p.d.tok_cap;
    const int32_t* table = t.table + (size_t)b * t.max_blocks;
    const int len = (int)min((long long)t.len[b], (long long)t.max_blocks << t.sh);
    const int n = hi - lo, nit = (n + QS_TOK - 1) / QS_TOK;

    const auto raw_q = Q8Warp<D, GQ, FMT, 1>::fetch_q(
        Q8Warp<D, GQ, FMT, 1>::q_row(p.d.q, p.c.dtype, (size_t)b * p.d.Hq + h0), p.c.dtype, lane);

    // Two tiles' entries are a window, one entry a lane.  The copies of a window
    // need its positions and their blocks: loaded two and one windows ahead, and
    // only looked at by the copies themselves, so that no load is waited for where
    // it is issued.
    auto position = [&](int w) { return w * 32 + lane < n ? toks[lo + w * 32 + lane] : -1; };
    auto inside = [&](int pos) { return (unsigned)pos < (unsigned)max(len, 0); };
    auto block_of = [&](int pos) { return inside(pos) ? table[pos >> t.sh] : -1; };
    int pos0 = position(0), pos1 = position(1);
    int id0 = block_of(pos0);
    int row_cur = -1;  // this window's entry's row of the pool; -1: not attended
    // the tiles' scales (lanes 0..15 K's, 16..31 V's) and masks, newest first
    float scales[QS_STAGES];
    unsigned masks[QS_STAGES];
    const float* slane = lane < 16 ? p.c.k_scale : p.c.v_scale;
    const unsigned ring32 = smem_addr32(ring);
    unsigned stage_in = 0;
    auto issue = [&](int i) {
#pragma unroll
        for (int k = QS_STAGES - 1; k > 0; --k) {
            scales[k] = scales[k - 1];
            masks[k] = masks[k - 1];
        }
        if (i < nit) {
            if ((i & 1) == 0) {
                row_cur = -1;
                if (inside(pos0) && (unsigned)id0 < (unsigned)t.n_blocks)
                    row_cur = ((id0 * p.c.Hkv + kvh) << t.sh) + (pos0 & (t.block - 1));
                else if (i * QS_TOK + lane < n)
                    atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
                pos0 = pos1;
                id0 = block_of(pos0);
                pos1 = position((i >> 1) + 2);
            }
            const unsigned sm = ring32 + stage_in * QG::SLOT;
            const int base = (i & 1) << 4;
            const int mine = __shfl_sync(FULL, row_cur, base + (lane & 15));
            scales[0] = mine >= 0 ? slane[mine >> t.sh] : 0.f;
            masks[0] = __ballot_sync(FULL, mine >= 0) & 0xffffu;
#pragma unroll
            for (int x = 0; x < QG::HALF / 512; ++x) {
                const int idx = x * 32 + lane, r = idx / QG::CH, c = idx % QG::CH;
                const int row = __shfl_sync(FULL, row_cur, base + r);
                const int size = row >= 0 ? 16 : 0;
                const size_t src = (size_t)max(row, 0) * D + c * 16;
                const unsigned dst = sm + q8_swz<D>(r, c);
                cp_async_16s(dst, static_cast<const char*>(p.c.k) + src, size);
                cp_async_16s(dst + QG::V, static_cast<const char*>(p.c.v) + src, size);
            }
        }
        stage_in = stage_in + 1 == QS_STAGES ? 0 : stage_in + 1;
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < QS_STAGES - 1; ++s) issue(s);
    Q8Warp<D, GQ, FMT, 1> st;
    st.set_q(raw_q, p.c.dtype, p.d.scale_log2, lane);
    st.reset();
    float* lamu = p.d.ws.lam + (size_t)u * p.d.ws.lam_cap + lo;
    unsigned stage_out = 0;
    auto step = [&](auto nbr) {
        for (int i = 0; i < nit; ++i) {
            __syncwarp();  // every lane is done reading the slot refilled next
            issue(i + QS_STAGES - 1);
            cp_async_wait<QS_STAGES - 1>();
            __syncwarp();  // what the other lanes copied is visible
            const unsigned mask = masks[QS_STAGES - 1];
            if constexpr (decltype(nbr)::value) {
                // an all-invalid tile has no logits of its own to store
                if (mask == 0u && lane < QS_TOK && i * QS_TOK + lane < n) lamu[i * QS_TOK + lane] = -INFINITY;
            }
            st.template tile<false, decltype(nbr)::value>(
                ring32 + stage_out * QG::SLOT, mask, scales[QS_STAGES - 1], lane, [&](int k, float x) {
                    if (i * QS_TOK + k < n) lamu[i * QS_TOK + k] = x;
                });
            stage_out = stage_out + 1 == QS_STAGES ? 0 : stage_out + 1;
        }
    };
    if (p.d.want_nbr) step(std::true_type{});
    else step(std::false_type{});
    cp_async_wait<0>();
    __syncwarp();
    st.write(p.d.ws.m + (size_t)slot * GQ, p.d.ws.l + (size_t)slot * GQ, p.d.ws.acc + (size_t)slot * GQ * D, lane);
}

template <int D, int GQ, int FMT>
__global__ void __launch_bounds__(QS_WARPS * 32, QS_CTAS) sparse_q8_kernel(const __grid_constant__ SparseQ8Params p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_warp[33];
    constexpr int RING = QS_STAGES * Q8Geom<D, 1>::SLOT;
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char* ring = smem + warp * RING;
    int* s_pre = reinterpret_cast<int*>(smem + QS_WARPS * RING);
    const int U = p.d.U;
    {
        // exclusive prefix of the lists' lengths; block 0 publishes it for the merge
        const int seg = (U + blockDim.x - 1) / blockDim.x;
        const int b0 = min(U, (int)threadIdx.x * seg), b1 = min(U, b0 + seg);
        int own = 0;
        for (int i = b0; i < b1; ++i) {
            const int x = max(0, min(p.d.n_tok[i], p.d.tok_cap));
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
        if (threadIdx.x == 0) s_pre[U] = all;
        __syncthreads();
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i <= U; i += blockDim.x) p.d.unit_prefix[i] = s_pre[i];
    }
    const int total = s_pre[U];
    if (total <= 0) return;
    const DynSplit sp = dyn_split(total, p.d.W, false);
    auto run_range = [&](int start, int end, int sbase) {
        int u = 0, c = U;
        while (c - u > 1) {
            const int mid = (u + c) >> 1;
            if (s_pre[mid] <= start) u = mid;
            else c = mid;
        }
        while (true) {
            const int lo = max(start, s_pre[u]), hi = min(end, s_pre[u + 1]);
            if (lo < hi) sparse_q8_segment<D, GQ, FMT>(p, u, lo - s_pre[u], hi - s_pre[u], sbase + u, ring, lane);
            if (end <= s_pre[u + 1] || u + 1 >= U) break;
            ++u;
        }
    };
    // one loop, so the segment's code is there once: the static slice (slots
    // [0, W + U)), then chunks by ticket (slots [W + U, W + 2U + nch))
    const int w = blockIdx.x * QS_WARPS + warp;
    int start = w * sp.per_s, end = min(start + sp.per_s, sp.R), sbase = w;
    while (true) {
        if (start < end) run_range(start, end, sbase);
        int c = 0;
        if (lane == 0) c = atomicAdd(p.d.ws.ticket, 1);
        c = __shfl_sync(FULL, c, 0);
        if (c >= sp.nch) break;
        start = sp.R + c * sp.chk;
        end = min(start + sp.chk, total);
        sbase = p.d.W + U + c;
    }
}

template <int D, int GQ, int FMT>
static cudaError_t launch_sparse_q8_t(SparseQ8Params p, cudaStream_t st) {
    static LaunchCache lc;
    auto kern = sparse_q8_kernel<D, GQ, FMT>;
    const size_t smem = QS_WARPS * QS_STAGES * Q8Geom<D, 1>::SLOT + ((size_t)p.d.U + 1) * 4;
    int per_sm = 0, sms = 0;
    cudaError_t e = prepare_launch(kern, lc, smem, QS_WARPS * 32, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    if (sms <= 0 || per_sm <= 0) return cudaErrorInvalidConfiguration;
    const int blocks = min(sms * per_sm, MAX_DECODE_WARPS / QS_WARPS);
    p.d.W = blocks * QS_WARPS;
    e = launch_pdl(KK_ATTENTION, kern, dim3(blocks), dim3(QS_WARPS * 32), smem, st, p);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.d.U), block(D + 32 * NBR_WARPS);
    if (p.c.dtype == CKV_DTYPE_BF16)
        return launch_pdl(KK_MERGE, decode_merge<__nv_bfloat16, D, GQ, false, true>, grid, block, 0, st, p.d);
    return launch_pdl(KK_MERGE, decode_merge<float, D, GQ, false, true>, grid, block, 0, st, p.d);
}

cudaError_t launch_sparse_decode_q8(const Q8View& c, const GraphView& g, const SelView& s, const void* q, float* out,
                                    int32_t* nbr8, const void* k_new, int32_t* assigned, void* ws, cudaStream_t st) {
    SparseQ8Params p{};
    p.c = c;
    DecodeParams& d = p.d;
    d.q = q;
    d.Hq = c.Hq;
    d.Hkv = c.Hkv;
    d.G = g.G;
    d.U = c.t.B * g.G;
    d.per_head = g.mode == CKV_GRAPH_PER_HEAD;
    d.S = g.S;
    d.sel_tok = s.sel_tok;
    d.tok_cap = s.tok_cap;
    d.T_cap = g.T_cap;
    d.dev_err = g.dev_err;
    d.unit_prefix = s.unit_prefix;
    d.n_tok = s.n_tok;
    d.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d);
    d.ws = carve_decode_ws(ws, WS_RESERVED + Q8_COUNTER_BYTES, d.U, g.gq, c.d, s.tok_cap);
    d.want_nbr = nbr8 != nullptr || k_new != nullptr;
    d.out = out;
    d.nbr8 = nbr8;
    d.len = c.t.len;
    if (k_new) {
        CacheView v{};
        v.B = c.t.B;
        v.Hkv = c.Hkv;
        v.Hq = c.Hq;
        v.d = c.d;
        v.T_cap = g.T_cap;
        v.dtype = c.dtype;
        d.append = 1;
        d.ap = make_assign_params(v, g, 0, nullptr, nullptr, nullptr, assigned);
        d.ap.k = k_new;  // nothing is written to a cache here: k_dst stays NULL
        d.ap.sb = (int64_t)c.Hkv * c.d;
        d.ap.sh = c.d;
    }
    if (!d.want_nbr) {
        BlocksQ8Params b{};
        b.c = c;
        b.q = q;
        b.out = out;
        b.scale_log2 = d.scale_log2;
        b.U = d.U;
        b.G = d.G;
        b.per_head = d.per_head;
        b.tok_cap = d.tok_cap;
        b.sel_tok = d.sel_tok;
        b.n_tok = d.n_tok;
        carve_blocks_ws(b, ws, g.gq);
        const long long tiles = (long long)d.U * (d.tok_cap / (QD_MIN_PIECE * 16) + 1);
#define CKV_QL(DD, GG)                                                                  \
        if (c.d == DD && g.gq == GG)                                                    \
            return c.format == Q8_I8 ? launch_blocks_q8_t<DD, GG, Q8_I8, true>(b, tiles, st) \
                                     : launch_blocks_q8_t<DD, GG, Q8_E4, true>(b, tiles, st);
        CKV_QL(64, 1) CKV_QL(64, 2) CKV_QL(64, 4) CKV_QL(64, 8)
        CKV_QL(128, 1) CKV_QL(128, 2) CKV_QL(128, 4) CKV_QL(128, 8)
#undef CKV_QL
        return cudaErrorInvalidValue;
    }
#define CKV_QS(DD, GG)             \
    if (c.d == DD && g.gq == GG)   \
        return c.format == Q8_I8 ? launch_sparse_q8_t<DD, GG, Q8_I8>(p, st) : launch_sparse_q8_t<DD, GG, Q8_E4>(p, st);
    CKV_QS(64, 1) CKV_QS(64, 2) CKV_QS(64, 4) CKV_QS(64, 8)
    CKV_QS(128, 1) CKV_QS(128, 2) CKV_QS(128, 4) CKV_QS(128, 8)
#undef CKV_QS
    return cudaErrorInvalidValue;
}

}  // namespace ckv
