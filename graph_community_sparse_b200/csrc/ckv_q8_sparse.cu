// Attention over the selected positions of the paged 8-bit cache, sm_100a
// (ckv_sparse_decode_q8): CommunityKV's exact attention over the selected
// communities plus the sinks ("CommunityKV: Efficient Long-Context Decoding via
// Graph Partitioning", rit.work summary, section "A graph of tokens replaces
// re-clustering", paragraphs 4-5), read in place from a cache in 8 bits.  The
// block-split kernel (ckv_q8_blocks.cuh) attends; when neighbours are wanted it also
// stores each entry's graph logit, and a small kernel launched as its programmatic
// dependent searches them and runs the fused update, a block per graph unit (the
// search of ckv_decode.cuh): a chain of dependent loads, 4 to 9 us after the attention
// (8 lists of 2052 tokens 11.5 -> 15.8 us, 256 of them 51 -> 60 us), and the update 3 to
// 5 us more.
#include "ckv_q8_blocks.cuh"

namespace ckv {

template <typename T, int D>
__global__ void __launch_bounds__(NBR_THREADS) neighbours_q8_kernel(const __grid_constant__ DecodeParams p) {
    pdl_wait();  // the logits are complete and visible
    const int u = blockIdx.x, t = threadIdx.x;
    const int n = max(0, min(p.n_tok[u], p.tok_cap));
    JoinAt at;
    if (p.append) {
        at.len = p.len[u / p.G];
        if (p.built) at.built = p.built[u];
        const int tl = min(p.ap.tail_len[u], p.ap.max_tail);
        if (tl > 0) at.last = p.ap.tail_tok[(size_t)u * p.ap.max_tail + tl - 1];
    }
    if (n > 0) {
        search_neighbours<T, D, true>(p, u, n, t, at);
        return;
    }
    if (p.nbr8 && t < CKV_NEIGHBOURS) p.nbr8[(size_t)u * CKV_NEIGHBOURS + t] = -1;
    if (p.append) {
        __shared__ int s_none[CKV_NEIGHBOURS];
        if (t < CKV_NEIGHBOURS) s_none[t] = -1;
        merge_assign<T, D, true>(p, u, s_none, t, at);  // no neighbour: the token joins nothing
    }
}

// A graph after its requests' lengths went down, or did not go up as a join
// expected (ckv_trim_graph_q8): a block per unit.  Nothing to do is the rule: 2
// dependent loads.
constexpr int TRIM_THREADS = 128;

struct TrimParams {
    TableView t;
    AssignParams ap;
    int32_t* offs;
    int32_t* num_comm;
    int32_t* built;
};

template <int D>
__global__ void __launch_bounds__(TRIM_THREADS) trim_graph_kernel(const __grid_constant__ TrimParams p) {
    pdl_wait();
    const AssignParams& ap = p.ap;
    const int u = blockIdx.x, tid = threadIdx.x;
    const int n = p.t.len[u / ap.G], built = p.built[u];
    if (n < 0 || n > (long long)p.t.max_blocks << p.t.sh) {
        if (tid == 0) atomicOr(p.t.dev_err, CKV_DEVERR_BLOCK);
        return;
    }
    if (n >= built) {
        if (tid < 32) untail_unit<D>(ap, u, n, tid);
        return;
    }
    // members of the build are gone: their communities cannot be kept
    for (int i = tid; i < ap.Cmax; i += TRIM_THREADS) {
        ap.cnt[(size_t)u * ap.Cmax + i] = 0;
        p.offs[(size_t)u * (ap.Cmax + 1) + i + 1] = 0;
    }
    for (int i = tid; i < ap.T_cap; i += TRIM_THREADS) ap.comm_of[(size_t)u * ap.T_cap + i] = -1;
    __syncthreads();  // everybody has read built
    if (tid == 0) {
        p.num_comm[u] = 0;
        ap.tail_len[u] = 0;
        p.built[u] = 0;
        if (n > 0) atomicOr(ap.dev_err, CKV_DEVERR_CUT);
    }
}

cudaError_t launch_trim_graph_q8(const Q8View& c, const GraphView& g, cudaStream_t st) {
    CacheView v{};
    v.B = c.t.B;
    v.Hkv = c.Hkv;
    v.Hq = c.Hq;
    v.d = c.d;
    v.dtype = c.dtype;
    const TrimParams p{c.t, make_assign_params(v, g, 0, nullptr, nullptr, nullptr, nullptr), g.offs, g.num_comm, g.built};
    const dim3 grid(p.ap.U), block(TRIM_THREADS);
    if (c.d == 128) return launch_pdl(KK_UPDATE, trim_graph_kernel<128>, grid, block, 0, st, p);
    return launch_pdl(KK_UPDATE, trim_graph_kernel<64>, grid, block, 0, st, p);
}

template <int D, int GQ, int FMT>
static cudaError_t launch_sparse_q8_t(const BlocksQ8Params& b, const DecodeParams& d, long long most, cudaStream_t st) {
    if (!d.want_nbr) return launch_blocks_q8_t<D, GQ, FMT, true>(b, most, st);
    const cudaError_t e = launch_blocks_q8_t<D, GQ, FMT, true, true>(b, most, st);
    if (e != cudaSuccess) return e;
    if (b.c.dtype == CKV_DTYPE_BF16)
        return launch_pdl(KK_MERGE, neighbours_q8_kernel<__nv_bfloat16, D>, dim3(d.U), dim3(NBR_THREADS), 0, st, d);
    return launch_pdl(KK_MERGE, neighbours_q8_kernel<float, D>, dim3(d.U), dim3(NBR_THREADS), 0, st, d);
}

cudaError_t launch_sparse_decode_q8(const Q8View& c, const GraphView& g, const SelView& s, const void* q, float* out,
                                    int32_t* nbr8, const void* k_new, int32_t* assigned, void* ws, cudaStream_t st) {
    BlocksQ8Params b{};
    b.c = c;
    b.q = q;
    b.out = out;
    b.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d);
    b.U = c.t.B * g.G;
    b.G = g.G;
    b.per_head = g.mode == CKV_GRAPH_PER_HEAD;
    b.S = g.S;
    b.tok_cap = s.tok_cap;
    b.sel_tok = s.sel_tok;
    b.n_tok = s.n_tok;
    carve_blocks_ws(b, ws, g.gq, c.d);
    DecodeParams d{};  // what the neighbour search and the update read
    d.G = g.G;
    d.U = b.U;
    d.S = g.S;
    d.sel_tok = s.sel_tok;
    d.tok_cap = s.tok_cap;
    d.n_tok = s.n_tok;
    d.ws.lam = b.lam;
    d.ws.lam_cap = s.tok_cap;
    d.want_nbr = nbr8 != nullptr || k_new != nullptr;
    d.nbr8 = nbr8;
    d.len = c.t.len;
    d.built = g.built;
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
    const long long most = (long long)d.U * (d.tok_cap / (QD_WARPS * QdShape<64, true>::TOK) + 1);
#define CKV_QS(DD, GG)                                                            \
    if (c.d == DD && g.gq == GG)                                                  \
        return c.format == Q8_I8 ? launch_sparse_q8_t<DD, GG, Q8_I8>(b, d, most, st) \
                                 : launch_sparse_q8_t<DD, GG, Q8_E4>(b, d, most, st);
    CKV_QS(64, 1) CKV_QS(64, 2) CKV_QS(64, 4) CKV_QS(64, 8)
    CKV_QS(128, 1) CKV_QS(128, 2) CKV_QS(128, 4) CKV_QS(128, 8)
#undef CKV_QS
    return cudaErrorInvalidValue;
}

}  // namespace ckv
