// Attention over the selected positions of the paged 8-bit cache, sm_100a
// (ckv_sparse_decode_q8): CommunityKV's exact attention over the selected
// communities plus the sinks ("CommunityKV: Efficient Long-Context Decoding via
// Graph Partitioning", rit.work summary, section "A graph of tokens replaces
// re-clustering", paragraphs 4-5), read in place from a cache in 8 bits.  The
// block-split kernel (ckv_q8_blocks.cuh) attends; when neighbours are wanted it also
// stores each entry's graph logit, and a small kernel launched as its programmatic
// dependent searches them and runs the fused update, a block per graph unit (the
// search of ckv_decode.cuh): a chain of dependent loads, 4 to 8 us after the attention
// (8 lists of 2052 tokens 11.5 -> 15.5 us, 256 of them 50 -> 59 us).
#include "ckv_q8_blocks.cuh"

namespace ckv {

template <typename T, int D>
__global__ void __launch_bounds__(NBR_THREADS) neighbours_q8_kernel(const __grid_constant__ DecodeParams p) {
    pdl_wait();  // the logits are complete and visible
    const int u = blockIdx.x, t = threadIdx.x;
    const int n = max(0, min(p.n_tok[u], p.tok_cap));
    if (n > 0) {
        search_neighbours<T, D, true>(p, u, n, t);
        return;
    }
    if (p.nbr8 && t < CKV_NEIGHBOURS) p.nbr8[(size_t)u * CKV_NEIGHBOURS + t] = -1;
    if (p.append) {
        __shared__ int s_none[CKV_NEIGHBOURS];
        if (t < CKV_NEIGHBOURS) s_none[t] = -1;
        merge_assign<T, D, true>(p, u, s_none, t);  // no neighbour: the token joins nothing
    }
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
