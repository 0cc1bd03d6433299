// Decode attention over all tokens of a ragged batch in the paged 8-bit cache,
// sm_100a (ckv_dense_decode_q8): the dense comparator of ckv_decode.cu for this
// cache.  The kernel and its work split: ckv_q8_blocks.cuh.
#include "ckv_q8_blocks.cuh"

namespace ckv {

size_t q8_blocks_ws_bytes(int gq, int d) {
    return align256((size_t)2 * QD_MAX_GRID * gq * 4) * 2 + align256((size_t)2 * QD_MAX_GRID * gq * d * 4);
}

cudaError_t launch_dense_decode_q8(const Q8View& c, const void* q, float* out, void* ws, cudaStream_t st) {
    BlocksQ8Params p{};
    p.c = c;
    p.q = q;
    p.out = out;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d);
    const int gq = c.Hq / c.Hkv;
    carve_blocks_ws(p, ws, gq, c.d);
    const long long units = (long long)c.t.B * c.Hkv;
    const long long most = units * ((long long)c.t.max_blocks * c.t.block / (QD_WARPS * QdShape<64, false>::TOK) + 1);
#define CKV_QD(DD, GG)                                                                \
    if (c.d == DD && gq == GG)                                                        \
        return c.format == Q8_I8 ? launch_blocks_q8_t<DD, GG, Q8_I8, false>(p, most, st) \
                                 : launch_blocks_q8_t<DD, GG, Q8_E4, false>(p, most, st);
    CKV_QD(64, 1) CKV_QD(64, 2) CKV_QD(64, 4) CKV_QD(64, 8)
    CKV_QD(128, 1) CKV_QD(128, 2) CKV_QD(128, 4) CKV_QD(128, 8)
#undef CKV_QD
    return cudaErrorInvalidValue;
}

}  // namespace ckv
