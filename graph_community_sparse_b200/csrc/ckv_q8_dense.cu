// Decode attention over all tokens of a ragged batch in the paged 8-bit cache,
// sm_100a (ckv_dense_decode_q8): the dense comparator of ckv_decode.cu for this
// cache.  The tile arithmetic and what bounds it: ckv_q8_attend.cuh.
//
// Work split: every (request, KV head) is a unit of ceil(len/16) tiles; the
// units are laid end to end and each block takes one equal range of tiles,
// whatever units it crosses, so one long request and many short ones fill the
// grid alike.  Inside a unit's segment the block's warps take tiles in turn,
// each with its own ring of staged tiles and its own softmax state, which the
// block joins in shared memory.  A unit that one block holds whole is finished
// there; otherwise the blocks write partials and the last of them to arrive (a
// counter per unit, returned to zero) joins them in slot order: the result does
// not depend on which block that is, no block waits for another, and the whole
// call is one launch.
#include "ckv_q8_attend.cuh"

namespace ckv {

constexpr int QD_WARPS = 8;
constexpr int QD_THREADS = QD_WARPS * 32;
constexpr int QD_STAGES = 3;
constexpr int QD_CTAS = 2;         // resident blocks per SM
constexpr int QD_MIN_TILES = 16;   // least tiles per block: below it more blocks cost more to join than they save
constexpr int QD_MAX_GRID = 1024;
constexpr int QD_LANES = 32;       // tiles per index window

struct DenseQ8Params {
    Q8View c;
    const void* q;
    float* out;
    float scale_log2;
    int* count;  // [units], zero between calls
    float* m;    // partials: 2 slots per block
    float* l;
    float* acc;
};

size_t q8_counter_bytes(int units) { return align256((size_t)units * 4); }
size_t q8_dense_ws_bytes(int gq, int d) {
    return align256((size_t)2 * QD_MAX_GRID * gq * 4) * 2 + align256((size_t)2 * QD_MAX_GRID * gq * d * 4);
}

template <int D, int GQ>
struct DenseQ8Smem {
    static constexpr int RING = QD_STAGES * Q8Geom<D>::SLOT;  // per warp
    static constexpr int ROW = GQ * D * 4;                    // a warp's accumulators
    static constexpr int WARP = RING > ROW ? RING : ROW;
    static constexpr int FIXED = QD_WARPS * WARP + 2 * QD_WARPS * GQ * 4;
};

template <int D, int GQ, int FMT>
__global__ void __launch_bounds__(QD_THREADS, QD_CTAS) dense_q8_kernel(const __grid_constant__ DenseQ8Params p) {
    using QG = Q8Geom<D>;
    using SM = DenseQ8Smem<D, GQ>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_scan[33];
    __shared__ int s_last;
    const TableView& t = p.c.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = t.B, Hkv = p.c.Hkv, bs = t.block;
    unsigned char* ring = smem + warp * SM::WARP;
    float* wm = reinterpret_cast<float*>(smem + QD_WARPS * SM::WARP);  // [warps][GQ]
    float* wl = wm + QD_WARPS * GQ;
    int* s_pre = reinterpret_cast<int*>(smem + SM::FIXED);             // [B + 1] tiles per head before request b
    pdl_wait();

    {
        const int seg = (B + QD_THREADS - 1) / QD_THREADS;
        const int b0 = min(B, tid * seg), b1 = min(B, b0 + seg);
        int own = 0;
        for (int b = b0; b < b1; ++b) {
            int n = t.len[b];
            if (n < 0 || n > (long long)t.max_blocks * bs) {
                if (blockIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
                n = 0;
            }
            const int x = (n + Q8_TOK - 1) / Q8_TOK;
            s_pre[b] = x;
            own += x;
        }
        int all;
        int run = block_exclusive_scan(own, s_scan, &all);
        for (int b = b0; b < b1; ++b) {
            const int x = s_pre[b];
            s_pre[b] = run;
            run += x;
        }
        if (tid == 0) s_pre[B] = all;
        __syncthreads();
    }
    for (int b = blockIdx.x; b < B; b += gridDim.x)
        if (s_pre[b] == s_pre[b + 1])  // nothing to attend to
            for (int i = tid; i < p.c.Hq * D; i += QD_THREADS) p.out[(size_t)b * p.c.Hq * D + i] = 0.f;
    const int total = s_pre[B] * Hkv;
    const int per = max(QD_MIN_TILES, (total + (int)gridDim.x - 1) / (int)gridDim.x);
    const int start = min((long long)blockIdx.x * per, (long long)total), end = min(start + per, total);
    if (start >= end) return;

    int b = 0;  // the request of the first tile
    {
        int hi = B;
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (s_pre[mid] * Hkv <= start) b = mid;
            else hi = mid;
        }
    }
    Q8Warp<D, GQ, FMT> st;
    for (int at = start; at < end;) {
        while (s_pre[b + 1] * Hkv <= at) ++b;
        const int nt = s_pre[b + 1] - s_pre[b];             // tiles of one unit of this request
        const int h = (at - s_pre[b] * Hkv) / nt;
        const int ubeg = s_pre[b] * Hkv + h * nt, uend = ubeg + nt;
        const int stop = min(end, uend);
        const int lo = at - ubeg, hi = stop - ubeg;         // the segment's tiles of the unit
        const int n = t.len[b];
        const int32_t* table = t.table + (size_t)b * t.max_blocks;

        const int nit = (hi - lo - warp + QD_WARPS - 1) / QD_WARPS;  // this warp's tiles: lo + warp + QD_WARPS i
        auto block_of = [&](int i) {
            const int tile = lo + warp + QD_WARPS * i;
            return i < nit ? table[(tile * Q8_TOK) >> t.sh] : 0;
        };
        int win_cur = block_of(lane), win_nxt = block_of(QD_LANES + lane);
        int stage_in = 0;
        auto issue = [&](int i) {
            if (i < nit) {
                if (i > 0 && (i & (QD_LANES - 1)) == 0) {
                    win_cur = win_nxt;
                    win_nxt = block_of(i + QD_LANES + lane);
                }
                unsigned char* sm = ring + stage_in * QG::SLOT;
                const int id = __shfl_sync(FULL, win_cur, i & (QD_LANES - 1));
                const bool ok = (unsigned)id < (unsigned)t.n_blocks;
                const int pos = (lo + warp + QD_WARPS * i) * Q8_TOK;
                const int rem = ok ? min(n - pos, Q8_TOK) : 0;
                const int64_t unit = ok ? (int64_t)id * Hkv + h : 0;
                const int64_t src = ((unit << t.sh) + (pos & (bs - 1))) * D;
                const char* ksrc = static_cast<const char*>(p.c.k) + src;
                const char* vsrc = static_cast<const char*>(p.c.v) + src;
#pragma unroll
                for (int x = 0; x < QG::TILE / 512; ++x) {
                    const int idx = x * 32 + lane, r = idx / QG::CH, c = idx % QG::CH;
                    const int dst = q8_swz<D>(r, c);
                    cp_async_16(sm + dst, ksrc + idx * 16, r < rem);
                    cp_async_16(sm + QG::TILE + dst, vsrc + idx * 16, r < rem);
                }
                // one scale each for the tile's tokens, K's to the first half
                cp_async_4z(sm + QG::SCALES + lane * 4, (lane < 16 ? p.c.k_scale : p.c.v_scale) + unit, ok);
                if (lane == 0) {
                    *reinterpret_cast<unsigned*>(sm + QG::MASK) = rem > 0 ? 0xffffu >> (16 - rem) : 0u;
                    if (!ok) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
                }
            }
            stage_in = stage_in + 1 == QD_STAGES ? 0 : stage_in + 1;
            cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < QD_STAGES - 1; ++s) issue(s);
        st.load_q(static_cast<const char*>(p.q) +
                      ((size_t)b * p.c.Hq + h * GQ) * D * (p.c.dtype == CKV_DTYPE_BF16 ? 2 : 4),
                  p.c.dtype, p.scale_log2, lane);
        st.reset();
        int stage_out = 0;
        for (int i = 0; i < nit; ++i) {
            __syncwarp();  // every lane is done reading the slot refilled next
            issue(i + QD_STAGES - 1);
            cp_async_wait<QD_STAGES - 1>();
            __syncwarp();  // what the other lanes copied is visible
            st.template tile<false>(ring + stage_out * QG::SLOT, lane, [](int, float) {});
            stage_out = stage_out + 1 == QD_STAGES ? 0 : stage_out + 1;
        }
        cp_async_wait<0>();
        __syncwarp();
        // the warps' states through their rings' memory
        st.write(wm + warp * GQ, wl + warp * GQ, reinterpret_cast<float*>(ring), lane);
        __syncthreads();
        const bool whole = lo == 0 && hi == nt;
        const int slot = 2 * blockIdx.x + (at == start ? 0 : 1);
        float* out = p.out + ((size_t)b * p.c.Hq + h * GQ) * D;
        for (int x = tid; x < GQ * D; x += QD_THREADS) {
            const int hh = x / D;
            float M = Q8_M_INIT;
#pragma unroll
            for (int k = 0; k < QD_WARPS; ++k) M = fmaxf(M, wm[k * GQ + hh]);
            float L = 0.f, A = 0.f;
#pragma unroll
            for (int k = 0; k < QD_WARPS; ++k) {
                const float f = exp2_approx(wm[k * GQ + hh] - M);
                L = fmaf(wl[k * GQ + hh], f, L);
                A = fmaf(reinterpret_cast<const float*>(smem + k * SM::WARP)[x], f, A);
            }
            if (whole) {
                out[x] = L == 0.f ? 0.f : A / L;  // no weight: every block of the unit was out of range
            } else {
                p.acc[(size_t)slot * GQ * D + x] = A;
                if (x % D == 0) {
                    p.m[slot * GQ + hh] = M;
                    p.l[slot * GQ + hh] = L;
                }
            }
        }
        if (!whole) {
            const int unit = b * Hkv + h;
            const int c0 = ubeg / per, c1 = (uend - 1) / per;  // the blocks that hold the unit
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(p.count + unit, 1) == c1 - c0;
            __syncthreads();
            if (s_last) {
                __threadfence();
                if (tid == 0) p.count[unit] = 0;
                auto slot_of = [&](int c) { return 2 * c + (c == c0 && ubeg % per != 0 ? 1 : 0); };
                for (int x = tid; x < GQ * D; x += QD_THREADS) {
                    const int hh = x / D;
                    float M = Q8_M_INIT;
                    for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(p.m + slot_of(c) * GQ + hh));
                    float L = 0.f, A = 0.f;
#pragma unroll 8
                    for (int c = c0; c <= c1; ++c) {
                        const int s = slot_of(c);
                        const float f = exp2_approx(__ldcg(p.m + s * GQ + hh) - M);
                        L = fmaf(__ldcg(p.l + s * GQ + hh), f, L);
                        A = fmaf(__ldcg(p.acc + (size_t)s * GQ * D + x), f, A);
                    }
                    out[x] = L == 0.f ? 0.f : A / L;
                }
            }
        }
        __syncthreads();  // the rings are free again
        at = stop;
    }
}

template <int D, int GQ, int FMT>
static cudaError_t launch_dense_q8_t(const DenseQ8Params& p, cudaStream_t st) {
    static LaunchCache lc;
    auto kern = dense_q8_kernel<D, GQ, FMT>;
    const size_t smem = DenseQ8Smem<D, GQ>::FIXED + ((size_t)p.c.t.B + 1) * 4;
    int per_sm = 0, sms = 0;
    cudaError_t e = prepare_launch(kern, lc, smem, QD_THREADS, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    if (sms <= 0 || per_sm <= 0) return cudaErrorInvalidConfiguration;
    const long long tiles = (long long)p.c.t.B * p.c.Hkv * p.c.t.max_blocks * (p.c.t.block / Q8_TOK);
    const int grid = (int)min((long long)min(sms * per_sm, QD_MAX_GRID), (tiles + QD_MIN_TILES - 1) / QD_MIN_TILES);
    return launch_pdl(KK_ATTENTION, kern, dim3(grid), dim3(QD_THREADS), smem, st, p);
}

cudaError_t launch_dense_decode_q8(const Q8View& c, const void* q, float* out, void* ws, cudaStream_t st) {
    DenseQ8Params p{};
    p.c = c;
    p.q = q;
    p.out = out;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d);
    const int gq = c.Hq / c.Hkv;
    char* w = static_cast<char*>(ws) + WS_RESERVED;
    p.count = reinterpret_cast<int*>(w);
    w += q8_counter_bytes(c.t.B * c.Hkv);
    p.m = reinterpret_cast<float*>(w);
    w += align256((size_t)2 * QD_MAX_GRID * gq * 4);
    p.l = reinterpret_cast<float*>(w);
    w += align256((size_t)2 * QD_MAX_GRID * gq * 4);
    p.acc = reinterpret_cast<float*>(w);
#define CKV_QD(DD, GG)               \
    if (c.d == DD && gq == GG)       \
        return c.format == Q8_I8 ? launch_dense_q8_t<DD, GG, Q8_I8>(p, st) : launch_dense_q8_t<DD, GG, Q8_E4>(p, st);
    CKV_QD(64, 1) CKV_QD(64, 2) CKV_QD(64, 4) CKV_QD(64, 8)
    CKV_QD(128, 1) CKV_QD(128, 2) CKV_QD(128, 4) CKV_QD(128, 8)
#undef CKV_QD
    return cudaErrorInvalidValue;
}

}  // namespace ckv
