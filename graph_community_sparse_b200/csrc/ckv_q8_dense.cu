// Decode attention over all tokens of a ragged batch in the paged 8-bit cache,
// sm_100a (ckv_dense_decode_q8): the dense comparator of ckv_decode.cu for this
// cache.  The tile arithmetic and what bounds it: ckv_q8_attend.cuh.
//
// Work split: every (request, KV head) is a unit of ceil(len/16) tiles; each
// block has one range of tiles, found by every block for itself from the lengths.
// Where pieces of about an equal share that do not cross units are no more than
// the blocks, each block has one piece, and so one start and one join; otherwise
// the units are laid end to end and cut into equal ranges, which may cross units.
// The second way costs a block that crosses a unit about 16 tiles' time (a new
// query, an empty ring, a join), the first the difference between the longest
// piece and the share: the smaller loss decides.  (Finer pieces by ticket, for the
// SMs' 10 % difference in bandwidth, lost more by their starts: 8 requests of
// 128K tokens 357 against 350 us, 8 heads a group at 64K 249 against 200.)
//
// Inside a segment of a unit the warps take tiles in turn, each with its own ring of
// staged tiles and its own softmax state, joined in shared memory.  A unit that
// one block holds whole is finished there; otherwise the blocks write partials
// and the last one to arrive (a counter per unit, returned to zero) joins them in
// order: the result does not depend on which block that is, no block waits for
// another, and the whole call is one launch.
#include "ckv_q8_attend.cuh"

namespace ckv {

constexpr int QD_WARPS = 4;
constexpr int QD_THREADS = QD_WARPS * 32;
constexpr int QD_CTAS = 4;          // resident blocks per SM
constexpr int QD_MAX_GRID = 640;    // >= QD_CTAS * SMs
constexpr int QD_MIN_PIECE = 16;    // tiles: below it more partials cost more than they save
constexpr int QD_CROSS = 16;        // tiles: what crossing a unit costs a block
constexpr int QD_LANES = 32;        // tiles per index window

template <int D>
struct QdStages {
    static constexpr int v = D == 128 ? 3 : 5;  // 16 warps x 2 (4) tiles ahead: at least 64 KB in flight per SM
};

struct DenseQ8Params {
    Q8View c;
    const void* q;
    float* out;
    float scale_log2;
    int* count;   // [units], zero between calls
    float* m;     // partials: two slots a block
    float* l;
    float* acc;
};

size_t q8_counter_bytes(int units) { return align256((size_t)units * 4); }
size_t q8_dense_ws_bytes(int gq, int d) {
    return align256((size_t)2 * QD_MAX_GRID * gq * 4) * 2 + align256((size_t)2 * QD_MAX_GRID * gq * d * 4);
}

template <int D, int GQ>
struct DenseQ8Smem {
    static constexpr int WARP = QdStages<D>::v * Q8Geom<D>::SLOT;  // a warp's ring, then its accumulators
    static constexpr int FIXED = QD_WARPS * WARP + 2 * QD_WARPS * GQ * 4;
    static_assert(GQ * D * 4 <= WARP, "a warp's accumulators fit its ring");
    // the join of a unit's partials: weights and sums of JOIN slots at a time
    static constexpr int JOIN = 512;
    static_assert(2 * JOIN * GQ * 4 + QD_THREADS * 16 <= QD_WARPS * WARP, "the join fits the rings");
};

// Joins the partials of a unit that blocks c0 .. c0 + np - 1 share into out, JOIN
// at a time.  A block's first segment has its even slot, its last (when that is
// another) the odd one: `odd` for block c0.  References
// and sums first, all at once, then the weighted rows with the slots shared out
// over the threads.
template <int D, int GQ>
__device__ __forceinline__ void join_partials(const DenseQ8Params& p, int c0, int np, int odd, float* out,
                                              unsigned char* smem, float* s_head, int tid) {
    constexpr int JOIN = DenseQ8Smem<D, GQ>::JOIN;
    constexpr int VECS = GQ * D / 4;  // float4 of an output
    constexpr int SHARE = QD_THREADS / VECS > 0 ? QD_THREADS / VECS : 1;
    constexpr int PER = VECS > QD_THREADS ? VECS / QD_THREADS : 1;
    const int lane = tid & 31, warp = tid >> 5;
    float* s_f = reinterpret_cast<float*>(smem);  // [JOIN][GQ] references, then weights
    float* s_l = s_f + JOIN * GQ;                 // [JOIN][GQ] sums
    float4* s_part = reinterpret_cast<float4*>(s_l + JOIN * GQ);
    float* s_m = s_head;                          // [GQ] running reference, sum and the old rows' factor
    float* s_sum = s_head + GQ;
    __shared__ float s_old[GQ];
    if (tid < GQ) {
        s_m[tid] = Q8_M_INIT;
        s_sum[tid] = 0.f;
    }
    const int part = tid / VECS;
    float4 A[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) A[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < np; i0 += JOIN) {
        const int n = min(np - i0, JOIN);
        __syncthreads();
        auto slot_of = [&](int i) { return 2 * (c0 + i0 + i) + (i0 + i == 0 ? odd : 0); };
        for (int x = tid; x < n * GQ; x += QD_THREADS) {
            const int at = slot_of(x / GQ) * GQ + x % GQ;
            s_f[x] = __ldcg(p.m + at);
            s_l[x] = __ldcg(p.l + at);
        }
        __syncthreads();
        for (int h = warp; h < GQ; h += QD_WARPS) {
            float M = s_m[h], L = 0.f;
            const float before = M;
            for (int i = lane; i < n; i += 32) M = fmaxf(M, s_f[i * GQ + h]);
#pragma unroll
            for (int k = 16; k >= 1; k >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, k));
            for (int i = lane; i < n; i += 32) {
                const float f = exp2_approx(s_f[i * GQ + h] - M);
                s_f[i * GQ + h] = f;
                L = fmaf(s_l[i * GQ + h], f, L);
            }
#pragma unroll
            for (int k = 16; k >= 1; k >>= 1) L += __shfl_xor_sync(FULL, L, k);
            if (lane == 0) {
                const float f = exp2_approx(before - M);
                s_old[h] = f;
                s_m[h] = M;
                s_sum[h] = fmaf(s_sum[h], f, L);
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int x = tid % VECS + k * QD_THREADS, h = x / (D / 4);
            const float4* acc = reinterpret_cast<const float4*>(p.acc) + x;
            const float fo = s_old[h];
            A[k].x *= fo;
            A[k].y *= fo;
            A[k].z *= fo;
            A[k].w *= fo;
#pragma unroll 8
            for (int i = part; i < n; i += SHARE) {
                const float4 v = __ldcg(acc + (size_t)slot_of(i) * VECS);
                const float f = s_f[i * GQ + h];
                A[k].x = fmaf(v.x, f, A[k].x);
                A[k].y = fmaf(v.y, f, A[k].y);
                A[k].z = fmaf(v.z, f, A[k].z);
                A[k].w = fmaf(v.w, f, A[k].w);
            }
        }
    }
    if constexpr (SHARE > 1) {
        s_part[tid] = A[0];
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int k = 1; k < SHARE; ++k) {
                const float4 v = s_part[k * VECS + tid];
                A[0].x += v.x;
                A[0].y += v.y;
                A[0].z += v.z;
                A[0].w += v.w;
            }
        }
    }
    if (part == 0) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int x = tid + k * QD_THREADS;
            const float L = s_sum[x / (D / 4)];
            const float inv = L == 0.f ? 0.f : 1.f / L;  // no weight: every block of the unit was out of range
            reinterpret_cast<float4*>(out)[x] = make_float4(A[k].x * inv, A[k].y * inv, A[k].z * inv, A[k].w * inv);
        }
    }
}

// A whole tile, K and V, each 16 D contiguous bytes (k, v: lane's first 16 of them).
// Rows 4 apart (d = 128) or 8 apart (d = 64) differ in the swizzle by one bit, or none.
template <int D>
__device__ __forceinline__ void copy_tile(unsigned sm, const char* k, const char* v, int lane) {
    constexpr int TILE = Q8Geom<D>::TILE;
    const unsigned even = sm + q8_swz<D>(lane / Q8Geom<D>::CH, lane % Q8Geom<D>::CH);
    cp_async_16i<0, 0>(even, k);
    cp_async_16i<TILE, 0>(even, v);
    if constexpr (D == 128) {
        const unsigned odd = sm + (q8_swz<D>(lane / 8, lane % 8) ^ 64);
        cp_async_16i<512, 512>(odd, k);
        cp_async_16i<1024, 1024>(even, k);
        cp_async_16i<1536, 1536>(odd, k);
        cp_async_16i<TILE + 512, 512>(odd, v);
        cp_async_16i<TILE + 1024, 1024>(even, v);
        cp_async_16i<TILE + 1536, 1536>(odd, v);
    } else {
        cp_async_16i<512, 512>(even, k);
        cp_async_16i<TILE + 512, 512>(even, v);
    }
}

template <int D, int GQ, int FMT>
__global__ void __launch_bounds__(QD_THREADS, QD_CTAS) dense_q8_kernel(const __grid_constant__ DenseQ8Params p) {
    using QG = Q8Geom<D>;
    using SM = DenseQ8Smem<D, GQ>;
    constexpr int STAGES = QdStages<D>::v;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_scan[33];
    __shared__ int s_last;
    const TableView& t = p.c.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = t.B, Hkv = p.c.Hkv, bs = t.block, grid = gridDim.x;
    unsigned char* ring = smem + warp * SM::WARP;
    float* wm = reinterpret_cast<float*>(smem + QD_WARPS * SM::WARP);  // [warps][GQ]
    float* wl = wm + QD_WARPS * GQ;
    int* s_nt = reinterpret_cast<int*>(smem + SM::FIXED);              // B > 32: [B] tiles of a unit of request b
    int* s_pre = s_nt + B;                                             // [B] positions or items before request b
    pdl_wait();

    auto tiles_of = [&](int b) {
        const int n = t.len[b];
        if (n >= 0 && n <= (long long)t.max_blocks * bs) return (n + Q8_TOK - 1) / Q8_TOK;
        if (blockIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
        return 0;
    };
    auto ceil_div = [](int a, int b) { return (int)(((unsigned)a + b - 1) / (unsigned)b); };
    // Up to 32 requests every warp works with one a lane, without a block barrier;
    // more are shared out over the threads.
    const bool small = B <= 32;
    const int seg = ceil_div(B, QD_THREADS);
    const int b0 = min(B, tid * seg), b1 = min(B, b0 + seg);
    int my_nt = 0, my_pre = 0, all = 0;
    if (small) {
        my_nt = lane < B ? tiles_of(lane) : 0;
        all = __reduce_add_sync(FULL, my_nt);
    } else {
        int own = 0;
        for (int b = b0; b < b1; ++b) own += s_nt[b] = tiles_of(b);
        block_exclusive_scan(own, s_scan, &all);
    }
    const int total = all * Hkv;
    if (total == 0) {
        for (int i = blockIdx.x * QD_THREADS + tid; i < B * p.c.Hq * D; i += grid * QD_THREADS) p.out[i] = 0.f;
        return;
    }
    const int share = ceil_div(total, grid);
    // pieces of at most `piece` tiles: 0 where the units are laid end to end instead
    const int per = max(share, QD_MIN_PIECE);
    const int most = per + max(QD_CROSS, share >> 4);
    const int step = max(1, (most - per) / (small ? 8 : 3));
    int piece = per, items = 0;
    while (true) {
        int own = 0;
        if (small) {
            own = __reduce_add_sync(FULL, ceil_div(my_nt, piece));
        } else {
            int mine = 0;
            for (int b = b0; b < b1; ++b) mine += ceil_div(s_nt[b], piece);
            block_exclusive_scan(mine, s_scan, &own);
        }
        items = own * Hkv;
        if (items <= grid) break;
        if (piece >= most) {
            piece = 0;
            break;
        }
        piece = min(piece + step, most);
    }
    // [start, end): this block's range, in pieces or in tiles, and what comes before each request
    const int start = piece ? (int)blockIdx.x : (int)min((long long)blockIdx.x * per, (long long)total);
    const int end = piece ? min(start + 1, items) : min(start + per, total);
    if (small) {
        const int own = piece ? ceil_div(my_nt, piece) : my_nt;
        my_pre = own;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int y = __shfl_up_sync(FULL, my_pre, k);
            if (lane >= k) my_pre += y;
        }
        my_pre = (my_pre - own) * Hkv;
    } else {
        int own = 0, none;
        for (int b = b0; b < b1; ++b) own += piece ? ceil_div(s_nt[b], piece) : s_nt[b];
        int run = block_exclusive_scan(own, s_scan, &none);
        for (int b = b0; b < b1; ++b) {
            s_pre[b] = run * Hkv;
            run += piece ? ceil_div(s_nt[b], piece) : s_nt[b];
        }
        __syncthreads();
    }
    for (int b = blockIdx.x; b < B; b += grid)
        if ((small ? __shfl_sync(FULL, my_nt, b & 31) : s_nt[b]) == 0)  // nothing to attend to
            for (int i = tid; i < p.c.Hq * D; i += QD_THREADS) p.out[(size_t)b * p.c.Hq * D + i] = 0.f;

    Q8Warp<D, GQ, FMT> st;
    for (int at = start; at < end;) {
        // the segment: tiles [lo, hi) of KV head h of request b, the unit shared by the blocks c0 .. c0 + np - 1
        int b, nt, pre;
        if (small) {
            b = 31 - __clz(__ballot_sync(FULL, lane < B && my_nt > 0 && my_pre <= at));
            nt = __shfl_sync(FULL, my_nt, b);
            pre = __shfl_sync(FULL, my_pre, b);
        } else {
            int hi = B;
            b = 0;
            while (hi - b > 1) {
                const int mid = (b + hi) >> 1;
                if (s_pre[mid] <= at) b = mid;
                else hi = mid;
            }
            while (s_nt[b] == 0) --b;  // empty requests share their place with the one before
            nt = s_nt[b];
            pre = s_pre[b];
        }
        int h, lo, hi, c0, np, odd = 0, slot = 2 * blockIdx.x;
        if (piece) {
            np = ceil_div(nt, piece);
            h = (at - pre) / np;
            const int i = (at - pre) - h * np;
            lo = (int)((long long)nt * i / np);
            hi = (int)((long long)nt * (i + 1) / np);
            c0 = blockIdx.x - i;
            at = end;
        } else {
            h = (at - pre) / nt;
            const int ubeg = pre + h * nt;
            lo = at - ubeg;
            hi = min(end - ubeg, nt);
            c0 = ubeg / per;
            np = (ubeg + nt - 1) / per - c0 + 1;
            odd = ubeg - c0 * per != 0 ? 1 : 0;
            slot += at == start ? 0 : 1;
            at = ubeg + hi;
        }
        const auto raw_q = Q8Warp<D, GQ, FMT>::fetch_q(
            Q8Warp<D, GQ, FMT>::q_row(p.q, p.c.dtype, (size_t)b * p.c.Hq + h * GQ), p.c.dtype, lane);
        const int n = t.len[b];
        const int32_t* table = t.table + (size_t)b * t.max_blocks;

        const int nit = (hi - lo - warp + QD_WARPS - 1) / QD_WARPS;  // this warp's tiles: lo + warp + QD_WARPS i
        auto block_of = [&](int x) {
            const int tile = lo + warp + QD_WARPS * x;
            return x < nit ? table[(tile * Q8_TOK) >> t.sh] : 0;
        };
        int win_cur = block_of(lane), win_nxt = block_of(QD_LANES + lane);
        const unsigned ring32 = smem_addr32(ring);
        const char* klane = static_cast<const char*>(p.c.k) + lane * 16;
        const char* vlane = static_cast<const char*>(p.c.v) + lane * 16;
        const float* slane = lane == 0 ? p.c.k_scale : p.c.v_scale;  // lanes 0 and 1 copy the scales
        unsigned stage_in = 0;
        unsigned bad = 0;  // staged tiles, by ring slot, whose block is out of range
        auto issue = [&](int x) {
            if (x < nit) {
                if ((x & (QD_LANES - 1)) == 0 && x > 0) {
                    win_cur = win_nxt;
                    win_nxt = block_of(x + QD_LANES + lane);
                }
                const unsigned sm = ring32 + stage_in * QG::SLOT;
                const int id = __shfl_sync(FULL, win_cur, x & (QD_LANES - 1));
                const int pos = (lo + warp + QD_WARPS * x) * Q8_TOK;
                bad &= ~(1u << stage_in);
                if ((unsigned)id < (unsigned)t.n_blocks) {
                    const unsigned unit = id * Hkv + h;
                    const size_t src = (size_t)((unit << t.sh) + (pos & (bs - 1))) * D;
                    if (pos + Q8_TOK <= n) {
                        copy_tile<D>(sm, klane + src, vlane + src, lane);
                    } else {
#pragma unroll
                        for (int y = 0; y < QG::TILE / 512; ++y) {
                            const int idx = y * 32 + lane, row = idx / QG::CH, c = idx % QG::CH;
                            const unsigned dst = sm + q8_swz<D>(row, c);
                            const int size = pos + row < n ? 16 : 0;
                            cp_async_16s(dst, klane + src + y * 512, size);
                            cp_async_16s(dst + QG::TILE, vlane + src + y * 512, size);
                        }
                    }
                    cp_async_4p(sm + QG::SCALES + lane * 64, slane + unit, lane < 2);
                } else {
                    bad |= 1u << stage_in;
                    if (lane == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
                }
            }
            stage_in = stage_in + 1 == STAGES ? 0 : stage_in + 1;
            cp_async_commit();
        };
#pragma unroll
        for (int x = 0; x < STAGES - 1; ++x) issue(x);
        st.set_q(raw_q, p.c.dtype, p.scale_log2, lane);
        st.reset();
        unsigned stage_out = 0;
        int left = n - (lo + warp) * Q8_TOK;  // tokens from this tile's first on
        for (int x = 0; x < nit; ++x) {
            __syncwarp();  // every lane is done reading the slot refilled next
            issue(x + STAGES - 1);
            cp_async_wait<STAGES - 1>();
            __syncwarp();  // what the other lanes copied is visible
            const unsigned mask = bad >> stage_out & 1u ? 0u : left >= Q8_TOK ? 0xffffu : 0xffffu >> (Q8_TOK - left);
            st.template tile<true, false>(ring32 + stage_out * QG::SLOT, mask, lane, [](int, float) {});
            left -= QD_WARPS * Q8_TOK;
            stage_out = stage_out + 1 == STAGES ? 0 : stage_out + 1;
        }
        cp_async_wait<0>();
        __syncwarp();
        // the warps' states through their rings' memory
        st.write(wm + warp * GQ, wl + warp * GQ, reinterpret_cast<float*>(ring), lane);
        __syncthreads();
        float* out = p.out + ((size_t)b * p.c.Hq + h * GQ) * D;
        for (int x = tid; x < GQ * D; x += QD_THREADS) {
            const int hh = x / D;
            float M = Q8_M_INIT;
#pragma unroll
            for (int w = 0; w < QD_WARPS; ++w) M = fmaxf(M, wm[w * GQ + hh]);
            float L = 0.f, A = 0.f;
#pragma unroll
            for (int w = 0; w < QD_WARPS; ++w) {
                const float f = exp2_approx(wm[w * GQ + hh] - M);
                L = fmaf(wl[w * GQ + hh], f, L);
                A = fmaf(reinterpret_cast<const float*>(smem + w * SM::WARP)[x], f, A);
            }
            if (np == 1) {
                out[x] = L == 0.f ? 0.f : A / L;  // no weight: every block of the unit was out of range
            } else {
                p.acc[(size_t)slot * GQ * D + x] = A;
                if (x % D == 0) {
                    p.m[slot * GQ + hh] = M;
                    p.l[slot * GQ + hh] = L;
                }
            }
        }
        if (np > 1) {
            const int unit = b * Hkv + h;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                s_last = atomicAdd(p.count + unit, 1) == np - 1;
                if (s_last) p.count[unit] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_partials<D, GQ>(p, c0, np, odd, out, smem, wm, tid);
            }
        }
        __syncthreads();  // the rings are free again
    }
}

template <int D, int GQ, int FMT>
static cudaError_t launch_dense_q8_t(const DenseQ8Params& p, cudaStream_t st) {
    static LaunchCache lc;
    auto kern = dense_q8_kernel<D, GQ, FMT>;
    const size_t smem = DenseQ8Smem<D, GQ>::FIXED + 2 * (size_t)p.c.t.B * 4;
    int per_sm = 0, sms = 0;
    cudaError_t e = prepare_launch(kern, lc, smem, QD_THREADS, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    if (sms <= 0 || per_sm <= 0) return cudaErrorInvalidConfiguration;
    const long long tiles = (long long)p.c.t.B * p.c.Hkv * p.c.t.max_blocks * (p.c.t.block / Q8_TOK);
    const int grid = (int)min((long long)min(sms * per_sm, QD_MAX_GRID), (tiles + QD_MIN_PIECE - 1) / QD_MIN_PIECE);
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
