// Decode attention over all tokens of a ragged batch in the paged 8-bit cache,
// sm_100a (ckv_dense_decode_q8): the dense comparator of ckv_decode.cu for this
// cache.  The tile arithmetic and what bounds it: ckv_q8_attend.cuh.
//
// Work split: every (request, KV head) is a unit of ceil(len/32) tiles; each
// block has one range of tiles, found by every block for itself from the lengths.
// Where pieces of about an equal share that do not cross units are no more than
// the blocks, each block has one piece, and so one start and one join; otherwise
// the units are laid end to end and cut into equal ranges, which may cross units.
// The second way costs a block that crosses a unit about 12 tiles' time (a new
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

constexpr int QD_TOK = 32;          // tokens of a tile
constexpr int QD_WARPS = 4;
constexpr int QD_THREADS = QD_WARPS * 32;
constexpr int QD_CTAS = 3;          // resident blocks per SM
constexpr int QD_MAX_GRID = 480;    // >= QD_CTAS * SMs
constexpr int QD_MIN_PIECE = 12;    // tiles: below it more partials cost more than they save
constexpr int QD_CROSS = 12;        // tiles: what crossing a unit costs a block

template <int D>
struct QdStages {
    static constexpr int v = D == 128 ? 2 : 4;  // 12 warps x 1 (3) tiles ahead: 96 KB in flight per SM
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
    static constexpr int WARP = QdStages<D>::v * Q8Geom<D, 2>::SLOT;  // a warp's ring, then its accumulators
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
    constexpr int SHARE = QD_THREADS / VECS > 0 ? QD_THREADS / VECS : 1;      // threads to a float4
    constexpr int PER = SHARE > 1 ? 1 : (VECS + QD_THREADS - 1) / QD_THREADS;  // float4 to a thread
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
    const int part = SHARE > 1 ? tid / VECS : 0, x0 = SHARE > 1 ? tid % VECS : tid;
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
            const int x = x0 + k * QD_THREADS, h = x / (D / 4);
            if (x >= VECS || part >= SHARE) continue;
            const float4* acc = reinterpret_cast<const float4*>(p.acc) + x;
            const float fo = s_old[h];
            A[k].x *= fo;
            A[k].y *= fo;
            A[k].z *= fo;
            A[k].w *= fo;
#pragma unroll 16
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
            const int x = x0 + k * QD_THREADS;
            if (x >= VECS) continue;
            const float L = s_sum[x / (D / 4)];
            const float inv = L == 0.f ? 0.f : 1.f / L;  // no weight: every block of the unit was out of range
            reinterpret_cast<float4*>(out)[x] = make_float4(A[k].x * inv, A[k].y * inv, A[k].z * inv, A[k].w * inv);
        }
    }
}

// 16 whole rows of K and of V, each 16 D contiguous bytes (k, v: lane's first 16 of
// them), to sm + SO.  Rows 4 apart (d = 128) differ in the swizzle by one bit.
template <int D, int SO>
__device__ __forceinline__ void copy_half(unsigned sm, const char* k, const char* v, int lane) {
    constexpr int V = Q8Geom<D, 2>::V + SO;
    const unsigned even = sm + q8_swz<D>(lane / Q8Geom<D, 2>::CH, lane % Q8Geom<D, 2>::CH);
    cp_async_16i<SO, 0>(even, k);
    cp_async_16i<V, 0>(even, v);
    if constexpr (D == 128) {
        const unsigned odd = sm + (q8_swz<D>(lane / 8, lane % 8) ^ 64);
        cp_async_16i<SO + 512, 512>(odd, k);
        cp_async_16i<SO + 1024, 1024>(even, k);
        cp_async_16i<SO + 1536, 1536>(odd, k);
        cp_async_16i<V + 512, 512>(odd, v);
        cp_async_16i<V + 1024, 1024>(even, v);
        cp_async_16i<V + 1536, 1536>(odd, v);
    } else {
        cp_async_16i<SO + 512, 512>(even, k);
        cp_async_16i<V + 512, 512>(even, v);
    }
}

template <int D, int GQ, int FMT>
__global__ void __launch_bounds__(QD_THREADS, QD_CTAS) dense_q8_kernel(const __grid_constant__ DenseQ8Params p) {
    using QG = Q8Geom<D, 2>;
    using SM = DenseQ8Smem<D, GQ>;
    constexpr int STAGES = QdStages<D>::v;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_last;
    const TableView& t = p.c.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = t.B, Hkv = p.c.Hkv, bs = t.block, grid = gridDim.x;
    unsigned char* ring = smem + warp * SM::WARP;
    float* wm = reinterpret_cast<float*>(smem + QD_WARPS * SM::WARP);  // [warps][GQ]
    float* wl = wm + QD_WARPS * GQ;
    int* s_nt = reinterpret_cast<int*>(smem + SM::FIXED);              // [B] tiles of a unit of request b
    pdl_wait();

    for (int b = tid; b < B; b += QD_THREADS) {
        const int n = t.len[b];
        const bool ok = n >= 0 && n <= (long long)t.max_blocks * bs;
        if (!ok && blockIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
        s_nt[b] = ok ? (n + QD_TOK - 1) / QD_TOK : 0;
    }
    __syncthreads();
    // from here every warp works for itself, 32 requests at a time
    auto ceil_div = [](int a, int b) { return (int)(((unsigned)a + b - 1) / (unsigned)b); };
    auto sum_over = [&](auto f) {
        int own = 0;
        for (int b = lane; b < B; b += 32) own += f(s_nt[b]);
        return __reduce_add_sync(FULL, own);
    };
    const int total = sum_over([](int nt) { return nt; }) * Hkv;
    if (total == 0) {
        for (int i = blockIdx.x * QD_THREADS + tid; i < B * p.c.Hq * D; i += grid * QD_THREADS) p.out[i] = 0.f;
        return;
    }
    const int share = ceil_div(total, grid);
    // pieces of at most `piece` tiles: 0 where the units are laid end to end instead
    const int per = max(share, QD_MIN_PIECE);
    const int most = per + max(QD_CROSS, share >> 4);
    int piece = per, items = 0;
    while (true) {
        items = sum_over([&](int nt) { return ceil_div(nt, piece); }) * Hkv;
        if (items <= grid) break;
        if (piece >= most || B * Hkv > 2 * grid) {
            piece = 0;
            break;
        }
        piece = min(piece + max(1, (most - per) >> 2), most);
    }
    // [start, end): this block's range, in pieces or in tiles
    const int start = piece ? (int)blockIdx.x : (int)min((long long)blockIdx.x * per, (long long)total);
    const int end = piece ? min(start + 1, items) : min(start + per, total);
    for (int b = blockIdx.x; b < B; b += grid)
        if (s_nt[b] == 0)  // nothing to attend to
            for (int i = tid; i < p.c.Hq * D; i += QD_THREADS) p.out[(size_t)b * p.c.Hq * D + i] = 0.f;

    Q8Warp<D, GQ, FMT, 2> st;
    for (int at = start; at < end;) {
        // the segment: tiles [lo, hi) of KV head h of request b, the unit shared by the blocks c0 .. c0 + np - 1
        int b = 0, pre = 0;  // pre: what comes before request b
        for (int k = 0;; k += 32) {
            const int x = k + lane < B ? s_nt[k + lane] : 0;
            int own = (piece ? ceil_div(x, piece) : x) * Hkv, inc = own;
#pragma unroll
            for (int y = 1; y < 32; y <<= 1) {
                const int z = __shfl_up_sync(FULL, inc, y);
                if (lane >= y) inc += z;
            }
            const int chunk = __shfl_sync(FULL, inc, 31);
            if (at < pre + chunk) {  // the first request that ends past `at`
                const int l = __ffs(__ballot_sync(FULL, at < pre + inc)) - 1;
                b = k + l;
                pre += __shfl_sync(FULL, inc - own, l);
                break;
            }
            pre += chunk;
        }
        const int nt = s_nt[b];
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
        const auto raw_q = Q8Warp<D, GQ, FMT, 2>::fetch_q(
            Q8Warp<D, GQ, FMT, 2>::q_row(p.q, p.c.dtype, (size_t)b * p.c.Hq + h * GQ), p.c.dtype, lane);
        const int n = t.len[b];
        const int32_t* table = t.table + (size_t)b * t.max_blocks;

        const int nit = (hi - lo - warp + QD_WARPS - 1) / QD_WARPS;  // this warp's tiles: lo + warp + QD_WARPS i
        // a window of 16 tiles: lane 2 i + j holds the block of half j of this warp's tile i
        auto block_of = [&](int x) {
            const int pos = (lo + warp + QD_WARPS * (x + (lane >> 1))) * QD_TOK + (lane & 1) * Q8_HALF;
            return x + (lane >> 1) < nit && pos < n ? table[pos >> t.sh] : 0;
        };
        int win_cur = block_of(0), win_nxt = block_of(16);
        const unsigned ring32 = smem_addr32(ring);
        const char* klane = static_cast<const char*>(p.c.k) + lane * 16;
        const char* vlane = static_cast<const char*>(p.c.v) + lane * 16;
        const float* slane = lane < 2 ? p.c.k_scale : p.c.v_scale;  // lanes 0..3 copy the halves' scales
        unsigned stage_in = 0;
        unsigned bad = 0;  // bit 2 s + j: the block of half j of the tile in ring slot s is out of range
        auto issue = [&](int x) {
            if (x < nit) {
                if ((x & 15) == 0 && x > 0) {
                    win_cur = win_nxt;
                    win_nxt = block_of(x + 16);
                }
                const unsigned sm = ring32 + stage_in * QG::SLOT;
                const int id0 = __shfl_sync(FULL, win_cur, 2 * (x & 15)), id1 = __shfl_sync(FULL, win_cur, 2 * (x & 15) + 1);
                const int pos = (lo + warp + QD_WARPS * x) * QD_TOK;
                const bool ok0 = (unsigned)id0 < (unsigned)t.n_blocks, ok1 = (unsigned)id1 < (unsigned)t.n_blocks;
                const unsigned unit0 = id0 * Hkv + h, unit1 = id1 * Hkv + h;
                const size_t src0 = (size_t)((unit0 << t.sh) + (pos & (bs - 1))) * D;
                const size_t src1 = (size_t)((unit1 << t.sh) + ((pos + Q8_HALF) & (bs - 1))) * D;
                if (pos + QD_TOK <= n && ok0 && ok1) {
                    copy_half<D, 0>(sm, klane + src0, vlane + src0, lane);
                    copy_half<D, QG::HALF>(sm, klane + src1, vlane + src1, lane);
                    bad &= ~(3u << 2 * stage_in);
                    cp_async_4p(sm + QG::SCALES + 8 * (lane & 1) + 4 * (lane >> 1), slane + (lane & 1 ? unit1 : unit0), lane < 4);
                } else {
                    // the end of the request, or a block out of range: zeros where there is nothing
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const bool ok = j ? ok1 : ok0;
                        const size_t src = ok ? (j ? src1 : src0) : 0;
                        const int rows = ok ? n - pos - j * Q8_HALF : 0;
#pragma unroll
                        for (int y = 0; y < QG::HALF / 512; ++y) {
                            const int idx = y * 32 + lane, row = idx / QG::CH, c = idx % QG::CH;
                            const unsigned dst = sm + j * QG::HALF + q8_swz<D>(row, c);
                            const int size = row < rows ? 16 : 0;
                            const size_t from = size ? src + y * 512 : 0;
                            cp_async_16s(dst, klane + from, size);
                            cp_async_16s(dst + QG::V, vlane + from, size);
                        }
                        if (lane < 2)
                            cp_async_4s(sm + QG::SCALES + 8 * j + 4 * lane,
                                        (lane ? p.c.v_scale : p.c.k_scale) + (rows > 0 ? (j ? unit1 : unit0) : 0),
                                        rows > 0 ? 4 : 0);
                    }
                    bad = (bad & ~(3u << 2 * stage_in)) | ((ok0 ? 0u : 1u) | (ok1 ? 0u : 2u)) << 2 * stage_in;
                    if (lane == 0 && !(ok0 && ok1)) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
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
        int left = n - (lo + warp) * QD_TOK;  // tokens from this tile's first on
        for (int x = 0; x < nit; ++x) {
            __syncwarp();  // every lane is done reading the slot refilled next
            issue(x + STAGES - 1);
            cp_async_wait<STAGES - 1>();
            __syncwarp();  // what the other lanes copied is visible
            unsigned mask = 0xffffffffu;
            if (left < QD_TOK) mask >>= QD_TOK - left;
            if (bad) mask &= ~((bad >> 2 * stage_out & 1u) * 0xffffu | (bad >> 2 * stage_out & 2u) * 0x7fff8000u);
            st.template tile<true, false>(ring32 + stage_out * QG::SLOT, mask, 0.f, lane, [](int, float) {});
            left -= QD_WARPS * QD_TOK;
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
    const size_t smem = DenseQ8Smem<D, GQ>::FIXED + (size_t)p.c.t.B * 4;
    int per_sm = 0, sms = 0;
    cudaError_t e = prepare_launch(kern, lc, smem, QD_THREADS, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    if (sms <= 0 || per_sm <= 0) return cudaErrorInvalidConfiguration;
    const long long tiles = (long long)p.c.t.B * p.c.Hkv * p.c.t.max_blocks * p.c.t.block / QD_TOK + (long long)p.c.t.B * p.c.Hkv;
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
