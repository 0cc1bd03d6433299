// The block-split attention over an 8-bit cache, sm_100a: all tokens of a ragged batch
// (LIST false; ckv_q8_dense.cu) or a selected list per graph unit (LIST true;
// ckv_q8_sparse.cu).  The tile arithmetic and what bounds it: ckv_q8_attend.cuh.
//
// Work split: a unit (a KV head of a request; a graph unit with its list) is
// ceil(tokens / TOK) tiles; each block has one range of tiles, found by every
// block for itself from the lengths.
// Where pieces of about an equal share that do not cross units are no more than
// the blocks, each block has one piece, and so one start and one join; otherwise
// the units are laid end to end and cut into equal ranges, which may cross units.
// The second way costs a block that crosses a unit about 12 tiles' time (a new
// query, an empty ring, a join), the first the difference between the longest
// piece and the share: the smaller loss decides (33 ragged requests 40.6 us, by ranges
// 50.6, one of 32K tokens 23.5 and 26.5; 8 requests of 128K tokens, whose pieces do not
// fit, 341, by pieces 355 with 342 beside it).
// (Finer pieces by ticket, for the SMs' 10 % difference in bandwidth, lost more by
// their starts: 8 requests of 128K tokens 357 against 350 us, 8 heads a group at 64K
// 249 against 200.)
//
// Inside a segment of a unit the warps take tiles in turn, each with its own ring of
// staged tiles and its own softmax state, joined in shared memory.  A unit that
// one block holds whole is finished there; otherwise the blocks write partials
// and the last one to arrive (a counter per unit, returned to zero) joins them in
// order: the result does not depend on which block that is, no block waits for
// another, and the whole call is one launch.
//
// A list entry's position goes through the request's block table, a window of 32
// entries ahead of the copies, and each row brings its own two scales.
//
// What bounds it: all tokens, HBM: 8 requests of 128K tokens, 8 heads of 128, in
// int8 332 to 367 us for 2.15 GB, 0.98 to 0.89 of the copy rate; 4 requests in e4m3
// 178 us, 0.92; d = 64 0.83; 8 query heads a KV head 0.90.  Short work has about 13 us
// on top of its bytes: the launch, the chain length - block - rows, the join (1
// request of 32K tokens 24 us, 33 ragged ones up to 9000 tokens 40 us).  Lists: 256 of
// 2052 tokens of 128K, one a query head: 50 us.  Their rows are scattered 128 bytes,
// of which HBM gives 4.4 to 4.7 TB/s (29 us for these); the rest is the start, the
// join and two scale loads a row.  8 lists of 2052 tokens: 11.5 us, of 8000: 17.2, one
// of 132: 7 us.
#pragma once

#include "ckv_q8_attend.cuh"

namespace ckv {

constexpr int QD_WARPS = 4;
constexpr int QD_THREADS = QD_WARPS * 32;
constexpr int QD_MAX_GRID = 640;    // >= resident blocks
constexpr int QD_WHOLE = 12;        // tiles: a unit up to this long stays whole
constexpr int QD_MIN_RANGE = 8;     // tiles: least range where units are laid end to end
constexpr int QD_CROSS = 12;        // tiles: what crossing a unit costs a block

// Least piece of a unit of nt tiles, for each warp equally many.  A unit's time is
// a piece's plus its join's, about a nt / np + b np for np pieces, so that the best
// piece grows about with the root of nt.  Few units, pieces of 4, 8, 16, 32 tiles:
// 16 tiles 10.3, 11.0, 12.8, 14.2 us; 32 tiles 8.9, 9.5, 10.5, 10.7; 128 tiles 13.0,
// 11.5, 13.1, 16.4; 313 tiles (8, 16, 32) 16.1, 15.3, 17.1; 1024 tiles 20.9, 18.2,
// 18.3; 4096 tiles 41.9, 34.1, 28.4; 500 tiles of lists (8, 16, 24) 19.3, 16.6, 17.8.
__device__ __forceinline__ int least_piece(int nt) {
    return QD_WARPS << (nt < 64 ? 0 : nt < 256 ? 1 : nt < 2048 ? 2 : 3);
}

// Rows in order: tiles of two halves, 12 warps an SM (64K tokens with 8 heads a group
// 182 us, d = 64 99 us; one half, 16 warps: 200 and 118).  Lists, which wait longer for
// scattered rows: one half, 16 warps (256 lists of 128K tokens 53 us; two halves 59).
template <int D, bool LIST>
struct QdShape {
    static constexpr int NH = LIST ? 1 : 2;
    static constexpr int TOK = NH * Q8_HALF;              // tokens of a tile
    static constexpr int CTAS = LIST ? 4 : 3;             // resident blocks per SM
    static constexpr int STAGES = LIST ? (D == 128 ? 3 : 5) : (D == 128 ? 2 : 4);
};

struct BlocksQ8Params {
    Q8View c;
    const void* q;
    float* out;
    float scale_log2;
    // LIST: U units, G per request
    int U, G, per_head, S, tok_cap;
    const int32_t* sel_tok;
    const int32_t* n_tok;
    float* lam;   // NBR: [U, tok_cap] graph logit of every entry, -inf where it is skipped
    int* count;   // [units], zero between calls
    float* m;     // partials: two slots a block
    float* l;
    float* acc;
};

template <int D, int GQ, bool LIST>
struct BlocksQ8Smem {
    static constexpr int WARP = QdShape<D, LIST>::STAGES * Q8Geom<D, QdShape<D, LIST>::NH>::SLOT;  // a warp's ring, then its accumulators
    static constexpr int FIXED = QD_WARPS * WARP + 2 * QD_WARPS * GQ * 4;
    static_assert(GQ * D * 4 <= WARP, "a warp's accumulators fit its ring");
    // the join of a unit's partials: JOIN rows at a time, with their references and sums
    static constexpr int FIT = (QD_WARPS * WARP - QD_THREADS * 16) / (GQ * D * 4 + 2 * GQ * 4);
    static constexpr int JOIN = FIT < 64 ? FIT / 4 * 4 : 64;
    static_assert(JOIN >= 8, "the join fits the rings");
};

// Joins the partials of a unit that blocks c0 .. c0 + np - 1 share into out.  A
// block's first segment has its even slot, its last (when that is another) the odd
// one: `odd` for block c0.  A chunk of rows at a time comes into the rings' memory
// by asynchronous copies, all in flight at once, with the references and sums
// (loads into registers, 16 at a time, took 2 us longer for 55 rows).
template <int D, int GQ, bool LIST>
__device__ __forceinline__ void join_partials(const BlocksQ8Params& p, int c0, int np, int odd, float* out,
                                              unsigned char* smem, float* s_head, int tid) {
    using SM = BlocksQ8Smem<D, GQ, LIST>;
    constexpr int VECS = GQ * D / 4;  // float4 of an output
    constexpr int SHARE = QD_THREADS / VECS > 0 ? QD_THREADS / VECS : 1;      // threads to a float4
    constexpr int PER = SHARE > 1 ? 1 : (VECS + QD_THREADS - 1) / QD_THREADS;  // float4 to a thread
    const int lane = tid & 31, warp = tid >> 5;
    float* s_f = reinterpret_cast<float*>(smem);  // [JOIN][GQ] references, then weights
    float* s_l = s_f + SM::JOIN * GQ;             // [JOIN][GQ] sums
    float4* s_part = reinterpret_cast<float4*>(s_l + SM::JOIN * GQ);
    float4* s_rows = s_part + QD_THREADS;         // [JOIN][VECS]
    float* s_m = s_head;                          // [GQ] running reference, then sum
    float* s_sum = s_head + GQ;
    __shared__ float s_old[GQ];                   // the old rows' factor
    if (tid < GQ) {
        s_m[tid] = Q8_M_INIT;
        s_sum[tid] = 0.f;
    }
    const int part = SHARE > 1 ? tid / VECS : 0, x0 = SHARE > 1 ? tid % VECS : tid;
    float4 A[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) A[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < np; i0 += SM::JOIN) {
        const int n = min(np - i0, SM::JOIN);
        auto slot_of = [&](int i) { return 2 * (c0 + i0 + i) + (i0 + i == 0 ? odd : 0); };
        __syncthreads();
        const float4* acc = reinterpret_cast<const float4*>(p.acc);
        for (int x = tid; x < n * VECS; x += QD_THREADS)
            cp_async_16i<0, 0>(smem_addr32(s_rows + x), acc + (size_t)slot_of(x / VECS) * VECS + x % VECS);
        cp_async_commit();
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
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int x = x0 + k * QD_THREADS, h = x / (D / 4);
            if (x >= VECS || part >= SHARE) continue;
            const float fo = s_old[h];
            A[k].x *= fo;
            A[k].y *= fo;
            A[k].z *= fo;
            A[k].w *= fo;
#pragma unroll 4
            for (int i = part; i < n; i += SHARE) {
                const float4 v = s_rows[i * VECS + x];
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

template <int D, int GQ, int FMT, bool LIST, bool NBR, bool QLO>
__global__ void __launch_bounds__(QD_THREADS, QdShape<D, LIST>::CTAS) blocks_q8_kernel(const __grid_constant__ BlocksQ8Params p) {
    using SH = QdShape<D, LIST>;
    using QG = Q8Geom<D, SH::NH>;
    using W = Q8Warp<D, GQ, FMT, SH::NH, QLO>;
    using SM = BlocksQ8Smem<D, GQ, LIST>;
    constexpr int STAGES = SH::STAGES, TOK = SH::TOK;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_last, s_red[2][QD_WARPS], s_at[2];
    const TableView& t = p.c.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // groups of units of one length: requests with Hkv units each, or single lists
    const int B = LIST ? p.U : t.B, H = LIST ? 1 : p.c.Hkv;
    const int Hkv = p.c.Hkv, bs = t.block, grid = gridDim.x;
    unsigned char* ring = smem + warp * SM::WARP;
    float* wm = reinterpret_cast<float*>(smem + QD_WARPS * SM::WARP);  // [warps][GQ]
    float* wl = wm + QD_WARPS * GQ;
    int* s_n = reinterpret_cast<int*>(smem + SM::FIXED);               // [B] tokens of a unit of group b
    pdl_wait();

    // thread i has the groups [b0, b1)
    const int seg = (B + QD_THREADS - 1) / QD_THREADS;
    const int b0 = min(B, tid * seg), b1 = min(B, b0 + seg);
    for (int b = b0; b < b1; ++b) {
        int n;
        if constexpr (LIST) {
            n = max(0, min(p.n_tok[b], p.tok_cap));
        } else {
            n = t.len[b];
            if (n < 0 || n > (long long)t.max_blocks * bs) {
                if (blockIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
                n = 0;
            }
        }
        s_n[b] = n;
    }
    auto tiles_of = [&](int b) { return (int)(((unsigned)s_n[b] + TOK - 1) / TOK); };
    auto ceil_div = [](int a, int b) { return (int)(((unsigned)a + b - 1) / (unsigned)b); };
    auto pieces = [&](int nt, int piece) {
        return nt <= QD_WHOLE ? min(nt, 1) : ceil_div(nt, max(piece, least_piece(nt)));
    };
    // the block's sum of f over the groups' tiles; one barrier (two buffers: a thread
    // that runs ahead to the next sum does not touch what others still read)
    int turn = 0;
    auto sum_over = [&](auto f) {
        int own = 0;
        for (int b = b0; b < b1; ++b) own += f(tiles_of(b));
        own = __reduce_add_sync(FULL, own);
        if (lane == 0) s_red[turn][warp] = own;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < QD_WARPS; ++w) all += s_red[turn][w];
        turn ^= 1;
        return all;
    };
    const int total = sum_over([](int nt) { return nt; }) * H;
    if (total == 0) {
        for (int i = blockIdx.x * QD_THREADS + tid; i < t.B * p.c.Hq * D; i += grid * QD_THREADS) p.out[i] = 0.f;
        return;
    }
    const int share = ceil_div(total, grid);
    // pieces of at most `piece` tiles: 0 where the units are laid end to end instead
    const int per = max(share, QD_MIN_RANGE);
    const int most = share + max(QD_CROSS, share >> 4);
    int piece = share, items = 0;
    while (true) {
        items = sum_over([&](int nt) { return pieces(nt, piece); }) * H;
        if (items <= grid) break;
        if (piece >= most || B * H > 2 * grid) {
            piece = 0;
            break;
        }
        piece = min(piece + max(1, (most - share) >> 2), most);
    }
    // [start, end): this block's range, in pieces or in tiles
    const int start = piece ? (int)blockIdx.x : (int)min((long long)blockIdx.x * per, (long long)total);
    const int end = piece ? min(start + 1, items) : min(start + per, total);
    // The query rows of a unit: in LIST mode group b is graph unit b, and `kvh` its KV head
    auto first_row = [&](int b, int h, int& kvh) {
        if constexpr (LIST) {
            const int s = b / p.G, g = b - s * p.G;
            kvh = p.per_head ? g / (p.c.Hq / Hkv) : g;
            return (size_t)s * p.c.Hq + g * GQ;
        } else {
            kvh = h;
            return (size_t)b * p.c.Hq + h * GQ;
        }
    };
    for (int b = blockIdx.x; b < B; b += grid)
        if (s_n[b] == 0) {  // nothing to attend to
            int kvh;
            float* o = p.out + first_row(b, 0, kvh) * D;
            for (int i = tid; i < H * GQ * D; i += QD_THREADS) o[i] = 0.f;
        }

    if (start >= end) return;
    // the group of `start`, and what comes before it: the thread whose groups hold it finds it
    {
        auto weight = [&](int b) { return (piece ? pieces(tiles_of(b), piece) : tiles_of(b)) * H; };
        int own = 0;
        for (int b = b0; b < b1; ++b) own += weight(b);
        int inc = own;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const int z = __shfl_up_sync(FULL, inc, y);
            if (lane >= y) inc += z;
        }
        if (lane == 31) s_red[turn][warp] = inc;
        __syncthreads();
        int pre = inc - own;
#pragma unroll
        for (int w = 0; w < QD_WARPS; ++w) pre += w < warp ? s_red[turn][w] : 0;
        if (pre <= start && start < pre + own) {
            int b = b0;
            while (start >= pre + weight(b)) pre += weight(b++);
            s_at[0] = b;
            s_at[1] = pre;
        }
        __syncthreads();
    }
    int b = s_at[0], pre = s_at[1];  // the group, and what comes before it

    W st;
    for (int at = start; at < end;) {
        // the segment: tiles [lo, hi) of unit h of group b, the unit shared by the blocks c0 .. c0 + np - 1
        while (at >= pre + tiles_of(b) * H && !piece) pre += tiles_of(b++) * H;
        const int n = s_n[b], nt = tiles_of(b);
        int h, lo, hi, c0, np, odd = 0, slot = 2 * blockIdx.x;
        if (piece) {
            np = pieces(nt, piece);
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
        int kvh;
        const size_t row0 = first_row(b, h, kvh);
        const auto raw_q = W::fetch_q(W::q_row(p.q, p.c.dtype, row0), p.c.dtype, lane);
        const int seq = LIST ? b / p.G : b;
        const int32_t* table = t.table + (size_t)seq * t.max_blocks;

        const int nit = (hi - lo - warp + QD_WARPS - 1) / QD_WARPS;  // this warp's tiles: lo + warp + QD_WARPS i
        const unsigned ring32 = smem_addr32(ring);
        unsigned stage_in = 0;
        // a window of 16 tiles: lane 2 i + j holds the block of half j of this warp's tile i
        auto rows_block = [&](int x) {
            const int pos = (lo + warp + QD_WARPS * (x + (lane >> 1))) * TOK + (lane & 1) * Q8_HALF;
            return x + (lane >> 1) < nit && pos < n ? table[pos >> t.sh] : 0;
        };
        int win_cur = 0, win_nxt = 0;
        if constexpr (!LIST) {
            win_cur = rows_block(0);
            win_nxt = rows_block(16);
        }
        const char* klane = static_cast<const char*>(p.c.k) + lane * 16;
        const char* vlane = static_cast<const char*>(p.c.v) + lane * 16;
        const float* slane = lane < 2 ? p.c.k_scale : p.c.v_scale;  // lanes 0..3 copy the halves' scales
        unsigned bad = 0;  // bit 2 s + j: the block of half j of the tile in ring slot s is out of range
        auto issue_rows = [&](int x) {
            if (x < nit) {
                if ((x & 15) == 0 && x > 0) {
                    win_cur = win_nxt;
                    win_nxt = rows_block(x + 16);
                }
                const unsigned sm = ring32 + stage_in * QG::SLOT;
                const int id0 = __shfl_sync(FULL, win_cur, 2 * (x & 15)), id1 = __shfl_sync(FULL, win_cur, 2 * (x & 15) + 1);
                const int pos = (lo + warp + QD_WARPS * x) * TOK;
                const bool ok0 = (unsigned)id0 < (unsigned)t.n_blocks, ok1 = (unsigned)id1 < (unsigned)t.n_blocks;
                const unsigned unit0 = id0 * Hkv + h, unit1 = id1 * Hkv + h;
                const size_t src0 = (size_t)((unit0 << t.sh) + (pos & (bs - 1))) * D;
                const size_t src1 = (size_t)((unit1 << t.sh) + ((pos + Q8_HALF) & (bs - 1))) * D;
                if (pos + TOK <= n && ok0 && ok1) {
                    copy_half<D, 0>(sm, klane + src0, vlane + src0, lane);
                    copy_half<D, Q8Geom<D, 2>::HALF>(sm, klane + src1, vlane + src1, lane);
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
        // Two tiles' entries of this warp are a window, one entry a lane.  The copies of
        // a window need its positions and their blocks: loaded two and one windows ahead,
        // and only looked at by the copies themselves, so that no load is waited for
        // where it is issued.
        int len = LIST ? t.len[seq] : 0;
        if (LIST && len > (long long)t.max_blocks << t.sh) len = 0;  // a bad length: every entry is out of range
        const int32_t* toks = LIST ? p.sel_tok + (size_t)b * p.tok_cap : nullptr;
        auto entry = [&](int w) {  // of this lane in window w
            return (lo + warp + QD_WARPS * (2 * w + (lane >> 4))) * TOK + (lane & 15);
        };
        auto position = [&](int w) { return 2 * w + (lane >> 4) < nit && entry(w) < n ? toks[entry(w)] : -1; };
        auto inside = [&](int pos) { return pos >= 0 && pos < len; };
        auto list_block = [&](int pos) { return inside(pos) ? table[pos >> t.sh] : -1; };
        // every list starts with the sinks, also that of a request too short to hold them
        auto missing_sink = [&](int e, int pos) {
            const int held = t.len[seq];
            return e < p.S && pos == e && held >= 0 && held <= e;
        };
        int pos0 = 0, pos1 = 0, id0 = 0, row_cur = -1;  // row_cur: the entry's row of the pool; -1: not attended
        // the tiles' scales (lanes 0..15 K's, 16..31 V's) and masks, newest first
        float scales[STAGES];
        unsigned masks[STAGES];
        const float* lscale = lane < 16 ? p.c.k_scale : p.c.v_scale;
        if constexpr (LIST) {
            pos0 = position(0);
            pos1 = position(1);
            id0 = list_block(pos0);
        }
        auto issue_list = [&](int x) {
#pragma unroll
            for (int k = STAGES - 1; k > 0; --k) {
                scales[k] = scales[k - 1];
                masks[k] = masks[k - 1];
            }
            if (x < nit) {
                if ((x & 1) == 0) {
                    row_cur = -1;
                    if (inside(pos0) && (unsigned)id0 < (unsigned)t.n_blocks)
                        row_cur = ((id0 * Hkv + kvh) << t.sh) + (pos0 & (bs - 1));
                    else if (x + (lane >> 4) < nit && entry(x >> 1) < n && !missing_sink(entry(x >> 1), pos0))
                        atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
                    pos0 = pos1;
                    id0 = list_block(pos0);
                    pos1 = position((x >> 1) + 2);
                }
                const unsigned sm = ring32 + stage_in * QG::SLOT;
                const int base = (x & 1) << 4;
                const int mine = __shfl_sync(FULL, row_cur, base + (lane & 15));
                scales[0] = mine >= 0 ? lscale[mine >> t.sh] : 0.f;
                masks[0] = __ballot_sync(FULL, mine >= 0) & 0xffffu;
#pragma unroll
                for (int y = 0; y < QG::HALF / 512; ++y) {
                    const int idx = y * 32 + lane, r = idx / QG::CH, c = idx % QG::CH;
                    const int row = __shfl_sync(FULL, row_cur, base + r);
                    const int size = row >= 0 ? 16 : 0;
                    const size_t src = (size_t)max(row, 0) * D + c * 16;
                    const unsigned dst = sm + q8_swz<D>(r, c);
                    cp_async_16s(dst, static_cast<const char*>(p.c.k) + src, size);
                    cp_async_16s(dst + QG::V, static_cast<const char*>(p.c.v) + src, size);
                }
            }
            stage_in = stage_in + 1 == STAGES ? 0 : stage_in + 1;
            cp_async_commit();
        };
        auto issue = [&](int x) {
            if constexpr (LIST) issue_list(x);
            else issue_rows(x);
        };
#pragma unroll
        for (int x = 0; x < STAGES - 1; ++x) issue(x);
        st.set_q(raw_q, p.c.dtype, p.scale_log2, lane);
        st.reset();
        unsigned stage_out = 0;
        int left = n - (lo + warp) * TOK;  // tokens from this tile's first on
        for (int x = 0; x < nit; ++x) {
            __syncwarp();  // every lane is done reading the slot refilled next
            issue(x + STAGES - 1);
            cp_async_wait<STAGES - 1>();
            __syncwarp();  // what the other lanes copied is visible
            unsigned mask;
            if constexpr (LIST) {
                mask = masks[STAGES - 1];
            } else {
                mask = 0xffffffffu;
                if (left < TOK) mask >>= TOK - left;
                if (bad) mask &= ~((bad >> 2 * stage_out & 1u) * 0xffffu | (bad >> 2 * stage_out & 2u) * 0x7fff8000u);
                left -= QD_WARPS * TOK;
            }
            [[maybe_unused]] const int entry0 = (lo + warp + QD_WARPS * x) * TOK;  // the tile's first list entry
            [[maybe_unused]] float* lamu = NBR ? p.lam + (size_t)b * p.tok_cap + entry0 : nullptr;
            if constexpr (NBR) {
                // a tile of skipped entries has no logits of its own to store
                if (mask == 0u && lane < TOK && entry0 + lane < n) lamu[lane] = -INFINITY;
            }
            st.template tile<!LIST, NBR>(ring32 + stage_out * QG::SLOT, mask, LIST ? scales[STAGES - 1] : 0.f, lane,
                                         [&](int k, float x) {
                                             if (entry0 + k < n) lamu[k] = x;
                                         });
            stage_out = stage_out + 1 == STAGES ? 0 : stage_out + 1;
        }
        cp_async_wait<0>();
        __syncwarp();
        // the warps' states through their rings' memory
        st.write(wm + warp * GQ, wl + warp * GQ, reinterpret_cast<float*>(ring), lane);
        __syncthreads();
        float* out = p.out + row0 * D;
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
            const int unit = b * H + h;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                s_last = atomicAdd(p.count + unit, 1) == np - 1;
                if (s_last) p.count[unit] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_partials<D, GQ, LIST>(p, c0, np, odd, out, smem, wm, tid);
            }
        }
        __syncthreads();  // the rings are free again
    }
}

// Resident blocks, but no more than there can be pieces (`most`).
template <int D, int GQ, int FMT, bool LIST, bool NBR, bool QLO>
static cudaError_t launch_blocks_q8_q(const BlocksQ8Params& p, long long most, cudaStream_t st) {
    static LaunchCache lc;
    auto kern = blocks_q8_kernel<D, GQ, FMT, LIST, NBR, QLO>;
    const size_t smem = BlocksQ8Smem<D, GQ, LIST>::FIXED + (size_t)(LIST ? p.U : p.c.t.B) * 4;
    int per_sm = 0, sms = 0;
    cudaError_t e = prepare_launch(kern, lc, smem, QD_THREADS, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    if (sms <= 0 || per_sm <= 0) return cudaErrorInvalidConfiguration;
    const int grid = (int)min((long long)min(sms * per_sm, QD_MAX_GRID), most);
    return launch_pdl(KK_ATTENTION, kern, dim3(grid), dim3(QD_THREADS), smem, st, p);
}

template <int D, int GQ, int FMT, bool LIST, bool NBR = false>
static cudaError_t launch_blocks_q8_t(const BlocksQ8Params& p, long long most, cudaStream_t st) {
    if constexpr (GQ == 8) {  // 33 ragged requests 40 us, with lo parts 44; 8 of 64K tokens 182, with them 189
        if (p.c.dtype == CKV_DTYPE_BF16) return launch_blocks_q8_q<D, GQ, FMT, LIST, NBR, false>(p, most, st);
    }
    return launch_blocks_q8_q<D, GQ, FMT, LIST, NBR, true>(p, most, st);
}

// The workspace's parts after its head: the units' counters, the partials, then the
// lists' graph logits.
inline void carve_blocks_ws(BlocksQ8Params& p, void* ws, int gq, int d) {
    char* w = static_cast<char*>(ws) + WS_RESERVED;
    p.count = reinterpret_cast<int*>(w);
    w += Q8_COUNTER_BYTES;
    p.m = reinterpret_cast<float*>(w);
    w += align256((size_t)2 * QD_MAX_GRID * gq * 4);
    p.l = reinterpret_cast<float*>(w);
    w += align256((size_t)2 * QD_MAX_GRID * gq * 4);
    p.acc = reinterpret_cast<float*>(w);
    w += align256((size_t)2 * QD_MAX_GRID * gq * d * 4);
    p.lam = reinterpret_cast<float*>(w);
}

}  // namespace ckv
