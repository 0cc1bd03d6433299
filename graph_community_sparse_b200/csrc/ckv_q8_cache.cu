// The paged 8-bit cache's bookkeeping and rows, sm_100a: block tables and slot
// maps from request lengths (ckv_plan_blocks), new rows quantised into their
// blocks (ckv_quant_append), rows read back (ckv_q8_read).  CommunityKV keeps the
// cache whole (rit.work summary, section "A graph of tokens replaces
// re-clustering", paragraph 5); this is that cache in 8 bits.
#include "ckv_q8.cuh"

namespace ckv {

// ---------------------------------------------------------------------------
// block-wide exclusive scan of one 64-bit integer per thread
// ---------------------------------------------------------------------------
__device__ __forceinline__ long long block_exclusive_scan64(long long x, long long* s_warp, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(FULL, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const long long w = lane < nw ? s_warp[lane] : 0;
        long long wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL, wi, o);
            if (lane >= o) wi += y;
        }
        if (lane < nw) s_warp[lane] = wi - w;
        if (lane == 31) s_warp[32] = wi;
    }
    __syncthreads();
    const long long r = s_warp[warp] + inc - x;
    *total = s_warp[32];
    __syncthreads();
    return r;
}

// Largest i in [0, n) with a[i] <= x, given a[0] <= x (a ascending).
__device__ __forceinline__ int last_le(const int* a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// plan.  Latency-bound: a few words per request and per block moved, 4 bytes
// per row of the slot map.  Every block of one cluster works the whole plan
// out for itself from len and add (two scans over the requests, kept in shared
// memory), so nothing has to be handed on between blocks; the cluster then
// shares the writes.  A cluster barrier separates what is read from the state
// from what is written to it, and the blocks given back from those taken.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 512;
constexpr int PLAN_CLUSTER = 8;

struct PlanParams {
    TableView t;
    PlanView p;
    const int32_t* add;
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const __grid_constant__ PlanParams q) {
    extern __shared__ int s_plan[];
    __shared__ long long s_warp[33];
    const TableView& t = q.t;
    const int B = t.B, bs = t.block, sh = t.sh, W = t.max_blocks;
    int* s_n1 = s_plan;             // [B] tokens after the drops
    int* s_n2 = s_n1 + B;           // [B] tokens after the growth
    int* s_gone = s_n2 + B;         // [B + 1] blocks given back before request b
    int* s_need = s_gone + B + 1;   // [B + 1] blocks taken before request b
    int* s_start = s_need + B + 1;  // [B + 1] first row of request b
    pdl_wait();
    const int tid = threadIdx.x;
    const int gthreads = gridDim.x * PLAN_THREADS, gtid = blockIdx.x * PLAN_THREADS + tid;
    const int n_free = max(0, min(*t.n_free, t.n_blocks));
    const long long cap = (long long)W << sh;
    auto blocks = [&](int n) { return (int)(((long long)n + bs - 1) >> sh); };

    // drops, and the rows asked for.  Thread i handles requests [b0, b1).
    const int seg = (B + PLAN_THREADS - 1) / PLAN_THREADS;
    const int b0 = min(B, tid * seg), b1 = min(B, b0 + seg);
    long long gone = 0, up = 0;
    for (int b = b0; b < b1; ++b) {
        const int n0 = t.len[b], a = q.add[b];
        const bool bad = n0 < 0 || n0 > cap;
        if (bad && blockIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
        const int n1 = bad ? 0 : a < 0 ? (int)max(0ll, (long long)n0 + a) : n0;
        s_n1[b] = n1;
        s_gone[b] = bad ? 0 : blocks(n0) - blocks(n1);
        gone += s_gone[b];
        up += max(a, 0);
    }
    long long total_up, total_gone, total_need;
    long long run_up = block_exclusive_scan64(up, s_warp, &total_up);
    long long run_gone = block_exclusive_scan64(gone, s_warp, &total_gone);
    const int freed = (int)min(total_gone, (long long)t.n_blocks - n_free);  // less only when the state is corrupt
    const int avail = n_free + freed;

    // growth that fits the table and the slot map, and the blocks it needs
    long long need = 0;
    for (int b = b0; b < b1; ++b) {
        const int a = max(q.add[b], 0), n0 = t.len[b];
        const bool bad = n0 < 0 || n0 > cap;
        s_start[b] = (int)min(run_up, 0x7fffffffll);
        const int g = s_gone[b];
        s_gone[b] = (int)min(run_gone, 0x7fffffffll);
        run_up += a;
        run_gone += g;
        const bool fits = !bad && (long long)s_n1[b] + a <= cap && run_up <= q.p.n_rows;
        s_n2[b] = fits ? s_n1[b] + a : -1;
        const int x = fits ? blocks(s_n2[b]) - blocks(s_n1[b]) : 0;
        s_need[b] = x;
        need += x;
    }
    long long run_need = block_exclusive_scan64(need, s_warp, &total_need);
    for (int b = b0; b < b1; ++b) {
        const int x = s_need[b];
        s_need[b] = (int)min(run_need, (long long)avail);
        run_need += x;
        if (s_n2[b] >= 0 && x > 0 && run_need > avail) s_n2[b] = -1;
        if (s_n2[b] < 0) {
            if (blockIdx.x == 0 && q.add[b] > 0) atomicOr(t.dev_err, CKV_DEVERR_PLAN);
            s_n2[b] = s_n1[b];
        }
    }
    if (tid == 0) {
        s_start[B] = (int)min(total_up, 0x7fffffffll);
        s_gone[B] = freed;
        s_need[B] = (int)min(total_need, (long long)avail);
    }
    __syncthreads();

    // blocks given back: the k-th of them at free_list[avail - 1 - k]
    for (int k = gtid; k < freed; k += gthreads) {
        const int b = last_le(s_gone, B + 1, k);
        const size_t at = (size_t)b * W + blocks(s_n1[b]) + (k - s_gone[b]);
        t.free_list[avail - 1 - k] = t.table[at];
        t.table[at] = -1;
    }
    // everybody has read len, add and n_free and given blocks back
    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();

    // blocks taken: the k-th is free_list[avail - 1 - k].  A refused request's
    // range of k is empty or belongs to nobody (all needs after the first
    // refusal for want of blocks are refused).
    const int taken = s_need[B];
    for (int k = gtid; k < taken; k += gthreads) {
        const int b = last_le(s_need, B + 1, k);
        const int j = blocks(s_n1[b]) + (k - s_need[b]);
        if (j < blocks(s_n2[b])) t.table[(size_t)b * W + j] = __ldcg(t.free_list + avail - 1 - k);
    }
    // the slot of every row: the block from the table where the request held
    // it already, else from the free list (the table entry may not be there yet)
    const int rows = q.p.n_rows, rows_in = s_start[B];
    for (int r = gtid; r < rows; r += gthreads) {
        int slot = -1;
        if (r < rows_in) {
            const int b = last_le(s_start, B + 1, r);
            const int n1 = s_n1[b], pos = n1 + (r - s_start[b]);
            if (pos < s_n2[b]) {
                const int j = pos >> sh, held = blocks(n1);
                const int id = j < held ? __ldcg(t.table + (size_t)b * W + j)
                                        : __ldcg(t.free_list + avail - 1 - (s_need[b] + j - held));
                slot = (int)((unsigned)id << sh) | (pos & (bs - 1));
                if ((unsigned)id >= (unsigned)t.n_blocks) {
                    atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
                    slot = -1;
                }
            }
        }
        q.p.slot[r] = slot;
    }
    if (blockIdx.x != 0) return;
    int took = 0;
    for (int b = b0; b < b1; ++b) {
        const int n0 = t.len[b];
        q.p.start[b] = s_start[b];
        const bool bad = n0 < 0 || n0 > cap;
        q.p.granted[b] = bad ? 0 : s_n2[b] - n0;
        if (!bad) {
            t.len[b] = s_n2[b];
            took += blocks(s_n2[b]) - blocks(s_n1[b]);
        }
    }
    long long total_took;
    block_exclusive_scan64(took, s_warp, &total_took);
    if (tid == 0) {
        q.p.start[B] = s_start[B];
        *t.n_free = avail - (int)total_took;
    }
}

cudaError_t launch_plan_blocks(const TableView& t, const int32_t* add, const PlanView& p, cudaStream_t st) {
    static LaunchCache lc;
    const PlanParams q{t, p, add};
    const size_t smem = (5 * (size_t)t.B + 3) * 4;
    cudaError_t e = prepare_launch(plan_kernel, lc, smem, PLAN_THREADS, nullptr, nullptr);
    if (e != cudaSuccess) return e;
    // one block until its threads write several slots each, then the cluster
    const int ctas = p.n_rows > 4 * PLAN_THREADS ? PLAN_CLUSTER : 1;
    const bool timed = timing_enabled();
    if (timed && (e = timing_mark(KK_UPDATE, true, st)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(PLAN_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, plan_kernel, q);
    if (timed && e == cudaSuccess) e = timing_mark(KK_UPDATE, false, st);
    return e;
}

// ---------------------------------------------------------------------------
// append.  One pass over the new rows, bound by their bytes: an item is one
// block's new rows of one head, K or V, kept in registers between the
// largest-magnitude reduction and the codes.  Items of the ragged batch are
// laid end to end (a scan over the requests in every block), so long and short
// requests share the grid evenly.
// ---------------------------------------------------------------------------
constexpr int APP_THREADS = 256;

struct AppendParams {
    Q8View c;
    PlanView p;
    RowsView r;
};

template <typename T>
__device__ __forceinline__ void vec16_values(const uint4& w, float (&x)[16 / ElemBytes<T>::v]) {
    if constexpr (ElemBytes<T>::v == 2) {
        x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
        x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
    } else {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
}

template <typename T, int D, int BS, int FMT>
__global__ void __launch_bounds__(APP_THREADS) append_kernel(const __grid_constant__ AppendParams q) {
    extern __shared__ int s_items[];  // [B + 1] touched blocks before request b
    __shared__ int s_warp[33];
    __shared__ unsigned s_max[APP_THREADS / 32];
    constexpr int V = 16 / ElemBytes<T>::v;           // values of a 16-byte load
    constexpr int TPR = D / V;                        // threads per row
    constexpr int RPP = APP_THREADS / TPR;            // rows per pass
    constexpr int NP = BS > RPP ? BS / RPP : 1;       // passes
    const TableView& t = q.c.t;
    const int B = t.B, Hkv = q.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();

    const int seg = (B + APP_THREADS - 1) / APP_THREADS;
    const int b0 = min(B, tid * seg), b1 = min(B, b0 + seg);
    int own = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = t.len[b], a = q.p.granted[b];
        int x = 0;
        if (a > 0) {
            const bool ok = n >= a && (long long)n <= (long long)t.max_blocks * BS &&
                            (q.r.T_rows ? a <= q.r.T_rows
                                        : q.p.start[b] >= 0 && (long long)q.p.start[b] + a <= q.p.n_rows);
            if (ok) x = (n - 1) / BS - (n - a) / BS + 1;
            else if (blockIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
        }
        s_items[b] = x;
        own += x;
    }
    int total;
    int run = block_exclusive_scan(own, s_warp, &total);
    for (int b = b0; b < b1; ++b) {
        const int x = s_items[b];
        s_items[b] = run;
        run += x;
    }
    if (tid == 0) s_items[B] = total;
    __syncthreads();

    const int r0 = tid / TPR, part = tid % TPR;
    const long long items = (long long)total * Hkv * 2;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int is_v = (int)(it & 1);
        const int h = (int)((it >> 1) % Hkv), blk_no = (int)((it >> 1) / Hkv);
        int b = 0;
        {
            int hi = B;
            while (hi - b > 1) {
                const int mid = (b + hi) >> 1;
                if (s_items[mid] <= blk_no) b = mid;
                else hi = mid;
            }
        }
        const int n = t.len[b], a = q.p.granted[b], start = q.p.start[b];
        const int n_old = n - a;
        const int j = n_old / BS + (blk_no - s_items[b]);
        const int lo = max(n_old - j * BS, 0), hi = min(n - j * BS, BS);  // new rows of the block: [lo, hi)
        const int first = j * BS + lo - n_old;                            // the first one's index among the request's
        const int slot = q.p.slot[start + first];
        const int id = slot / BS;
        if (slot < 0 || id >= t.n_blocks || slot % BS != lo) {  // uniform over the block
            if (tid == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
            continue;
        }
        const T* src = static_cast<const T*>(is_v ? q.r.v : q.r.k) + h * q.r.sh + part * V +
                       (q.r.T_rows ? b * q.r.sb + first * q.r.st : (int64_t)(start + first) * q.r.st);
        uint4 w[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int r = p * RPP + r0;
            w[p] = make_uint4(0, 0, 0, 0);
            if (r >= lo && r < hi) w[p] = *reinterpret_cast<const uint4*>(src + (int64_t)(r - lo) * q.r.st);
        }
        float* scale = (is_v ? q.c.v_scale : q.c.k_scale) + (size_t)id * Hkv + h;
        const float s_old = lo > 0 ? *scale : 0.f;
        unsigned amax = 0;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            float x[V];
            vec16_values<T>(w[p], x);
#pragma unroll
            for (int i = 0; i < V; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
        }
        amax = __reduce_max_sync(FULL, amax);
        if (lane == 0) s_max[warp] = amax;
        __syncthreads();
        amax = __reduce_max_sync(FULL, s_max[lane % (APP_THREADS / 32)]);
        __syncthreads();  // s_max is free for the next item; every thread has the old scale
        float s = q8c_scale<FMT>(amax);
        if (lo > 0 && !(s_old <= s)) s = s_old != s_old || s_old > s ? s_old : s;  // a NaN on either side stays
        const float inv = __fdiv_rn(1.f, s);
        unsigned char* dst = static_cast<unsigned char*>(is_v ? q.c.v : q.c.k) +
                             ((size_t)id * Hkv + h) * (BS * D) + part * V;
        if (lo > 0 && s != s_old) {
            // the block's older codes move to the larger scale
            const float f = __fmul_rn(s_old, inv);
            for (int r = r0; r < lo; r += RPP) {
                unsigned* c = reinterpret_cast<unsigned*>(dst + r * D);
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    float x[4];
                    q8c_values<FMT>(c[i], x);
                    c[i] = q8c_codes<FMT>(x[0], x[1], x[2], x[3], f);
                }
            }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int r = p * RPP + r0;
            if (r >= lo && r < hi) {
                float x[V];
                vec16_values<T>(w[p], x);
                unsigned c[V / 4];
#pragma unroll
                for (int i = 0; i < V / 4; ++i)
                    c[i] = q8c_codes<FMT>(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], inv);
                if constexpr (V == 8) *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<unsigned*>(dst + r * D) = c[0];
            }
        }
        if (tid == 0) *scale = s;
    }
}

template <typename T, int D, int BS, int FMT>
cudaError_t launch_append_t(const AppendParams& q, cudaStream_t st) {
    static LaunchCache lc;
    auto kern = append_kernel<T, D, BS, FMT>;
    const size_t smem = ((size_t)q.c.t.B + 1) * 4;
    int per_sm = 0, sms = 0;
    cudaError_t e = prepare_launch(kern, lc, smem, APP_THREADS, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    // a request touches at most its rows / BS + 2 blocks (the slot map bounds the rows)
    const long long bound = ((long long)q.p.n_rows / BS + 2ll * q.c.t.B) * q.c.Hkv * 2;
    const int grid = (int)min((long long)sms * per_sm, bound);
    return launch_pdl(KK_UPDATE, kern, dim3(grid), dim3(APP_THREADS), smem, st, q);
}

cudaError_t launch_quant_append(const Q8View& c, const PlanView& p, const RowsView& r, cudaStream_t st) {
    const AppendParams q{c, p, r};
#define CKV_APP4(TT, DD, BB)                                                                       \
    if (c.d == DD && c.t.block == BB)                                                              \
        return c.format == Q8_I8 ? launch_append_t<TT, DD, BB, Q8_I8>(q, st) : launch_append_t<TT, DD, BB, Q8_E4>(q, st);
#define CKV_APP(TT) \
    CKV_APP4(TT, 64, 16) CKV_APP4(TT, 64, 32) CKV_APP4(TT, 64, 64) CKV_APP4(TT, 64, 128) \
    CKV_APP4(TT, 128, 16) CKV_APP4(TT, 128, 32) CKV_APP4(TT, 128, 64) CKV_APP4(TT, 128, 128)
    if (c.dtype == CKV_DTYPE_BF16) {
        CKV_APP(__nv_bfloat16)
    } else {
        CKV_APP(float)
    }
#undef CKV_APP
#undef CKV_APP4
    return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// read back.  A thread takes 8 codes of a row (K, then V) for READ_PASS rows,
// all loads issued before the first is used; bound by the rows written.
// ---------------------------------------------------------------------------
constexpr int READ_THREADS = 256;
constexpr int READ_PASS = 4;

struct ReadParams {
    Q8View c;
    RowsView r;
    const int32_t* first;
    int R;
    int chunks;  // row chunks per (request, head)
};

template <typename T, int FMT>
__device__ __forceinline__ void store_row8(T* dst, const uint2& w, float s) {
    float x[4], y[4];
    q8c_values<FMT>(w.x, x);
    q8c_values<FMT>(w.y, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] *= s;
        y[i] *= s;
    }
    if constexpr (ElemBytes<T>::v == 2) {
        __nv_bfloat162 o[4] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3]),
                               __floats2bfloat162_rn(y[0], y[1]), __floats2bfloat162_rn(y[2], y[3])};
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
    } else {
        reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(y[0], y[1], y[2], y[3]);
    }
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(READ_THREADS) read_kernel(const __grid_constant__ ReadParams q) {
    constexpr int TPR = D / 8, RPP = READ_THREADS / TPR;
    pdl_wait();
    const TableView& t = q.c.t;
    const int chunk = blockIdx.x % q.chunks, bh = blockIdx.x / q.chunks;
    const int b = bh / q.c.Hkv, h = bh - b * q.c.Hkv;
    const int part = threadIdx.x % TPR, r0 = chunk * (RPP * READ_PASS) + threadIdx.x / TPR;
    const long long cap = (long long)t.max_blocks << t.sh;
    const int n = t.len[b];
    const bool bad_len = n < 0 || n > cap;
    if (bad_len && threadIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
    const int first = q.first ? q.first[b] : 0;
    int64_t row[READ_PASS];  // row of the pool, -1: zeros
#pragma unroll
    for (int p = 0; p < READ_PASS; ++p) {
        const int r = r0 + p * RPP;
        const long long pos = (long long)first + r;
        row[p] = -1;
        if (r < q.R && !bad_len && pos >= 0 && pos < n) {
            const int id = t.table[(size_t)b * t.max_blocks + (pos >> t.sh)];
            if ((unsigned)id < (unsigned)t.n_blocks)
                row[p] = (((int64_t)id * q.c.Hkv + h) << t.sh) + (pos & (t.block - 1));
            else
                atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
        }
    }
    uint2 kw[READ_PASS], vw[READ_PASS];
    float ks[READ_PASS], vs[READ_PASS];
#pragma unroll
    for (int p = 0; p < READ_PASS; ++p) {
        kw[p] = vw[p] = make_uint2(0, 0);
        ks[p] = vs[p] = 0.f;
        if (row[p] >= 0) {
            kw[p] = reinterpret_cast<const uint2*>(static_cast<const char*>(q.c.k) + row[p] * D)[part];
            vw[p] = reinterpret_cast<const uint2*>(static_cast<const char*>(q.c.v) + row[p] * D)[part];
            ks[p] = q.c.k_scale[row[p] >> t.sh];
            vs[p] = q.c.v_scale[row[p] >> t.sh];
        }
    }
    T* ko = static_cast<T*>(q.r.k) + b * q.r.sb + h * q.r.sh + part * 8;
    T* vo = static_cast<T*>(q.r.v) + b * q.r.sb + h * q.r.sh + part * 8;
#pragma unroll
    for (int p = 0; p < READ_PASS; ++p) {
        const int r = r0 + p * RPP;
        if (r >= q.R) continue;
        store_row8<T, FMT>(ko + r * q.r.st, kw[p], ks[p]);
        store_row8<T, FMT>(vo + r * q.r.st, vw[p], vs[p]);
    }
}

template <typename T, int D, int FMT>
static cudaError_t launch_read_t(ReadParams q, cudaStream_t st) {
    constexpr int ROWS = READ_THREADS / (D / 8) * READ_PASS;
    q.chunks = (q.R + ROWS - 1) / ROWS;
    const long long grid = (long long)q.chunks * q.c.t.B * q.c.Hkv;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_pdl(KK_UPDATE, read_kernel<T, D, FMT>, dim3((unsigned)grid), dim3(READ_THREADS), 0, st, q);
}

cudaError_t launch_q8_read(const Q8View& c, const int32_t* first, int R, const RowsView& r, cudaStream_t st) {
    const ReadParams q{c, r, first, R, 0};
#define CKV_READ(TT, DD)     \
    if (c.d == DD)           \
        return c.format == Q8_I8 ? launch_read_t<TT, DD, Q8_I8>(q, st) : launch_read_t<TT, DD, Q8_E4>(q, st);
    if (c.dtype == CKV_DTYPE_BF16) {
        CKV_READ(__nv_bfloat16, 64) CKV_READ(__nv_bfloat16, 128)
    } else {
        CKV_READ(float, 64) CKV_READ(float, 128)
    }
#undef CKV_READ
    return cudaErrorInvalidValue;
}

}  // namespace ckv
