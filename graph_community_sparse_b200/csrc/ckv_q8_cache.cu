// The paged 8-bit cache's bookkeeping and rows, sm_100a: block tables and slot
// maps from request lengths (ckv_plan_blocks), new rows quantised into their
// blocks (ckv_quant_append), rows read back (ckv_q8_read).  CommunityKV keeps the
// cache whole (rit.work summary, section "A graph of tokens replaces
// re-clustering", paragraph 5); this is that cache in 8 bits.
#include "ckv_q8.cuh"

namespace ckv {

// ---------------------------------------------------------------------------
// block-wide exclusive scan of N 64-bit integers per thread, their totals in
// total; one barrier, and s_warp ([N][32]) must not be in use still
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ void block_exclusive_scan64(long long (&x)[N], long long* s_warp, long long (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    long long inc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        inc[i] = x[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL, inc[i], o);
            if (lane >= o) inc[i] += y;
        }
        if (lane == 31) s_warp[i * 32 + warp] = inc[i];
    }
    __syncthreads();
    // every warp scans the warps' totals for itself
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const long long w = lane < nw ? s_warp[i * 32 + lane] : 0;
        long long wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL, wi, o);
            if (lane >= o) wi += y;
        }
        total[i] = __shfl_sync(FULL, wi, 31);
        x[i] = __shfl_sync(FULL, wi - w, warp) + inc[i] - x[i];
    }
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
// from what is written to it, and the blocks given back from those taken.  32
// requests that grow by a few tokens: 4.3 us a call; 48 prompts of 500 to 6000
// tokens that end and come again: 17.5 us for the two calls.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_CLUSTER = 8;

struct PlanParams {
    TableView t;
    PlanView p;
    const int32_t* add;
    int rows_here;  // rows whose slots the plan kernel writes itself
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const __grid_constant__ PlanParams q) {
    extern __shared__ int s_plan[];
    __shared__ long long s_warp[128];
    const TableView& t = q.t;
    const int B = t.B, bs = t.block, sh = t.sh, W = t.max_blocks, threads = blockDim.x;
    int* s_n1 = s_plan;             // [B] tokens after the drops
    int* s_n2 = s_n1 + B;           // [B] tokens after the growth
    int* s_gone = s_n2 + B;         // [B + 1] blocks given back before request b
    int* s_need = s_gone + B + 1;   // [B + 1] blocks taken before request b
    int* s_start = s_need + B + 1;  // [B + 1] first row of request b
    pdl_wait();
    const int tid = threadIdx.x;
    const int gthreads = gridDim.x * threads, gtid = blockIdx.x * threads + tid;
    const int n_free = max(0, min(*t.n_free, t.n_blocks));
    const long long cap = (long long)W << sh;
    auto blocks = [&](int n) { return (int)(((long long)n + bs - 1) >> sh); };

    // drops, and the rows asked for.  Thread i handles requests [b0, b1).
    const int seg = (B + threads - 1) / threads;
    const int b0 = min(B, tid * seg), b1 = min(B, b0 + seg);
    long long gu[2] = {0, 0};  // blocks given back, rows asked for
    for (int b = b0; b < b1; ++b) {
        const int n0 = t.len[b], a = q.add[b];
        const bool bad = n0 < 0 || n0 > cap;
        if (bad && blockIdx.x == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
        const int n1 = bad ? 0 : a < 0 ? (int)max(0ll, (long long)n0 + a) : n0;
        s_n1[b] = n1;
        s_gone[b] = bad ? 0 : blocks(n0) - blocks(n1);
        gu[0] += s_gone[b];
        gu[1] += max(a, 0);
    }
    long long totals[2];
    block_exclusive_scan64<2>(gu, s_warp, totals);
    long long run_gone = gu[0], run_up = gu[1];
    const long long total_gone = totals[0], total_up = totals[1];
    const int freed = (int)min(total_gone, (long long)t.n_blocks - n_free);  // less only when the state is corrupt
    const int avail = n_free + freed;

    // growth that fits the table and the slot map, and the blocks it needs
    long long need[1] = {0}, need_all[1];
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
        need[0] += x;
    }
    block_exclusive_scan64<1>(need, s_warp + 64, need_all);
    long long run_need = need[0];
    const long long total_need = need_all[0];
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

    // blocks given back: the k-th of them at free_list[avail - 1 - k].  A thread
    // takes 4 consecutive ones: one search, the loads independent of each other.
    for (int k0 = gtid * 4; k0 < freed; k0 += gthreads * 4) {
        int b = last_le(s_gone, B + 1, k0);
        size_t at[4];
        int id[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = min(k0 + i, freed - 1);
            while (k >= s_gone[b + 1]) ++b;
            at[i] = (size_t)b * W + blocks(s_n1[b]) + (k - s_gone[b]);
            id[i] = t.table[at[i]];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (k0 + i >= freed) break;
            t.free_list[avail - 1 - (k0 + i)] = id[i];
            t.table[at[i]] = -1;
        }
        const unsigned top = max(max((unsigned)id[0], (unsigned)id[1]), max((unsigned)id[2], (unsigned)id[3]));
        if (top >= (unsigned)t.n_blocks) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
    }
    // everybody has read len, add and n_free and given blocks back
    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();

    // blocks taken: the k-th is free_list[avail - 1 - k].  A refused request's
    // range of k is empty or belongs to nobody (all needs after the first
    // refusal for want of blocks are refused).  An id out of range is flagged
    // with the slots of its rows.
    const int taken = s_need[B];
    for (int k0 = gtid * 4; k0 < taken; k0 += gthreads * 4) {
        int b = last_le(s_need, B + 1, k0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + i;
            if (k >= taken) break;
            while (k >= s_need[b + 1]) ++b;
            const int j = blocks(s_n1[b]) + (k - s_need[b]);
            if (j < blocks(s_n2[b])) t.table[(size_t)b * W + j] = __ldcg(t.free_list + avail - 1 - k);
        }
    }
    // the slot of every row, where they are few (else slots_kernel): the block
    // from the table where the request held it already, else from the free list
    // (the table entry may not be there yet)
    const int rows_in = s_start[B];
    for (int r = gtid; r < q.rows_here; r += gthreads) {
        int slot = -1;
        if (r < rows_in) {
            const int b = last_le(s_start, B + 1, r);
            const int n1 = s_n1[b], pos = n1 + (r - s_start[b]);
            if (pos < s_n2[b]) {
                const int j = pos >> sh, held = blocks(n1);
                const int id = __ldcg(j < held ? t.table + (size_t)b * W + j
                                               : t.free_list + avail - 1 - (s_need[b] + j - held));
                if ((unsigned)id < (unsigned)t.n_blocks) slot = (id << sh) | (pos & (bs - 1));
                else atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
            }
        }
        q.p.slot[r] = slot;
    }
    if (blockIdx.x != 0) return;
    long long took[1] = {0}, total_took[1];
    for (int b = b0; b < b1; ++b) {
        const int n0 = t.len[b];
        q.p.start[b] = s_start[b];
        const bool bad = n0 < 0 || n0 > cap;
        q.p.granted[b] = bad ? 0 : s_n2[b] - n0;
        if (!bad) {
            t.len[b] = s_n2[b];
            took[0] += blocks(s_n2[b]) - blocks(s_n1[b]);
        }
    }
    block_exclusive_scan64<1>(took, s_warp + 96, total_took);
    if (tid == 0) {
        q.p.start[B] = s_start[B];
        *t.n_free = avail - (int)total_took[0];
    }
}

// The slot map of many rows, after the plan kernel: every request's blocks are in
// the table by then.  A thread takes 8 consecutive rows: one search, the loads
// independent of each other.  (On the plan kernel's 8 SMs this phase was 10 us of
// a call's 13 for 151K rows.)
constexpr int SLOT_THREADS = 256;

__global__ void __launch_bounds__(SLOT_THREADS) slots_kernel(const __grid_constant__ PlanParams q) {
    extern __shared__ int s_plan[];
    const TableView& t = q.t;
    const int B = t.B, tid = threadIdx.x, rows = q.p.n_rows;
    int* s_start = s_plan;  // [B + 1]
    pdl_wait();
    for (int b = tid; b <= B; b += SLOT_THREADS) s_start[b] = q.p.start[b];
    __syncthreads();
    const int rows_in = s_start[B];
    const bool vec = (reinterpret_cast<uintptr_t>(q.p.slot) & 15u) == 0;
    for (long long r0 = ((long long)blockIdx.x * SLOT_THREADS + tid) * 8; r0 < rows;
         r0 += (long long)gridDim.x * SLOT_THREADS * 8) {
        int pos[8], id[8];
        int b = r0 < rows_in ? last_le(s_start, B + 1, (int)r0) : B;
        int g = 0, n0 = -1;  // tokens granted to the request, and its length before
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = (int)r0 + k;
            pos[k] = -1;
            if (r0 + k < rows && r < rows_in) {
                if (n0 < 0 || r >= s_start[b + 1]) {
                    while (r >= s_start[b + 1]) ++b;
                    g = q.p.granted[b];
                    n0 = g > 0 ? t.len[b] - g : 0;
                }
                const int i = r - s_start[b];
                if (i < g) {  // else refused (a request granted tokens has a good length)
                    pos[k] = n0 + i;
                    id[k] = t.table[(size_t)b * t.max_blocks + (pos[k] >> t.sh)];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            int slot = -1;
            if (pos[k] >= 0) {
                if ((unsigned)id[k] < (unsigned)t.n_blocks) slot = (id[k] << t.sh) | (pos[k] & (t.block - 1));
                else atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
            }
            pos[k] = slot;
        }
        if (vec && r0 + 8 <= rows) {
            int4* dst = reinterpret_cast<int4*>(q.p.slot + r0);
            dst[0] = make_int4(pos[0], pos[1], pos[2], pos[3]);
            dst[1] = make_int4(pos[4], pos[5], pos[6], pos[7]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (r0 + k < rows) q.p.slot[r0 + k] = pos[k];
        }
    }
}

cudaError_t launch_plan_blocks(const TableView& t, const int32_t* add, const PlanView& p, cudaStream_t st) {
    static LaunchCache lc;
    // few rows: one block and one launch.  Many: a cluster for the blocks, then the
    // slot map on the whole GPU.
    const bool many = p.n_rows > 4 * PLAN_THREADS;
    const PlanParams q{t, p, add, many ? 0 : p.n_rows};
    const size_t smem = (5 * (size_t)t.B + 3) * 4;
    cudaError_t e = prepare_launch(plan_kernel, lc, smem, PLAN_THREADS, nullptr, nullptr);
    if (e != cudaSuccess) return e;
    // (a call that only drops may give back as many blocks as the table has)
    const bool drops = p.n_rows == 0 && (long long)t.B * t.max_blocks > 8 * PLAN_THREADS;
    const int ctas = many || drops || t.B > PLAN_THREADS ? PLAN_CLUSTER : 1;
    const int threads = t.B <= 256 && p.n_rows <= 1024 && ctas == 1 ? 256 : PLAN_THREADS;  // barriers of fewer warps: 0.6 us less
    const bool timed = timing_enabled();
    if (timed && (e = timing_mark(KK_UPDATE, true, st)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
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
    if (e != cudaSuccess || !many) return e;
    static LaunchCache slots_lc;
    int per_sm = 0, sms = 0;
    const size_t slots_smem = ((size_t)t.B + 1) * 4;
    e = prepare_launch(slots_kernel, slots_lc, slots_smem, SLOT_THREADS, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    const int grid = min(sms * per_sm, (p.n_rows + SLOT_THREADS * 8 - 1) / (SLOT_THREADS * 8));
    return launch_pdl(KK_UPDATE, slots_kernel, dim3(grid), dim3(SLOT_THREADS), slots_smem, st, q);
}

// ---------------------------------------------------------------------------
// append.  One pass over the new rows, bound by their bytes: an item is one
// block's new rows of one head, K or V, kept in registers between the
// largest-magnitude reduction and the codes.  Items of the ragged batch are
// laid end to end (a scan over the requests in every block), so long and short
// requests share the grid evenly.
// ---------------------------------------------------------------------------
// Small blocks: while some wait at the reduction's barrier, others load (32768 rows
// of 8 heads: 34 us, 0.90 of the copy rate; before the instructions an item costs
// were cut 37, 40 with 256 threads, 65 with 512, and 60 with 256 that load their next
// item ahead, for want of registers).  One token each of 8 requests: 3.4 us, the
// launch and the chain length - slot - row - scale.
constexpr int APP_THREADS = 128;

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

// The largest magnitude so far, with these values: fp32 bits, or two bf16s, whose
// order without the sign is that of 16-bit integers.
template <typename T>
__device__ __forceinline__ unsigned max_magnitude(unsigned m, const uint4& w) {
    if constexpr (ElemBytes<T>::v == 2) {
        constexpr unsigned ABS = 0x7fff7fffu;
        return __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & ABS, w.y & ABS), __vmaxu2(w.z & ABS, w.w & ABS)));
    } else {
        constexpr unsigned ABS = 0x7fffffffu;
        return max(m, max(max(w.x & ABS, w.y & ABS), max(w.z & ABS, w.w & ABS)));
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
            // (rows of their own for every request: the blocks counted here stay within 31 bits)
            const long long first = q.p.start[b], last = first + a;
            const bool ok = n >= a && (long long)n <= (long long)t.max_blocks * BS && first >= 0 &&
                            last <= q.p.n_rows && last <= q.p.start[b + 1] && (q.r.T_rows == 0 || a <= q.r.T_rows);
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
    const unsigned items = (unsigned)total * Hkv * 2;  // the pool has fewer than 2^31 rows, 16 or more to a block
    struct Item {
        int lo, hi;   // new rows of the block
        int unit;     // block id * Hkv + head; -1: a bad slot
        bool is_v;
    };
    auto load = [&](unsigned it, Item& x, uint4 (&w)[NP]) {
        const int blk_no = (int)((it >> 1) / (unsigned)Hkv), h = (int)((it >> 1) - (unsigned)blk_no * Hkv);
        const int b = last_le(s_items, B, blk_no);
        const int n = t.len[b], a = q.p.granted[b], start = q.p.start[b];
        const int n_old = n - a;
        const int j = n_old / BS + (blk_no - s_items[b]);
        x.is_v = it & 1;
        x.lo = max(n_old - j * BS, 0);
        x.hi = min(n - j * BS, BS);
        const int first = j * BS + x.lo - n_old;  // the first new row's index among the request's
        const int slot = q.p.slot[start + first], id = slot / BS;
        x.unit = slot < 0 || id >= t.n_blocks || slot % BS != x.lo ? -1 : id * Hkv + h;
        const T* src = static_cast<const T*>(x.is_v ? q.r.v : q.r.k) + h * q.r.sh + part * V +
                       (q.r.T_rows ? b * q.r.sb + first * q.r.st : (int64_t)(start + first) * q.r.st);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int r = p * RPP + r0;
            w[p] = make_uint4(0, 0, 0, 0);
            if (r >= x.lo && r < x.hi) w[p] = *reinterpret_cast<const uint4*>(src + (int64_t)(r - x.lo) * q.r.st);
        }
    };
    auto store = [&](const Item& x, const uint4 (&w)[NP]) {
        if (x.unit < 0) {  // uniform over the block
            if (tid == 0) atomicOr(t.dev_err, CKV_DEVERR_BLOCK);
            return;
        }
        float* scale = (x.is_v ? q.c.v_scale : q.c.k_scale) + x.unit;
        const float s_old = x.lo > 0 ? *scale : 0.f;
        unsigned amax = 0;
#pragma unroll
        for (int p = 0; p < NP; ++p) amax = max_magnitude<T>(amax, w[p]);
        if constexpr (ElemBytes<T>::v == 2) amax = max(amax & 0xffff0000u, amax << 16);
        amax = __reduce_max_sync(FULL, amax);
        if (lane == 0) s_max[warp] = amax;
        __syncthreads();
        amax = __reduce_max_sync(FULL, s_max[lane % (APP_THREADS / 32)]);
        __syncthreads();  // s_max is free for the next item; every thread has the old scale
        float s = q8c_scale<FMT>(amax);
        if (x.lo > 0 && !(s_old <= s)) s = s_old != s_old || s_old > s ? s_old : s;  // a NaN on either side stays
        const float inv = __fdiv_rn(1.f, s);
        unsigned char* dst = static_cast<unsigned char*>(x.is_v ? q.c.v : q.c.k) + (size_t)x.unit * (BS * D) + part * V;
        if (x.lo > 0 && s != s_old) {
            // the block's older codes move to the larger scale
            const float f = __fmul_rn(s_old, inv);
            for (int r = r0; r < x.lo; r += RPP) {
                unsigned* c = reinterpret_cast<unsigned*>(dst + r * D);
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    float y[4];
                    q8c_values<FMT>(c[i], y);
                    c[i] = q8c_codes<FMT>(y[0], y[1], y[2], y[3], f);
                }
            }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int r = p * RPP + r0;
            if (r >= x.lo && r < x.hi) {
                float y[V];
                vec16_values<T>(w[p], y);
                unsigned c[V / 4];
#pragma unroll
                for (int i = 0; i < V / 4; ++i)
                    c[i] = q8c_codes<FMT>(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3], inv);
                if constexpr (V == 8) *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<unsigned*>(dst + r * D) = c[0];
            }
        }
        if (tid == 0) *scale = s;
    };
    for (unsigned it = blockIdx.x; it < items; it += gridDim.x) {
        Item x;
        uint4 w[NP];
        load(it, x, w);
        store(x, w);
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
// all loads issued before the first is used; bound by the rows written, few ones by
// the chain of loads length - block - codes.  32768 rows of 8 heads: 35 us, 0.88 of
// the copy rate (256 threads of 4 passes 35.8, of 1 pass 37.3; 16 codes a thread 40
// to 45, whose stores leave half sectors); up to 1000 rows each of 13 requests 5.8 us
// (7.3 with 256 threads of 4 passes: fewer, longer blocks).
// ---------------------------------------------------------------------------
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
    q.chunks = (q.R + q8_read_rows(D) - 1) / q8_read_rows(D);
    const long long grid = q8_read_blocks(q.c.t.B, q.c.Hkv, D, q.R);  // below 2^31: checked by the caller
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
