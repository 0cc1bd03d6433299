// What the decode attention kernels share: the parameter pack, the work split
// and the merge kernel that follows them (the units' partials combined, the
// neighbour search over the stored graph logits, the fused community update).
// The attention over the 16/32-bit cache (ckv_decode.cu) uses all of it, the one
// over an 8-bit cache's selected tokens (ckv_q8_sparse.cu) the neighbour search.
#pragma once

#include <math.h>

#include "ckv_assign.cuh"
#include "ckv_internal.cuh"

namespace ckv {

// Work split of the attention kernel: the first 7/8 of the concatenated token
// lists are cut into one equal slice per warp; the last 1/8 is handed out in
// chunks of at least DYN_CHUNK_MIN tokens (at most NCH_MAX chunks) from an
// atomic ticket, so warps on SMs that run faster (the SMs of a GPC share its
// memory bandwidth unevenly) take more of it and all warps end together.
constexpr int DYN_DEN = 8;
constexpr int MIN_WARP_TOKENS = 64;
constexpr int DYN_CHUNK_MIN = 64;
constexpr int NCH_MAX = 4096;

struct DynSplit {
    int R;      // tokens of the static part, [0, R)
    int per_s;  // static tokens per warp
    int chk;    // dynamic chunk length
    int nch;    // dynamic chunks
};

// dense: static slices only (its units are long, so a dynamic tail would
// multiply the partials each merge block combines)
__host__ __device__ __forceinline__ DynSplit dyn_split(int total, int W, bool dense) {
    DynSplit d;
    const int dyn = dense ? 0 : total / DYN_DEN;
    d.chk = max(DYN_CHUNK_MIN, (dyn + NCH_MAX - 1) / NCH_MAX);
    d.nch = (dyn + d.chk - 1) / d.chk;
    d.R = total - dyn;
    // at least MIN_WARP_TOKENS per warp: small problems use fewer warps, so
    // each unit has fewer partials to merge
    d.per_s = max(MIN_WARP_TOKENS, (d.R + W - 1) / W);
    return d;
}

struct DecodeParams {
    const void* k;
    const void* v;
    int64_t sb, sh, st;
    const void* q;
    int Hq, Hkv;
    int U, G, per_head;
    int S;
    const int32_t* sel_tok;
    int tok_cap;
    int32_t* unit_prefix;   // written by block 0 of the attention kernel
    const int32_t* n_tok;
    int T;                  // dense only: tokens per unit
    int T_cap;              // rows per (sequence, KV head): debug checks of positions
    int32_t* dev_err;       // the graph's error word (debug checks; NULL for dense)
    float scale_log2;
    DecodeWs ws;
    int W;                  // warps in the grid
    int want_nbr;
    float* out;
    int32_t* nbr8;          // may be NULL when only the fused update needs them
    int append;             // fused community update (and K/V append) in the merge
    AssignParams ap;
    const int32_t* len;     // 8-bit cache: tokens per request, the position each request's new token joins at
    const int32_t* built;   // 8-bit cache: positions each unit was built over, or NULL
};

__device__ __forceinline__ void unit_heads(const DecodeParams& p, int u, int gq, bool dense,
                                           int& b, int& kvh, int& h0) {
    b = u / p.G;
    const int g = u - b * p.G;
    if (!dense && p.per_head) {
        kvh = g / (p.Hq / p.Hkv);
        h0 = g;
    } else {
        kvh = g;
        h0 = g * gq;
    }
}

// 2^x by the hardware approximation (PTX ex2.approx.ftz.f32, relative error
// about 2^-22).  Arguments here are <= 8; results below 2^-126 flush to zero,
// which only drops weights below 1e-38 of the running maximum.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Warps of the merge block that search the neighbours (sparse decode only).
constexpr int NBR_WARPS = 4;
// Spare partial slots after the last one: a merge chunk (<= 32 slots) may
// read past a unit's last slot without leaving the arrays.
constexpr int MERGE_PAD = 32;
constexpr int NBR_THREADS = NBR_WARPS * 32;
constexpr int NBR_KEEP = 16;  // list entries per thread held in registers
constexpr int NBR_CAP = 256;  // candidate slots in shared memory

// Neighbour ranking key: graph logit descending, then position ascending, as
// one unsigned 64-bit number (larger is better; 0 = no entry).  The logit is
// mapped to an order-preserving unsigned integer.
__device__ __forceinline__ unsigned long long nbr_key(float lam, int pos) {
    unsigned b = __float_as_uint(lam + 0.0f);  // -0 ranks as +0
    b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return ((unsigned long long)b << 32) | (unsigned)(0x7fffffff - pos);
}
__device__ __forceinline__ int nbr_pos(unsigned long long k) {
    return 0x7fffffff - (int)(unsigned)(k & 0xffffffffu);
}

// An 8-bit cache's unit before its new token joins: the request's length, the last
// tail member's position (-1: none) and the positions the unit was built over.
// Loaded ahead of the neighbour search, looked at after it.
struct JoinAt {
    int len = 0, last = -1, built = 0;
};

// The fused community update of unit u by the merge block's NBR_WARPS
// neighbour warps (thread xt of 32 NBR_WARPS), given its neighbour positions.
template <typename T, int D, bool Q8 = false>
__device__ __forceinline__ void merge_assign(const DecodeParams& p, int u, const int* nbpos, int xt,
                                             const JoinAt& at = JoinAt()) {
    __shared__ __align__(16) AssignScratch<D> s_as;
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(NBR_THREADS) : "memory"); };
    if constexpr (Q8) {
        // the requests of an 8-bit cache differ in length: each one's token
        // joins at its own end.  A position joins once: members at it or past it
        // (growth refused since, or tokens given back) leave first.
        AssignParams ap = p.ap;
        ap.pos = at.len;
        const bool stale = at.last >= ap.pos;
        const int err = ap.pos < 0 || ap.pos >= ap.T_cap || (stale && !ap.undo) ? CKV_DEVERR_INDEX
                        : ap.pos < at.built                                     ? CKV_DEVERR_CUT
                                                                                : 0;
        if (err) {
            if (xt == 0) {
                atomicOr(ap.dev_err, err);
                if (ap.assigned) ap.assigned[u] = -1;
            }
            return;
        }
        if (stale) {
            if (xt < 32) untail_unit<D>(ap, u, ap.pos, xt);
            sync();
        }
        assign_unit<T, D, NBR_WARPS, false>(ap, u, nbpos, xt, s_as, sync);
    } else {
        assign_unit<T, D, NBR_WARPS, false>(p.ap, u, nbpos, xt, s_as, sync);
    }
}

// The neighbours of unit u, a list of n >= 1 entries, and its fused update, by
// NBR_THREADS threads (xt of them).
template <typename T, int D, bool Q8 = false>
__device__ __forceinline__ void search_neighbours(const DecodeParams& p, int u, int n, int xt,
                                                  const JoinAt& at = JoinAt()) {
    // neighbour search over the graph logits the attention kernel stored,
    // for the unit's non-sink list entries [S, n).  Threshold filter:
    // theta = the 8th largest of the NBR_THREADS per-thread maxima is a
    // distinct entry's key with 7 larger ones, so every top-8 entry has
    // key >= theta; those few candidates are collected in shared memory
    // and sorted by one warp.
    __shared__ unsigned long long s_top[NBR_THREADS / 4];
    __shared__ unsigned long long s_cand[NBR_CAP];
    __shared__ int s_cnt;
    const int lane = xt & 31, xw = xt >> 5;
    const float* lamu = p.ws.lam + (size_t)u * p.ws.lam_cap;
    const int32_t* toks = p.sel_tok + (size_t)u * p.tok_cap;
    // an 8-bit cache's skipped entry (logit -inf) is no neighbour
    auto key_of = [&](float lam, int pos) { return Q8 && lam == -INFINITY ? 0ull : nbr_key(lam, pos); };
    auto key_at = [&](int i) { return key_of(lamu[i], __ldg(toks + i)); };
    // all loads first (clamped in-range indices, no branches), so the
    // 2 x NBR_KEEP loads are in flight together
    float lv[NBR_KEEP];
    int pv[NBR_KEEP];
#pragma unroll
    for (int k = 0; k < NBR_KEEP; ++k) {
        const int i = min(p.S + xt + k * NBR_THREADS, n - 1);
        lv[k] = lamu[i];
        pv[k] = __ldg(toks + i);
    }
    unsigned long long kk[NBR_KEEP];
#pragma unroll
    for (int k = 0; k < NBR_KEEP; ++k)
        kk[k] = p.S + xt + k * NBR_THREADS < n ? key_of(lv[k], pv[k]) : 0ull;
    unsigned long long mx = 0;
#pragma unroll
    for (int k = 0; k < NBR_KEEP; ++k) mx = kk[k] > mx ? kk[k] : mx;
    for (int i = p.S + xt + NBR_KEEP * NBR_THREADS; i < n; i += NBR_THREADS) {
        const unsigned long long k2 = key_at(i);
        mx = k2 > mx ? k2 : mx;
    }
    if (xt == 0) s_cnt = 0;
    const unsigned long long srt = warp_sort_desc(mx, lane);
    if (lane < 8) s_top[xw * 8 + lane] = srt;
    asm volatile("bar.sync 1, %0;" ::"n"(NBR_THREADS) : "memory");
    // every warp sorts the NBR_WARPS x 8 warp leaders itself (no extra barrier)
    const unsigned long long theta =
        __shfl_sync(FULL, warp_sort_desc(lane < NBR_WARPS * 8 ? s_top[lane] : 0ull, lane), 7);
    auto offer = [&](unsigned long long k2) {
        if (k2 != 0ull && k2 >= theta) {
            const int slot = atomicAdd(&s_cnt, 1);
            if (slot < NBR_CAP) s_cand[slot] = k2;
        }
    };
#pragma unroll
    for (int k = 0; k < NBR_KEEP; ++k) offer(kk[k]);
    for (int i = p.S + xt + NBR_KEEP * NBR_THREADS; i < n; i += NBR_THREADS) offer(key_at(i));
    asm volatile("bar.sync 1, %0;" ::"n"(NBR_THREADS) : "memory");
    __shared__ int s_nbpos[CKV_NEIGHBOURS];
    if (xw == 0) {
        const int cnt = s_cnt;
        int32_t* outn = p.nbr8 ? p.nbr8 + (size_t)u * 8 : nullptr;
        if (cnt <= 32) {
            const unsigned long long x = warp_sort_desc(lane < cnt ? s_cand[lane] : 0ull, lane);
            if (lane < 8) {
                const int np = x ? nbr_pos(x) : -1;
                s_nbpos[lane] = np;
                if (outn) outn[lane] = np;
            }
        } else {
            // many candidates (ties in the logits): 8 rounds, each taking
            // the best key below the previous winner, from the shared
            // list or, past its capacity, from the whole list
            unsigned long long prev = ~0ull;
            for (int r = 0; r < 8; ++r) {
                unsigned long long best = 0;
                if (cnt <= NBR_CAP) {
                    for (int c = lane; c < cnt; c += 32) {
                        const unsigned long long k2 = s_cand[c];
                        if (k2 < prev && k2 > best) best = k2;
                    }
                } else {
                    for (int i = p.S + lane; i < n; i += 32) {
                        const unsigned long long k2 = key_at(i);
                        if (k2 < prev && k2 > best) best = k2;
                    }
                }
                best = warp_max_u64(best);
                if (lane == 0) {
                    const int np = best ? nbr_pos(best) : -1;
                    s_nbpos[r] = np;
                    if (outn) outn[r] = np;
                }
                prev = best;  // 0 once the entries run out: every later round finds none
            }
        }
    }
    if (p.append) {
        asm volatile("bar.sync 1, %0;" ::"n"(NBR_THREADS) : "memory");  // s_nbpos complete
        merge_assign<T, D, Q8>(p, u, s_nbpos, xt, at);
    }
}

// One block per unit: threads 0..D-1 own one output dimension each (all the
// unit's heads); the NBR_WARPS extra warps search the top-8 neighbours.  Slots are
// combined in slot order, a chunk of slots at a time, by a per-thread online
// merge: no shared memory and no barriers, so the merge costs about two
// dependent rounds of loads.
template <typename T, int D, int GQ, bool DENSE>
__global__ void __launch_bounds__(D + (DENSE ? 0 : 32 * NBR_WARPS), 2) decode_merge(const __grid_constant__ DecodeParams p) {
    pdl_wait();  // the attention kernel's partials are complete and visible
    const int u = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    // no kernel of this call takes a ticket any more: return it to zero
    if (u == 0 && t == 0) *p.ws.ticket = 0;
    int b, kvh, h0;
    unit_heads(p, u, GQ, DENSE, b, kvh, h0);
    int ubeg, uend, total;
    if constexpr (DENSE) {
        ubeg = u * p.T;
        uend = ubeg + p.T;
        total = p.U * p.T;
    } else {
        ubeg = p.unit_prefix[u];
        uend = p.unit_prefix[u + 1];
        total = p.unit_prefix[p.U];
    }
    float* outu = p.out + ((size_t)b * p.Hq + h0) * D;
    // the new K/V rows go into the cache first, by the output threads (off
    // the neighbour search and update, which wait on more round trips)
    if (!DENSE && p.append && t < D) append_rows(p.ap, u, t, D);
    if (uend <= ubeg) {
        for (int i = t; i < GQ * D; i += blockDim.x) outu[i] = 0.f;
        if (!DENSE && p.want_nbr && p.nbr8 && t < 8) p.nbr8[(size_t)u * 8 + t] = -1;
        if (!DENSE && p.append && warp >= D / 32) {
            __shared__ int s_none[CKV_NEIGHBOURS];
            if (t - D < CKV_NEIGHBOURS) s_none[t - D] = -1;
            merge_assign<T, D>(p, u, s_none, t - D);  // no neighbour: the token joins nothing
        }
        return;
    }
    // the unit's partials: static slices [sA, sA + nA), then dynamic chunks
    // [sB, sB + nB) (the attention kernel's split, recomputed)
    const DynSplit sp = dyn_split(total, p.W, DENSE);
    int nA = 0, nB = 0;
    size_t sA = 0, sB = 0;
    if (ubeg < sp.R) {
        const int f = ubeg / sp.per_s, l = (min(uend, sp.R) - 1) / sp.per_s;
        sA = (size_t)f + u;
        nA = l - f + 1;
    }
    if (uend > sp.R) {
        const int f = (max(ubeg, sp.R) - sp.R) / sp.chk, l = (uend - 1 - sp.R) / sp.chk;
        sB = (size_t)p.W + p.U + f + u;
        nB = l - f + 1;
    }
    const DecodeWs& ws = p.ws;

    if (!DENSE && p.want_nbr && warp >= D / 32) {
        search_neighbours<T, D>(p, u, uend - ubeg, t - D);
        return;
    }

    if (t >= D) return;
    // online merge, in slot order, of this thread's output dimension for every
    // head: running max, rescaled sum and accumulator; all loads of a chunk of
    // slots are issued before any is used
    constexpr int CH = GQ >= 8 ? 4 : 32 / GQ;
    float M[GQ], Ls[GQ], A[GQ];
#pragma unroll
    for (int h = 0; h < GQ; ++h) {
        M[h] = -INFINITY;
        Ls[h] = 0.f;
        A[h] = 0.f;
    }
    for (int part = 0; part < 2; ++part) {
      const size_t s0 = part ? sB : sA;
      const int nslots = part ? nB : nA;
      for (int c0 = 0; c0 < nslots; c0 += CH) {
        float xm[CH][GQ], xl[CH][GQ], xa[CH][GQ];
        // unconditional loads at constant offsets from one base (the slot
        // arrays carry MERGE_PAD spare slots, so a chunk never reads past
        // them), masked afterwards by selects: every load of the chunk is in
        // flight before the first is used
        const float* mb = ws.m + (s0 + c0) * GQ;
        const float* lb = ws.l + (s0 + c0) * GQ;
        const float* ab = ws.acc + (s0 + c0) * GQ * D + t;
#pragma unroll
        for (int r = 0; r < CH; ++r) {
#pragma unroll
            for (int h = 0; h < GQ; ++h) {
                xm[r][h] = mb[r * GQ + h];
                xl[r][h] = lb[r * GQ + h];
                xa[r][h] = ab[(r * GQ + h) * D];
            }
        }
#pragma unroll
        for (int r = 0; r < CH; ++r) {
            const bool ok = c0 + r < nslots;
#pragma unroll
            for (int h = 0; h < GQ; ++h) {
                xm[r][h] = ok ? xm[r][h] : -INFINITY;
                xl[r][h] = ok ? xl[r][h] : 0.f;
                xa[r][h] = ok ? xa[r][h] : 0.f;
            }
        }
        // the chunk's maximum first, then independent weights: the dependent
        // chain per chunk is one rescale instead of one per slot
#pragma unroll
        for (int h = 0; h < GQ; ++h) {
            float mc = -INFINITY;
#pragma unroll
            for (int r = 0; r < CH; ++r) mc = fmaxf(mc, xm[r][h]);
            if (mc == -INFINITY) continue;
            const float mn = fmaxf(M[h], mc);
            const float fo = exp2_approx(M[h] - mn);
            float ls = 0.f, a = 0.f;
#pragma unroll
            for (int r = 0; r < CH; ++r) {
                const float f = exp2_approx(xm[r][h] - mn);
                ls = fmaf(xl[r][h], f, ls);
                a = fmaf(xa[r][h], f, a);
            }
            Ls[h] = fmaf(Ls[h], fo, ls);
            A[h] = fmaf(A[h], fo, a);
            M[h] = mn;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < GQ; ++h) outu[h * D + t] = A[h] / Ls[h];
}

}  // namespace ckv
