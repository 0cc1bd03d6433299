// The paged 8-bit cache: launch parameter packs and the code formats, shared by
// its kernels (ckv_q8_cache.cu, ckv_q8_dense.cu, ckv_q8_sparse.cu) and the build
// (ckv_build.cu).
#pragma once

#include <cuda_fp16.h>

#include "ckv_internal.cuh"

namespace ckv {

struct TableView {
    int B, block, n_blocks, max_blocks;
    int sh;  // log2(block)
    int32_t* table;
    int32_t* len;
    int32_t* free_list;
    int32_t* n_free;
    int32_t* dev_err;
};

struct Q8View {
    TableView t;
    int format, dtype, Hkv, Hq, d;
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
};

struct PlanView {
    int n_rows;
    int32_t* start;
    int32_t* slot;
    int32_t* granted;
};

struct RowsView {  // new rows in, or read-back rows out
    void* k;
    void* v;
    int64_t sb, st, sh;  // element strides: request, token, KV head
    int T_rows;          // append: rows per request when padded, 0 when packed
};

cudaError_t launch_plan_blocks(const TableView& t, const int32_t* add, const PlanView& p, cudaStream_t st);
cudaError_t launch_quant_append(const Q8View& c, const PlanView& p, const RowsView& r, cudaStream_t st);
// A block of the read takes READ_PASS rows a thread, D / 8 threads to a row.
constexpr int READ_THREADS = 128;
constexpr int READ_PASS = 2;
constexpr int q8_read_rows(int d) { return READ_THREADS / (d / 8) * READ_PASS; }
constexpr long long q8_read_blocks(int B, int Hkv, int d, long long R) {
    return (R + q8_read_rows(d) - 1) / q8_read_rows(d) * B * Hkv;
}
cudaError_t launch_q8_read(const Q8View& c, const int32_t* first, int R, const RowsView& r, cudaStream_t st);
// The attention's workspace: after the head, counters of the units (of the most there
// can be, so that they are in the same place for every cache), the partials, and the
// graph logits of the sparse call's lists.
constexpr size_t Q8_COUNTER_BYTES = (size_t)MAX_UNITS * 4;
size_t q8_blocks_ws_bytes(int gq, int d);
cudaError_t launch_dense_decode_q8(const Q8View& c, const void* q, float* out, void* ws, cudaStream_t st);
cudaError_t launch_sparse_decode_q8(const Q8View& c, const GraphView& g, const SelView& s, const void* q, float* out,
                                    int32_t* nbr8, const void* k_new, int32_t* assigned, void* ws, cudaStream_t st);
cudaError_t launch_build_q8(const Q8View& c, const GraphView& g, const int32_t* labels, int64_t labels_stride, int T,
                            const int32_t* which, void* ws, cudaStream_t st);
cudaError_t launch_trim_graph_q8(const Q8View& c, const GraphView& g, cudaStream_t st);

// ---------------------------------------------------------------------------
// formats.  int8: scale amax/127.  e4m3: a power-of-two scale, which costs a
// floating code no precision, makes x/s exact and re-scales codes with no
// second rounding (but for codes that become subnormal).
// ---------------------------------------------------------------------------
constexpr int Q8_I8 = CKV_Q8_INT8, Q8_E4 = CKV_Q8_E4M3;
constexpr float Q8_FLOOR = 7.88860905221011805e-31f;  // 2^-100: 1/s stays finite

// the scale that holds magnitudes up to amax (bits of a float >= 0; not finite: NaN)
template <int FMT>
__device__ __forceinline__ float q8c_scale(unsigned amax_bits) {
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    const float a = fmaxf(__uint_as_float(amax_bits), Q8_FLOOR);
    if constexpr (FMT == Q8_I8) {
        return __fdiv_rn(a, 127.f);
    } else {
        // a = m 2^E, m in [1, 2); 448 = 1.75 * 2^8
        const unsigned b = __float_as_uint(a);
        const unsigned e = (b >> 23) - 8u + ((b & 0x7fffffu) > 0x600000u ? 1u : 0u);
        return __uint_as_float(e << 23);
    }
}

// Four codes of x f.  int8: one fma adds 1.5 * 2^23, which rounds the exact
// product to the nearest integer, ties to even (x f rounded to fp32 first
// would turn near-ties, common with amax/2, into ties); the low byte of the sum
// is the code.  e4m3: f is a power of two, so the product is exact.  With a NaN
// f (a block made NaN) the codes mean nothing.
template <int FMT>
__device__ __forceinline__ unsigned q8c_codes(float x0, float x1, float x2, float x3, float f) {
    if constexpr (FMT == Q8_I8) {
        constexpr float MAGIC = 12582912.f;  // 1.5 * 2^23
        auto code = [&](float x) {
            const float y = fminf(fmaxf(__fmaf_rn(x, f, MAGIC), MAGIC - 127.f), MAGIC + 127.f);
            return __float_as_uint(y);
        };
        const unsigned lo = __byte_perm(code(x0), code(x1), 0x0040), hi = __byte_perm(code(x2), code(x3), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        auto pair = [&](float a, float b) {
            unsigned short r;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b * f), "f"(a * f));
            return (unsigned)r;
        };
        return pair(x0, x1) | (pair(x2, x3) << 16);
    }
}

// Two e4m3 codes (the low byte first) as fp16, exact.
__device__ __forceinline__ unsigned e4m3x2_half2(unsigned short c) {
    unsigned r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// Four codes as fp32 values (without the scale).
template <int FMT>
__device__ __forceinline__ void q8c_values(unsigned w, float (&x)[4]) {
    if constexpr (FMT == Q8_I8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int)(signed char)(w >> (8 * i));
    } else {
        const unsigned a = e4m3x2_half2((unsigned short)(w & 0xffffu)), b = e4m3x2_half2((unsigned short)(w >> 16));
        const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
        x[0] = fa.x; x[1] = fa.y; x[2] = fb.x; x[3] = fb.y;
    }
}

}  // namespace ckv
