// paged.cuh -- what the paged-cache kernels share: 8-bit conversions, the search for
// the sequence that owns a packed row, and the lookup of a position's page.
#pragma once

#include <cuda_fp8.h>

#include "kernels.h"

namespace attn {

// ------------------------------------------------------- 8-bit floating point
// Largest finite values 448 = 1.75 * 2^8 (e4m3) and 57344 = 1.75 * 2^15 (e5m2).
template <int CACHE> struct F8;
template <> struct F8<CACHE_E4M3> {
    static constexpr __nv_fp8_interpretation_t kKind = __NV_E4M3;
    static constexpr int kTopExp = 8;
};
template <> struct F8<CACHE_E5M2> {
    static constexpr __nv_fp8_interpretation_t kKind = __NV_E5M2;
    static constexpr int kTopExp = 15;
};
// two codes (low byte first) as two halves: every value of either type is a half
template <int CACHE>
__device__ __forceinline__ uint32_t f8x2_to_h2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, F8<CACHE>::kKind);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
// nearest codes of two floats; beyond the largest finite value, the largest; NaN stays NaN
template <int CACHE>
__device__ __forceinline__ uint32_t f8x2_from_f(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, F8<CACHE>::kKind);
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t h) { return __half22float2(*reinterpret_cast<__half2*>(&h)); }

// ------------------------------------------------------------------ searches
// Largest i in [0, n) with key(i) <= x for a non-decreasing key, or -1: by a whole warp,
// 32 probes a round (two dependent loads for up to 1024 entries).  Whatever the keys
// are, the result lies in [-1, n).
template <typename Key>
__device__ __forceinline__ int warp_last_le(int n, long long x, Key key) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;  // the answer lies in [lo - 1, lo + len)
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int i = lo + lane * step;  // first entry of this lane's stretch
        const bool le = i < lo + len && key(i) <= x;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        if (c == 0) return lo - 1;
        if (step == 1) return lo + c - 1;
        const int first = lo + (c - 1) * step;  // key(first) <= x: the answer is in its stretch
        const int end = min(lo + len, first + step);
        lo = first + 1;
        len = end - lo;
    }
    return lo - 1;
}

// A packed row's sequence and position, counted from the sequence's first row.
struct RowSeq {
    int b, first, end;  // rows [first, end) of the packed tensor are sequence b's; b < 0: none holds the row
};
__device__ __forceinline__ RowSeq row_seq(const PagedParams& P, int r) {
    RowSeq s;
    s.b = warp_last_le(P.B + 1, r, [&](int i) { return (long long)__ldg(P.cu + i); });
    s.first = s.end = 0;
    if (s.b >= P.B) s.b = -1;  // behind the last sequence
    if (s.b >= 0) {
        s.first = __ldg(P.cu + s.b);
        s.end = __ldg(P.cu + s.b + 1);
        // prefix sums that decrease or leave the tensor: no sequence
        if (s.first < 0 || s.first > r || s.end <= r || s.end > P.total) {
            if ((threadIdx.x & 31) == 0) atomicOr(P.status, ST_PAGED_BOUNDS);
            s.b = -1;
        }
    }
    return s;
}

// The page of block j (of max_pages) of sequence b, or -1 (flagged) outside the pool.
__device__ __forceinline__ int page_of(const PagedParams& P, int b, int j, bool flag) {
    int pg = -1;
    if (j >= 0 && j < P.max_pages) pg = __ldg(P.table + (long long)b * P.max_pages + j);
    if (pg < 0 || pg >= P.num_pages) {
        if (flag) atomicOr(P.status, ST_PAGED_BOUNDS);
        return -1;
    }
    return pg;
}
// first element of row `row` of page pg for KV head h
__device__ __forceinline__ long long cache_row(const PagedParams& P, int pg, int h, int row) {
    return ((((long long)pg * P.Hkv + h) << P.page_shift) + row) * P.hd;
}

}  // namespace attn
