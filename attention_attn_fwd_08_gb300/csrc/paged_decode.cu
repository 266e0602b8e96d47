// paged_decode.cu -- attention of a few query rows of each sequence over a paged cache.
//
// One CTA per (sequence, head, query row): four warps take every fourth key, each with a
// running maximum and sum, and merge at the end.
#include <math.h>

#include <type_traits>

#include "paged.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <bool BF16, int HD, int CACHE>
__global__ void __launch_bounds__(128) paged_decode_kernel(const PagedParams P) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int kPer = HD / 32;
    __shared__ float sm[4], sl[4], so[4][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long id = blockIdx.x;
    const int lq = (int)(id % P.Lq);
    id /= P.Lq;
    const int h = (int)(id % P.H), b = (int)(id / P.H), kvh = h / P.G;
    const int cap = P.max_pages << P.page_shift;
    const int raw = __ldg(P.lengths + b);
    if (raw > cap && threadIdx.x == 0) atomicOr(P.status, ST_PAGED_BOUNDS);
    const int len = min(max(raw, 0), cap);
    const int pos = len - P.Lq + lq;
    const int lo = P.wl >= 0 ? max(0, pos - P.wl) : 0;
    const int hi = P.wr >= 0 ? (int)min((long long)len, (long long)pos + P.wr + 1) : len;
    const long long qrow = (((long long)b * P.Lq + lq) * P.H + h) * HD;
    float q[kPer], o[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        q[e] = Elem<T>::to_f(static_cast<const T*>(P.q)[qrow + lane + 32 * e]);
        o[e] = 0.f;
    }
    auto value = [&](const void* cache, const float* scale, int pg, int row, int d) -> float {
        const long long at = cache_row(P, pg, kvh, row) + d;
        if constexpr (CACHE == CACHE_16) return Elem<T>::to_f(static_cast<const T*>(cache)[at]);
        else return h2_to_f2(f8x2_to_h2<CACHE>(static_cast<const uint8_t*>(cache)[at])).x *
                    scale[(long long)pg * P.Hkv + kvh];
    };
    float m = -INFINITY, l = 0.f;
    for (int j = lo + warp; j < hi; j += 4) {
        const int pg = page_of(P, b, j >> P.page_shift, lane == 0), row = j & (P.page_size - 1);
        if (pg < 0) continue;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) s += q[e] * value(P.k_cache, P.k_scale, pg, row, lane + 32 * e);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= P.scale;
        if (P.softcap > 0.f) s = P.softcap * tanh_accurate(s / P.softcap);
        s *= kLog2e;
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.f : fast_exp2(m - mn), p = fast_exp2(s - mn);
        m = mn;
        l = l * a + p;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = o[e] * a + p * value(P.v_cache, P.v_scale, pg, row, lane + 32 * e);
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int e = 0; e < kPer; ++e) so[warp][lane + 32 * e] = o[e];
    __syncthreads();
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float L = 0.f, w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        w[x] = sm[x] == -INFINITY ? 0.f : fast_exp2(sm[x] - M);
        L += w[x] * sl[x];
    }
    for (int d = threadIdx.x; d < HD; d += 128) {
        float acc = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) acc += w[x] * so[x][d];
        static_cast<T*>(P.o)[qrow + d] = Elem<T>::from_f(M == -INFINITY ? 0.f : acc / L);
    }
    if (P.lse && threadIdx.x == 0)
        P.lse[((long long)b * P.H + h) * P.Lq + lq] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <bool BF16, int HD, int CACHE>
cudaError_t decode_typed(const PagedParams& p, cudaStream_t s) {
    const long long n = (long long)p.B * p.H * p.Lq;
    if (n > INT32_MAX) return cudaErrorInvalidConfiguration;
    paged_decode_kernel<BF16, HD, CACHE><<<(unsigned)n, 128, 0, s>>>(p);
    return cudaGetLastError();
}

template <bool BF16, int HD>
cudaError_t by_cache(const PagedParams& p, int cache, cudaStream_t s) {
    if (cache == CACHE_E4M3) return decode_typed<BF16, HD, CACHE_E4M3>(p, s);
    if (cache == CACHE_E5M2) return decode_typed<BF16, HD, CACHE_E5M2>(p, s);
    return decode_typed<BF16, HD, CACHE_16>(p, s);
}
template <bool BF16>
cudaError_t by_hd(const PagedParams& p, int cache, cudaStream_t s) {
    if (p.hd == 64) return by_cache<BF16, 64>(p, cache, s);
    if (p.hd == 128) return by_cache<BF16, 128>(p, cache, s);
    return by_cache<BF16, 256>(p, cache, s);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedParams& p, bool bf16, int cache, cudaStream_t s) {
    return bf16 ? by_hd<true>(p, cache, s) : by_hd<false>(p, cache, s);
}

}  // namespace attn
