// paged.cu -- the paged key/value cache's writer and its bulk reader: new keys turned by
// their position and stored with their values in the sequences' pages (and the queries
// turned beside them), and pages read back into packed 16-bit rows.
//
// Turn: pair (x[i], x[i + hd/2]) of a head vector at position p turns by p * theta^(-2i/hd)
// (the rotate-half form of rope.cu).  Far positions need more than fp32 for the angle, so
// the frequency is held in turns as a 64-bit fixed-point fraction f of one turn, and p * f
// modulo 2^64 is the angle's fraction of a turn, exact to p * 2^-64: two 32-bit multiplies
// give its upper 32 bits, which become an angle in [-pi, pi) for the hardware sine and
// cosine (absolute error below 2^-21, under the rounding to 16 or 8 bits that follows).
//
// 8-bit pages: the scale of a (page, head) block is a power of two, the smallest s with
// max|x| <= top * s over the block's rows, so that dividing by it is exact, the code is the
// only rounding, and a block whose scale grows in a later call has its earlier rows
// divided by an exact power of two (only codes that become subnormal round again).
#include <math.h>

#include "paged.cuh"

namespace attn {
namespace {

struct TurnFreqs {
    unsigned long long f[128];  // theta^(-2i/hd) / (2 pi) turns, in units of 2^-64 turns
};

TurnFreqs turn_freqs(int hd, double theta) {
    TurnFreqs t;
    for (int i = 0; i < hd / 2; ++i) {
        // at most 1 / (2 pi) of a turn for theta >= 1; a theta below 1 turns faster than once
        // a position: only the fraction of a turn counts
        const double turns = pow(theta, -2.0 * i / hd) / 6.283185307179586476925286766559;
        t.f[i] = (unsigned long long)ldexp(turns - floor(turns), 64);
    }
    return t;
}

__device__ __forceinline__ void turn_sincos(unsigned int p, unsigned long long f, float& s, float& c) {
    const unsigned int fl = (unsigned int)f, fh = (unsigned int)(f >> 32);
    const int frac = (int)(__umulhi(p, fl) + p * fh);      // upper half of p * f mod 2^64
    const float a = (float)frac * 1.46291807926715968e-9f;  // 2 pi / 2^32
    s = __sinf(a);
    c = __cosf(a);
}

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
    else return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// 8 pairs (lo[e], hi[e]) of a head vector, its elements 8c .. and hd/2 + 8c ..
struct Pairs {
    float lo[8], hi[8];
};
template <bool BF16>
__device__ __forceinline__ void load_pairs(Pairs& x, const void* base, long long elem, int half) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + elem;
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + half);
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 u = unpack16<BF16>(aw[e]), v = unpack16<BF16>(bw[e]);
        x.lo[2 * e] = u.x;
        x.lo[2 * e + 1] = u.y;
        x.hi[2 * e] = v.x;
        x.hi[2 * e + 1] = v.y;
    }
}
template <bool BF16>
__device__ __forceinline__ void store_pairs(const Pairs& x, void* base, long long elem, int half) {
    uint16_t* p = static_cast<uint16_t*>(base) + elem;
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<BF16>(x.lo[0], x.lo[1]), pack2<BF16>(x.lo[2], x.lo[3]),
                                              pack2<BF16>(x.lo[4], x.lo[5]), pack2<BF16>(x.lo[6], x.lo[7]));
    *reinterpret_cast<uint4*>(p + half) = make_uint4(pack2<BF16>(x.hi[0], x.hi[1]), pack2<BF16>(x.hi[2], x.hi[3]),
                                                     pack2<BF16>(x.hi[4], x.hi[5]), pack2<BF16>(x.hi[6], x.hi[7]));
}
__device__ __forceinline__ void turn_pairs(Pairs& x, const float (&sn)[8], const float (&cs)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float a, b;
        rope_turn(x.lo[e], x.hi[e], cs[e], sn[e], a, b);
        x.lo[e] = a;
        x.hi[e] = b;
    }
}

constexpr int kWarps = 8;  // of a CTA, here and below

// ------------------------------------------------------- rows in 16 bits
// One warp per (row, group of heads): lane l owns the 8 pairs of chunk l mod (hd/16) of
// every head it meets, so that its sines and cosines serve all of them.  The heads are the
// row's query heads (if they are turned), then, for 16-bit pages, its keys and values.
template <bool BF16, int HD>
__device__ void append_rows(const PagedParams& P, bool kv, bool turn, int steps, int row_block, int group,
                            const TurnFreqs& fr) {
    constexpr int kChunks = HD / 16, kHeads = 32 / kChunks;  // lanes of a head, heads of a step
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = row_block * kWarps + warp;
    if (r >= P.total) return;
    const RowSeq sq = row_seq(P, r);
    if (sq.b < 0) return;
    const long long pos = (long long)__ldg(P.lengths + sq.b) - (sq.end - r);
    if (pos < 0) return;  // a padding slot's row
    const int nq = P.q ? P.H : 0;
    const int pg = pos <= INT32_MAX ? page_of(P, sq.b, (int)(pos >> P.page_shift), lane == 0)
                                    : page_of(P, sq.b, -1, lane == 0);
    if (pg < 0) return;
    const int row = (int)pos & (P.page_size - 1);
    const int c = lane % kChunks;
    float sn[8], cs[8];
    if (turn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_sincos((unsigned int)pos, fr.f[c * 8 + e], sn[e], cs[e]);
    }
    const int heads = nq + (kv ? 2 * P.Hkv : 0);
#pragma unroll 4
    for (int st = 0; st < steps; ++st) {
        const int h = (group * steps + st) * kHeads + lane / kChunks;
        if (h >= heads) break;
        Pairs x;
        if (h < nq) {
            load_pairs<BF16>(x, P.q, r * P.q_stride + h * HD + c * 8, HD / 2);
            if (turn) turn_pairs(x, sn, cs);
            store_pairs<BF16>(x, P.q_out, ((long long)r * P.H + h) * HD + c * 8, HD / 2);
        } else {
            const bool is_v = h - nq >= P.Hkv;
            const int hk = h - nq - (is_v ? P.Hkv : 0);
            load_pairs<BF16>(x, is_v ? P.v : P.k, r * (is_v ? P.v_stride : P.k_stride) + hk * HD + c * 8, HD / 2);
            if (turn && !is_v) turn_pairs(x, sn, cs);
            store_pairs<BF16>(x, is_v ? P.v_cache : P.k_cache, cache_row(P, pg, hk, row) + c * 8, HD / 2);
        }
    }
}

// ------------------------------------------------------- blocks in 8 bits
// One CTA per (sequence's page, KV head, keys or values): the block's scale needs the
// largest magnitude of all its new rows before the first code can be written.
//
// The pages that a call touches are numbered without a pass over the prefix sums:
// sequence b owns the numbers cu[b]/page + 2b .. cu[b+1]/page + 2b + 1, at least as many
// as the pages that its rows can touch, so a number finds its sequence by one search.
template <bool BF16, int HD, int CACHE>
__device__ void append_block(const PagedParams& P, bool turn, int number, int head, bool is_v, const TurnFreqs& fr) {
    constexpr int kChunks = HD / 16;
    constexpr int kThreads = kWarps * 32;
    __shared__ float red[kWarps];
    const int tid = threadIdx.x, page = P.page_size;
    const int b = warp_last_le(P.B, number,
                               [&](int i) { return (long long)(__ldg(P.cu + i) >> P.page_shift) + 2 * i; });
    if (b < 0) return;
    const int first = __ldg(P.cu + b), end = __ldg(P.cu + b + 1);
    if (first < 0 || end < first || end > P.total) {
        if (tid == 0 && end != first) atomicOr(P.status, ST_PAGED_BOUNDS);
        return;
    }
    if (first == end) return;
    const long long len = __ldg(P.lengths + b);
    const long long p0 = len - (end - first);  // position of the sequence's first new row
    const long long start = p0 < 0 ? 0 : p0;
    const long long j = (start >> P.page_shift) + (number - ((first >> P.page_shift) + 2 * b));
    const long long lo = max(start, j << P.page_shift), hi = min(len, (j + 1) << P.page_shift);
    if (lo >= hi) return;
    const int pg = page_of(P, b, j <= INT32_MAX ? (int)j : -1, tid == 0);
    if (pg < 0) return;
    const int n_old = (int)(lo - (j << P.page_shift));  // rows of the page that an earlier call stored
    const int rows = (int)(hi - lo);
    const void* src = is_v ? P.v : P.k;
    const long long src_stride = is_v ? P.v_stride : P.k_stride;
    const long long src_row = first + (lo - p0);
    uint8_t* cache = static_cast<uint8_t*>(is_v ? P.v_cache : P.k_cache) + cache_row(P, pg, head, 0);
    float* scale_at = (is_v ? P.v_scale : P.k_scale) + (long long)pg * P.Hkv + head;
    const bool turned = turn && !is_v;
    (void)page;

    const int tasks = rows * kChunks;
    auto load = [&](int t, Pairs& x) {
        const int i = t / kChunks, c = t % kChunks;
        load_pairs<BF16>(x, src, (src_row + i) * src_stride + head * HD + c * 8, HD / 2);
        if (turned) {
            float sn[8], cs[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) turn_sincos((unsigned int)(lo + i), fr.f[c * 8 + e], sn[e], cs[e]);
            turn_pairs(x, sn, cs);
        }
    };
    float amax = 0.f;
    for (int t = tid; t < tasks; t += kThreads) {
        Pairs x;
        load(t, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // what is not finite has no part in the scale
            const float a = fabsf(x.lo[e]), d = fabsf(x.hi[e]);
            amax = fmaxf(amax, a < INFINITY ? a : 0.f);
            amax = fmaxf(amax, d < INFINITY ? d : 0.f);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    const float old = n_old > 0 ? *scale_at : 0.f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, red[w]);
    // smallest power of two s with amax <= 1.75 * 2^kTopExp * s, at least 2^-64
    const uint32_t bits = __float_as_uint(amax);
    int ex = (int)(bits >> 23) - 127 - F8<CACHE>::kTopExp + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    ex = max(ex, -64);
    float s = __uint_as_float((uint32_t)(ex + 127) << 23);
    if (n_old > 0) {
        if (old >= s) {
            s = old;
        } else {
            // the rows that are there, in units of the grown scale
            const float ratio = old / s;
            uint32_t* w = reinterpret_cast<uint32_t*>(cache);
            for (int i = tid; i < n_old * HD / 4; i += kThreads) {
                const uint32_t x = w[i];
                const float2 u = h2_to_f2(f8x2_to_h2<CACHE>(x & 0xffffu)), v = h2_to_f2(f8x2_to_h2<CACHE>(x >> 16));
                w[i] = f8x2_from_f<CACHE>(u.x * ratio, u.y * ratio) |
                       (f8x2_from_f<CACHE>(v.x * ratio, v.y * ratio) << 16);
            }
        }
    }
    // a scale of this library is a power of two (its inverse exact); a block that another
    // program began may have any
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0u;
    const float inv = 1.f / s;
    for (int t = tid; t < tasks; t += kThreads) {
        Pairs x;
        load(t, x);
        if (pow2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x.lo[e] *= inv, x.hi[e] *= inv;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x.lo[e] /= s, x.hi[e] /= s;
        }
        const int i = t / kChunks, c = t % kChunks;
        uint8_t* out = cache + (n_old + i) * HD + c * 8;
        auto word = [](const float* y) {
            return f8x2_from_f<CACHE>(y[0], y[1]) | (f8x2_from_f<CACHE>(y[2], y[3]) << 16);
        };
        *reinterpret_cast<uint2*>(out) = make_uint2(word(x.lo), word(x.lo + 4));
        *reinterpret_cast<uint2*>(out + HD / 2) = make_uint2(word(x.hi), word(x.hi + 4));
    }
    if (tid == 0) *scale_at = s;
}

// One launch: CTAs below row_ctas turn rows, the others store 8-bit blocks.
template <bool BF16, int HD, int CACHE>
__global__ void __launch_bounds__(kWarps * 32)
    paged_append_kernel(const PagedParams P, int turn, int steps, int groups, int row_ctas,
                        const __grid_constant__ TurnFreqs fr) {
    if ((int)blockIdx.x < row_ctas) {
        append_rows<BF16, HD>(P, CACHE == CACHE_16, turn, steps, blockIdx.x / groups, blockIdx.x % groups, fr);
    } else if constexpr (CACHE != CACHE_16) {
        const int u = blockIdx.x - row_ctas, per = 2 * P.Hkv;
        append_block<BF16, HD, CACHE>(P, turn, u / per, (u % per) >> 1, u & 1, fr);
    }
}

// --------------------------------------------------------------- reading back
// One warp per packed row.
template <bool BF16, int HD, int CACHE>
__global__ void __launch_bounds__(kWarps * 32) paged_gather_kernel(const PagedParams P) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x * kWarps + warp;
    if (r >= P.total) return;
    const RowSeq sq = row_seq(P, r);
    if (sq.b < 0) return;
    const int pos = r - sq.first;
    const int pg = page_of(P, sq.b, pos >> P.page_shift, lane == 0);
    const int row = pos & (P.page_size - 1);
    const int n = P.Hkv * HD / 8;  // 16-byte pieces of an output row
    for (int i = lane; i < 2 * n; i += 32) {
        const bool is_v = i >= n;
        const int e = (is_v ? i - n : i) * 8, h = e / HD, d = e % HD;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (pg >= 0) {
            const long long at = cache_row(P, pg, h, row) + d;
            const void* cache = is_v ? P.v_cache : P.k_cache;
            if constexpr (CACHE == CACHE_16) {
                w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + at));
            } else {
                const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at));
                const float s = __ldg((is_v ? P.v_scale : P.k_scale) + (long long)pg * P.Hkv + h);
                auto two = [&](uint32_t c) {
                    const float2 f = h2_to_f2(f8x2_to_h2<CACHE>(c));
                    return pack2<BF16>(f.x * s, f.y * s);
                };
                w = make_uint4(two(x.x & 0xffffu), two(x.x >> 16), two(x.y & 0xffffu), two(x.y >> 16));
            }
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? P.v_out : P.k_out) + (long long)r * P.Hkv * HD + e) = w;
    }
}

template <bool BF16, int HD, int CACHE>
cudaError_t append_typed(const PagedParams& p, double theta, cudaStream_t s) {
    constexpr int kHeads = 32 / (HD / 16);
    TurnFreqs fr = {};
    if (theta > 0) fr = turn_freqs(HD, theta);
    const int heads = (p.q ? p.H : 0) + (CACHE == CACHE_16 ? 2 * p.Hkv : 0);
    const long long row_blocks = (p.total + kWarps - 1) / kWarps;
    const int all = (heads + kHeads - 1) / kHeads;
    int steps = 1;
    while (steps < 4 && row_blocks * ((all + steps - 1) / steps) > 152 * 8) steps *= 2;
    const int groups = (all + steps - 1) / steps;
    const long long row_ctas = row_blocks * groups;
    long long blocks = 0;
    if (CACHE != CACHE_16) blocks = ((long long)(p.total >> p.page_shift) + 2LL * p.B) * 2 * p.Hkv;
    if (row_ctas + blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (row_ctas + blocks == 0) return cudaSuccess;
    paged_append_kernel<BF16, HD, CACHE><<<(unsigned)(row_ctas + blocks), kWarps * 32, 0, s>>>(
        p, theta > 0 ? 1 : 0, steps, groups, (int)row_ctas, fr);
    return cudaGetLastError();
}

template <bool BF16, int HD, int CACHE>
cudaError_t gather_typed(const PagedParams& p, cudaStream_t s) {
    paged_gather_kernel<BF16, HD, CACHE><<<(p.total + kWarps - 1) / kWarps, kWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename F>
cudaError_t dispatch(const PagedParams& p, bool bf16, int cache, F f) {
    auto by_cache = [&](auto b, auto h) {
        if (cache == CACHE_E4M3) return f(b, h, std::integral_constant<int, CACHE_E4M3>());
        if (cache == CACHE_E5M2) return f(b, h, std::integral_constant<int, CACHE_E5M2>());
        return f(b, h, std::integral_constant<int, CACHE_16>());
    };
    auto by_hd = [&](auto b) {
        if (p.hd == 64) return by_cache(b, std::integral_constant<int, 64>());
        if (p.hd == 128) return by_cache(b, std::integral_constant<int, 128>());
        return by_cache(b, std::integral_constant<int, 256>());
    };
    return bf16 ? by_hd(std::true_type()) : by_hd(std::false_type());
}

}  // namespace

cudaError_t launch_paged_append(const PagedParams& p, bool bf16, int cache, double theta, cudaStream_t s) {
    return dispatch(p, bf16, cache, [&](auto b, auto h, auto c) {
        return append_typed<decltype(b)::value, decltype(h)::value, decltype(c)::value>(p, theta, s);
    });
}

cudaError_t launch_paged_gather(const PagedParams& p, bool bf16, int cache, cudaStream_t s) {
    return dispatch(p, bf16, cache, [&](auto b, auto h, auto c) {
        return gather_typed<decltype(b)::value, decltype(h)::value, decltype(c)::value>(p, s);
    });
}

}  // namespace attn
