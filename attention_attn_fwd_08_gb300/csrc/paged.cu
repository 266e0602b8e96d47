// paged.cu -- the paged key/value cache's writer and its bulk reader: new keys turned by
// their position and stored with their values in the sequences' pages (and the queries
// turned beside them), and pages read back into packed 16-bit rows.
//
// Turn: pair (x[i], x[i + hd/2]) of a head vector at position p turns by p * theta^(-2i/hd)
// (the rotate-half form of rope.cu).  Far positions need more than fp32 for the angle, so
// the frequency is held in turns as a 64-bit fixed-point fraction f of one turn (right to its
// last unit), and p * f modulo 2^64 is the angle's fraction of a turn, right to p * 2^-64: two
// 32-bit multiplies give its upper 32 bits, which become an angle in [-pi, pi) in fp32 (off by
// 3e-7 at most, near pi) for the hardware sine and cosine (off by 2^-21.4 and 2^-21.2 at most, by
// their documentation): 2^-20 in all at every position, under the rounding to 16 or 8 bits that
// follows.
//
// 8-bit pages: the scale of a (page, head) block is a power of two, the smallest s with
// max|x| <= top * s over the block's rows, so that dividing by it is exact, the code is the
// only rounding, and a block whose scale grows in a later call has its earlier rows
// divided by an exact power of two (only codes that become subnormal round again).
//
// All three move bytes: each element is read and written once.  What they reach (H32/8, hd 128):
// four prompts of 2048 tokens into bf16 pages 39 us (201 MB, 5.2 TB/s; the copy rate is 6.8),
// 12288 tokens in ragged chunks into e4m3 pages 54 us (277 MB, 5.1 TB/s), 32768 e4m3 tokens read
// back as bf16 37 us (201 MB, 5.4 TB/s).  Between that and the copy rate stand about half of
// the issue slots (unpacking, turning and packing; gather 71 %) with 28 warps active on average of
// the 32 that an append's 64 registers a thread leave an SM.  At hd 256 the same chunks take 119 us
// (553 MB, 4.6 TB/s): one CTA of 1024 threads to an SM, its next head on the way.  A step of one
// token for each of 64 sequences takes 8.2 us, a launch and four dependent reads.
#include <math.h>

#include <type_traits>

#include "paged.cuh"
#include "turns.cuh"

namespace attn {
namespace {

TurnFreqs turn_freqs(int hd, double theta) {
    // hd / 2 is a power of two: theta^(-2/hd) is 1 / theta's root, that often squared
    Two r = {1 / theta, 0};
    r.lo = fma(-theta, r.hi, 1.0) / theta;
    for (int n = hd / 2; n > 1; n /= 2) r = two_sqrt(r);
    Two turns = kTurnsPerRadian;
    TurnFreqs t;
    for (int i = 0; i < hd / 2; ++i) {
        // At most 1 / (2 pi) of a turn for theta >= 1; a theta below 1 turns faster than once a
        // position (2^29.4 times for 2^-32, the least): only the fraction of a turn counts, and it
        // is right to 2^-64 still.
        t.f[i] = turn_fraction(turns);
        turns = two_mul(turns, r);
    }
    return t;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
    else return __half22float2(*reinterpret_cast<__half2*>(&w));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 8 pairs (lo[e], hi[e]) of a head vector, its elements 8c .. and hd/2 + 8c ..
struct Pairs {
    float lo[8], hi[8];
};
struct RawPairs {  // the same as loaded
    uint4 lo, hi;
};
__device__ __forceinline__ RawPairs load_raw(const void* base, long long elem, int half) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + elem;
    return RawPairs{*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + half)};
}
template <bool BF16>
__device__ __forceinline__ void unpack_pairs(Pairs& x, const RawPairs& r) {
    const uint32_t aw[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w}, bw[4] = {r.hi.x, r.hi.y, r.hi.z, r.hi.w};
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
__device__ __forceinline__ void store_raw(const RawPairs& r, void* base, long long elem, int half) {
    uint16_t* p = static_cast<uint16_t*>(base) + elem;
    *reinterpret_cast<uint4*>(p) = r.lo;
    *reinterpret_cast<uint4*>(p + half) = r.hi;
}
// (x.lo, x.hi) turned by the angles whose cosines and sines are cs and sn, as rope_turn does,
// two pairs to an instruction
__device__ __forceinline__ void turn_pairs(Pairs& x, const float (&sn)[8], const float (&cs)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t a = f2_make(x.lo[e], x.lo[e + 1]), b = f2_make(x.hi[e], x.hi[e + 1]);
        const uint64_t s = f2_make(sn[e], sn[e + 1]), c = f2_make(cs[e], cs[e + 1]), m = f2_make(-sn[e], -sn[e + 1]);
        f2_split(f2_fma(a, c, f2_mul(b, m)), x.lo[e], x.lo[e + 1]);
        f2_split(f2_fma(b, c, f2_mul(a, s)), x.hi[e], x.hi[e + 1]);
    }
}

// An append's CTA is as large as its largest team, 512 threads at least: 64 registers to a
// thread fill an SM.
constexpr int append_warps(int team) { return team > 512 ? team / 32 : 16; }
constexpr int blocks_ahead(int team) { return team > 512 ? 1 : 2; }  // heads of a team on their way: 32 KB of a CTA
constexpr int kSms = 152;

// ------------------------------------------------------- rows in 16 bits
// One warp per (row, group of heads): lane l owns the 8 pairs of chunk l mod (hd/16) of every
// head it meets.  The row's sines and cosines are formed once by the warp, each lane a few,
// and exchanged through shared memory.  The heads are the row's query heads (if they are
// turned), then, for 16-bit pages, its keys and values, kAhead at a time; the first ones are
// loaded before it is known where they go, so that the search and the page's lookup (four
// dependent reads) overlap the rows' own latency.
template <bool BF16, int HD, int kWarps>
__device__ void append_rows(uint4* smem, const PagedParams& P, bool kv, bool turn, int steps, int row_block, int group,
                            const TurnFreqs& fr) {
    constexpr int kChunks = HD / 16, kHeads = 32 / kChunks, kAhead = 2;  // lanes of a head, heads of a step
    float2 (*turns)[HD / 2 + 4] = reinterpret_cast<float2 (*)[HD / 2 + 4]>(smem);  // of each warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = row_block * kWarps + warp;
    if (r >= P.total) return;
    const int c = lane % kChunks;
    const int nq = P.q ? P.H : 0, heads = nq + (kv ? 2 * P.Hkv : 0);
    const int h0 = group * steps * kHeads + lane / kChunks, h1 = min(heads, (group + 1) * steps * kHeads);
    RawPairs raw[kAhead];
    auto load = [&](int st) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int h = h0 + (st + k) * kHeads;
            if (h >= h1) continue;
            const void* from = h < nq ? P.q : h < nq + P.Hkv ? P.k : P.v;
            const long long stride = h < nq ? P.q_stride : h < nq + P.Hkv ? P.k_stride : P.v_stride;
            const int hh = h < nq ? h : h < nq + P.Hkv ? h - nq : h - nq - P.Hkv;
            raw[k] = load_raw(from, r * stride + hh * HD + c * 8, HD / 2);
        }
    };
    load(0);
    const RowSeq sq = row_seq(P, r);
    if (sq.b < 0) return;
    const long long pos = (long long)__ldg(P.lengths + sq.b) - (sq.end - r);
    if (pos < 0) return;  // a padding slot's row
    const int pg = page_of(P, sq.b, pos <= INT32_MAX ? (int)(pos >> P.page_shift) : -1, lane == 0);
    if (pg < 0) return;
    const int row = (int)pos & (P.page_size - 1);
    float sn[8], cs[8];
    if (turn) {
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            float2 t;
            turn_sincos((unsigned int)pos, fr.f[lane + 32 * i], t.x, t.y);
            turns[warp][lane + 32 * i] = t;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float4 t = *reinterpret_cast<const float4*>(&turns[warp][c * 8 + e]);
            sn[e] = t.x, cs[e] = t.y, sn[e + 1] = t.z, cs[e + 1] = t.w;
        }
    }
    for (int st = 0; st < steps; st += kAhead) {
        if (st > 0) load(st);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int h = h0 + (st + k) * kHeads;
            if (h >= h1) continue;
            const bool is_v = h >= nq + P.Hkv;
            const int hk = h - nq - (is_v ? P.Hkv : 0);
            void* to = h < nq ? P.q_out : is_v ? P.v_cache : P.k_cache;
            const long long at = h < nq ? ((long long)r * P.H + h) * HD + c * 8 : cache_row(P, pg, hk, row) + c * 8;
            if (turn && !is_v) {
                Pairs x;
                unpack_pairs<BF16>(x, raw[k]);
                turn_pairs(x, sn, cs);
                store_pairs<BF16>(x, to, at, HD / 2);
            } else {
                store_raw(raw[k], to, at, HD / 2);
            }
        }
    }
}

// ------------------------------------------------------- blocks in 8 bits
// kTeam threads per (sequence's page, keys or values), for some KV heads one after the other:
// a head's block needs the largest magnitude of all its new rows before its first code can be
// written, and a thread's 16 elements stay in its registers from the one to the other.  A
// thread keeps its row and columns from head to head, so its sines and cosines serve them
// all, and the next heads' elements are fetched ahead.  A block of more than 16 kTeam elements
// (pages of 128 and 256 tokens with wide heads) is gone through piece by piece, twice.
//
// The pages that a call touches are numbered without a pass over the prefix sums:
// sequence b owns the numbers cu[b]/page + 2b .. cu[b+1]/page + 2b + 1, at least as many
// as the pages that its rows can touch, so a number finds its sequence by one search.
//
// A call with few rows to a sequence gives each number a warp, and leaves blocks of more than
// kFew pieces (a chunk of one sequence's prompt beside the others' single tokens) to teams of
// 512, which find them by a row (kByRow): of the rows that are the last of kFew / kChunks, one
// at least lies in such a block, and the first that does stands for it.
constexpr int kFew = 64;
template <bool BF16, int HD, int CACHE, int kTeam, bool kByRow>
__device__ void append_blocks(uint4* smem, const PagedParams& P, bool turn, int number, int head0, int head1, bool is_v,
                              const TurnFreqs& fr) {
    constexpr int kChunks = HD / 16, kStride = kFew / kChunks;
    constexpr int kWarps = append_warps(kTeam), kAhead = blocks_ahead(kTeam);
    __shared__ float red[2][kWarps];
    uint4* ring = smem;
    const int tid = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
    const int row = kByRow ? number * kStride + kStride - 1 : 0;
    const int b = kByRow ? warp_last_le(P.B + 1, row, [&](int i) { return (long long)__ldg(P.cu + i); })
                         : warp_last_le(P.B, number, [&](int i) { return (long long)(__ldg(P.cu + i) >> P.page_shift) + 2 * i; });
    if (b < 0 || b >= P.B) return;
    const int first = __ldg(P.cu + b), end = __ldg(P.cu + b + 1);
    const long long len = __ldg(P.lengths + b);
    if (first < 0 || end < first || end > P.total) {
        if (tid == 0 && end != first) atomicOr(P.status, ST_PAGED_BOUNDS);
        return;
    }
    if (first == end || (kByRow && (row < first || row >= end))) return;
    const long long p0 = len - (end - first);  // position of the sequence's first new row
    const long long start = p0 < 0 ? 0 : p0;
    const long long at = p0 + (row - first);  // of the row
    if (kByRow && at < 0) return;
    const long long j = kByRow ? at >> P.page_shift
                               : (start >> P.page_shift) + (number - ((first >> P.page_shift) + 2 * b));
    const long long lo = max(start, j << P.page_shift), hi = min(len, (j + 1) << P.page_shift);
    if (lo >= hi) return;
    if (kTeam == 32 && (hi - lo) * kChunks > kFew) return;
    if (kByRow && ((hi - lo) * kChunks <= kFew || at - lo >= kStride)) return;
    const int pg = page_of(P, b, j <= INT32_MAX ? (int)j : -1, tid == 0);
    if (pg < 0) return;
    const int n_old = (int)(lo - (j << P.page_shift));  // rows of the page that an earlier call stored
    const bool turned = turn && !is_v;
    const int tasks = (int)(hi - lo) * kChunks;  // of 16 elements each
    const bool once = tasks <= kTeam;
    const int c = tid % kChunks, pos = (int)lo + tid / kChunks;  // of the thread's first row
    const long long src_stride = is_v ? P.v_stride : P.k_stride;
    const uint16_t* src = static_cast<const uint16_t*>(is_v ? P.v : P.k) + (first + (pos - p0)) * src_stride + c * 8;

    float sn[8], cs[8];
    auto angles = [&](int t) {
        if (turned && t < tasks) {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn_sincos((unsigned int)(pos + (t - tid) / kChunks), fr.f[c * 8 + e], sn[e], cs[e]);
        }
    };
    auto fetch = [&](int h, int t, RawPairs& raw) {
        if (t < tasks) raw = load_raw(src, (t - tid) / kChunks * src_stride + h * HD, HD / 2);
    };
    // The elements of the next heads are on their way into shared memory, where a thread finds
    // only its own: what a head costs beside them (the maximum over the team, the stores) would
    // not cover their latency.
    const uint32_t mine = smem_u32(&ring[threadIdx.x]);
    auto stage = [&](int h) {
        if (tid < tasks && h < head1) {
            const uint32_t to = mine + (h & (kAhead - 1)) * (uint32_t)(2 * kWarps * 32 * 16);
            cp_async16(to, src + h * HD);
            cp_async16(to + kWarps * 32 * 16, src + h * HD + HD / 2);
        }
        cp_async_commit();
    };
    Pairs x;
    auto value = [&](int t, const RawPairs& raw) {
        if (t >= tasks) return;
        unpack_pairs<BF16>(x, raw);
        if (turned) turn_pairs(x, sn, cs);
    };
    RawPairs raw;
    if (once) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) stage(head0 + k);
    }
    angles(tid);
    for (int h = head0; h < head1; ++h) {
        if (once) {
            cp_async_wait<kAhead - 1>();
            const uint4* from = ring + (h & (kAhead - 1)) * (2 * kWarps * 32) + threadIdx.x;
            raw.lo = from[0];
            raw.hi = from[kWarps * 32];
        }
        float* scale_at = (is_v ? P.v_scale : P.k_scale) + (long long)pg * P.Hkv + h;
        const float old = n_old > 0 ? *scale_at : 0.f;
        float amax = 0.f;
        for (int t = tid; t - tid < tasks; t += kTeam) {
            if (!once) {
                fetch(h, t, raw);
                angles(t);
            }
            value(t, raw);
            if (t >= tasks) continue;
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x.lo[e]), fabsf(x.hi[e])));  // (passes NaN over)
            if (top == INFINITY) {
                // what is not finite has no part in the scale
                top = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = fabsf(x.lo[e]), d = fabsf(x.hi[e]);
                    top = fmaxf(top, fmaxf(a < INFINITY ? a : 0.f, d < INFINITY ? d : 0.f));
                }
            }
            amax = fmaxf(amax, top);
        }
        if (once) stage(h + kAhead);  // (the place that was just read)
#pragma unroll
        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if constexpr (kTeam > 32) {
            float* part = red[h & 1] + team * (kTeam / 32);
            if ((tid & 31) == 0) part[tid >> 5] = amax;
            named_bar_sync(1 + team, kTeam);
#pragma unroll
            for (int w = 0; w < kTeam / 32; ++w) amax = fmaxf(amax, part[w]);
        } else {
            __syncwarp();  // as that barrier: all lanes have read the old scale before one stores the new
        }
        // smallest power of two s with amax <= 1.75 * 2^kTopExp * s, at least 2^-64
        const uint32_t bits = __float_as_uint(amax);
        int ex = (int)(bits >> 23) - 127 - F8<CACHE>::kTopExp + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        ex = max(ex, -64);
        float s = __uint_as_float((uint32_t)(ex + 127) << 23);
        uint8_t* cache = static_cast<uint8_t*>(is_v ? P.v_cache : P.k_cache) + cache_row(P, pg, h, 0);
        if (n_old > 0) {
            if (fabsf(old) >= s) {
                s = old;  // (of either sign: another program's block)
            } else {
                // the rows that are there, in units of the grown scale
                const float ratio = old / s;
                uint32_t* w = reinterpret_cast<uint32_t*>(cache);
                for (int i = tid; i < n_old * HD / 4; i += kTeam) {
                    const uint32_t y = w[i];
                    const float2 u = h2_to_f2(f8x2_to_h2<CACHE>(y & 0xffffu)), v = h2_to_f2(f8x2_to_h2<CACHE>(y >> 16));
                    w[i] = f8x2_from_f<CACHE>(u.x * ratio, u.y * ratio) |
                           (f8x2_from_f<CACHE>(v.x * ratio, v.y * ratio) << 16);
                }
            }
        }
        // a scale of this library is a power of two (its inverse exact); a block that another
        // program began may have any
        const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0u;
        const float inv = 1.f / s;
        for (int t = tid; t < tasks; t += kTeam) {
            if (!once) {
                fetch(h, t, raw);
                angles(t);
                value(t, raw);
            }
            if (pow2) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    f2_split(f2_mul(f2_make(x.lo[e], x.lo[e + 1]), f2_make(inv, inv)), x.lo[e], x.lo[e + 1]);
                    f2_split(f2_mul(f2_make(x.hi[e], x.hi[e + 1]), f2_make(inv, inv)), x.hi[e], x.hi[e + 1]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x.lo[e] /= s, x.hi[e] /= s;
            }
            uint8_t* out = cache + (n_old + t / kChunks) * HD + c * 8;
            auto word = [](const float* y) {
                return f8x2_from_f<CACHE>(y[0], y[1]) | (f8x2_from_f<CACHE>(y[2], y[3]) << 16);
            };
            *reinterpret_cast<uint2*>(out) = make_uint2(word(x.lo), word(x.lo + 4));
            *reinterpret_cast<uint2*>(out + HD / 2) = make_uint2(word(x.hi), word(x.hi + 4));
        }
        if (tid == 0) *scale_at = s;
    }
}

// One launch: the last row_ctas CTAs turn rows, those before them store 8-bit blocks, `per`
// heads of a page's keys or values to each team (the blocks first: they take longer, and the
// rows' short CTAs fill the end; the chunks above: 53 us, the rows first 60).
template <bool BF16, int HD, int CACHE, int kTeam>
__global__ void __launch_bounds__(append_warps(kTeam) * 32, 32 / append_warps(kTeam))
    paged_append_kernel(const PagedParams P, int turn, int steps, int groups, int row_ctas, int units, int per,
                        int long_ctas, int long_per, const __grid_constant__ TurnFreqs fr) {
    constexpr int kWarps = append_warps(kTeam);
    constexpr int kTurns = kWarps * (HD / 2 + 4) / 2, kRing = CACHE == CACHE_16 ? 0 : blocks_ahead(kTeam) * 2 * kWarps * 32;
    __shared__ uint4 smem[kTurns > kRing ? kTurns : kRing];
    const int x = (int)blockIdx.x - ((int)gridDim.x - row_ctas);
    if (x >= 0) {
        append_rows<BF16, HD, kWarps>(smem, P, CACHE == CACHE_16, turn, steps, x / groups, x % groups, fr);
    } else if constexpr (CACHE != CACHE_16) {
        const bool by_row = kTeam == 32 && (int)blockIdx.x < long_ctas;
        const int u = by_row ? blockIdx.x : (blockIdx.x - long_ctas) * (kWarps * 32 / kTeam) + threadIdx.x / kTeam;
        const int n = by_row ? long_per : per, parts = (P.Hkv + n - 1) / n, which = u % (2 * parts);
        const int number = u / (2 * parts), h = (which >> 1) * n, h1 = min(P.Hkv, h + n);
        if (by_row) {
            if constexpr (kTeam == 32) append_blocks<BF16, HD, CACHE, 512, true>(smem, P, turn, number, h, h1, which & 1, fr);
        } else if (u < units) {
            append_blocks<BF16, HD, CACHE, kTeam, false>(smem, P, turn, number, h, h1, which & 1, fr);
        }
    }
}

// --------------------------------------------------------------- reading back
// One warp per packed row.
constexpr int kGatherWarps = 8;
template <bool BF16, int HD, int CACHE>
__global__ void __launch_bounds__(kGatherWarps * 32) paged_gather_kernel(const PagedParams P) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x * kGatherWarps + warp;
    if (r >= P.total) return;
    const RowSeq sq = row_seq(P, r);
    if (sq.b < 0) return;
    const int pos = r - sq.first;
    const int pg = page_of(P, sq.b, pos >> P.page_shift, lane == 0);
    const int row = pos & (P.page_size - 1);
    // Lane l owns 8 elements of every kStep-th head: the row's key heads, then its value heads,
    // kAhead of its pieces in flight.
    constexpr int kStep = 256 / HD, kAhead = 4;
    const int d = lane * 8 % HD, heads = 2 * P.Hkv;
    const long long head_at = (long long)P.page_size * HD;  // from head to head of a page
    const long long at = pg < 0 ? 0 : cache_row(P, pg, 0, row) + d, out = (long long)r * P.Hkv * HD + d;
    const long long scale_at = (long long)max(pg, 0) * P.Hkv;
#pragma unroll 1
    for (int x0 = lane * 8 / HD; x0 < heads; x0 += kStep * kAhead) {
        uint4 raw[kAhead];
        float scale[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int x = x0 + k * kStep, h = x < P.Hkv ? x : x - P.Hkv;
            if (x >= heads || pg < 0) continue;
            const void* cache = x < P.Hkv ? P.k_cache : P.v_cache;
            if constexpr (CACHE == CACHE_16) {
                raw[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + at + h * head_at));
            } else {
                const uint2 y = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at + h * head_at));
                raw[k].x = y.x, raw[k].y = y.y;
                scale[k] = __ldg((x < P.Hkv ? P.k_scale : P.v_scale) + scale_at + h);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int x = x0 + k * kStep, h = x < P.Hkv ? x : x - P.Hkv;
            if (x >= heads) continue;
            uint4 w = make_uint4(0, 0, 0, 0);  // a page outside the pool reads as zeros
            if (pg >= 0) {
                if constexpr (CACHE == CACHE_16) {
                    w = raw[k];
                } else {
                    auto two = [&](uint32_t c) {
                        const float2 f = h2_to_f2(f8x2_to_h2<CACHE>(c));
                        return pack2<BF16>(f.x * scale[k], f.y * scale[k]);
                    };
                    w = make_uint4(two(raw[k].x & 0xffffu), two(raw[k].x >> 16), two(raw[k].y & 0xffffu), two(raw[k].y >> 16));
                }
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(x < P.Hkv ? P.k_out : P.v_out) + out + h * HD) = w;
        }
    }
}

template <bool BF16, int HD, int CACHE>
cudaError_t append_typed(const PagedParams& p, double theta, cudaStream_t s) {
    constexpr int kPieces = HD / 16, kHeads = 32 / kPieces;
    TurnFreqs fr = {};
    if (theta > 0) fr = turn_freqs(HD, theta);
    const int heads = (p.q ? p.H : 0) + (CACHE == CACHE_16 ? 2 * p.Hkv : 0);
    const int tasks = p.page_size * kPieces;  // pieces of 16 elements in a page's block
    const long long numbers = (long long)(p.total >> p.page_shift) + 2LL * p.B;
    int team = 512;
    if (CACHE != CACHE_16) {
        // threads of a block: a warp where the call brings few rows to a sequence (and 512 for the
        // long blocks of such a call: one token of each of 127 sequences and 700 of another take
        // 18.5 us, with a warp to every block 32; a call without such a block pays for teams that
        // find none, one token of each of 128 10.2 against 8.2; four times as many rows to a
        // sequence would help such calls, 575 rows of 64 sequences 14 against 18 us, and cost those
        // of even chunks, 30 rows of each of 100 26 against 18), else as many as it has pieces, up to
        // 512; 1024 where
        // that spares a second pass (12288 tokens in chunks, hd 256, pages of 64: 121 against 182
        // us; hd 128, pages of 128: 63 against 67) and there are some blocks to an SM (one KV head,
        // pages of 128: 27 against 23 us)
        if ((long long)p.total * kPieces <= (long long)kFew * p.B) team = 32;
        else if (tasks <= 256) team = tasks <= 128 ? 128 : 256;
        else if (tasks == 1024 && numbers * 2 * p.Hkv >= kSms * 4LL) team = 1024;
    }
    const int warps = append_warps(team);
    const long long row_blocks = (p.total + warps - 1) / warps;
    const int all = (heads + kHeads - 1) / kHeads;
    // steps of a warp: two where that fills no more than the SMs' warps, else a row's heads in
    // equal parts of at most twelve (of four: the prompts above 41 against 39 us, the chunks 57
    // against 53)
    const int most = row_blocks * ((all + 1) / 2) > kSms * 4LL ? 12 : 2;
    const int groups = (all + most - 1) / most;
    const int steps = groups ? ((all + groups - 1) / groups + 1) / 2 * 2 : 2;  // (even: two are loaded at a time)
    const long long row_ctas = row_blocks * groups;
    long long units = 0, unit_ctas = 0, long_ctas = 0;
    int per = 1, long_per = 1;
    if (CACHE != CACHE_16) {
        // heads of a team, which share its angles and whose loads it overlaps: as many as leave
        // every SM 512 threads (the chunks with hd 64: 33 us, four times as many 37), or 1024 where
        // a CTA has them or goes through a block twice (pages of 128: 70 us, 512 threads 86)
        const long long least = kSms * (tasks > 512 ? 1024LL : 512LL);
        auto heads_of_team = [&](long long blocks, int threads) {
            int n = 1;
            while (n < 8 && n < p.Hkv && blocks * 2 * (p.Hkv / (2 * n)) * threads >= least) n *= 2;
            return n;
        };
        per = heads_of_team(numbers, team);
        if (team == 32 && tasks > kFew) {
            const long long rows = p.total / (kFew / kPieces);  // that may stand for a long block
            long_per = heads_of_team(rows, 512);
            long_ctas = rows * 2 * ((p.Hkv + long_per - 1) / long_per);
        }
        units = numbers * 2 * ((p.Hkv + per - 1) / per);
        unit_ctas = long_ctas + (units * team + warps * 32 - 1) / (warps * 32);
    }
    if (row_ctas + unit_ctas > INT32_MAX || units > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (row_ctas + unit_ctas == 0) return cudaSuccess;
    auto launch = [&](auto t) {
        paged_append_kernel<BF16, HD, CACHE, decltype(t)::value>
            <<<(unsigned)(row_ctas + unit_ctas), warps * 32, 0, s>>>(p, theta > 0 ? 1 : 0, steps, groups, (int)row_ctas,
                                                                     (int)units, per, (int)long_ctas, long_per, fr);
        return cudaGetLastError();
    };
    if constexpr (CACHE != CACHE_16) {
        if (team == 32) return launch(std::integral_constant<int, 32>());
        if (team == 128) return launch(std::integral_constant<int, 128>());
        if (team == 256) return launch(std::integral_constant<int, 256>());
        if (team == 1024) return launch(std::integral_constant<int, 1024>());
    }
    return launch(std::integral_constant<int, 512>());
}

template <bool BF16, int HD, int CACHE>
cudaError_t gather_typed(const PagedParams& p, cudaStream_t s) {
    paged_gather_kernel<BF16, HD, CACHE><<<(p.total + kGatherWarps - 1) / kGatherWarps, kGatherWarps * 32, 0, s>>>(p);
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
