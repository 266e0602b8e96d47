// paged_decode.cuh -- attention of a few query rows of each sequence over a paged cache:
// the kernels, instantiated per pool type in paged_decode_*.cu.
//
// For query row r of a (sequence, KV head) group: O = sum_j p_j v_j / sum_j p_j with
// p_j = exp(s_j - m), s_j = scale * ks * q . k_j (capped) over the visible keys, m a running
// maximum, ks and vs the scales of the key's page.
//
// Bound by HBM: every visible K and V byte is read once.  What the design does about it:
//   * The 64-key tiles of all (sequence, KV head) items are numbered in one row and dealt
//     out in equal stretches to a fixed number of CTAs that are all resident, so that
//     sequences of unlike lengths, one long sequence, or many short ones load every SM
//     alike; the numbering is made on the device from the lengths (each CTA sums them), so
//     the launch depends on none of them.  An item cut by a stretch's end leaves partial
//     (m, l, O) rows in the workspace, which paged_combine_kernel merges in a fixed order.
//   * A producer warp keeps a ring of tiles in flight (TMA, 128-byte swizzle, one box for
//     each run of a page's rows), page numbers and scales fetched 32 groups of 16 keys at a
//     time, one batch ahead, by the lanes that hold them.
//   * A team of four consumer warps (eight at hd 256) splits each tile by keys for S = Q K^T and
//     by columns of the head for O += P V (two teams of four share the tiles of many rows): the
//     probabilities go through shared memory, one barrier a tile, and no warp holds more than
//     its share of O, so that three CTAs fit an SM.
//   * p is relative to a reference of its row that the warps know alike and that moves only
//     when a score passes it by far, so that in the usual tile no maximum is exchanged and P V
//     accumulates in the products themselves; a page's vs enters as an addend of the exponent,
//     relative to the item's first.  Masked tiles, and scales too unlike for that, take a path
//     of their own with a factor for each group of 16 keys, applied in fp32.
//   * 8-bit pages: codes become fp16 in registers (exact for both types) and the products
//     run in fp16 with fp32 accumulation.  Q is brought to fp16 by a power of two for each
//     row (exact for all that matters: 2^-38 of the row's largest element is kept).  A
//     thread's 32 bits of a K fragment are four neighbouring columns, so the columns of Q
//     are stored in the order that makes the products match; for V, ldmatrix.trans moves
//     pairs of columns, and a byte permutation pairs the keys of the even and of the odd one.
// It takes (16 x 32768 tokens, H32/8, hd 128) 169 us over e4m3 pages with one query row, 0.93 of
// the measured copy rate, and 314 us over bf16 pages with four, all of it; 61 sequences of 5 to
// 9973 tokens 112 us, 0.82.  One short sequence takes 11.7 us, the merge included.
// mma.sync serves the 16 rows that a group usually has: as rows of tcgen05's M (64 at least) they
// would leave three quarters of it idle.  With 32 or 64 rows keys could be M and rows N, nothing
// idle, but 8-bit codes would go through shared memory once more; not built: 64 rows over the same
// cache take 490 us of either type, bound by the latency of a tile's chain at two warps a scheduler.
//
// Rounding: P goes into P V in 16 bits, as the tensor cores take it (half a step of each p, of the
// rows' type over 16-bit pages, of fp16 over 8-bit ones); sums, references, S and O are fp32, and l
// sums p unrounded.  Relative to 64 bits O is off by 0.0022 over the bf16 cache above, of which 0.0017
// is its own rounding to bf16, over the e4m3 one by 0.0017, over short fp16 ones by 2.6e-4 of
// which 2.1e-4 is its own.
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>

#include "paged.cuh"

namespace attn {
namespace {
namespace paged {

constexpr int kKeys = 64;                  // keys of a tile
constexpr int kSms = 152;
constexpr int kMaxCtasPerSm = 3;
constexpr int kMaxCtas = kSms * kMaxCtasPerSm;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFailed = INT32_MAX;
// p = 2^(score - ref) with ref `bias` below the largest score when it is set, and moved when a p
// would pass 2^top (half of fp16's largest value).  In bf16, whose exponent is fp32's, p stays
// at most 1, so that P V passes fp32's range no sooner than the unweighted sum of V.
template <bool kBf>
struct PRange {
    static constexpr float bias = kBf ? -9.f : 6.f, top = kBf ? 0.f : 15.f;
};
// In the usual tile p is multiplied by its group's vs / vref before it is rounded (8-bit pages): with
// that ratio at least kRatioLo, fp16's finest step (2^-24) lies 2^-24 or more below the largest p's
// product, as without a scale; with it at most kRatioHi, scores may pass the reference's by 2^4
// before the product leaves fp16's range and the reference moves.
constexpr float kRatioLo = 1.f / 64, kRatioHi = 32.f;

// Bytes of workspace: (m, l), then O, of two slots of R partial rows for each CTA (a stretch
// can begin in the middle of one item and end in the middle of another).
__host__ __device__ inline size_t ws_o_offset(int R) { return (size_t)kMaxCtas * 2 * R * 8; }
inline size_t ws_bytes(int R, int hd) { return ws_o_offset(R) + (size_t)kMaxCtas * 2 * R * hd * 4; }

template <int HD, int CACHE, int kRowTiles>
struct DecShape {
    static constexpr bool k8 = CACHE != CACHE_16;
    static constexpr int kEs = k8 ? 1 : 2;
    static constexpr int kRowBytes = HD * kEs < 128 ? HD * kEs : 128;  // of a box
    static constexpr int kBoxes = HD * kEs / kRowBytes;                // side by side
    static constexpr int kTileBytes = kKeys * HD * kEs;                // of K or of V
    static constexpr int kStageBytes = 2 * kTileBytes;
    // Teams of consumer warps that share the ring, each with half of the rows, and row tiles of
    // 16 of each team: two where one team's warps would hold too many rows' state and be too few
    // to hide their latencies (16 x 32768 tokens, hd 128, 64 rows: 490 us, one team 524 (e4m3) and
    // 517 (bf16); 32 rows, bf16: 334 against 346; e5m2, hd 256, 32 x 8192 tokens: 32 rows 142
    // against 154, 48 rows 310 against 379).  One team converts each code once, which decides for
    // 32 rows of 8-bit pages at hd 128 (222 against 357) and at hd 64 (64 rows: 586 against 693).
    static constexpr bool kSplitTwo = HD == 256 || (HD == 128 && !k8);  // with two row tiles
    static constexpr int kTeams = (HD > 64 && kRowTiles == 4) || (kSplitTwo && kRowTiles == 2) ? 2 : 1;
    static constexpr int RT = kRowTiles / kTeams;
    static constexpr int kRows = RT * 16;
    // Warps of a team; keys of a tile that each scores; 8-column products of its share of the
    // head.  At hd 256 the ring leaves room for two CTAs: eight warps each, with half a tile's
    // work, hide its latencies better than four (e5m2, 32 x 8192 tokens: 95 against 129 us); at
    // hd 128 three CTAs of four warps do (e4m3, 16 x 32768 tokens: 170 against 277 us).
    static constexpr int kW = HD == 256 && kTeams == 1 ? 8 : 4;
    static constexpr int kConsumers = kTeams * kW * 32;
    static constexpr int kThreads = kConsumers + 32;
    static constexpr int kWk = kKeys / kW, kNt = kWk / 8;
    static constexpr int kN = HD / 8 / kW;
    static constexpr int kQPitch = HD * 2 + 16;  // 16 past a multiple of 128: eight rows' chunks in eight places
    static constexpr int kPPitch = kKeys * 2 + 16;
    static constexpr int kQBytes = kRows * kQPitch;      // of a team, as the next two
    static constexpr int kPBytes = 2 * kRows * kPPitch;
    static constexpr int kMlBytes = 2 * kRows * kW * 4;  // two buffers of a number by row and warp
    static constexpr int kFixed = kTeams * (kQBytes + kPBytes + kMlBytes + kRows * 4) + 2048;  // + row scales, alignment, barriers
    // The most CTAs of an SM whose ring keeps at least three tiles each, and whose warps have the
    // registers that more row tiles need: two with more than one tile (e4m3, hd 128, 32 rows over
    // 16 x 32768 tokens: 222 us, three 256; hd 64, 64 rows: 586, three 1019), one of two teams;
    // and the ring's depth.
    static constexpr int kMost = kTeams == 2 ? 1 : RT == 1 ? 3 : 2;
    static constexpr int stages(int ctas) {
        const int s = (227 * 1024 / ctas - 1024 - kFixed - 512) / kStageBytes;
        return s > 8 ? 8 : s;
    }
    static constexpr int kCtas = kMost == 3 && stages(3) >= 3 ? 3 : kMost >= 2 && stages(2) >= 3 ? 2 : 1;
    static constexpr int kStages = stages(kCtas);
    static constexpr int kBytes = kStages * kStageBytes + kFixed;
    // Q fragments stay in registers where they take at most 32
    static constexpr bool kQReg = kW == 4 && RT * HD <= 128;
    static_assert(kStages >= 2, "ring too shallow");
};

// D = A B + 0 and D += A B, m16n8k16 with fp32 accumulation
template <bool BF16>
__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
template <bool BF16>
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four codes of a K row (neighbouring columns) as the two halves of a B fragment, and four
// codes of V (two columns of two keys, as ldmatrix.trans leaves them) as one half of the
// even column's fragment and of the odd one's.  An e5m2 code is the upper byte of its fp16.
template <int CACHE>
__device__ __forceinline__ void codes_k(uint32_t c, uint32_t& h0, uint32_t& h1) {
    if constexpr (CACHE == CACHE_E4M3)
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
            : "=r"(h0), "=r"(h1)
            : "r"(c));
    else
        h0 = __byte_perm(c, 0, 0x1404), h1 = __byte_perm(c, 0, 0x3424);
}
template <int CACHE>
__device__ __forceinline__ void codes_v(uint32_t c, uint32_t& even, uint32_t& odd) {
    if constexpr (CACHE == CACHE_E4M3) codes_k<CACHE>(__byte_perm(c, 0, 0x3120), even, odd);
    else even = __byte_perm(c, 0, 0x2404), odd = __byte_perm(c, 0, 0x3414);
}
// the maximum, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}

// Sequence b: its visible tokens, the position of its first row, and the tiles that any
// of its rows sees.
struct SeqTiles {
    int len, p0, lo, hi, t0, n;
};
__device__ __forceinline__ SeqTiles seq_tiles(const PagedParams& P, int b) {
    SeqTiles s;
    s.len = min(max(__ldg(P.lengths + b), 0), P.max_pages << P.page_shift);
    s.p0 = s.len - P.Lq;
    key_range(P.wl, P.wr, s.len, s.p0, s.len - 1, &s.lo, &s.hi);
    s.t0 = s.lo / kKeys;
    s.n = s.hi > s.lo ? (s.hi + kKeys - 1) / kKeys - s.t0 : 0;
    return s;
}

// What an item costs beside its tiles (its rows of Q, its first and last tile, its results), in
// tiles: it is dealt out as that many more at its beginning.  (61 sequences of 5 to 9973 e4m3
// tokens: 125 us without, 115 with 2, 112 with 3 or 5; 128 of 100 to 2000: 79, 68, 66, 68.)
constexpr int kItemCost = 3;
__device__ __forceinline__ int item_cost(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }

// How the items' costs are dealt out: `all` of them, `share` to a CTA.
struct Deal {
    long long all, share;
};
// Sums over all sequences, by the whole CTA (`sums`: two shared numbers to a warp; ends after a
// barrier).  `before`: the cost of one KV head of the sequences before `upto`.
__device__ __forceinline__ Deal deal_tiles(const PagedParams& P, int ctas, long long (*sums)[2], int upto,
                                           long long& before) {
    const int lane = threadIdx.x & 31;
    long long sum = 0, part = 0;
#pragma unroll 4
    for (int b = threadIdx.x; b < P.B; b += blockDim.x) {
        const int n = item_cost(seq_tiles(P, b).n);
        sum += n;
        if (b < upto) part += n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        part += __shfl_xor_sync(0xffffffffu, part, o);
    }
    if (lane == 0) sums[threadIdx.x >> 5][0] = sum, sums[threadIdx.x >> 5][1] = part;
    __syncthreads();
    Deal d;
    d.all = before = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) d.all += sums[w][0], before += sums[w][1];
    d.all *= P.Hkv;
    d.share = (d.all + ctas - 1) / ctas;
    return d;
}
// Number x < all: number `off` of the `n` of item (b, h).
struct Place {
    int b, h, off, n;
};
__device__ __forceinline__ Place place_of(const PagedParams& P, long long x) {
    const int lane = threadIdx.x & 31;
    for (int base = 0;; base += 32) {
        const int b = base + lane;
        const int n = b < P.B ? item_cost(seq_tiles(P, b).n) : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned after = __ballot_sync(0xffffffffu, incl * P.Hkv > x);
        if (after) {
            const int at = __ffs(after) - 1;
            Place p;
            p.b = base + at;
            p.n = __shfl_sync(0xffffffffu, n, at);
            const long long in = x - (__shfl_sync(0xffffffffu, incl, at) - p.n) * P.Hkv;
            p.h = (int)(in / p.n);
            p.off = (int)(in % p.n);
            return p;
        }
        x -= __shfl_sync(0xffffffffu, incl, 31) * P.Hkv;
        if (base + 32 >= P.B) return Place{0, 0, 0, 0};  // (x was not below all)
    }
}
// The stretch's part of an item of `tiles` tiles that it enters at number `off`: sets off to
// the part's first tile, takes the part's cost from `left` and returns its tiles.
__device__ __forceinline__ int stretch_tiles(int tiles, int& off, long long& left) {
    const int end = (int)min((long long)tiles + kItemCost, off + left);
    left -= end - off;
    off = max(off - kItemCost, 0);
    return max(end - kItemCost - off, 0);
}
// the next item with tiles, by the whole warp: 32 sequences at a time
__device__ __forceinline__ void next_item(const PagedParams& P, int& b, int& h) {
    if (++h < P.Hkv) return;
    h = 0;
    const int lane = threadIdx.x & 31;
    for (++b; b < P.B; b += 32) {
        const unsigned some = __ballot_sync(0xffffffffu, b + lane < P.B && seq_tiles(P, b + lane).n > 0);
        if (some) {
            b += __ffs(some) - 1;
            return;
        }
    }
}

// kBf: the rows (and 16-bit pools) are bfloat16; over 8-bit pools a run-time choice
template <int HD, int CACHE, int kRowTiles, bool kBf>
__global__ void __launch_bounds__(DecShape<HD, CACHE, kRowTiles>::kThreads, DecShape<HD, CACHE, kRowTiles>::kCtas)
    paged_split_kernel(const PagedParams P, const int rows_bf16, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV) {
    using S = DecShape<HD, CACHE, kRowTiles>;
    constexpr int RT = S::RT;
    constexpr bool k8 = S::k8;
    constexpr bool kMmaBf = !k8 && kBf;  // type of the products
    constexpr PRange<kMmaBf> kRange{};
    const bool bf = k8 ? rows_bf16 != 0 : kBf;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* qs = smem + S::kStages * S::kStageBytes;
    __shared__ __align__(8) uint64_t bars[2 * S::kStages];
    __shared__ float4 meta[S::kStages][4];  // of the tile's groups of 16 keys: ks, vs / vref, its log2, its inverse
    __shared__ float vrefs[S::kStages];
    __shared__ int there[S::kStages];  // bits 0-3: groups that were loaded; bit 4: scales out of the usual
    __shared__ int raised_by[S::kTeams][2];  // the last tile (as the CTA counts them) with a score too high; kFailed: a wait ran out
    __shared__ int abort_flag;
    __shared__ long long sums[S::kThreads / 32][2];
    const uint32_t ring = smem_u32(smem);
    auto full_bar = [&](int s) { return smem_u32(bars + s); };
    auto empty_bar = [&](int s) { return smem_u32(bars + S::kStages + s); };
    const int lane = threadIdx.x & 31;
    const int R = P.G * P.Lq;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full_bar(s), k8 ? 2 : 1);  // the tile's bytes; over 8-bit pools, its scales
            mbar_init(empty_bar(s), S::kTeams * S::kW);
        }
        abort_flag = 0;
        for (int i = 0; i < S::kTeams; ++i) raised_by[i][0] = raised_by[i][1] = 0;
        fence_barrier_init();
    }
    long long before;
    const Deal deal = deal_tiles(P, gridDim.x, sums, 0, before);  // (its barrier publishes the ring's)
    // the merging kernel's CTAs may come up from here on (all of this kernel's are running)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long first = min(deal.all, (long long)blockIdx.x * deal.share);
    long long left = min(deal.share, deal.all - first);
    Place at = {0, 0, 0, 0};
    if (left > 0) at = place_of(P, first);
    int b = at.b, h = at.h, off = at.off;

    if (threadIdx.x >= S::kConsumers) {
        // ------------------------------------------------------------- producer
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        const uint64_t pol = policy_evict_first();  // streamed once
        const int box_rows = min(P.page_size, kKeys);
        const int subs = kKeys / box_rows, groups = box_rows / 16;  // boxes down a tile, groups of a box
        // this lane's box of a tile
        const int sub = lane % subs, bx = (lane / subs) % S::kBoxes, is_v = lane / subs / S::kBoxes;
        const bool has_box = is_v < 2;
        int stage = 0, phase = 1;  // a wait on a fresh barrier's other phase returns at once
        int made = 0;              // tiles produced, up to the ring's depth
        bool ok = true;
        while (left > 0 && ok) {
            const SeqTiles sq = seq_tiles(P, b);
            const int n = stretch_tiles(sq.n, off, left);
            // group l of batch k: the 16 keys from (t0 + off) * 64 + (32 k + l) * 16 on
            const int g0 = (sq.t0 + off) * 4;
            auto page_at = [&](int batch) {
                const int g = g0 + batch * 32 + lane;
                const long long key = (long long)g * 16;
                if (batch * 8 >= n || batch * 32 + lane >= n * 4 || key >= sq.hi || key + 16 <= sq.lo) return -2;
                return page_of(P, b, (int)(key >> P.page_shift), true);
            };
            auto scales_at = [&](int pg) {
                float2 s = make_float2(0.f, 0.f);
                if constexpr (k8) {
                    if (pg >= 0) {
                        const long long i = (long long)pg * P.Hkv + h;
                        s = make_float2(__ldg(P.k_scale + i), __ldg(P.v_scale + i));
                    }
                }
                return s;
            };
            int pg = page_at(0), pg_next = page_at(1);
            float2 sc = scales_at(pg);
            float vref = 0.f;  // scale of V that the item's O is held in: its first usable one
            for (int base = 0; base < n && ok; base += 8) {
                const float2 sc_next = scales_at(pg_next);
                const int pg_after = page_at(base / 8 + 2);
                const int m = min(8, n - base);
                const unsigned have = __ballot_sync(0xffffffffu, pg >= 0);
                // a box's page: that of any of its groups that is wanted
                int box = pg;
                if (groups > 1) box = max(box, __shfl_xor_sync(0xffffffffu, box, 1));
                if (groups > 2) box = max(box, __shfl_xor_sync(0xffffffffu, box, 2));
                float4 mine = make_float4(0.f, 0.f, 0.f, 0.f);
                unsigned odd = 0;
                for (int i = 0; i < m; ++i) {
                    const int s = stage;
                    if (!warp_wait(empty_bar(s), phase, P.status, ST_DEC_WAIT, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const int page = __shfl_sync(0xffffffffu, box, i * 4 + sub * groups);
                    const unsigned boxes = __ballot_sync(0xffffffffu, has_box && page >= 0);
                    if (lane == 0) {
                        if constexpr (!k8) there[s] = (int)(have >> (4 * i) & 0xfu);
                        mbar_expect_tx(full_bar(s), (uint32_t)(__popc(boxes) * box_rows * S::kRowBytes));
                    }
                    __syncwarp();
                    if (has_box && page >= 0) {
                        const uint32_t dst = ring + (uint32_t)(s * S::kStageBytes + is_v * S::kTileBytes +
                                                               bx * kKeys * S::kRowBytes + sub * box_rows * S::kRowBytes);
                        const int row = ((sq.t0 + off + base + i) * kKeys + sub * box_rows) & (P.page_size - 1);
                        const int y = ((page * P.Hkv + h) << P.page_shift) + row;
                        tma_load_2d(dst, is_v ? &tmV : &tmK, full_bar(s), bx * (S::kRowBytes / S::kEs), y, pol);
                    }
                    if constexpr (k8) {
                        if (i == 0) {  // the batch's scales, needed only now
                            if (vref == 0.f) {
                                // (from 2^-30 on: with a scale of 2^40 elsewhere and 2^31 codes of 2^16, times 2^6
                                // for p, the sums in its units stay below 2^123)
                                const unsigned fit = __ballot_sync(0xffffffffu, pg >= 0 && sc.y >= 0x1p-30f && sc.y < 1e18f);
                                vref = fit ? __shfl_sync(0xffffffffu, sc.y, __ffs(fit) - 1) : 1.f;
                            }
                            const float ratio = sc.y / vref;
                            // (a scale of 0, as of a block of zeros, has no logarithm: not the usual)
                            const bool usual = pg < 0 || (sc.x > 0.f && sc.x < 1e30f && ratio >= kRatioLo && ratio <= kRatioHi);
                            odd = __ballot_sync(0xffffffffu, !usual);
                            mine = pg < 0 ? make_float4(1.f, 1.f, 0.f, 1.f)
                                          : make_float4(sc.x, ratio, usual ? __log2f(ratio) : 0.f, 1.f / ratio);
                        }
                        if ((lane >> 2) == i) meta[s][lane & 3] = mine;
                        if (lane == 0) {
                            vrefs[s] = vref;
                            there[s] = (int)((have >> (4 * i) & 0xfu) | ((odd >> (4 * i) & 0xfu) ? 16u : 0u));
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full_bar(s));
                    }
                    made = min(made + 1, S::kStages);
                    if (++stage == S::kStages) stage = 0, phase ^= 1;
                }
                pg = pg_next;
                sc = sc_next;
                pg_next = pg_after;
            }
            off = 0;
            if (left > 0) next_item(P, b, h);
        }
        // no copy is in flight when the CTA ends
        for (int i = 0; i < made; ++i) {
            if (--stage < 0) stage = S::kStages - 1, phase ^= 1;
            mbar_wait(full_bar(stage), phase ^ 1, P.status, ST_DEC_WAIT | ST_TEARDOWN, nullptr);
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3, mi = lane >> 3, ri = lane & 7;
    const int team = threadIdx.x / (S::kW * 32), warp = (threadIdx.x >> 5) % S::kW;  // warp of its team
    const int row0 = team * S::kRows, bar = 1 + team;  // its first row, its barrier
    qs += team * S::kQBytes;
    uint8_t* ps = smem + S::kStages * S::kStageBytes + S::kTeams * S::kQBytes + team * S::kPBytes;
    float* maxima = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes + S::kTeams * (S::kQBytes + S::kPBytes) +
                                             team * S::kMlBytes);  // [2][rows][warps]
    float* qscale = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes +
                                             S::kTeams * (S::kQBytes + S::kPBytes + S::kMlBytes)) + row0;  // [rows]
    int* raised = raised_by[team];
    float2* ws_ml = reinterpret_cast<float2*>(P.ws);
    float* ws_o = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(P.ws) + ws_o_offset(R));
    int stage = 0, phase = 0, tiles = 0;
    bool failed = false;
    float vref = 1.f;
    // this thread's places in a tile: its K row's chunk, its V rows' chunks, its rows of P
    constexpr int kBoxBytes = kKeys * S::kRowBytes;
    auto chunk = [&](int row, int c) -> uint32_t {  // of 16 bytes, as the swizzle lays them
        if constexpr (S::kRowBytes == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
        else return (c >> 3) * kBoxBytes + sw128(row, c & 7);
    };
    // (4 warps: 16 keys by two chunks at a time; 8 warps: 8 keys by four)
    const uint32_t k_off = S::kNt == 2 ? chunk(warp * 16 + (mi & 1) * 8 + ri, mi >> 1) : chunk(warp * 8 + ri, mi);
    constexpr int kVc = k8 ? 16 : 8;  // columns of a chunk of V
    uint32_t v_off[S::kN / 2];
#pragma unroll
    for (int c = 0; c < S::kN; c += 2) {
        const int first = (warp * S::kN + c) * 8 / kVc;
        v_off[c / 2] = S::kTileBytes + (k8 ? chunk(mi * 8 + ri, first) : chunk((mi & 1) * 8 + ri, first + (mi >> 1)));
    }
    uint8_t* p_out = ps + g * S::kPPitch + (warp * S::kWk + 2 * t) * 2;
    const float cap_inv = P.softcap > 0.f ? 1.f / P.softcap : 0.f;
    while (left > 0) {
        const SeqTiles sq = seq_tiles(P, b);
        const int n = stretch_tiles(sq.n, off, left);
        if (n == 0) break;  // (the stretch ends before the item's first tile)
        // ---- Q of the group into shared memory: row r is (head r / Lq, query row r % Lq)
        constexpr int kPer = HD / 64;  // pairs of a lane
        uint32_t qw[S::kRows / S::kW][kPer];
#pragma unroll
        for (int i = 0; i < S::kRows / S::kW; ++i) {
            const int r = row0 + warp + S::kW * i, gg = r / P.Lq, lq = r - gg * P.Lq;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                static_cast<const uint16_t*>(P.q) + (((long long)b * P.Lq + lq) * P.H + h * P.G + gg) * HD);
#pragma unroll
            for (int e = 0; e < kPer; ++e) qw[i][e] = r < R ? __ldg(src + lane + 32 * e) : 0u;
        }
        named_bar_sync(bar, S::kW * 32);  // no warp reads the last item's rows any more
#pragma unroll
        for (int i = 0; i < S::kRows / S::kW; ++i) {
            const int r = warp + S::kW * i;
            uint32_t (&w)[kPer] = qw[i];
            if constexpr (k8) {
                // to fp16 by a power of two that brings the row's largest element to 2^13 .. 2^14
                float2 f[kPer];
                float big = 0.f;
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    f[e] = bf ? __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w[e])) : h2_to_f2(w[e]);
                    big = max_nan(big, max_nan(fabsf(f[e].x), fabsf(f[e].y)));
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
                int ex = (int)(__float_as_uint(big) >> 23) - 127;
                ex = big > 0.f && big < INFINITY ? max(ex, -100) : 13;
                const float mul = __uint_as_float((uint32_t)(13 - ex + 127) << 23);
                if (lane == 0) qscale[r] = __uint_as_float((uint32_t)(ex - 13 + 127) << 23);
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    // columns 4c .. 4c+3 of each 16 go where a fragment's thread c finds them
                    const int c = 2 * (lane + 32 * e), in = c & 15;
                    const int at = (c & ~15) + 2 * (in >> 2) + ((in & 2) ? 8 : 0);
                    *reinterpret_cast<uint32_t*>(qs + r * S::kQPitch + at * 2) = pack2<false>(f[e].x * mul, f[e].y * mul);
                }
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    *reinterpret_cast<uint32_t*>(qs + r * S::kQPitch + 4 * (lane + 32 * e)) = w[e];
            }
        }
        named_bar_sync(bar, S::kW * 32);
        const uint32_t qaddr = smem_u32(qs) + ((mi & 1) * 8 + ri) * S::kQPitch + (mi >> 1) * 16;
        uint32_t qa[S::kQReg ? RT : 1][S::kQReg ? HD / 16 : 1][4];
        if constexpr (S::kQReg) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks)
                    ldsm_x4(qaddr + rt * 16 * S::kQPitch + ks * 32, qa[rt][ks][0], qa[rt][ks][1], qa[rt][ks][2],
                            qa[rt][ks][3]);
        }
        // this thread's rows 16 rt + g (e < 2) and + 8: visible keys [vlo, vhi), score factor
        int vlo[RT][2], vhi[RT][2];
        float qf[RT][2], ref[RT][2];  // and the reference: p = 2^(score - ref)
        float o[RT][S::kN][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int in = rt * 16 + g + 8 * e, r = row0 + in, pos = sq.p0 + r % P.Lq;
                vlo[rt][e] = r < R && P.wl >= 0 ? max(0, pos - P.wl) : 0;
                vhi[rt][e] = r < R && P.wr >= 0 ? (int)min((long long)sq.len, (long long)pos + P.wr + 1) : sq.len;
                qf[rt][e] = P.scale * (k8 ? qscale[in] : 1.f) * (P.softcap > 0.f ? 1.f : kLog2e);
                ref[rt][e] = -INFINITY;
            }
        // tiles from full_lo to full_hi on are seen whole by every row (tile_full over j0)
        const int full_lo = P.wl >= 0 ? max(0, sq.len - 1 - P.wl) : 0;
        const int full_hi = (P.wr >= 0 ? (int)min((long long)sq.len, (long long)sq.p0 + P.wr + 1) : sq.len) - kKeys;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < S::kN; ++i) o[rt][i][0] = o[rt][i][1] = o[rt][i][2] = o[rt][i][3] = 0.f;

        float l[RT][2];  // this thread's part of the sums
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) l[rt][0] = l[rt][1] = 0.f;

        for (int i = 0; i < n; ++i) {
            // A warp whose wait ran out says so before the tile's first barrier, and all stop there
            // (another way and some would wait at a barrier that the others never reach).
            if (!warp_wait(full_bar(stage), phase, P.status, ST_DEC_WAIT, &abort_flag)) atomicMax(&raised[i & 1], kFailed);
            const int j0 = (sq.t0 + off + i) * kKeys, have = there[stage], buf = i & 1;
            const uint32_t base = ring + (uint32_t)(stage * S::kStageBytes);
            if (k8 && i == 0) vref = vrefs[stage];

            // ---- S = Q K^T for this warp's keys, 8 to a column tile
            // (one row tile alone: the even and the odd steps' products apart, for shorter chains)
            constexpr int kNt = S::kNt, kChains = RT == 1 ? 2 : 1;
            float sc[RT][kNt][4], odd[kNt][4];
#pragma unroll
            for (int x = 0; x < kNt; ++x) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) sc[rt][x][0] = sc[rt][x][1] = sc[rt][x][2] = sc[rt][x][3] = 0.f;
                odd[x][0] = odd[x][1] = odd[x][2] = odd[x][3] = 0.f;
            }
            const uint32_t kt = base + k_off;
            // steps of 16 columns that one ldmatrix.x4 (8-bit) or kNt of them (16-bit) serve
            constexpr int kStep = kNt == 2 || !k8 ? 2 : 4;
#pragma unroll
            for (int ks = 0; ks < HD / 16; ks += kStep) {
                uint32_t kb[kStep][kNt][2];  // [step][column tile][fragment half]
                if constexpr (k8) {
                    uint32_t r[4];
                    ldsm_x4((kt ^ ((ks & 7) << 4)) + (ks >> 3) * kBoxBytes, r[0], r[1], r[2], r[3]);
#pragma unroll
                    for (int x = 0; x < kStep; ++x)
#pragma unroll
                        for (int y = 0; y < kNt; ++y) codes_k<CACHE>(r[x * kNt + y], kb[x][y][0], kb[x][y][1]);
                } else if constexpr (kNt == 2) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int c = 2 * (ks + x);
                        ldsm_x4((kt ^ ((c & 7) << 4)) + (c >> 3) * kBoxBytes, kb[x][0][0], kb[x][1][0], kb[x][0][1],
                                kb[x][1][1]);
                    }
                } else {
                    const int c = 2 * ks;
                    ldsm_x4((kt ^ ((c & 7) << 4)) + (c >> 3) * kBoxBytes, kb[0][0][0], kb[0][0][1], kb[1][0][0],
                            kb[1][0][1]);
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int x = 0; x < kStep; ++x) {
                        uint32_t a[4];
                        if constexpr (S::kQReg) {
                            a[0] = qa[rt][ks + x][0], a[1] = qa[rt][ks + x][1], a[2] = qa[rt][ks + x][2],
                            a[3] = qa[rt][ks + x][3];
                        } else {
                            ldsm_x4(qaddr + rt * 16 * S::kQPitch + (ks + x) * 32, a[0], a[1], a[2], a[3]);
                        }
#pragma unroll
                        for (int y = 0; y < kNt; ++y) {
                            if (kChains == 2 && (x & 1)) mma_add<kMmaBf>(odd[y], a, kb[x][y][0], kb[x][y][1]);
                            else mma_add<kMmaBf>(sc[rt][y], a, kb[x][y][0], kb[x][y][1]);
                        }
                    }
            }
            if constexpr (kChains == 2) {
#pragma unroll
                for (int x = 0; x < kNt; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[0][x][e] += odd[x][e];
            }

            const int grp = warp * S::kWk / 16;               // the group of 16 keys that they lie in
            float4 own = make_float4(1.f, 1.f, 0.f, 1.f);  // its ks, vs / vref, the log2 of that, its inverse
            if constexpr (k8) own = meta[stage][grp];
            // the score in log2 units, before any mask
            auto score = [&](float raw, float c) {
                const float y = raw * c;
                return P.softcap > 0.f ? P.softcap * tanh_accurate(y * cap_inv) * kLog2e : y;
            };
            auto group_maxima = [&](const float* of_row, float (&mw)[4]) {
                const float4 u = *reinterpret_cast<const float4*>(of_row);
                if constexpr (S::kW == 4) {
                    mw[0] = u.x, mw[1] = u.y, mw[2] = u.z, mw[3] = u.w;
                } else {
                    const float4 v = *reinterpret_cast<const float4*>(of_row + 4);
                    mw[0] = max_nan(u.x, u.y), mw[1] = max_nan(u.z, u.w), mw[2] = max_nan(v.x, v.y), mw[3] = max_nan(v.z, v.w);
                }
            };
            const uint32_t paddr = smem_u32(ps) + (buf * S::kRows + (mi & 1) * 8 + ri) * S::kPPitch + (mi >> 1) * 16;
            uint8_t* p_to = p_out + buf * S::kRows * S::kPPitch;
            auto load_v = [&](int kp, int c, uint32_t (&vb)[2][2][2]) {  // [group][8-column product][fragment half]
                if constexpr (k8) {
                    // 16 columns: even ones are product c, odd ones c + 1
                    uint32_t r[2][2];
                    ldsm_x4_t(base + v_off[c / 2] + kp * 16 * S::kRowBytes, r[0][0], r[0][1], r[1][0], r[1][1]);
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int z = 0; z < 2; ++z) codes_v<CACHE>(r[y][z], vb[y][0][z], vb[y][1][z]);
                } else {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        ldsm_x4_t(base + v_off[c / 2] + (kp + y) * 16 * S::kRowBytes, vb[y][0][0], vb[y][0][1],
                                  vb[y][1][0], vb[y][1][1]);
                }
            };

            // ---- the usual tile: seen whole by every row, scales near the item's first, and no
            // score so far above the rows' references that p would leave fp16's range
            bool done = false;
            ++tiles;
            const bool unmasked = (have & 0xf) == 0xf && j0 >= full_lo && j0 <= full_hi;
            const bool usual = have == 0xf && unmasked;
            if (usual) {
                if (i == 0) {
                    // nothing is summed yet: the rows' references from this tile's maxima
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float c = qf[rt][r] * own.x;
                            float m = score(sc[rt][0][2 * r], c);
#pragma unroll
                            for (int e = 1; e < 2 * kNt; ++e) m = max_nan(m, score(sc[rt][e >> 1][2 * r + (e & 1)], c));
                            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
                            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
                            if (t == 0) maxima[(buf * S::kRows + rt * 16 + g + 8 * r) * S::kW + warp] = m;
                        }
                    named_bar_sync(bar, S::kW * 32);
                    if ((failed = raised[buf] == kFailed)) break;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float mw[4];
                            group_maxima(maxima + (buf * S::kRows + rt * 16 + g + 8 * r) * S::kW, mw);
                            ref[rt][r] = max_nan(max_nan(mw[0], mw[1]), max_nan(mw[2], mw[3])) - kRange.bias;
                        }
                }
                float part[RT][2];
                bool high = false;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float c = qf[rt][r] * own.x, shift = own.z - ref[rt][r];
                        float y[2 * kNt];
#pragma unroll
                        for (int e = 0; e < 2 * kNt; ++e) {
                            const float raw = sc[rt][e >> 1][2 * r + (e & 1)];
                            y[e] = P.softcap > 0.f ? score(raw, c) + shift : fmaf(raw, c, shift);
                            high |= !(y[e] <= kRange.top);
                        }
                        uint8_t* to = p_to + (rt * 16 + 8 * r) * S::kPPitch;
                        const float p0 = fast_exp2(y[0]), p1 = fast_exp2(y[1]);
                        *reinterpret_cast<uint32_t*>(to) = pack2<kMmaBf>(p0, p1);
                        part[rt][r] = p0 + p1;
                        if constexpr (kNt == 2) {
                            const float p2 = fast_exp2(y[2]), p3 = fast_exp2(y[3]);
                            *reinterpret_cast<uint32_t*>(to + 16) = pack2<kMmaBf>(p2, p3);
                            part[rt][r] += p2 + p3;
                        }
                    }
                if (high) atomicMax(&raised[buf], tiles);
                named_bar_sync(bar, S::kW * 32);
                const int last = raised[buf];
                done = last < tiles;
                if ((failed = last == kFailed)) break;
                if (done) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        l[rt][0] = fmaf(part[rt][0], own.w, l[rt][0]);
                        l[rt][1] = fmaf(part[rt][1], own.w, l[rt][1]);
                    }
#pragma unroll
                    for (int kp = 0; kp < 4; kp += 2) {
                        uint32_t pa[2][RT][4];
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                ldsm_x4(paddr + rt * 16 * S::kPPitch + (kp + y) * 32, pa[y][rt][0], pa[y][rt][1],
                                        pa[y][rt][2], pa[y][rt][3]);
                        // all columns of one group, then of the other: a sum waits for no product before its own
                        uint32_t vb[S::kN / 2][2][2][2];
#pragma unroll
                        for (int c = 0; c < S::kN; c += 2) load_v(kp, c, vb[c / 2]);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int c = 0; c < S::kN; c += 2)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
#pragma unroll
                                    for (int rt = 0; rt < RT; ++rt)
                                        mma_add<kMmaBf>(o[rt][c + x], pa[y][rt], vb[c / 2][y][x][0], vb[c / 2][y][x][1]);
                    }
                }
            }

            // ---- any other tile: masks, a new reference, a factor for each group of 16 keys
            if (!done) {
                float mx[RT][2];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        mx[rt][r] = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 2 * kNt; ++e) {
                            float& y = sc[rt][e >> 1][2 * r + (e & 1)];
                            y = score(y, qf[rt][r] * own.x);
                            const int j = j0 + warp * S::kWk + (e >> 1) * 8 + 2 * t + (e & 1);
                            if (!unmasked && (j < vlo[rt][r] || j >= vhi[rt][r] || !((have >> grp) & 1))) y = -INFINITY;
                            mx[rt][r] = max_nan(mx[rt][r], y);
                        }
                        mx[rt][r] = max_nan(mx[rt][r], __shfl_xor_sync(0xffffffffu, mx[rt][r], 1));
                        mx[rt][r] = max_nan(mx[rt][r], __shfl_xor_sync(0xffffffffu, mx[rt][r], 2));
                        if (t == 0) maxima[(buf * S::kRows + rt * 16 + g + 8 * r) * S::kW + warp] = mx[rt][r];
                    }
                if constexpr (kNt == 1) {  // two warps to a group
                    named_bar_sync(bar, S::kW * 32);
                    if ((failed = raised[buf] == kFailed)) break;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            mx[rt][r] = max_nan(mx[rt][r], maxima[(buf * S::kRows + rt * 16 + g + 8 * r) * S::kW + (warp ^ 1)]);
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        // p relative to the group's own maximum
                        const float to0 = mx[rt][r] == -INFINITY ? 0.f : mx[rt][r];
                        float p[2 * kNt];
#pragma unroll
                        for (int e = 0; e < 2 * kNt; ++e) p[e] = fast_exp2(sc[rt][e >> 1][2 * r + (e & 1)] - to0);
                        uint8_t* to = p_to + (rt * 16 + 8 * r) * S::kPPitch;
                        *reinterpret_cast<uint32_t*>(to) = pack2<kMmaBf>(p[0], p[1]);
                        sc[rt][0][2 * r] = p[0] + p[1];
                        if constexpr (kNt == 2) {
                            *reinterpret_cast<uint32_t*>(to + 16) = pack2<kMmaBf>(p[2], p[3]);
                            sc[rt][0][2 * r] += p[2] + p[3];
                        }
                    }
                named_bar_sync(bar, S::kW * 32);
                if ((failed = raised[buf] == kFailed)) break;
                float f[RT][2][4];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float mw[4];
                        group_maxima(maxima + (buf * S::kRows + rt * 16 + g + 8 * r) * S::kW, mw);
                        const float top = max_nan(max_nan(mw[0], mw[1]), max_nan(mw[2], mw[3])) - kRange.bias;
                        const float next = max_nan(ref[rt][r], top), to0 = next == -INFINITY ? 0.f : next;
                        const float alpha = fast_exp2(ref[rt][r] - to0);  // 0 before the row's first key
                        ref[rt][r] = next;
                        l[rt][r] = fmaf(fast_exp2(mx[rt][r] - to0), sc[rt][0][2 * r], l[rt][r] * alpha);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            // a row that sees none of the group takes nothing of it, whatever its scale
                            f[rt][r][w] = fast_exp2(mw[w] - to0);
                            if constexpr (k8) f[rt][r][w] = mw[w] == -INFINITY ? 0.f : f[rt][r][w] * meta[stage][w].y;
                        }
#pragma unroll
                        for (int c = 0; c < S::kN; ++c) o[rt][c][2 * r] *= alpha, o[rt][c][2 * r + 1] *= alpha;
                    }
                // Keys that no row sees may hold any bytes: they are masked out of V.  A value
                // that is not finite may be seen by one row and not by another, whose P of 0 would
                // not keep it out of a product: such a tile goes through one key of each group at a
                // time, and a row takes the products of the keys that it sees.
                auto keep_of = [&](int k, int y) {  // halves of group y's fragment words: keys k + 2t, k + 2t + 1
                    const int j = j0 + y * 16 + k + 2 * t;
                    const bool in = (have >> y) & 1;
                    return (in && j >= sq.lo && j < sq.hi ? 0xffffu : 0u) |
                           (in && j + 1 >= sq.lo && j + 1 < sq.hi ? 0xffff0000u : 0u);
                };
                bool wild = false;
#pragma unroll 1
                for (int kp = unmasked || P.Lq == 1 ? 4 : 0; kp < 4; kp += 2) {  // (rows of one position see alike)
                    const uint32_t keep[2][2] = {{keep_of(0, kp), keep_of(8, kp)}, {keep_of(0, kp + 1), keep_of(8, kp + 1)}};
#pragma unroll
                    for (int c = 0; c < S::kN; c += 2) {
                        uint32_t vb[2][2][2];
                        load_v(kp, c, vb);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    constexpr uint32_t kInf = kMmaBf ? 0x7f80u : 0x7c00u;
                                    const uint32_t w = vb[y][x][z] & keep[y][z];
                                    wild |= (w & kInf) == kInf || ((w >> 16) & kInf) == kInf;
                                }
                    }
                }
                wild = __any_sync(0xffffffffu, wild);
#pragma unroll 1
                for (int k = wild ? 0 : 16; k < (wild ? 16 : 17); ++k) {
                    // k = 16: all keys at once; below: key k of each group
                    const uint32_t one = (k & 1) ? 0xffff0000u : 0xffffu;
                    const uint32_t lo8 = k == 16 ? 0xffffffffu : (k < 8 && (k >> 1) == t ? one : 0u);
                    const uint32_t hi8 = k == 16 ? 0xffffffffu : (k >= 8 && ((k - 8) >> 1) == t ? one : 0u);
#pragma unroll
                    for (int kp = 0; kp < 4; kp += 2) {
                        uint32_t pa[2][RT][4];
                        bool takes[2][RT][2];
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) {
                                ldsm_x4(paddr + rt * 16 * S::kPPitch + (kp + y) * 32, pa[y][rt][0], pa[y][rt][1],
                                        pa[y][rt][2], pa[y][rt][3]);
                                const int j = j0 + (kp + y) * 16 + k;
#pragma unroll
                                for (int r = 0; r < 2; ++r) takes[y][rt][r] = k == 16 || (j >= vlo[rt][r] && j < vhi[rt][r]);
                            }
                        const uint32_t keep[2][2] = {{keep_of(0, kp) & lo8, keep_of(8, kp) & hi8},
                                                     {keep_of(0, kp + 1) & lo8, keep_of(8, kp + 1) & hi8}};
#pragma unroll
                        for (int c = 0; c < S::kN; c += 2) {
                            uint32_t vb[2][2][2];
                            load_v(kp, c, vb);
#pragma unroll
                            for (int y = 0; y < 2; ++y)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
#pragma unroll
                                    for (int rt = 0; rt < RT; ++rt) {
                                        float d[4];
                                        mma_zero<kMmaBf>(d, pa[y][rt], vb[y][x][0] & keep[y][0], vb[y][x][1] & keep[y][1]);
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (takes[y][rt][e >> 1])
                                                o[rt][c + x][e] = fmaf(f[rt][e >> 1][kp + y], d[e], o[rt][c + x][e]);
                                    }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar(stage));
            if (++stage == S::kStages) stage = 0, phase ^= 1;
        }

        if (failed) break;

        // ---- the rows' sums: a row's quad, then the warps
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[rt][r] += __shfl_xor_sync(0xffffffffu, l[rt][r], 1);
                l[rt][r] += __shfl_xor_sync(0xffffffffu, l[rt][r], 2);
                // (the half of the buffers that the last tile did not use)
                if (t == 0) maxima[(((n & 1) * S::kRows) + rt * 16 + g + 8 * r) * S::kW + warp] = l[rt][r];
            }
        named_bar_sync(bar, S::kW * 32);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float4* u =
                    reinterpret_cast<const float4*>(maxima + (((n & 1) * S::kRows) + rt * 16 + g + 8 * r) * S::kW);
                l[rt][r] = 0.f;
#pragma unroll
                for (int w = 0; w < S::kW / 4; ++w) l[rt][r] += (u[w].x + u[w].y) + (u[w].z + u[w].w);
            }

        // ---- the item's rows, whole or partial
        const bool begins = off == 0, ends = off + n == sq.n;
        const bool whole = begins && ends;
        const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row0 + rt * 16 + g + 8 * e;
                if (r >= R) continue;
                const int gg = r / P.Lq, lq = r - gg * P.Lq;
                const int hq = h * P.G + gg;
                const bool none = ref[rt][e] == -INFINITY;
                // O / vref in units of 2^ref, l in units of 2^ref
                const float mul = whole ? (none ? 0.f : vref / l[rt][e]) : vref;
                uint16_t* od = static_cast<uint16_t*>(P.o) + (((long long)b * P.Lq + lq) * P.H + hq) * HD;
                float* wd = ws_o + ((long long)slot * R + r) * HD;
                auto two = [&](float x, float y) { return bf ? pack2<true>(x, y) : pack2<false>(x, y); };
                if constexpr (k8) {
#pragma unroll
                    for (int c = 0; c < S::kN; c += 2) {
                        const int d = (warp * S::kN + c) * 8 + 4 * t;
                        const float x0 = o[rt][c][2 * e] * mul, x1 = o[rt][c + 1][2 * e] * mul,
                                    x2 = o[rt][c][2 * e + 1] * mul, x3 = o[rt][c + 1][2 * e + 1] * mul;
                        if (whole) *reinterpret_cast<uint2*>(od + d) = make_uint2(two(x0, x1), two(x2, x3));
                        else *reinterpret_cast<float4*>(wd + d) = make_float4(x0, x1, x2, x3);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < S::kN; ++c) {
                        const int d = (warp * S::kN + c) * 8 + 2 * t;
                        const float x0 = o[rt][c][2 * e] * mul, x1 = o[rt][c][2 * e + 1] * mul;
                        if (whole) *reinterpret_cast<uint32_t*>(od + d) = two(x0, x1);
                        else *reinterpret_cast<float2*>(wd + d) = make_float2(x0, x1);
                    }
                }
                if (warp == 0 && t == 0) {
                    if (whole) {
                        if (P.lse)
                            P.lse[((long long)b * P.H + hq) * P.Lq + lq] =
                                none ? -INFINITY : (ref[rt][e] + log2f(l[rt][e])) * 0.6931471805599453f;
                    } else {
                        ws_ml[(long long)slot * R + r] = make_float2(ref[rt][e], l[rt][e]);
                    }
                }
            }
        off = 0;
        if (left > 0) next_item(P, b, h);
    }

    // sequences of which no row sees a key
    for (int e = blockIdx.x; e < P.B; e += gridDim.x) {
        if (threadIdx.x == 0 && __ldg(P.lengths + e) > (P.max_pages << P.page_shift)) atomicOr(P.status, ST_PAGED_BOUNDS);
        if (seq_tiles(P, e).n > 0) continue;
        uint4* od = reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.o) + (long long)e * P.Lq * P.H * HD);
        for (int i = threadIdx.x; i < P.Lq * P.H * HD / 8; i += S::kConsumers) od[i] = make_uint4(0, 0, 0, 0);
        if (P.lse)
            for (int i = threadIdx.x; i < P.Lq * P.H; i += S::kConsumers) P.lse[(long long)e * P.Lq * P.H + i] = -INFINITY;
    }
}

// Merges the partial rows of the items that stretches cut: CTA (x, y) those of the item
// that begins in stretch x and does not end in it (by_item: of item x; there are then no
// more items than stretches), rows_per_cta rows of it, several warps to a row.  It finds its item from the lengths while the split kernel still runs.  The
// order of the sums is that of the stretches.
template <int HD>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams P, const int rows_bf16, const int ctas,
                                                            const int by_item, const int rows_per_cta) {
    constexpr int kPer = HD / 32;  // columns of a lane
    __shared__ float part[8][HD];
    __shared__ long long sums[8][2];
    int b, h, cta;      // the item, and the stretch that it begins in
    int n = 0;          // its parts: that stretch's end, and the beginnings of the next ones
    long long before;
    const Deal deal = deal_tiles(P, ctas, sums, by_item ? blockIdx.x / P.Hkv : 0, before);
    if (by_item) {
        b = blockIdx.x / P.Hkv, h = blockIdx.x % P.Hkv;
        const int tiles = seq_tiles(P, b).n;
        if (tiles > 0) {
            const long long first = before * P.Hkv + (long long)h * item_cost(tiles) + kItemCost;  // its first tile
            cta = (int)(first / deal.share);
            n = (int)((first + tiles - 1) / deal.share) - cta + 1;
        }
    } else {
        cta = blockIdx.x;
        const long long first = (long long)cta * deal.share, last = min(deal.all, first + deal.share) - 1;
        if (first <= last) {
            const Place at = place_of(P, last);
            b = at.b, h = at.h;
            // the stretch's last item, if its first tile lies in the stretch
            if (at.off >= kItemCost && at.off - kItemCost <= last - first) n = 1 + (int)((at.n - 1 - at.off + deal.share - 1) / deal.share);
        }
    }
    // Every CTA waits for the split kernel, also those with nothing to merge: this kernel's
    // end then stands for both.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n <= 1) return;  // whole in one stretch: written by it
    const int R = P.G * P.Lq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wpr = 8 / rows_per_cta;  // warps of a row
    const int r = blockIdx.y * rows_per_cta + warp / wpr, w = warp % wpr;
    const bool live = r < R;
    const float2* ml = reinterpret_cast<const float2*>(P.ws);
    const float* wo = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(P.ws) + ws_o_offset(R));
    auto slot = [&](int i) { return (long long)(2 * (cta + i) + (i == 0 ? 1 : 0)) * R + r; };
    float M = -INFINITY, L = 0.f;
    float acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    if (live) {
        // 32 parts at a time, relative to the maximum so far; this warp's every wpr-th of them
        for (int base = 0; base < n; base += 32) {
            const int i = base + lane;
            const float2 x = i < n ? ml[slot(i)] : make_float2(-INFINITY, 0.f);
            const int m = min(32, n - base);
            float mx = max_nan(M, x.x);
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float ref = mx == -INFINITY ? 0.f : mx;
            const float alpha = fast_exp2(M - ref), f = fast_exp2(x.x - ref);
            M = mx;
            L = L * alpha + f * x.y;  // of this lane's parts
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] *= alpha;
#pragma unroll 4
            for (int j = w; j < m; j += wpr) {
                const float* src = wo + slot(base + j) * HD + lane * kPer;
                float y[kPer];
                if constexpr (kPer == 2) {
                    const float2 v = *reinterpret_cast<const float2*>(src);
                    y[0] = v.x, y[1] = v.y;
                } else {
#pragma unroll
                    for (int q = 0; q < kPer / 4; ++q) {
                        const float4 v = reinterpret_cast<const float4*>(src)[q];
                        y[4 * q] = v.x, y[4 * q + 1] = v.y, y[4 * q + 2] = v.z, y[4 * q + 3] = v.w;
                    }
                }
                const float fj = __shfl_sync(0xffffffffu, f, j);
                // a part whose row saw nothing holds zeros
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[e] = fmaf(fj, y[e], acc[e]);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    }
    if (wpr > 1) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) part[warp][lane * kPer + e] = acc[e];
        __syncthreads();
        if (w == 0)
            for (int x = 1; x < wpr; ++x)
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[e] += part[warp + x][lane * kPer + e];
    }
    if (!live || w != 0) return;
    const int gg = r / P.Lq, lq = r - gg * P.Lq, hq = h * P.G + gg;
    const bool none = M == -INFINITY;
    const float inv = none ? 0.f : 1.f / L;
    uint32_t* od = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(P.o) +
                                               (((long long)b * P.Lq + lq) * P.H + hq) * HD + lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
        const float x = none ? 0.f : acc[e] * inv, y = none ? 0.f : acc[e + 1] * inv;
        od[e / 2] = rows_bf16 ? pack2<true>(x, y) : pack2<false>(x, y);
    }
    if (P.lse && lane == 0)
        P.lse[((long long)b * P.H + hq) * P.Lq + lq] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Dynamic shared memory of a kernel, asked for once on each device.
template <typename K>
cudaError_t allow_smem(K k, int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <int HD, int CACHE, int kRowTiles, bool kBf>
cudaError_t decode_launch(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s) {
    using S = DecShape<HD, CACHE, kRowTiles>;
    auto k = paged_split_kernel<HD, CACHE, kRowTiles, kBf>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(k, S::kBytes, done);
    if (e != cudaSuccess) return e;
    constexpr int kGrid = kSms * S::kCtas;
    k<<<kGrid, S::kThreads, S::kBytes, s>>>(p, bf16 ? 1 : 0, maps.k, maps.v);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // launched early: its CTAs come up while the split kernel's last ones run, and wait there
    cudaLaunchConfig_t cfg = {};
    // by item where there are few; rows to a CTA so that there are not many more CTAs than SMs
    const int by_item = (long long)p.B * p.Hkv <= kGrid ? 1 : 0, R = p.G * p.Lq;
    const int x = by_item ? p.B * p.Hkv : kGrid;
    int per = 1;
    while (per < 8 && x * ((R + per - 1) / per) > 2 * kSms) per *= 2;
    cfg.gridDim = dim3(x, (R + per - 1) / per);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_combine_kernel<HD>, p, bf16 ? 1 : 0, kGrid, by_item, per);
}

template <int HD, int CACHE, bool kBf>
cudaError_t decode_rows(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s) {
    const int R = p.G * p.Lq;
    if (R <= 16) return decode_launch<HD, CACHE, 1, kBf>(p, bf16, maps, s);
    if (R <= 32) return decode_launch<HD, CACHE, 2, kBf>(p, bf16, maps, s);
    return decode_launch<HD, CACHE, 4, kBf>(p, bf16, maps, s);
}
template <int CACHE, bool kBf>
cudaError_t decode_hd(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s) {
    if (p.hd == 64) return decode_rows<64, CACHE, kBf>(p, bf16, maps, s);
    if (p.hd == 128) return decode_rows<128, CACHE, kBf>(p, bf16, maps, s);
    return decode_rows<256, CACHE, kBf>(p, bf16, maps, s);
}

}  // namespace paged
}  // namespace
}  // namespace attn
