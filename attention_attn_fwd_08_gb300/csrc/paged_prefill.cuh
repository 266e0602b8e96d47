// paged_prefill.cuh -- attention of a chunk of new tokens of each sequence over its pages: the
// kernels, instantiated per row and pool type in paged_prefill_*.cu.
//
// Row (token i of sequence b's n, query head hq) at position p = L - n + i: O = sum_j p_j v_j / sum_j p_j,
// p_j = exp(scale * q . k_j (capped)) over the keys j < L that the window lets it see.
//
// The rows of a KV head's G query heads share its keys, so a query tile is 128 / G tokens by G heads
// (rows token * G + head), and an item is two such tiles (one at hd 256) that share every K/V tile: the
// keys are read once for all heads of the group, and a chunk of a few dozen tokens still fills the 128
// rows of the tensor cores' M.
//   paged_plan_kernel lists the items of all sequences (first row, position, key tiles) from the
//   device's lengths and prefix sums, with the running sum of their key tiles.
//   paged_prefill_kernel: the key tiles of all (KV head, item) pairs stand in one row that is cut into
//   equal stretches, one to each of 152 CTAs, so that unlike lengths, one long sequence or few
//   rows load every SM alike; the launch depends on none of them.  An item cut by a stretch's end leaves
//   partial (m, l, O) rows in the workspace.
//   paged_prefill_merge_kernel joins those in a fixed order.
//
// What bounds it: with many rows the chain S, softmax, P V of two tiles that share an SM (the tensor work of both products
// is 561 us of the 816 that 2048 tokens over 32768 take, 32 heads of 128 on 8 in bf16: 1.32 PFLOP/s; with nearly all of the
// softmax left out 640 remain).  Beside that the instructions themselves: all roles together fit the
// instruction cache only where their loops are rolled up, and over 8-bit pages, whose widening warps
// issue beside the softmax, that was worth more than anything else (the same chunk over e4m3 pages: 2537 us with the
// softmax and the issue unrolled, 1472 rolled, 1299 now; with a quarter of the widening it would be 5 % less, with a quarter of
// the softmax 970).  The widening keeps up: of 4460 cycles that a K and a V tile take it, 1730 are waits for a free
// stage, while a softmax works 3000 of a tile's 4600.  With few rows the launches: of the 24.6 us that 64 tokens
// over 777 take, the plan is 4.5, the merge 6.6, and a CTA's first fetch of each path some of the rest.
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>

#include "paged.cuh"

namespace attn {
namespace {
namespace prefill {

constexpr int kM = 128;  // rows of a query tile
constexpr float kLog2e = 1.4426950408889634f;
// What an item costs beside its key tiles, in tiles, dealt out at its beginning.
constexpr int kItemCost = 2;
// The least that a stretch holds.  (64 new tokens over 777, 32 heads on 8: 35.2 us at 8, 27.5 at 4, 24.5 at 2; larger
// calls have more than that in each stretch anyway.)
constexpr int kMinShare = 2;

// p = 2^(x - ref): a row's reference is moved when its largest p would pass 2^top, or, before it has
// seen anything, when it would stay below 2^(top - 10); it is then put at 2^(top - 8).  fp16 p have room up
// to 2^8 and no more exponents to lose below; bf16 ones stay at most 1, so that P V passes fp32's range
// no sooner than the sum of V does.
template <bool BF16>
struct PRange {
    static constexpr float top = BF16 ? 0.f : 8.f;
};

template <int HD, bool F8>
struct Cfg {
    static constexpr int NT = HD == 256 ? 1 : 2;     // query tiles of an item (O in TMEM: NT * HD columns)
    static constexpr int BN = HD == 256 ? 64 : 128;  // keys of a tile
    static constexpr int kBoxes = HD / 64;           // 128-byte columns of a 16-bit tile
    static constexpr int kQBytes = kM * HD * 2, kTileBytes = BN * HD * 2;
    // K and V tiles in turn go through one ring, 16 bits to an element; 8-bit tiles come into a
    // ring of their own and are widened into it (room for 4 wide and 2 bare ones: 2048 over 32768 e4m3 tokens 1302 us, with
    // 3 and 4 1316)
    static constexpr int kRawRow = HD < 128 ? HD : 128, kRawBoxes = HD / kRawRow;
    static constexpr int kRawBytes = F8 ? BN * HD : 0;
    static constexpr int kStages = F8 ? (HD == 64 ? 6 : 4) : (HD == 64 ? 8 : 5);
    static constexpr int kRaw = F8 ? (HD == 64 ? 4 : 2) : 0;
    static_assert(!F8 || kStages == 3 || kStages % 2 == 0, "which use of a stage comes before a V tile's");
    static constexpr int kRingOff = NT * kQBytes;
    static constexpr int kRawOff = kRingOff + kStages * kTileBytes;
    static constexpr int kBarOff = kRawOff + kRaw * kRawBytes;
    // barriers, in this order
    static constexpr int Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, P_FULL = 6, O_DONE = 8, O_EMPTY = 10, PV_DONE = 12,
                         MMA_DONE = 14, FULL = 15, EMPTY = FULL + kStages, V_OK = EMPTY + kStages, RAW_FULL = V_OK + kStages,
                         RAW_EMPTY = RAW_FULL + kRaw, Q_WIDE = RAW_EMPTY + kRaw, kBars = Q_WIDE + (F8 ? 2 : 0);
    // (8-bit pools) exponents that the rows of Q are held by, of two parts and both tiles
    static constexpr int kQexpOff = kBarOff + kBars * 8 + 16, kQexpBytes = F8 ? 2 * 2 * kM * 2 : 0;
    static constexpr int kBytes = kQexpOff + kQexpBytes + 1024;  // (1024: alignment)
    static_assert(kBytes + 256 <= 227 * 1024, "shared memory");
    // Warpgroups: softmax of tile A; of tile B (at hd 256 the widening warps instead); loads and MMA
    // issue; the widening warps beside two tiles.
    static constexpr bool kWideB = F8 && NT == 1, kWide4 = F8 && NT == 2;
    static constexpr int kThreads = kWide4 ? 512 : 384;
    static constexpr int kWide0 = kWide4 ? 12 : 4;  // first widening warp
    // registers: shares of what the launch holds (512 x 128, 384 x 168)
    static constexpr int kRegsSoftmax = kWide4 ? 200 : 216, kRegsLoad = kWide4 ? 48 : 72, kRegsWide = kWide4 ? 64 : 120;
    static constexpr int kRegsB = NT == 2 ? kRegsSoftmax : F8 ? kRegsWide : 168;
    static_assert((kRegsSoftmax + kRegsB + kRegsLoad + (kWide4 ? kRegsWide : 0)) * 128 <= kThreads * (kWide4 ? 128 : 168),
                  "register split exceeds the launch");
};

// ------------------------------------------------------------------- the plan
// An item: `ntok` tokens of a sequence from packed row `row` on, the first at position `pos`; `len` valid
// keys; key tiles t0 .. t0 + tiles - 1.
struct Item {
    int b, row, ntok, pos, len, t0, tiles, pad;
};
struct Plan {
    long long* all;  // sum of one KV head's costs
    int* count;      // items of one KV head
    int* base;       // [B + 1] items before a sequence
    Item* items;
    long long* cum;  // [count + 1] costs before an item
    int4* split;     // of a stretch: the item that begins in it and does not end in it: its first row, tokens, KV head, parts
    float* part;     // partial rows
};
__host__ __device__ __forceinline__ long long plan_items(int total, int B, int tokens) { return (long long)total / tokens + B; }
__host__ __device__ __forceinline__ size_t round256(size_t n) { return (n + 255) / 256 * 256; }
// bytes before the partial rows
__host__ __device__ __forceinline__ size_t plan_bytes(int total, int B, int tokens) {
    const size_t n = (size_t)plan_items(total, B, tokens);
    return 256 + round256(kPrefillCtas * sizeof(int4)) + round256(((size_t)B + 1) * 4) + round256(n * sizeof(Item)) + round256((n + 1) * 8);
}
__device__ __forceinline__ Plan plan_of(const PagedParams& P, int tokens) {
    uint8_t* w = reinterpret_cast<uint8_t*>(P.ws);
    const size_t n = (size_t)plan_items(P.total, P.B, tokens);
    Plan p;
    p.all = reinterpret_cast<long long*>(w);
    p.count = reinterpret_cast<int*>(w + 8);
    w += 256;
    p.split = reinterpret_cast<int4*>(w);
    w += round256(kPrefillCtas * sizeof(int4));
    p.base = reinterpret_cast<int*>(w);
    w += round256(((size_t)P.B + 1) * 4);
    p.items = reinterpret_cast<Item*>(w);
    w += round256(n * sizeof(Item));
    p.cum = reinterpret_cast<long long*>(w);
    w += round256((n + 1) * 8);
    p.part = reinterpret_cast<float*>(w);
    return p;
}
// partial rows: slot s (two to a stretch: 2c for the item that begins before stretch c, 2c + 1 for the one
// that ends behind it) holds (m, l) of its rows, and all slots' O follow
constexpr int kSlots = 2 * kPrefillCtas;
__host__ __device__ __forceinline__ size_t part_bytes(int rows, int hd) { return (size_t)kSlots * rows * (8 + (size_t)hd * 4); }
__device__ __forceinline__ float2* part_ml(const Plan& p, int slot, int rows) {
    return reinterpret_cast<float2*>(p.part) + (size_t)slot * rows;
}
__device__ __forceinline__ float* part_o(const Plan& p, int slot, int rows, int hd) {
    return p.part + (size_t)kSlots * rows * 2 + (size_t)slot * rows * hd;
}

// inclusive sum over the block's 1024 threads; total in *all
__device__ __forceinline__ long long block_scan(long long x, long long* sums, long long* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // (sums of an earlier scan have been read)
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *all = __shfl_sync(0xffffffffu, s, 31);
    const long long before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
    return x + (warp > 0 ? before : 0);
}

// new tokens of sequence b: rows first .. first + n - 1 (n = 0 where the prefix sums leave the rows)
__device__ __forceinline__ int seq_rows(const PagedParams& P, int b, int& first, bool flag) {
    const int a0 = __ldg(P.cu + b), a1 = __ldg(P.cu + b + 1);
    first = a0;
    if (a0 < 0 || a1 < a0 || a1 > P.total) {
        if (flag) atomicOr(P.status, ST_PAGED_BOUNDS);
        return 0;
    }
    return a1 - a0;
}

constexpr int kPlanThreads = 1024;
// tokens: of an item; bn: keys of a tile.  One block: the sums over sequences and items are small.
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedParams P, const int tokens, const int bn) {
    __shared__ long long sums[32];
    __shared__ int base_s[kPlanThreads + 1];
    const Plan plan = plan_of(P, tokens);
    const long long most = plan_items(P.total, P.B, tokens);
    const bool small = P.B <= kPlanThreads;
    int* base = small ? base_s : plan.base;
    long long carry = 0, all;
    for (int b0 = 0; b0 < P.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int n = 0, first;
        if (b < P.B) {
            n = (seq_rows(P, b, first, true) + tokens - 1) / tokens;
            // (without any page, no length is out of range: nothing is attended)
            if (P.max_pages > 0 && __ldg(P.lengths + b) > (P.max_pages << P.page_shift)) atomicOr(P.status, ST_PAGED_BOUNDS);
        }
        const long long incl = block_scan(n, sums, &all);
        if (b < P.B) base[b] = (int)min(carry + incl - n, most);
        carry += all;
    }
    // (prefix sums that go back and forth, which are flagged, could name more items than there is room for)
    const int count = (int)min(carry, most);
    __syncthreads();
    // the main kernel's CTAs come up meanwhile
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    carry = 0;
    for (int e0 = 0; e0 < count; e0 += kPlanThreads) {
        const int e = e0 + threadIdx.x;
        Item it = {};
        long long cost = 0;
        if (e < count) {
            int lo = 0, hi = P.B;  // the last b with base[b] <= e lies in [lo, hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (base[mid] <= e) lo = mid;
                else hi = mid;
            }
            int first;
            const int n = seq_rows(P, lo, first, false), i0 = (e - base[lo]) * tokens;
            it.b = lo;
            it.row = first + i0;
            it.ntok = min(tokens, n - i0);
            it.len = min(max(__ldg(P.lengths + lo), 0), P.max_pages << P.page_shift);
            it.pos = it.len - n + i0;
            int klo, khi;
            key_range(P.wl, P.wr, it.len, it.pos, it.pos + it.ntok - 1, &klo, &khi);
            it.t0 = klo / bn;
            it.tiles = khi > klo ? (khi + bn - 1) / bn - it.t0 : 0;
            cost = it.tiles + kItemCost;
            plan.items[e] = it;
        }
        const long long incl = block_scan(cost, sums, &all);
        if (e < count) plan.cum[e] = carry + incl - cost;
        carry += all;
    }
    if (threadIdx.x == 0) {
        *plan.all = carry;
        *plan.count = count;
        plan.cum[count] = carry;
    }
}

// ------------------------------------------------------------------- stretches
struct Deal {
    long long all, share;  // of all KV heads; of a stretch
};
__device__ __forceinline__ Deal deal_of(const PagedParams& P, long long per_head) {
    Deal d;
    d.all = per_head * P.Hkv;
    d.share = max((d.all + kPrefillCtas - 1) / kPrefillCtas, (long long)kMinShare);
    return d;
}
// A CTA's walk along its stretch, the same in every warp: `next` gives the next item of which the stretch
// holds key tiles (or that has none and ends in it), tiles [begin, end) of it.
struct Walk {
    int left;   // of the stretch (a stretch of 2^31 tiles would take days)
    int share;
    int off;    // where it enters item e
    int h, e, count;
};
struct Part {
    Item it;
    int h, begin, end;
    __device__ bool whole() const { return begin == 0 && end == it.tiles; }
};
__device__ __forceinline__ Walk walk_of(const PagedParams& P, const Plan& plan) {
    Walk w;
    const long long per_head = *plan.all;
    const Deal d = deal_of(P, per_head);
    const long long first = min(d.all, (long long)blockIdx.x * d.share);
    w.share = (int)min(d.share, (long long)INT32_MAX);
    w.left = (int)min((long long)w.share, d.all - first);
    w.count = *plan.count;
    w.h = w.e = 0;
    w.off = 0;
    if (w.left > 0) {
        w.h = (int)(first / per_head);
        const long long in = first - w.h * per_head;
        w.e = warp_last_le(w.count, in, [&](int i) { return plan.cum[i]; });
        w.off = (int)(in - plan.cum[w.e]);
    }
    return w;
}
__device__ __forceinline__ bool next_part(const Plan& plan, Walk& w, Part& p) {
    while (w.left > 0) {
        p.it = plan.items[w.e];
        p.h = w.h;
        const int cost = p.it.tiles + kItemCost, take = min(cost - w.off, w.left), end = w.off + take;
        p.begin = max(w.off - kItemCost, 0);
        p.end = max(end - kItemCost, 0);
        w.left -= take;
        w.off = 0;
        if (++w.e == w.count) w.e = 0, ++w.h;
        if (p.end > p.begin || (p.it.tiles == 0 && end == cost)) return true;
    }
    return false;
}

// Query tile u of a part: its tokens, and the tiles [t0, t0 + n) of the part that any of its rows sees.
struct Tiles {
    int ntok, pos, t0, n;
};
template <int BN>
__device__ __forceinline__ Tiles tiles_of(const PagedParams& P, const Part& p, int u, int tm) {
    Tiles t;
    t.ntok = min(max(p.it.ntok - u * tm, 0), tm);
    t.pos = p.it.pos + u * tm;
    t.t0 = t.n = 0;
    if (t.ntok > 0) {
        int lo, hi;
        key_range(P.wl, P.wr, p.it.len, t.pos, t.pos + t.ntok - 1, &lo, &hi);
        const int a = max(lo / BN, p.it.t0 + p.begin), b = min((hi + BN - 1) / BN, p.it.t0 + p.end);
        if (hi > lo && b > a) t.t0 = a, t.n = b - a;
    }
    return t;
}

// Bounded waits as mbar_wait and warp_wait, but a waiting warp sleeps until the phase completes (for up to a
// millisecond at a time) instead of asking again and again: the others' asking took 40 % of the issue slots.
__device__ __forceinline__ bool sleep_wait(uint32_t bar, uint32_t parity, unsigned int* status, unsigned int code,
                                           volatile int* abort_flag) {
    if (mbar_test_wait(bar, parity)) return true;
    unsigned long long t0 = 0;
#pragma unroll 1
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(1000000u)
            : "memory");
        if (ok) return true;
        if (abort_flag && *abort_flag) return false;
        const unsigned long long t = globaltimer();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            atomicOr(status, code);
            if (abort_flag) *abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool warp_sleep_wait(uint32_t bar, uint32_t parity, unsigned int* status, unsigned int code,
                                                volatile int* abort_flag) {
    return __all_sync(0xffffffffu, sleep_wait(bar, parity, status, code, abort_flag));
}

__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------ 8-bit pools
// The products run in fp16, whose values hold both types' codes exactly.  Q becomes fp16 by a power of two for each
// row that brings its largest element to 2^13 (exact for all that matters: 2^-38 of that element is kept).  A
// key's scale multiplies its scores in fp32.  A value's enters its fp16 element as vs / vref, vref a power of two
// beside the part's first usable scale, and O is multiplied by vref at the end: exact where the scale is a power
// of two, else off by half a step of fp16 for the ratio and for the product.  A tile with a ratio outside
// [2^-14, 2^7] (e5m2, whose codes reach fp16's end: [2^-14, 1]), zero but for, keeps its bare codes, and the softmax
// warps make its product in fp32, as that of a tile with values that are not finite.  (A load of P and its wait for each
// key and 32 columns: 2048 tokens over 8192 take 335 us, with a tile in four like that 2880, with all 10200.)
struct VRef {
    float ref, inv, most;  // vref, its inverse, and the largest ratio
};
// of the tile whose boxes' scales the first `subs` lanes hold: whether one is usable, and vref by it
__device__ __forceinline__ bool vref_of(float vs, int subs, bool e4m3, VRef& v) {
    const int lane = threadIdx.x & 31;
    const float a = fabsf(vs);
    const unsigned fit = __ballot_sync(0xffffffffu, lane < subs && a >= 0x1p-100f && a <= 0x1p90f);
    v.ref = v.inv = 1.f;
    v.most = e4m3 ? 0x1p7f : 1.f;
    if (!fit) return false;
    const float first = __shfl_sync(0xffffffffu, a, __ffs(fit) - 1);
    const int e = (int)(__float_as_uint(first) >> 23) - 127 + (e4m3 ? 4 : 8);  // nominal ratios of 2^-4, 2^-8 .. 2 times that
    v.ref = __uint_as_float((uint32_t)(e + 127) << 23);
    v.inv = __uint_as_float((uint32_t)(127 - e) << 23);
    return true;
}
// lanes (of the first `subs`) whose box's values do not fit in fp16 beside vref
__device__ __forceinline__ unsigned odd_scales(float vs, int subs, const VRef& v) {
    const float r = fabsf(vs * v.inv);
    return __ballot_sync(0xffffffffu, (int)(threadIdx.x & 31) < subs && !(r == 0.f || (r >= 0x1p-14f && r <= v.most)));
}
// four codes as two words of two halves
template <bool E4M3>
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& w0, uint32_t& w1) {
    if constexpr (E4M3)
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
            : "=r"(w0), "=r"(w1)
            : "r"(c));
    else
        w0 = __byte_perm(c, 0, 0x1404), w1 = __byte_perm(c, 0, 0x3424);  // an e5m2 code is its fp16's upper byte
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// n bits from bit i on (i + n <= 32)
__device__ __forceinline__ uint32_t bit_range(int i, int n) {
    uint32_t m;
    asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(i), "r"(n));
    return m;
}
// 32 bytes to global memory, aligned to them
__device__ __forceinline__ void store_32(void* at, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// ------------------------------------------------------------------ the kernel
// Roles (warps): softmax of tile u, one thread to a row (0-3, 4-7); loads (8); MMA issue of tile u (9 + u); looking
// V over (11); over 8-bit pools, widening (Cfg::kWide0 ...).  With two tiles one's softmax runs while the tensor cores
// work on the other's P V and next S; each has one S buffer, and a completed S(n), issued after
// P(n-1) V(n-1), also means that O stands still.  Over 16-bit pages the softmaxes take turns, so that they do not end
// up in step with the tensor cores idle behind both (long chunks 819 us, 1056 without turns); over 8-bit ones the
// widening warps' rate spaces them and a turn only waits (ragged chunks 1267 us, 1395 with turns).  With one tile (hd 256)
// there are two S buffers instead, S(n+1) is issued before P(n) V(n), and the softmax may be done with P(n+1)
// before that product is issued: S, P and the product have a barrier for each buffer.
//
// What a row does not see has no effect on it.  Warp 11 looks over each tile of V before its product is
// issued: rows of V that no row of the item sees (behind the sequence, in a page that does not exist) become
// zeros in shared memory, and of those that some rows see it notes whether a value is not finite; if so, the
// softmax warps of a tile that does not see all of it make its product themselves, row by row over the
// keys that the row sees, in place of the MMA.
template <bool BF16, int HD, bool F8, bool CAP>
__global__ void __launch_bounds__(Cfg<HD, F8>::kThreads, 1)
    paged_prefill_kernel(const PagedParams P, const int e4m3, const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = Cfg<HD, F8>;
    constexpr int NT = C::NT, BN = C::BN, NS = C::kStages;
    constexpr bool MB = BF16 && !F8;  // the products' type is bfloat16
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
    const uint32_t bar0 = smem_u32(bars);
    auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    __shared__ int abort_flag;
    __shared__ int done_count[2];  // warps that have finished a softmax of tile u
    __shared__ int bad_v[NS];      // of V tile n, at n mod NS, as its barrier: a value that not every row sees is not finite
    __shared__ int v_loads;        // (16-bit pools) V tiles whose load has been asked for
    __shared__ int skip_pv[2][2];  // by the parity of the tile: the softmax warps make this product
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tm = kM / P.G;  // tokens of a query tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kBars; ++i) {
            uint32_t n = 1;
            if ((i >= C::P_FULL && i < C::P_FULL + 2) || (i >= C::O_EMPTY && i < C::O_EMPTY + 2))
                n = 4;  // softmax warps of a tile
            if ((i >= C::EMPTY && i < C::EMPTY + NS) || i == C::MMA_DONE) n = NT;  // MMA issuers
            if (F8 && ((i >= C::FULL && i < C::FULL + NS) || (i >= C::RAW_EMPTY && i < C::RAW_EMPTY + C::kRaw)))
                n = 4;  // widening warps
            if (F8 && i >= C::Q_WIDE && i < C::Q_WIDE + 2) n = 4;
            mbar_init(BAR(i), n);
        }
        abort_flag = v_loads = 0;
        for (int u = 0; u < 2; ++u) done_count[u] = 0, skip_pv[u][0] = skip_pv[u][1] = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    // the plan is there from here on; the merging kernel's CTAs may come up
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Plan plan = plan_of(P, NT * tm);
    // rows of a box of keys, and how many stand below each other in a tile
    const int box_shift = min(P.page_shift, 6), box_rows = 1 << box_shift, subs = BN >> box_shift;
    // The table's entry for the box of keys from `key` on, -1 if no row of [lo, hi) lies in it; what is no page is told
    // by page_ok, later, so that nothing waits for the entry when it is asked for.
    auto box_page = [&](const Part& p, int key, int lo, int hi) {
        if (key >= hi || key + box_rows <= lo) return -1;
        return __ldg(P.table + (long long)p.it.b * P.max_pages + (key >> P.page_shift));
    };
    auto page_ok = [&](int pg) { return (unsigned)pg < (unsigned)P.num_pages; };
    auto key_span = [&](const Part& p, int& lo, int& hi) {
        key_range(P.wl, P.wr, p.it.len, p.it.pos, p.it.pos + p.it.ntok - 1, &lo, &hi);
    };

    // (8-bit pools) the scales of a page's keys and values for the part's KV head; and vref of a part
    auto scales_at = [&](const Part& p, int pg) {
        if (!F8 || !page_ok(pg)) return make_float2(0.f, 0.f);
        const long long i = (long long)pg * P.Hkv + p.h;
        return make_float2(__ldg(P.k_scale + i), __ldg(P.v_scale + i));
    };
    auto first_vref = [&](const Part& p, int tile0, int n, int lo, int hi) {
        VRef v = {1.f, 1.f, 1.f};
        if constexpr (F8) {
            const int sub = lane < subs ? lane : 0;
#pragma unroll 1
            for (int i = 0; i < n; ++i)
                if (vref_of(scales_at(p, box_page(p, (tile0 + i) * BN + sub * box_rows, lo, hi)).y, subs, e4m3 != 0, v)) break;
        }
        return v;
    };

    if (warp >= 8 && warp < 12) {
        regs_dec<C::kRegsLoad>();
        if (warp == 8) {
            // ------------------------------------------------------------ loads
            if (elect_one()) {
                prefetch_tmap(&tmQ);
                if (P.max_pages > 0) {  // (there are no other maps without a page)
                    prefetch_tmap(&tmK);
                    prefetch_tmap(&tmV);
                }
            }
            constexpr int kCols = F8 ? C::kRawBoxes : C::kBoxes, kRowBytes = F8 ? C::kRawRow : 128;
            constexpr int kBytes = F8 ? C::kRawBytes : C::kTileBytes, kDepth = F8 ? C::kRaw : NS;
            constexpr int kFull = F8 ? C::RAW_FULL : C::FULL, kEmpty = F8 ? C::RAW_EMPTY : C::EMPTY;
            constexpr int kOff = F8 ? C::kRawOff : C::kRingOff;
            const int sub = lane % subs, col = lane / subs;
            bool ok = true;
            int stage = 0, phase = 1, made = 0;  // (a wait on a fresh barrier's other phase returns at once)
            int qn[2] = {0, 0};
            Walk w = walk_of(P, plan);
            Part p;
            while (ok && next_part(plan, w, p)) {
                int lo, hi;
                key_span(p, lo, hi);
                Tiles tu[2];
                for (int u = 0; u < NT; ++u) tu[u] = tiles_of<BN>(P, p, u, tm);
                const int tile0 = p.it.t0 + p.begin, n = p.end - p.begin;
                int pg = n > 0 && col < kCols ? box_page(p, tile0 * BN + sub * box_rows, lo, hi) : -1;
                for (int u = 0; ok && u < NT; ++u) {
                    if (tu[u].n == 0) continue;
                    if (qn[u] > 0 && !warp_sleep_wait(BAR(C::Q_EMPTY + u), (qn[u] - 1) & 1, P.status, ST_FWD_PRODUCER, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) mbar_expect_tx(BAR(C::Q_FULL + u), C::kBoxes * P.G * tm * 128);
                    for (int bx = 0; bx < C::kBoxes; ++bx)
                        if (elect_one())
                            tma_load_3d(sbase + u * C::kQBytes + bx * (kM * 128), &tmQ, BAR(C::Q_FULL + u), bx * 64, p.h * P.G,
                                        p.it.row + u * tm);
                    ++qn[u];
                }
                for (int i = 0; ok && i < n; ++i) {
                    const int key = (tile0 + i) * BN + sub * box_rows;
                    const int next = i + 1 < n && col < kCols ? box_page(p, key + BN, lo, hi) : -1;
                    const bool load = page_ok(pg);
                    if (!load && col < kCols && key < hi && key + box_rows > lo) atomicOr(P.status, ST_PAGED_BOUNDS);
                    const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, load)) * box_rows * kRowBytes);
                    const int y = load ? ((pg * P.Hkv + p.h) << P.page_shift) + (key & (P.page_size - 1)) : 0;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (!warp_sleep_wait(BAR(kEmpty + stage), phase, P.status, ST_FWD_PRODUCER, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) {
                            mbar_expect_tx(BAR(kFull + stage), bytes);
                            if (!F8 && kv) atomicAdd(&v_loads, 1);
                        }
                        __syncwarp();
                        if (load)
                            load_2d(sbase + kOff + stage * kBytes + col * (BN * kRowBytes) + sub * box_rows * kRowBytes,
                                    kv ? &tmV : &tmK, BAR(kFull + stage), col * (F8 ? kRowBytes : 64), y);
                        __syncwarp();
                        made = min(made + 1, kDepth);
                        if (++stage == kDepth) stage = 0, phase ^= 1;
                    }
                    pg = next;
                }
            }
            // every copy in flight lands before the CTA ends
            for (int u = 0; u < NT; ++u)
                if (qn[u] > 0) sleep_wait(BAR(C::Q_FULL + u), (qn[u] - 1) & 1, P.status, ST_TEARDOWN, nullptr);
            for (int i = 0; i < made; ++i) {
                if (--stage < 0) stage = kDepth - 1, phase ^= 1;
                sleep_wait(BAR(kFull + stage), phase ^ 1, P.status, ST_TEARDOWN, nullptr);
            }
        } else if (warp <= 8 + NT) {
            // -------------------------------------------------------- MMA issue
            // (its loops are rolled up: a product takes longer than the loop's turn, and the fewer instructions all
            // roles' loops have, the fewer are fetched again and again)
            const int u = warp - 9;
            constexpr uint32_t idS = idesc_f16(MB, kM, BN, false, false), idPV = idesc_f16(MB, kM, HD, false, true);
            const uint64_t qdesc = sdesc_sw128(sbase + u * C::kQBytes, 16, 1024);
            const uint64_t kdesc0 = sdesc_sw128(sbase + C::kRingOff, 16, 1024);
            const uint64_t vdesc0 = sdesc_sw128(sbase + C::kRingOff, BN * 128, 1024);
            const uint32_t tO = tbase + 256 + u * HD;
            auto wait = [&](int bar, uint32_t parity) { return warp_sleep_wait(BAR(bar), parity, P.status, ST_FWD_MMA, &abort_flag); };
            bool ok = true;
            int rs = 0, vs = 0;           // stage of the ring that comes next, and V tile's place among the looked over
            uint32_t rph = 0, vph = 0;    // their phases
            int sc = 0, pc = 0, act = 0;  // S issued, P taken, parts in which this tile was active
            auto advance = [&]() {
                if (++rs == NS) rs = 0, rph ^= 1;
            };
            // (by the one elected lane, as the rest of the issue)
            auto issue_s = [&](int stage, bool last) {
                const int buf = NT == 2 ? 0 : (sc & 1);
                uint64_t qd = qdesc, kd = kdesc0 + (uint32_t)(stage * C::kTileBytes >> 4);
#pragma unroll 1
                for (int kk = 0; kk < HD / 16; ++kk) {
                    mma_ss(tbase + (NT == 2 ? u * 128 : buf * 64), qd, kd, idS, kk > 0 ? 1u : 0u);
                    const bool box = (kk & 3) == 3;  // the next 64 columns
                    qd += box ? (kM * 128 - 96) >> 4 : 2;
                    kd += box ? (BN * 128 - 96) >> 4 : 2;
                }
                mma_commit(BAR(C::S_FULL + (NT == 2 ? u : buf)));
                if (last) mma_commit(BAR(C::Q_EMPTY + u));
            };
            Walk w = walk_of(P, plan);
            Part p;
            while (ok && next_part(plan, w, p)) {
                const int n = p.end - p.begin, tile0 = p.it.t0 + p.begin;
                if (n <= 0) continue;
                const Tiles my = tiles_of<BN>(P, p, u, tm);
                const int i0 = my.t0 - tile0, i1 = i0 + my.n;  // the tiles of the part that this query tile takes
                // A tile's release is committed only after the wait for its data, also for tiles that
                // this query tile skips, so that no arrival belongs to a later use of the stage.
                if (my.n > 0 && !wait((F8 && BF16 ? C::Q_WIDE : C::Q_FULL) + u, act & 1)) break;
                for (int i = -1; i < n; ++i) {
                    // tile i's product with V, and S of tile i + 1: after it, or (one tile) before
                    const bool now = i >= i0 && i < i1 && i >= 0, more = i + 1 < n, next = more && i + 1 >= i0 && i + 1 < i1;
                    const bool first = i == i0, last = i == i1 - 1, next_last = i + 1 == i1 - 1;
                    int vstage = 0;
                    if (i >= 0) {
                        vstage = rs;
                        advance();
                    }
                    if (more && !(ok = wait(C::FULL + rs, rph))) break;
                    if (NT == 1 || i < 0) {
                        tc_fence_after();
                        if (more && elect_one()) {
                            if (next) issue_s(rs, next_last);
                            mma_commit(BAR(C::EMPTY + rs));
                        }
                        __syncwarp();
                        if (next) ++sc;
                    }
                    if (i >= 0) {
                        if (!(ok = wait(C::V_OK + vs, vph))) break;
                        if (++vs == NS) vs = 0, vph ^= 1;
                        // the first product overwrites O: the last part's epilogue must have read it
                        if (now && first && act > 0 && !(ok = wait(C::O_EMPTY + u, (act - 1) & 1))) break;
                        const int pb = NT == 2 ? u : (pc & 1);
                        if (now && !(ok = wait(C::P_FULL + pb, (NT == 2 ? pc : pc >> 1) & 1))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            if (now) {
                                if (!*static_cast<volatile int*>(&skip_pv[u][pc & 1])) {
                                    const uint32_t tS = tbase + (NT == 2 ? u * 128 : (pc & 1) * 64);
                                    const uint64_t vd = vdesc0 + (uint32_t)(vstage * C::kTileBytes >> 4);
#pragma unroll 1
                                    for (int kk = 0; kk < BN / 16; ++kk)
                                        mma_ts(tO, tS + kk * 8, vd + kk * 128, idPV, (!first || kk > 0) ? 1u : 0u);
                                }
                                if constexpr (NT == 1) mma_commit(BAR(C::PV_DONE + (pc & 1)));
                                if (last) mma_commit(BAR(C::O_DONE + u));
                            }
                            if (NT == 2 && next) issue_s(rs, next_last);
                            mma_commit(BAR(C::EMPTY + vstage));
                            if (NT == 2 && more) mma_commit(BAR(C::EMPTY + rs));
                        }
                        __syncwarp();
                        if (now) ++pc;
                        if (NT == 2 && next) ++sc;
                    }
                    if (more) advance();
                }
                if (my.n > 0) ++act;
            }
            mma_commit_e(BAR(C::MMA_DONE));
            sleep_wait(BAR(C::MMA_DONE), 0, P.status, ST_TEARDOWN, nullptr);
        } else if (warp == 11) {
            // ------------------------------------------------------ V looked over
            const int sub = lane < subs ? lane : 0;
            bool ok = true;
            unsigned g = 0;  // ring position of the part's first K tile
            Walk w = walk_of(P, plan);
            Part p;
            int4 split = make_int4(0, 0, 0, 0);
            while (ok && next_part(plan, w, p)) {
                const int n = p.end - p.begin, tile0 = p.it.t0 + p.begin;
                if (p.begin == 0 && p.end < p.it.tiles)  // the item goes on in the next stretches
                    split = make_int4(p.it.row, p.it.ntok, p.h, 1 + (p.it.tiles - p.end - 1) / w.share + 1);
                int lo, hi;
                key_span(p, lo, hi);
                // keys that every row of the item sees
                const long long last = (long long)p.it.pos + p.it.ntok - 1;
                const int all_lo = P.wl >= 0 ? (int)max(0ll, last - P.wl) : 0;
                const int all_hi = P.wr >= 0 ? (int)max(min((long long)p.it.len, (long long)p.it.pos + P.wr + 1), 0ll) : p.it.len;
                int pg = n > 0 ? box_page(p, tile0 * BN + sub * box_rows, lo, hi) : -1;
                for (int i = 0; ok && i < n; ++i) {
                    const int j0 = (tile0 + i) * BN;
                    const unsigned there = __ballot_sync(0xffffffffu, lane < subs && page_ok(pg));
                    if (i + 1 < n) pg = box_page(p, j0 + BN + sub * box_rows, lo, hi);
                    // A phase that has not begun looks like one that is over, so V's is asked for only when the stage's use
                    // before it is known to be: over 8-bit pages the tiles come in order and that was a V tile, or the
                    // K tile before one that has been seen; over 16-bit ones V's load, once asked for, shows it.  K tiles are
                    // not waited for: their stages are filled again without a look at V, so that a late wait could
                    // find its phase two uses back, which looks like one that is still to come.
                    const unsigned gv = g + 2 * i + 1, stage = gv % NS;
                    if (!F8) {
                        ok = count_wait(&v_loads, (int)(g / 2 + i + 1), P.status, ST_FWD_PRODUCER, &abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                    }
                    ok = ok && warp_sleep_wait(BAR(C::FULL + stage), (gv / NS) & 1, P.status, ST_FWD_PRODUCER, &abort_flag);
                    if (!ok) break;
                    bool bad = false;
                    if (j0 < all_lo || j0 + BN > all_hi || there != (1u << subs) - 1u) {
                        uint8_t* vt = smem + C::kRingOff + stage * C::kTileBytes;
                        auto zero_rows = [&](int r0, int r1) {
                            for (int x = r0 * 8 + lane; x < r1 * 8; x += 32)
#pragma unroll
                                for (int bx = 0; bx < C::kBoxes; ++bx)
                                    *reinterpret_cast<uint4*>(vt + bx * (BN * 128) + x * 16) = make_uint4(0, 0, 0, 0);
                        };
                        auto check_rows = [&](int r0, int r1) {
#pragma unroll 2
                            for (int x = r0 * 8 + lane; x < r1 * 8; x += 32)
#pragma unroll
                                for (int bx = 0; bx < C::kBoxes; ++bx) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(vt + bx * (BN * 128) + x * 16);
                                    // an exponent of all ones carries into its sign's place
                                    constexpr uint32_t kExp = MB ? 0x7f807f80u : 0x7c007c00u, kOne = MB ? 0x00800080u : 0x04000400u;
                                    const uint32_t c = ((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne);
                                    bad = bad || (c & 0x80008000u);
                                }
                        };
                        auto in_tile = [&](int j) { return min(max(j - j0, 0), BN); };
                        const int a = in_tile(lo), b = in_tile(hi);
                        zero_rows(0, a);
                        zero_rows(b, BN);
                        if (there != (1u << subs) - 1u)
                            for (int x = 0; x < subs; ++x)
                                if (!((there >> x) & 1u)) zero_rows(max(x * box_rows, a), min((x + 1) * box_rows, b));
                        __syncwarp();
                        const int c = min(max(in_tile(all_lo), a), b), d = max(min(in_tile(all_hi), b), c);
                        check_rows(a, c);
                        check_rows(d, b);
                        fence_proxy_async_smem();  // the zeros, before the product
                    }
                    bad = __any_sync(0xffffffffu, bad);
                    if (lane == 0) {
                        const unsigned v = (g / 2 + i) % NS;
                        bad_v[v] = bad ? 1 : 0;
                        mbar_arrive(BAR(C::V_OK + v));
                    }
                    __syncwarp();
                }
                g += 2 * n;
            }
            if (lane == 0) plan.split[blockIdx.x] = split;
        }
    } else if (F8 && warp >= C::kWide0 && warp < C::kWide0 + 4) {
        // ---------------------------------------------------------------- widening
        if constexpr (F8) {
            regs_dec<C::kRegsWide>();
            const int ww = warp - C::kWide0;
            constexpr int kChunks = C::kRawRow / 16;            // 16-byte chunks of a box's row
            constexpr int kSteps = BN * HD / 16 / 128;          // chunks of a lane, of a tile
            const int sub = lane % subs;
            bool ok = true;
            int stage = 0, phase = 1, raw = 0, raw_phase = 0;
            // This lane's chunk of 16 codes (columns 16c .. of a box's row) in steps of kRowsStep rows, the warp's 32 rows
            // together: where it lies, and the two chunks of a 128-byte column of the wide tile that it becomes, by the
            // step's parity.  Lanes of either half of a row store those in the other order, so that eight lanes
            // meet no bank twice.
            constexpr int kRowsStep = 32 / kChunks, kStepRaw = kRowsStep * C::kRawRow;
            const int c = lane % kChunks, row0 = ww * 32 % BN, box = ww * 32 / BN;
            const bool swap = (c >> 2) & 1;
            uint32_t from[2], to0[2], to1[2];
#pragma unroll
            for (int o2 = 0; o2 < 2; ++o2) {
                const int row = row0 + o2 * kRowsStep + lane / kChunks, c2 = (2 * c) & 7;
                from[o2] = box * (BN * C::kRawRow) + row * C::kRawRow + (C::kRawRow == 128 ? (c ^ (row & 7)) << 4 : (c ^ ((row >> 1) & 3)) << 4);
                const uint32_t to = (box * (kChunks / 4) + (c >> 2)) * (BN * 128) + row * 128;
                to0[o2] = to + (((c2 + (swap ? 1 : 0)) ^ (row & 7)) << 4);
                to1[o2] = to + (((c2 + (swap ? 0 : 1)) ^ (row & 7)) << 4);
            }
            int qn[2] = {0, 0};  // parts in which a tile was active
            Walk w = walk_of(P, plan);
            Part p;
            while (ok && next_part(plan, w, p)) {
                int lo, hi;
                key_span(p, lo, hi);
                const int tile0 = p.it.t0 + p.begin, n = p.end - p.begin;
                // the rows of Q in fp16, a thread to a row
                if constexpr (BF16) {
                    for (int u = 0; ok && u < NT; ++u) {
                        if (tiles_of<BN>(P, p, u, tm).n == 0) continue;
                        const int at = u ? qn[1]++ : qn[0]++;
                        ok = warp_sleep_wait(BAR(C::Q_FULL + u), at & 1, P.status, ST_FWD_PRODUCER, &abort_flag);
                        if (!ok) break;
                        const int r = ww * 32 + lane;
                        uint8_t* row = smem + u * C::kQBytes + r * 128;
                        float big = 0.f;
#pragma unroll 2
                        for (int c = 0; c < 8 * C::kBoxes; ++c) {
                            const uint4 x = *reinterpret_cast<const uint4*>(row + (c >> 3) * (kM * 128) + (((c & 7) ^ (r & 7)) << 4));
                            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                big = max3f(big, fabsf(__uint_as_float(xw[e] << 16)), fabsf(__uint_as_float(xw[e] & 0xffff0000u)));
                        }
                        int ex = (int)(__float_as_uint(big) >> 23) - 127;
                        ex = big > 0.f && big < INFINITY ? max(ex, -100) : 13;
                        const float mul = __uint_as_float((uint32_t)(13 - ex + 127) << 23);
#pragma unroll 2
                        for (int c = 0; c < 8 * C::kBoxes; ++c) {
                            uint4* q = reinterpret_cast<uint4*>(row + (c >> 3) * (kM * 128) + (((c & 7) ^ (r & 7)) << 4));
                            const uint4 x = *q;
                            auto half = [&](uint32_t v) {
                                return pack2<false>(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xffff0000u) * mul);
                            };
                            *q = make_uint4(half(x.x), half(x.y), half(x.z), half(x.w));
                        }
                        reinterpret_cast<short*>(smem + C::kQexpOff)[((at & 1) * 2 + u) * kM + r] = (short)(ex - 13);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(BAR(C::Q_WIDE + u));
                    }
                }
                auto page_at = [&](int i) { return i < n ? box_page(p, (tile0 + i) * BN + sub * box_rows, lo, hi) : -1; };
                VRef vref = first_vref(p, tile0, n, lo, hi);
                int pg = page_at(1);
                float vs = scales_at(p, page_at(0)).y;
                for (int i = 0; ok && i < n; ++i) {
                    const float vs_next = scales_at(p, pg).y;
                    pg = page_at(i + 2);
                    const unsigned odd = odd_scales(vs, subs, vref);
                    const float r = odd ? 1.f : vs * vref.inv;
                    const uint32_t ratio = pack2<false>(r, r);  // of this lane's box
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        ok = warp_sleep_wait(BAR(C::RAW_FULL + raw), raw_phase, P.status, ST_FWD_PRODUCER, &abort_flag) &&
                             warp_sleep_wait(BAR(C::EMPTY + stage), phase, P.status, ST_FWD_PRODUCER, &abort_flag);
                        if (!ok) break;
                        const uint8_t* src = smem + C::kRawOff + raw * C::kRawBytes;
                        const uint32_t dst = sbase + C::kRingOff + stage * C::kTileBytes;
                        const uint32_t factor = kv ? ratio : pack2<false>(1.f, 1.f);
                        auto widen = [&](auto e4m3c) {
#pragma unroll 1
                            for (int t = 0; t < kSteps; t += 2) {
#pragma unroll
                                for (int o2 = 0; o2 < 2; ++o2) {
                                    const uint4 x = *reinterpret_cast<const uint4*>(src + from[o2] + t * kStepRaw);
                                    const uint32_t f = __shfl_sync(0xffffffffu, factor, (row0 + (t + o2) * kRowsStep) >> box_shift);
                                    uint32_t o[8];
                                    widen4<decltype(e4m3c)::value>(swap ? x.z : x.x, o[0], o[1]);
                                    widen4<decltype(e4m3c)::value>(swap ? x.w : x.y, o[2], o[3]);
                                    widen4<decltype(e4m3c)::value>(swap ? x.x : x.z, o[4], o[5]);
                                    widen4<decltype(e4m3c)::value>(swap ? x.y : x.w, o[6], o[7]);
#pragma unroll
                                    for (int e = 0; e < 8; ++e) o[e] = mul_h2(o[e], f);
                                    st_shared_v4(dst + to0[o2] + t * (kRowsStep * 128), o[0], o[1], o[2], o[3]);
                                    st_shared_v4(dst + to1[o2] + t * (kRowsStep * 128), o[4], o[5], o[6], o[7]);
                                }
                            }
                        };
                        if (e4m3) widen(std::true_type());
                        else widen(std::false_type());
                        fence_proxy_async_smem();  // the tensor cores read the tile through the async proxy
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(BAR(C::FULL + stage));
                            mbar_arrive(BAR(C::RAW_EMPTY + raw));
                        }
                        if (++stage == NS) stage = 0, phase ^= 1;
                        if (++raw == C::kRaw) raw = 0, raw_phase ^= 1;
                    }
                    vs = vs_next;
                }
            }
        }
    } else if (warp < 4 * NT) {
        regs_inc<C::kRegsSoftmax>();
        // -------------------------------------------------- softmax, epilogue of tile u
        const int u = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t tO = tbase + 256 + u * HD + lane_off;
        const int tok = r / P.G, head = r - tok * P.G;  // of this thread's row
        const float sl2 = P.scale * kLog2e;
        const uint64_t sl2_2 = f2_make(sl2, sl2);
        const float cap_in = P.scale / fmaxf(P.softcap, 1e-30f), cap_out = P.softcap * kLog2e;
        constexpr float kTop = PRange<MB>::top;
        constexpr int NC = BN / 32;
        auto wait = [&](int bar, uint32_t parity) {
            return __all_sync(0xffffffffu, sleep_wait(BAR(bar), parity, P.status, ST_FWD_SOFTMAX, &abort_flag));
        };
        bool ok = true;
        int sc = 0, act = 0;  // tiles done, parts in which this tile was active
        // (one tile) the product of the tile before this one is complete.  At most that one can still be on
        // its way, since this tile's S was issued after the one before it, and it cannot be overtaken.
        auto wait_pv = [&]() { return wait(C::PV_DONE + ((sc - 1) & 1), ((sc - 1) >> 1) & 1); };
        int base[2] = {0, 0};         // softmaxes of both tiles in earlier parts
        unsigned g = 0;               // ring position of the part's first K tile
        // x = score * log2(e) - m of a pair of raw scores; mode 0: plain; with a softcap 1: the fitted polynomial, for
        // scores in its range; 2: by exp outside it.  A score's form is its own, so that no other's bytes change its bits.
        const CapPoly cp = cap_poly(P.scale, P.softcap);
        // (the fit's highest coefficient is an eighth power of scale / softcap: where fp32 might not hold it, nothing fits, not even 0)
        const float fit_max = P.scale <= 1e4f * P.softcap ? cp.r_max : -1.f;
        float lead, lead_;  // the coefficient as it enters: where it is 0, a masked -inf would become NaN
        f2_split(f2_mul(cp.s3, sl2_2), lead, lead_);
        const bool inf_fits = lead > 0.f;
        auto to_x = [&](auto modec, uint64_t rr, uint64_t nm) -> uint64_t {
            constexpr int kMode = decltype(modec)::value;
            if constexpr (kMode == 0) return f2_fma(rr, sl2_2, nm);
            const uint64_t uu = f2_mul(rr, rr);
            uint64_t sp = f2_fma(uu, f2_mul(cp.s3, sl2_2), f2_mul(cp.s2, sl2_2));
            sp = f2_fma(uu, sp, f2_mul(cp.s1, sl2_2));
            sp = f2_fma(uu, sp, f2_mul(cp.s0, sl2_2));
            const uint64_t fit = f2_fma(rr, f2_fma(uu, sp, sl2_2), nm);
            if constexpr (kMode == 1) return fit;
            float r0, r1, m0, m1, x0, x1;
            f2_split(rr, r0, r1);
            f2_split(nm, m0, m1);
            f2_split(fit, x0, x1);
            // a masked score is -inf, and softcap * tanh(-inf) would be finite
            const float y0 = r0 == -INFINITY ? -INFINITY : fmaf(cap_out, tanh_accurate(r0 * cap_in), m0);
            const float y1 = r1 == -INFINITY ? -INFINITY : fmaf(cap_out, tanh_accurate(r1 * cap_in), m1);
            return f2_make(fabsf(r0) <= fit_max ? x0 : y0, fabsf(r1) <= fit_max ? x1 : y1);
        };
        using M0 = std::integral_constant<int, 0>;
        using M1 = std::integral_constant<int, 1>;
        using M2 = std::integral_constant<int, 2>;
        Walk w = walk_of(P, plan);
        Part p;
        while (ok && next_part(plan, w, p)) {
            const int n = p.end - p.begin, tile0 = p.it.t0 + p.begin;
            const Tiles my = tiles_of<BN>(P, p, u, tm);
            const Tiles other = NT == 2 ? tiles_of<BN>(P, p, 1 - u, tm) : my;
            const int nA = u == 0 ? my.n : other.n, nB = u == 0 ? other.n : my.n, bA = base[0], bB = base[1];
            // (a tile whose keys begin more than one tile before the other's would wait for a turn that needs a
            // stage of the ring that only its own product frees; 128 rows apart they never do)
            const bool alt = NT == 2 && !F8 && abs(my.t0 - other.t0) <= 1;
            base[0] += nA;
            base[1] += nB;
            const unsigned g0 = g;
            g += 2 * n;
            if (my.ntok == 0) continue;
            int lo, hi;  // keys that any row of the item sees
            key_span(p, lo, hi);
            const bool row_live = tok < my.ntok;
            const int pos = my.pos + tok;
            float m = 8.f - kTop, l = 0.f;
            // the first keys of the tiles that every row sees whole: from full_lo to full_hi
            const int full_lo = P.wl >= 0 ? (int)max((long long)my.pos + my.ntok - 1 - P.wl, 0ll) : 0;
            const int full_hi = (P.wr >= 0 ? (int)min((long long)p.it.len, max((long long)my.pos + P.wr + 1, 0ll)) : p.it.len) - BN;
            const int sub = lane < subs ? lane : 0;
            int pg = my.n > 0 ? box_page(p, my.t0 * BN + sub * box_rows, lo, hi) : -1;
            // (8-bit pools) vref, the scales of the tile's boxes, those of the next, and this row's factor
            const VRef vref = first_vref(p, tile0, n, lo, hi);
            float2 scale = scales_at(p, pg), scale_next = make_float2(0.f, 0.f);
            int pg_next = my.n > 1 ? box_page(p, (my.t0 + 1) * BN + sub * box_rows, lo, hi) : -1;
            float qf = 1.f;
            for (int k = 0; k < my.n; ++k) {
                const int j0 = (my.t0 + k) * BN;
                // boxes of this tile that are there (bit = box)
                const unsigned there = __ballot_sync(0xffffffffu, lane < subs && page_ok(pg));
                const unsigned odd = F8 ? odd_scales(scale.y, subs, vref) : 0u;
                if constexpr (F8) {
                    pg = pg_next;
                    scale_next = scales_at(p, pg);
                    if (k + 2 < my.n) pg_next = box_page(p, j0 + 2 * BN + sub * box_rows, lo, hi);
                } else {
                    if (k + 1 < my.n) pg = box_page(p, j0 + BN + sub * box_rows, lo, hi);
                }
                const bool full = there == (1u << subs) - 1u && j0 >= full_lo && j0 <= full_hi;
                const int sbuf = NT == 2 ? u : (sc & 1);
                const uint32_t tS = tbase + (NT == 2 ? u * 128 : (sc & 1) * 64) + lane_off;
                if (!wait(C::S_FULL + sbuf, NT == 2 ? sc & 1 : (sc >> 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // Two tiles over 16-bit pages hold a row's 128 scores in registers, with the chunks unrolled; elsewhere they are
                // loaded chunk by chunk in rolled loops.  Held, the loops take three times the instructions:
                // alone they still fit the instruction cache (long chunks 821 us, rolled 990), beside the widening's they do
                // not (2048 tokens over 8192 of e4m3: 428 us, rolled 365), nor with both forms of a softcap (of 50, the
                // same over bf16 pages: 507 us, rolled 400).
                constexpr bool kHold = !F8 && NT == 2 && !CAP;
                uint32_t sv[kHold ? NC : 1][32];
                if constexpr (kHold)
#pragma unroll
                    for (int c = 0; c < NC; ++c) tmem_ld32(tS + c * 32, sv[c]);
                if (alt && (u == 0 ? (k >= 1 && k - 1 < nB) : (k < nA))) {
                    const int need = 4 * (u == 0 ? bB + k : bA + k + 1);
                    const bool rr = count_wait(&done_count[u ^ 1], need, P.status, ST_FWD_SOFTMAX, &abort_flag);
                    if (!__all_sync(0xffffffffu, rr)) {
                        if constexpr (kHold) tmem_ld_wait_only();
                        ok = false;
                        break;
                    }
                }
                if constexpr (kHold) {
                    tmem_ld_wait_only();
#pragma unroll
                    for (int c = 0; c < NC; ++c) tmem_pin(sv[c]);
                }
                if (F8 && BF16 && k == 0) {
                    const int ex = reinterpret_cast<const volatile short*>(smem + C::kQexpOff)[((act & 1) * 2 + u) * kM + r];
                    qf = __uint_as_float((uint32_t)(ex + 127) << 23);
                }
                // ---- the keys of the tile that this row sees: [va, vb), in boxes that are there
                int va = 0, vb = BN;
                if (!full) {
                    long long x = lo - j0, y = hi - j0;
                    if (P.wl >= 0) x = max(x, (long long)pos - P.wl - j0);
                    if (P.wr >= 0) y = min(y, (long long)pos + P.wr - j0 + 1);
                    va = (int)min(max(x, 0ll), (long long)BN);
                    vb = row_live ? (int)min(max(y, (long long)va), (long long)BN) : va;
                }
                // (8-bit pools) a raw score in units of 1: the scale of the keys' page, and the power of two of the row of Q
                // (applied as the scores are loaded where a softcap or a mask follows, else with the factor log2(e) scale)
                auto page_unit = [&](int c, int half) { return __shfl_sync(0xffffffffu, scale.x, (32 * c + 16 * half) >> box_shift) * qf; };
                auto scaled = [&](uint32_t (&x)[32], int c) {
                    const float f0 = page_unit(c, 0), f1 = page_unit(c, 1);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float f = e < 16 ? f0 : f1;
                        float y, z;
                        f2_split(f2_mul(f2_make(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), f2_make(f, f)), y, z);
                        x[e] = __float_as_uint(y);
                        x[e + 1] = __float_as_uint(z);
                    }
                };
                auto prepare = [&](uint32_t (&x)[32], int c) {
                    if (F8) scaled(x, c);
                    if (__builtin_expect(!full, 0)) {
                        const int c0 = min(max(va - 32 * c, 0), 32), c1 = min(max(vb - 32 * c, 0), 32);
                        uint32_t see = bit_range(c0, c1 - c0);
                        if (there != (1u << subs) - 1u) {  // boxes of 16, 32 or 64 keys
                            const int q = (32 * c) >> box_shift;
                            uint32_t have = ((there >> q) & 1u) ? 0xffffffffu : 0u;
                            if (box_rows == 16) have = (have & 0xffffu) | (((there >> (q + 1)) & 1u) ? 0xffff0000u : 0u);
                            see &= have;
                        }
                        if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = (see >> e) & 1u ? x[e] : 0xff800000u;  // -inf
                        }
                    }
                };
                auto chunks = [&](auto fn) {
                    if constexpr (kHold) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) fn(sv[c], c);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < NC; ++c) {
                            uint32_t x[32];
                            tmem_ld32(tS + c * 32, x);
                            tmem_ld_wait(x);
                            prepare(x, c);
                            fn(x, c);
                        }
                    }
                };
                auto largest = [&](const uint32_t (&x)[32]) {
                    float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; e += 2) y[(e >> 1) & 1] = max3f(y[(e >> 1) & 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    return fmaxf(y[0], y[1]);
                };
                auto largest_abs = [&](const uint32_t (&x)[32]) {
                    float y[2] = {0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        y[(e >> 1) & 1] = max3f(y[(e >> 1) & 1], fabsf(__uint_as_float(x[e])), fabsf(__uint_as_float(x[e + 1])));
                    return fmaxf(y[0], y[1]);
                };
                bool o_stands = NT == 2;  // the product of the tile before is complete
                // ---- (8-bit pools) the scores in one pass, 32 kAt keys at a time: their maximum, then their p over S.  A move
                // of the reference, rare after the first keys, also scales the P of the tile's earlier keys, by a power of two.
                // 2048 tokens over 32768 e4m3 ones take 1314 us with 64 keys at a time, 1320 with 32, 1664 with the whole tile
                // (more instructions than stay in their cache), and 1410 in two passes of 32.
                auto one_pass = [&](auto wholec) {
                    constexpr bool kWhole = decltype(wholec)::value;
                    constexpr int kAt = 2;
                    float low = l == 0.f && row_live ? kTop - 10.f : -INFINITY;
                    uint64_t nm = f2_make(-m, -m), rs0 = f2_make(0.f, 0.f), rs1 = rs0;
                    const float top = row_live ? kTop : INFINITY;
                    auto add_up = [&]() {
                        float a0, a1, b0, b1;
                        f2_split(rs0, a0, a1);
                        f2_split(rs1, b0, b1);
                        l += (a0 + b0) + (a1 + b1);
                        rs0 = rs1 = f2_make(0.f, 0.f);
                    };
#pragma unroll 1
                    for (int c = 0; c < NC; c += kAt) {
                        uint32_t x[kAt][32];
                        float f[kAt][2];
                        float xm = -INFINITY;
#pragma unroll
                        for (int d = 0; d < kAt; ++d) tmem_ld32(tS + (c + d) * 32, x[d]);
                        tmem_ld_wait_only();
#pragma unroll
                        for (int d = 0; d < kAt; ++d) {
                            tmem_pin(x[d]);
                            if constexpr (!kWhole) prepare(x[d], c + d);
                            f[d][0] = (kWhole ? page_unit(c + d, 0) : 1.f) * sl2;
                            f[d][1] = (kWhole ? page_unit(c + d, 1) : 1.f) * sl2;
                            float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < 32; e += 2) y[e >> 4] = max3f(y[e >> 4], __uint_as_float(x[d][e]), __uint_as_float(x[d][e + 1]));
                            if (__builtin_expect(f[d][0] < 0.f || f[d][1] < 0.f, 0)) {  // (the same for all of a warp's rows)
                                float z[2] = {INFINITY, INFINITY};
#pragma unroll
                                for (int e = 0; e < 32; ++e) z[e >> 4] = fminf(z[e >> 4], __uint_as_float(x[d][e]));
                                if (f[d][0] < 0.f) y[0] = z[0];
                                if (f[d][1] < 0.f) y[1] = z[1];
                            }
                            // (nothing seen is -inf also where the page's scale is 0)
                            xm = max3f(xm, y[0] == -INFINITY ? y[0] : fmaf(y[0], f[d][0], -m), y[1] == -INFINITY ? y[1] : fmaf(y[1], f[d][1], -m));
                        }
                        const bool move = xm > top || (xm < low && xm != -INFINITY);
                        if (__builtin_expect(__any_sync(0xffffffffu, move), 0)) {
                            add_up();
                            // rows that have seen nothing hold O = 0: their reference may move by any amount
                            const float by = ceilf(xm - (kTop - 8.f));
                            const float alpha = fast_exp2(move && l > 0.f ? -by : 0.f);
                            if (move) {
                                m += by;
                                l *= alpha;
                            }
                            nm = f2_make(-m, -m);
                            if (c > 0) tmem_st_wait();
#pragma unroll 1
                            for (int q = 0; q < c / 2; ++q) {
                                uint32_t pk[32];
                                tmem_ld32(tS + q * 32, pk);
                                tmem_ld_wait(pk);
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const float2 h = h2_to_f2(pk[e]);
                                    pk[e] = pack2<false>(h.x * alpha, h.y * alpha);
                                }
                                tmem_st32(tS + q * 32, pk);
                            }
                            if (k > 0) {
                                if (!o_stands) {
                                    ok = wait_pv() && ok;
                                    o_stands = true;
                                    tc_fence_after();
                                }
#pragma unroll 1
                                for (int q = 0; q < HD / 32; ++q) {
                                    uint32_t orr[32];
                                    tmem_ld32(tO + q * 32, orr);
                                    tmem_ld_wait(orr);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
                                    tmem_st32(tO + q * 32, orr);
                                }
                            }
                        }
                        if (xm != -INFINITY) low = -INFINITY;
#pragma unroll
                        for (int d = 0; d < kAt; ++d) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float x0, x1;
                                const float g = f[d][e >> 3];
                                f2_split(f2_fma(f2_make(__uint_as_float(x[d][2 * e]), __uint_as_float(x[d][2 * e + 1])), f2_make(g, g), nm), x0, x1);
                                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);  // 2^-inf = 0
                                if (e & 1) rs1 = f2_add(rs1, f2_make(p0, p1));
                                else rs0 = f2_add(rs0, f2_make(p0, p1));
                                pk[e] = pack2<false>(p0, p1);
                            }
                            tmem_st16(tS + (c + d) * 16, pk);
                        }
                    }
                    add_up();
                };
                auto two_passes = [&]() {
                    if (kHold && !full) {
#pragma unroll
                        for (int c = 0; c < (kHold ? NC : 0); ++c) prepare(sv[c], c);
                    }
                    // ---- the row's largest score, as x against its reference
                    float rmax = -INFINITY;
                    chunks([&](uint32_t (&x)[32], int) { rmax = fmaxf(rmax, largest(x)); });
                    float xm, xm_;
                    {
                        const uint64_t r2 = f2_make(rmax, rmax), n2 = f2_make(-m, -m);
                        uint64_t x2;
                        if (!CAP) x2 = to_x(M0(), r2, n2);
                        else x2 = to_x(M2(), r2, n2);
                        f2_split(x2, xm, xm_);
                    }
                    if (rmax == -INFINITY) xm = -INFINITY;
                    const bool move = row_live && (xm > kTop || (l == 0.f && xm < kTop - 10.f && xm != -INFINITY));
                    if (__builtin_expect(__any_sync(0xffffffffu, move), 0)) {
                        // rows that have seen nothing hold O = 0: their reference may move by any amount
                        const float by = xm - (kTop - 8.f);
                        const float alpha = fast_exp2(move && l > 0.f ? -by : 0.f);
                        if (move) {
                            m += by;
                            l *= alpha;
                        }
                        if (k > 0) {
                            if (!o_stands) {
                                ok = wait_pv() && ok;
                                o_stands = true;
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int c = 0; c < HD / 32; ++c) {
                                uint32_t orr[32];
                                tmem_ld32(tO + c * 32, orr);
                                tmem_ld_wait(orr);
#pragma unroll
                                for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
                                tmem_st32(tO + c * 32, orr);
                            }
                        }
                    }
                    // ---- p over S, behind the scores that have been loaded: rounded to the products' type, summed in fp32 before.
                    // With a softcap, 32 keys at a time that the warp's rows see within the fit's range take the fit alone (2048 tokens
                    // over 8192 of bf16, softcap 50: 382 us; of 8, half of which a score in 16 000 passes: 612, 2: 1300).
                    const uint64_t nm = f2_make(-m, -m);
                    uint64_t rs0 = f2_make(0.f, 0.f), rs1 = f2_make(0.f, 0.f);
                    chunks([&](uint32_t (&x)[32], int c) {
                        auto put = [&](auto modec) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float x0, x1;
                                f2_split(to_x(modec, f2_make(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), nm), x0, x1);
                                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);  // 2^-inf = 0
                                if (e & 1) rs1 = f2_add(rs1, f2_make(p0, p1));
                                else rs0 = f2_add(rs0, f2_make(p0, p1));
                                pk[e] = pack2<MB>(p0, p1);
                            }
                            tmem_st16(tS + c * 16, pk);
                        };
                        if constexpr (!CAP) {
                            put(M0());
                        } else {
                            float amax = 0.f;
                            if (full) {
                                amax = largest_abs(x);
                            } else {  // (-inf: not seen)
#pragma unroll
                                for (int e = 0; e < 32; ++e) amax = fmaxf(amax, x[e] == 0xff800000u ? 0.f : fabsf(__uint_as_float(x[e])));
                            }
                            if (__all_sync(0xffffffffu, amax <= fit_max || !row_live) && (full || inf_fits)) put(M1());
                            else put(M2());
                        }
                    });
                    float a0, a1, b0, b1;
                    f2_split(rs0, a0, a1);
                    f2_split(rs1, b0, b1);
                    l += (a0 + b0) + (a1 + b1);
                };
                if constexpr (F8 && !CAP) {
                    if (full) one_pass(std::true_type());
                    else one_pass(std::false_type());
                } else {
                    two_passes();
                }
                if (!ok) break;
                // ---- a tile that is not whole: is all of V finite that some row does not see
                bool by_row = false;
                if (!full || odd) {
                    const int i = my.t0 + k - tile0;  // its place in the part
                    const unsigned gv = g0 + 2 * i + 1, vn = g0 / 2 + i;
                    if (!wait(C::V_OK + vn % NS, (vn / NS) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint8_t* vt = smem + C::kRingOff + (gv % NS) * C::kTileBytes;
                    by_row = (!full && *static_cast<volatile int*>(&bad_v[vn % NS]) != 0) || odd;
                    if (by_row) {
                        tmem_st_wait();
                        if (!o_stands && k > 0) {
                            if (!wait_pv()) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c = 0; c < HD / 32; ++c) {
                            uint32_t orr[32];
                            if (k > 0) {
                                tmem_ld32(tO + c * 32, orr);
                                tmem_ld_wait(orr);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) orr[e] = 0u;
                            }
                            const uint8_t* col = vt + (c >> 1) * (BN * 128);
#pragma unroll 1
                            for (int j = 0; j < BN; ++j) {
                                uint32_t pw;
                                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(pw) : "r"(tS + (j >> 1)));
                                asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(pw)::"memory");
                                float p0, p1;
                                if constexpr (MB) {
                                    p0 = __uint_as_float(pw << 16);
                                    p1 = __uint_as_float(pw & 0xffff0000u);
                                } else {
                                    const float2 f = h2_to_f2(pw);
                                    p0 = f.x, p1 = f.y;
                                }
                                float pj = (j & 1) ? p1 : p0;
                                if (F8 && odd) pj *= __shfl_sync(0xffffffffu, scale.y * vref.inv, j >> box_shift);
                                const bool see = j >= va && j < vb && ((there >> (j >> box_shift)) & 1u);
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(col + j * 128 + ((((c & 1) * 4 + q) ^ (j & 7)) << 4));
                                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        float v0, v1;
                                        if constexpr (MB) {
                                            v0 = __uint_as_float(vw[e] << 16);
                                            v1 = __uint_as_float(vw[e] & 0xffff0000u);
                                        } else {
                                            const float2 f = h2_to_f2(vw[e]);
                                            v0 = f.x, v1 = f.y;
                                        }
                                        uint32_t& o0 = orr[8 * q + 2 * e];
                                        uint32_t& o1 = orr[8 * q + 2 * e + 1];
                                        if (see) {
                                            o0 = __float_as_uint(fmaf(pj, v0, __uint_as_float(o0)));
                                            o1 = __float_as_uint(fmaf(pj, v1, __uint_as_float(o1)));
                                        }
                                    }
                                }
                            }
                            tmem_st32(tO + c * 32, orr);
                        }
                    }
                }
                if (wq == 0 && lane == 0) *static_cast<volatile int*>(&skip_pv[u][sc & 1]) = by_row ? 1 : 0;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(BAR(C::P_FULL + (NT == 2 ? u : (sc & 1))));
                    if constexpr (NT == 2) atomicAdd(&done_count[u], 1);
                }
                ++sc;
                scale = scale_next;
            }
            // ------------------------------------------------------------ epilogue
            const bool have_o = ok && my.n > 0 && wait(C::O_DONE + u, act & 1);
            if (my.n > 0) ++act;
            if (!ok || (my.n > 0 && !have_o)) {
                ok = false;
                break;
            }
            if (have_o) tc_fence_after();
            const bool whole = p.whole();
            const bool none = l == 0.f, o32 = (reinterpret_cast<uintptr_t>(P.o) & 31u) == 0;
            const float inv = (none ? 0.f : 1.f / l) * vref.ref;
            const int slot = 2 * blockIdx.x + (p.begin == 0 ? 1 : 0), rows = NT * kM;
            const long long orow = (long long)(p.it.row + u * tm + tok);
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.o) + (orow * P.H + p.h * P.G + head) * HD);
            float4* part = reinterpret_cast<float4*>(part_o(plan, slot, rows, HD) + (size_t)(u * kM + r) * HD);
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t orr[32];
                if (have_o) {
                    tmem_ld32(tO + c * 32, orr);
                    tmem_ld_wait(orr);
                }
                if (row_live && whole) {
                    uint32_t pk[2][8];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pk[e >> 3][e & 7] = none ? 0u : pack2<BF16>(__uint_as_float(orr[2 * e]) * inv, __uint_as_float(orr[2 * e + 1]) * inv);
                    // (a row's sector at a time, where O is aligned to them)
                    if (o32) {
                        store_32(out + c * 4, pk[0]);
                        store_32(out + c * 4 + 2, pk[1]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            out[c * 4 + q] = make_uint4(pk[q >> 1][4 * (q & 1)], pk[q >> 1][4 * (q & 1) + 1], pk[q >> 1][4 * (q & 1) + 2],
                                                        pk[q >> 1][4 * (q & 1) + 3]);
                    }
                } else if (row_live && !none) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = F8 ? __float_as_uint(__uint_as_float(orr[8 * q + e]) * vref.ref) : orr[8 * q + e];
                        store_32(part + c * 8 + q * 2, f);
                    }
                }
                __syncwarp();
            }
            // O is in registers or out: the next part's first product may overwrite it
            if (have_o) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(C::O_EMPTY + u));
            }
            if (row_live) {
                if (!whole) part_ml(plan, slot, rows)[u * kM + r] = make_float2(m, l);
                else if (P.lse)
                    P.lse[(long long)(p.h * P.G + head) * P.total + orow] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// ------------------------------------------------------------------- the merge
// Joins the partial rows of the items that stretches cut, a warp to a row, in the order of the stretches.
constexpr int kMergeCtas = 8 * kPrefillCtas;
template <int HD>
__global__ void __launch_bounds__(256) paged_prefill_merge_kernel(const PagedParams P, const int bf16) {
    constexpr int NT = HD == 256 ? 1 : 2, rows = NT * kM, kPer = HD / 32;
    static_assert(kPrefillCtas <= 256, "a thread to a stretch");
    __shared__ int4 split_s[kPrefillCtas];
    __shared__ int before_s[kPrefillCtas];  // rows of the items that earlier stretches cut
    __shared__ int sums[8];
    const int tm = kM / P.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Plan plan = plan_of(P, NT * tm);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 mine = threadIdx.x < kPrefillCtas ? plan.split[threadIdx.x] : make_int4(0, 0, 0, 0);
    const int count = mine.y * P.G;  // (no tokens: nothing is cut)
    int incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int all = 0;
    for (int i = 0; i < 8; ++i) {
        if (i < warp) incl += sums[i];
        all += sums[i];
    }
    if (threadIdx.x < kPrefillCtas) split_s[threadIdx.x] = mine, before_s[threadIdx.x] = incl - count;
    __syncthreads();
    for (int x = blockIdx.x * 8 + warp; x < all; x += kMergeCtas * 8) {
        const int c = warp_last_le(kPrefillCtas, x, [&](int i) { return (long long)before_s[i]; });
        const int4 it = split_s[c];
        const int y = x - before_s[c], n = it.w;
        const int t = y / P.G, head = y - t * P.G, u = t / tm, r = u * kM + (t - u * tm) * P.G + head;
        auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
        float M = -INFINITY, L = 0.f;
        float acc[kPer];
#pragma unroll
        for (int q = 0; q < kPer; ++q) acc[q] = 0.f;
        for (int base = 0; base < n; base += 32) {
            const int i = base + lane;
            const float2 ml = i < n ? part_ml(plan, slot(i), rows)[r] : make_float2(0.f, 0.f);
            const bool some = ml.y != 0.f;  // a part whose row saw nothing holds no O
            float mx = some ? ml.x : -INFINITY;
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const unsigned use = __ballot_sync(0xffffffffu, some);
            if (use == 0) continue;
            const float ref = fmaxf(M, mx), alpha = M == -INFINITY ? 0.f : fast_exp2(M - ref);
            const float f = some ? fast_exp2(ml.x - ref) : 0.f;
            M = ref;
            L = L * alpha + (some ? f * ml.y : 0.f);  // of this lane's parts
#pragma unroll
            for (int q = 0; q < kPer; ++q) acc[q] *= alpha;
            const int m = min(32, n - base);
#pragma unroll 4
            for (int j = 0; j < m; ++j) {
                const float* src = part_o(plan, slot(base + j), rows, HD) + (size_t)r * HD + lane * kPer;
                const float fj = __shfl_sync(0xffffffffu, f, j);
                const bool has = (use >> j) & 1u;
#pragma unroll
                for (int q = 0; q < kPer; q += 2) {
                    const float2 v = *reinterpret_cast<const float2*>(src + q);
                    acc[q] = has ? fmaf(fj, v.x, acc[q]) : acc[q];
                    acc[q + 1] = has ? fmaf(fj, v.y, acc[q + 1]) : acc[q + 1];
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        const bool none = M == -INFINITY;
        const float inv = none ? 0.f : 1.f / L;
        const long long orow = it.x + t;
        const int hq = it.z * P.G + head;
        uint32_t* od = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(P.o) + (orow * P.H + hq) * HD + lane * kPer);
#pragma unroll
        for (int q = 0; q < kPer; q += 2)
            od[q / 2] = bf16 ? pack2<true>(acc[q] * inv, acc[q + 1] * inv) : pack2<false>(acc[q] * inv, acc[q + 1] * inv);
        if (P.lse && lane == 0) P.lse[(long long)hq * P.total + orow] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
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
inline void early(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at) {
    at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
}

template <bool BF16, int HD, bool F8, bool CAP>
cudaError_t launch_one(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s) {
    using C = Cfg<HD, F8>;
    auto k = paged_prefill_kernel<BF16, HD, F8, CAP>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(k, C::kBytes, done);
    if (e != cudaSuccess) return e;
    paged_plan_kernel<<<1, kPlanThreads, 0, s>>>(p, C::NT * (kM / p.G), C::BN);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3(kPrefillCtas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = s;
    early(cfg, at);
    if ((e = cudaLaunchKernelEx(&cfg, k, p, cache == CACHE_E4M3 ? 1 : 0, maps.q, maps.k, maps.v)) != cudaSuccess) return e;
    cfg.gridDim = dim3(kMergeCtas);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, paged_prefill_merge_kernel<HD>, p, BF16 ? 1 : 0);
}
template <bool BF16, bool F8>
cudaError_t launch_hd(const PagedParams& p, int cache, const PrefillMaps& m, cudaStream_t s) {
    const bool cap = p.softcap > 0.f;
    if (p.hd == 64) return cap ? launch_one<BF16, 64, F8, true>(p, cache, m, s) : launch_one<BF16, 64, F8, false>(p, cache, m, s);
    if (p.hd == 128) return cap ? launch_one<BF16, 128, F8, true>(p, cache, m, s) : launch_one<BF16, 128, F8, false>(p, cache, m, s);
    return cap ? launch_one<BF16, 256, F8, true>(p, cache, m, s) : launch_one<BF16, 256, F8, false>(p, cache, m, s);
}

}  // namespace prefill
}  // namespace
}  // namespace attn
