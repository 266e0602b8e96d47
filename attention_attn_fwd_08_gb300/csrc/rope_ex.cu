// rope_ex.cu -- rotary positions in every form: rows [rows][H*hd] of which `rd` elements of each
// head, from element `rs` on, are turned in pairs by the row's position.
//
// With f_i the frequency of pair i < rd/2, p the row's position and A an amplitude, the pair (a, b)
// becomes A (a cos pf_i - b sin pf_i, b cos pf_i + a sin pf_i); backward, the transposed map, has
// -sin in place of sin.  Half layout: pair i is elements (rs + i, rs + rd/2 + i); interleaved:
// (rs + 2i, rs + 2i + 1).  The other elements of a head are copied, or, in place, left alone.
//
// Bound by HBM: each element is read and written once, beside 4 bytes of position a row.  The
// angle is an integer product (turns.cuh), formed once for each (row, pair) of a CTA and shared by
// its heads through shared memory, so that no fp64 arithmetic and few sines are left.  A thread
// moves chunks of up to 16 bytes, several in flight.  16-bit elements take the hardware sine and
// cosine (2^-20 of the pair's length, under the 2^-12 at least of the rounding that follows),
// fp32 ones sincospif of the angle's distance to the nearest quarter turn (2^-22).
// 4 x 2048 rows of 32 heads of 128 in bf16 (134 MB) take 22.8 us, 0.87 of the copy rate, in either layout and
// direction; 5003 rows of 16 heads of 256 in fp32, 64 elements turned, 30.9 (0.78).  64 rows of 40 heads: 2.6 us.
#include <math.h>

#include "kernels.h"
#include "turns.cuh"

namespace attn {
namespace {

// of a CTA, which takes about four items a thread: 16-bit rows gain from more and smaller CTAs in different stages at a time
// (4 x 2048 rows of 32 heads in bf16 22.7 us, 25.4 with 256), fp32 rows, whose sines take longer, do not (32.0, and 30.9 with 256)
template <typename T>
constexpr int kThreadsOf = sizeof(T) == 4 ? 256 : 128;
constexpr int kSms = 152;
constexpr int kTableBytes = 20 * 1024;
constexpr int kMaxRows = 8;       // of a CTA
constexpr int kMaxItems = 65536;  // of a CTA (fast_div)

struct RopeExArgs {
    const void* x;
    void* y;
    long long xs, ys;  // elements from row to row
    const int* positions;
    int pos, period;  // without positions: row r sits at pos + r % period
    int rows, H, hd, rd, rs;
    int lo_step, hi_off;      // element of a head: rs + lo_step * slot, and its partner's distance
    int rows_cta, heads_cta;  // of a CTA
    int turned, slots;        // chunks (or pairs of chunks) of a head that are turned, and all that are touched
    unsigned inv_slots, inv_heads, inv_heads_last;
    float amplitude, sign;
    TurnFreqs fr;
};

// n / d for n, d < 2^16 and m = 2^32 / d rounded up (0 for d = 1)
__device__ __forceinline__ int fast_div(int n, unsigned m) { return m ? (int)__umulhi((unsigned)n, m) : n; }

template <typename T>
__device__ __forceinline__ float2 turn_of(int p, unsigned long long f) {
    const unsigned long long frac = (unsigned long long)(long long)p * f;
    float s, c;
    if constexpr (sizeof(T) == 4) {
        // nearest quarter turn q, and the rest in (-1/8, 1/8] of a turn, right to 2^-24 of itself
        const unsigned q = (unsigned)((frac + (1ull << 61)) >> 62);
        const float rest = (float)(long long)(frac - ((unsigned long long)q << 62)) * 0x1p-63f;
        float s0, c0;
        sincospif(rest, &s0, &c0);
        s = (q & 1) ? c0 : s0;
        c = (q & 1) ? s0 : c0;
        if (q & 2) s = -s;
        if ((q + 1) & 2) c = -c;
    } else {
        const float a = (float)(int)(frac >> 32) * 1.46291807926715968e-9f;  // 2 pi / 2^32
        s = __sinf(a);
        c = __cosf(a);
    }
    return make_float2(c, s);
}

template <int kBytes> struct Chunk;
template <> struct Chunk<16> { using U = uint4; };
template <> struct Chunk<8> { using U = uint2; };
template <> struct Chunk<4> { using U = uint32_t; };
template <> struct Chunk<2> { using U = uint16_t; };

// kPair: a chunk's pairs lie inside it (interleaved); otherwise an item is two chunks, the first
// and the second elements of its pairs (with one element to a chunk, of either layout).
template <typename T, int kBytes, bool kPair>
__global__ void __launch_bounds__(kThreadsOf<T>) rope_ex_kernel(const __grid_constant__ RopeExArgs P) {
    constexpr int kThreads = kThreadsOf<T>;
    constexpr int V = kBytes / (int)sizeof(T);  // elements of a chunk
    constexpr int kAngles = kPair ? V / 2 : V;  // of an item
    constexpr int kAhead = kPair ? 4 : 2;       // items of a thread in flight
    // an item's angles lie together, padded so that eight items' 16-byte reads meet no bank twice
    constexpr int kSlotBytes = kAngles >= 2 ? kAngles * 8 + 16 : 8;
    static_assert(!kPair || V >= 2, "a pair needs two elements");
    using U = typename Chunk<kBytes>::U;
    union Vec {
        U u;
        T t[V];
    };
    __shared__ __align__(16) unsigned char table[kTableBytes];
    const int r0 = blockIdx.x * P.rows_cta, nrows = min(P.rows_cta, P.rows - r0);
    const int h0 = blockIdx.y * P.heads_cta, heads = min(P.heads_cta, P.H - h0);
    const unsigned inv_heads = blockIdx.y == gridDim.y - 1 ? P.inv_heads_last : P.inv_heads;
    const int items = nrows * heads * P.slots, row_bytes = P.turned * kSlotBytes;
    const T* xr = static_cast<const T*>(P.x) + r0 * P.xs + (long long)h0 * P.hd;
    T* yr = static_cast<T*>(P.y) + r0 * P.ys + (long long)h0 * P.hd;
    Vec a[kAhead], b[kAhead];
    int row[kAhead], at[kAhead], slot[kAhead];  // at: the chunk's first element, from the row's
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = base + k * kThreads;
            if (i >= items) continue;
            const int t = fast_div(i, P.inv_slots);
            slot[k] = i - t * P.slots;
            row[k] = fast_div(t, inv_heads);
            int e;
            if (slot[k] < P.turned) {
                e = P.rs + slot[k] * P.lo_step;
            } else {
                e = (slot[k] - P.turned) * V;
                if (e >= P.rs) e += P.rd;
            }
            at[k] = (t - row[k] * heads) * P.hd + e;
            const T* src = xr + row[k] * P.xs + at[k];
            a[k].u = *reinterpret_cast<const U*>(src);
            if constexpr (!kPair)
                if (slot[k] < P.turned) b[k].u = *reinterpret_cast<const U*>(src + P.hi_off);
        }
    };
    load(threadIdx.x);  // on the way while the angles are formed
    for (int i = threadIdx.x; i < nrows * (P.rd / 2); i += kThreads) {
        const int r = i / (P.rd / 2), j = i - r * (P.rd / 2);
        const int p = P.positions ? __ldg(P.positions + r0 + r) : P.pos + (r0 + r) % P.period;
        float2 cs = turn_of<T>(p, P.fr.f[j]);
        cs.x *= P.amplitude;
        cs.y *= P.amplitude * P.sign;
        *reinterpret_cast<float2*>(table + r * row_bytes + j / kAngles * kSlotBytes + j % kAngles * 8) = cs;
    }
    __syncthreads();
    for (int base = threadIdx.x; base < items; base += kAhead * kThreads) {
        if (base != (int)threadIdx.x) load(base);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (base + k * kThreads >= items) continue;
            T* dst = yr + row[k] * P.ys + at[k];
            if (slot[k] < P.turned) {
                const unsigned char* e = table + row[k] * row_bytes + slot[k] * kSlotBytes;
                float2 cs[kAngles];
                if constexpr (kAngles >= 2) {
#pragma unroll
                    for (int j = 0; j < kAngles; j += 2) {
                        const float4 w = *reinterpret_cast<const float4*>(e + j * 8);
                        cs[j] = make_float2(w.x, w.y);
                        cs[j + 1] = make_float2(w.z, w.w);
                    }
                } else {
                    cs[0] = *reinterpret_cast<const float2*>(e);
                }
#pragma unroll
                for (int j = 0; j < kAngles; ++j) {
                    T& lo = kPair ? a[k].t[2 * j] : a[k].t[j];
                    T& hi = kPair ? a[k].t[2 * j + 1] : b[k].t[j];
                    float u, v;
                    rope_turn(Elem<T>::to_f(lo), Elem<T>::to_f(hi), cs[j].x, cs[j].y, u, v);
                    lo = Elem<T>::from_f(u);
                    hi = Elem<T>::from_f(v);
                }
                if constexpr (!kPair) *reinterpret_cast<U*>(dst + P.hi_off) = b[k].u;
            }
            *reinterpret_cast<U*>(dst) = a[k].u;
        }
    }
}

unsigned inverse(int d) { return d == 1 ? 0u : (unsigned)((0x100000000ull + d - 1) / d); }

template <typename T, int kBytes, bool kPair>
cudaError_t rope_ex_typed(RopeExArgs a, bool interleaved, cudaStream_t s) {
    constexpr int V = kBytes / (int)sizeof(T);
    a.turned = kPair ? a.rd / V : a.rd / 2 / V;
    a.slots = a.turned + (a.x != a.y ? (a.hd - a.rd) / V : 0);
    a.lo_step = !kPair && interleaved ? 2 : V;
    a.hi_off = interleaved ? 1 : a.rd / 2;
    a.inv_slots = inverse(a.slots);
    // About four items a thread to a CTA: as few rows as hold them, or, where there are few rows, as few of
    // a row's heads as leave two CTAs to an SM, down to one item a thread.
    constexpr int kThreads = kThreadsOf<T>, kItems = 4 * kThreads;
    const long long row_items = (long long)a.H * a.slots;
    long long rows = kItems / row_items;
    rows = rows < 1 ? 1 : rows > kMaxRows ? kMaxRows : rows;
    while (rows > 1 && (a.rows + rows - 1) / rows < 2 * kSms) --rows;
    a.rows_cta = (int)rows;
    long long heads = a.H;
    while (heads > 1 && rows * heads * a.slots > kThreads &&
           (rows * heads * a.slots >= kMaxItems ||
            (a.rows + rows - 1) / rows * ((a.H + heads - 1) / heads) < 2 * kSms || rows * heads * a.slots > 2 * kItems))
        heads = (heads + 1) / 2;
    a.heads_cta = (int)heads;
    const int groups = (a.H + a.heads_cta - 1) / a.heads_cta;
    a.inv_heads = inverse(a.heads_cta);
    a.inv_heads_last = inverse(a.H - (groups - 1) * a.heads_cta);
    const dim3 grid((a.rows + a.rows_cta - 1) / a.rows_cta, groups);
    rope_ex_kernel<T, kBytes, kPair><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// The widest chunks that every address and every part of a head is a multiple of.
template <typename T>
cudaError_t rope_ex_widths(const RopeExArgs& a, bool interleaved, cudaStream_t s) {
    constexpr int E = (int)sizeof(T);
    auto fits = [&](int bytes) {
        const int v = bytes / E;
        const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
        return at % bytes == 0 && a.xs % v == 0 && a.ys % v == 0 && a.hd % v == 0 && a.rs % v == 0 &&
               (interleaved ? a.rd : a.rd / 2) % v == 0;
    };
    if (interleaved) {
        if (fits(16)) return rope_ex_typed<T, 16, true>(a, true, s);
        if (fits(8)) return rope_ex_typed<T, 8, true>(a, true, s);
        if constexpr (E == 2)
            if (fits(4)) return rope_ex_typed<T, 4, true>(a, true, s);
        return rope_ex_typed<T, E, false>(a, true, s);
    }
    if (fits(16)) return rope_ex_typed<T, 16, false>(a, false, s);
    if (fits(8)) return rope_ex_typed<T, 8, false>(a, false, s);
    if constexpr (E == 2)
        if (fits(4)) return rope_ex_typed<T, 4, false>(a, false, s);
    return rope_ex_typed<T, E, false>(a, false, s);
}

}  // namespace

cudaError_t launch_rope_ex(const RopeExCall& c, int dt, cudaStream_t s) {
    RopeExArgs a = {};
    a.x = c.x; a.y = c.y; a.xs = c.x_stride; a.ys = c.y_stride;
    a.positions = c.positions; a.pos = c.pos; a.period = c.period;
    a.rows = c.rows; a.H = c.H; a.hd = c.hd; a.rd = c.rotary_dim; a.rs = c.rotary_start;
    a.amplitude = c.amplitude;
    a.sign = c.backward ? -1.f : 1.f;
    for (int i = 0; i < a.rd / 2; ++i) {
        const double f = c.inv_freq[i];
        const unsigned long long t = turn_fraction(two_mul(Two{fabs(f), 0}, kTurnsPerRadian));
        a.fr.f[i] = f < 0 ? 0ull - t : t;
    }
    if (dt == 0) return rope_ex_widths<float>(a, c.interleaved, s);
    if (dt == 1) return rope_ex_widths<__half>(a, c.interleaved, s);
    return rope_ex_widths<__nv_bfloat16>(a, c.interleaved, s);
}

}  // namespace attn
