// New keys and values into a paged cache of 8-bit integers on gfx950, the
// position rotation applied on the way.
//
// A page and head of the cache has one scale 2^e for its keys and one for its
// values; the integer q stands for (q + 1/2) 2^e.  With x running over every
// value that the page and head holds,
//
//   e = min { e >= -126 : -128 <= x / 2^e < 128 for all x },   q = floor(x / 2^e)
//
// (scale 0, q 0 where all x are 0).  floor(floor(x / 2^a) / 2^b) = floor(x /
// 2^(a+b)), so a page whose scale grows keeps its tokens by an arithmetic shift
// and its bits depend on its contents alone, not on how many calls brought
// them; no value is ever off by more than half a step of the final scale.
//
// Rotation of a pair (a, b) at a position with cosine c and sine s:
// (a c - b s, b c + a s), in 64 bits, where the products of a 16-bit value and
// a 32-bit one are exact and the one rounding (2^-53) does not show.  floor and
// the range test need no more than that value rounded down to fp32: the
// integers n 2^e, |n| <= 128, are fp32 values, so x >= n 2^e exactly when its
// fp32 value rounded down is.  Rotation takes bf16 values past fp32's range, up to
// whose end, 128 times 2^127, there is a scale for them: so everything below stands
// 2^8 lower, x 2^-8 for a key x (n 2^(e-8) are fp32 values as well).
//
// HBM bounds long calls: 7100 tokens of 8 heads of 128 with their 32 query heads move
// 164 MB in 39 us (4.2 TB/s; a large copy 4.9).  The launch and one dependent chain of
// loads (batch, page table, tokens, scale) bound short ones: one token 6.5 us.  A
// workgroup takes the new tokens of one page and head, keys or values: the page's
// exponent needs all of them, and they stay in registers between the two looks at them
// (a second pass over the tokens where they do not fit).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb.h"
#include "mnb_cache.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kKeyUnits = 4;     // units of sixteen keys' elements that a thread keeps between its two looks at them
constexpr int kValueUnits = 2;   // the same of 8 elements of four tokens

struct AppendParams {
    CacheBatch b;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;        // or null
    uint16_t* q_out;
    const float* cos;         // [rows][rot / 2], or null with rot == 0
    const float* sin;
    int8_t* k_pages;          // [pages][heads][P][D]
    int8_t* v_pages;          // [pages][heads][D][P]
    float* k_scales;          // [pages][heads]
    float* v_scales;
    int64_t k_stride, v_stride, q_stride, q_out_stride;   // elements between tokens
    int32_t heads, q_heads, rot;
    int32_t slots;            // page slots of the grid
    int32_t narrow;           // workgroups of one wave
    int32_t by_token;         // slot of a sequence's first page: its first token, else see slot_base
};

// A sequence of n tokens touches at most n pages, and at most floor((n - 1) /
// P) + 2.  Its slots start at its first token, or at floor(t0 / P) + 2 s, which
// leaves room for that many whatever the sequences before it hold.
__device__ __forceinline__ int64_t slot_base(const AppendParams& p, int32_t t0, int32_t s)
{
    return p.by_token ? t0 : (int64_t)(t0 >> p.b.page_bits) + 2 * (int64_t)s;
}

// The fp32 value at or below x (where x lies past fp32's range, something past
// 2^126, which range_bits takes for not finite).
__device__ __forceinline__ float round_down(double x)
{
    const float f = (float)x;
    const uint32_t b = __float_as_uint(f);
    const uint32_t lower = (b << 1) == 0 ? 0x80000001u : (b >> 31) ? b + 1 : b - 1;
    return (double)f > x ? __uint_as_float(lower) : f;
}

// Bits whose maximum over the page gives its exponent: those of |x|, less one
// step for negative x (-128 * 2^e still fits, 128 * 2^e does not), at least 1
// where x is not zero; 0x7F800000 where no scale fits (x past 128 * 2^127, or not
// finite).
__device__ __forceinline__ uint32_t range_bits(float x)
{
    const uint32_t b = __float_as_uint(x), m = b & 0x7FFFFFFFu, less = (b >> 31) && m > 1 ? m - 1 : m;
    return less >= 0x7E800000u ? 0x7F800000u : less;
}

// (0x00400000 is 2^-127, 2^8 times which is 64 * 2^-125.)
__device__ __forceinline__ int exponent_of(uint32_t bits) { return bits < 0x00400000u ? -126 : (int)(bits >> 23) - 125; }

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// floor(x 2^by) of a value in range.  (The product is exact unless it falls below
// fp32's range, where only its sign counts.)
__device__ __forceinline__ int quantize(float x, int by)
{
    const float y = __builtin_amdgcn_ldexpf(x, by);
    return (int)floorf(y) - ((__float_as_uint(y) << 1) == 0 && x < 0.f ? 1 : 0);
}

// The bytes of w shifted right arithmetically by d (1 <= d <= 7): with u = q +
// 128, floor(q / 2^d) = floor(u / 2^d) - 128 / 2^d.
__device__ __forceinline__ uint32_t shift_bytes(uint32_t w, int d)
{
    const uint32_t u = ((w ^ 0x80808080u) >> d) & (0x01010101u * (0xFFu >> d));
    return ((u | 0x80808080u) - 0x01010101u * (0x80u >> d)) ^ 0x80808080u;
}

// Sixteen elements, unit j of a token's head: two pieces of eight, rotated
// where the unit lies in the first rot elements.
template <bool NEAR>
__device__ __forceinline__ void unit_of(int j, int rot, int* first, int* second)
{
    const bool halves = !NEAR && 16 * j < rot;
    *first = halves ? 8 * j : 16 * j;
    *second = halves ? rot / 2 + 8 * j : 16 * j + 8;
}

template <bool BF16>
__device__ __forceinline__ float element(const u32x4& a, int i)
{
    const uint32_t w = a[i >> 1];
    return widen16(i & 1 ? w >> 16 : w & 0xFFFFu, BF16);
}

// The cosines and sines of unit j at a position: 1 and 0 where it is not rotated.
__device__ __forceinline__ void load_turn(const AppendParams& p, int64_t position, int j, float4_t (&c)[2], float4_t (&s)[2])
{
    c[0] = c[1] = float4_t{1.f, 1.f, 1.f, 1.f};
    s[0] = s[1] = float4_t{0.f, 0.f, 0.f, 0.f};
    if (16 * j < p.rot) {
        const float4_t* cp = reinterpret_cast<const float4_t*>(p.cos + position * (p.rot / 2) + 8 * j);
        const float4_t* sp = reinterpret_cast<const float4_t*>(p.sin + position * (p.rot / 2) + 8 * j);
        c[0] = cp[0];
        c[1] = cp[1];
        s[0] = sp[0];
        s[1] = sp[1];
    }
}

// The pieces a and b turned, value(n, x) called with each of the sixteen in 64 bits,
// n = 0 .. 7 of the first piece, then the second's; DOWN: times 2^-8.  A unit that is
// not rotated keeps its values whatever they are (0 times infinity would not).
template <bool BF16, bool NEAR, bool DOWN, class F>
__device__ __forceinline__ void turn(const u32x4& a, const u32x4& b, const float4_t (&c)[2], const float4_t (&s)[2],
                                     bool turned, F value)
{
    constexpr float by = DOWN ? 0x1p-8f : 1.f;      // (exact: 16-bit values go down to 2^-133)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e0 = NEAR ? 2 * i : i, e1 = NEAR ? 2 * i + 1 : 8 + i;
        const float x0 = by * (NEAR ? (i < 4 ? element<BF16>(a, 2 * (i & 3)) : element<BF16>(b, 2 * (i & 3)))
                                    : element<BF16>(a, i));
        const float x1 = by * (NEAR ? (i < 4 ? element<BF16>(a, 2 * (i & 3) + 1) : element<BF16>(b, 2 * (i & 3) + 1))
                                    : element<BF16>(b, i));
        const double co = c[i >> 2][i & 3], si = s[i >> 2][i & 3];
        const double y0 = (double)x0 * co - (double)x1 * si, y1 = (double)x1 * co + (double)x0 * si;
        value(e0, turned ? y0 : (double)x0);
        value(e1, turned ? y1 : (double)x1);
    }
}

// The largest of a workgroup's values, in every thread.
template <int kThreads>
__device__ __forceinline__ uint32_t workgroup_max(uint32_t v, uint32_t* part)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    if (kThreads == 64) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) v = part[w] > v ? part[w] : v;
    return v;
}

// What a page's old scale says: the bits whose maximum with the new values'
// gives the new exponent (0: zeros only), and the old exponent.
struct OldScale {
    uint32_t bits;
    int e;
};
__device__ __forceinline__ OldScale old_scale(float scale)
{
    const uint32_t b = __float_as_uint(scale) & 0x7FFFFFFFu;
    if (b == 0) return OldScale{0, 0};
    if (b >= 0x7F800000u) return OldScale{0x7F800000u, 0};
    const int e = (int)(b >> 23) - 127;
    return OldScale{max(__float_as_uint(0.25f * __uint_as_float(b)), 1u), e < -126 ? -126 : e};      // 64 * 2^-8
}

// One page of one head: the tokens of positions first + a .. first + b - 1, whose
// rows follow each other; `row` is that of position first.  page is looked at
// only once the new values are on their way.
template <int D, bool BF16, bool NEAR, int kThreads>
__device__ __forceinline__ void store_keys(const AppendParams& p, int32_t page, int head, int64_t first, int a, int b,
                                           int64_t row, uint32_t* part)
{
    constexpr int UNITS = D / 16;
    const int count = (b - a) * UNITS;
    const uint16_t* src = p.k + row * p.k_stride + (int64_t)head * D;
    // Units i, i + 256, ... of a thread share their place in the head.
    const int j = threadIdx.x % UNITS;
    int piece0, piece1;
    unit_of<NEAR>(j, p.rot, &piece0, &piece1);
    const bool turned = 16 * j < p.rot;
    uint32_t top = 0;
    float kept[kKeyUnits][16];
    auto look = [&](int i, float (&x)[16]) {
        const int off = a + i / UNITS;
        const u32x4 va = *reinterpret_cast<const u32x4*>(src + off * p.k_stride + piece0);
        const u32x4 vb = *reinterpret_cast<const u32x4*>(src + off * p.k_stride + piece1);
        float4_t c[2], s[2];
        load_turn(p, first + off, j, c, s);
        turn<BF16, NEAR, true>(va, vb, c, s, turned, [&](int n, double y) { x[n] = round_down(y); });
    };
    const bool keep = count <= kKeyUnits * kThreads;
    if (keep) {
#pragma unroll
        for (int u = 0; u < kKeyUnits; ++u) {
            const int i = threadIdx.x + u * kThreads;
            if (i < count) {
                look(i, kept[u]);
#pragma unroll
                for (int n = 0; n < 16; ++n) top = max(top, range_bits(kept[u][n]));
            }
        }
    } else {
        for (int i = threadIdx.x; i < count; i += kThreads) {
            look(i, kept[0]);
#pragma unroll
            for (int n = 0; n < 16; ++n) top = max(top, range_bits(kept[0][n]));
        }
    }
    if (page < 0 || page >= p.b.pages) return;
    const int64_t at = (int64_t)page * p.heads + head;
    int8_t* dst = p.k_pages + (at << p.b.page_bits) * D;
    const OldScale old = a > 0 ? old_scale(p.k_scales[at]) : OldScale{0, 0};
    top = workgroup_max<kThreads>(max(top, old.bits), part);
    const bool finite = top < 0x7F800000u;
    const int e = exponent_of(top);
    if (threadIdx.x == 0) p.k_scales[at] = !finite ? __uint_as_float(0x7FC00000u) : top == 0 ? 0.f : power_of_two(e);
    if (old.bits && finite && e > old.e) {
        const int d = e - old.e < 7 ? e - old.e : 7;
        uint32_t* w = reinterpret_cast<uint32_t*>(dst);
        for (int i = threadIdx.x; i < a * D / 4; i += kThreads) w[i] = shift_bytes(w[i], d);
    }
    auto store = [&](int i, const float (&x)[16]) {
        uint32_t w[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            uint32_t r = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m) r |= (uint32_t)(quantize(x[4 * n + m], 8 - e) & 255) << (8 * m);
            w[n] = finite ? r : 0;
        }
        int8_t* to = dst + (a + i / UNITS) * D;
        *reinterpret_cast<u32x2*>(to + piece0) = u32x2{w[0], w[1]};
        *reinterpret_cast<u32x2*>(to + piece1) = u32x2{w[2], w[3]};
    };
    if (keep) {
#pragma unroll
        for (int u = 0; u < kKeyUnits; ++u)
            if ((int)threadIdx.x + u * kThreads < count) store(threadIdx.x + u * kThreads, kept[u]);
    } else {
        for (int i = threadIdx.x; i < count; i += kThreads) {
            look(i, kept[0]);
            store(i, kept[0]);
        }
    }
}

// The largest of |x|, and of |x| less a step where x is negative, of pairs of 16-bit
// values.  (Their bits are in the order of their size; a step less takes a power of
// two into the range below, as range_bits does.)
__device__ __forceinline__ void range16(uint32_t w, uint32_t& most, uint32_t& less)
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const uint32_t m = w & 0x7FFF7FFFu;
    const u16x2 sign = __builtin_bit_cast(u16x2, w) >> (uint16_t)15;
    most = max_u16x2(most, m);
    less = max_u16x2(less, __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, m), sign)));
}

__device__ __forceinline__ uint32_t range_of(uint32_t most, uint32_t less, int bf16)
{
    most = max(most & 0xFFFFu, most >> 16);
    less = max(less & 0xFFFFu, less >> 16);
    if (most >= (bf16 ? 0x7F80u : 0x7C00u)) return 0x7F800000u;
    // (A step below the type's smallest value is zero, which says nothing of its range.)
    return most == 0 ? 0u : max(__float_as_uint(0x1p-9f * widen16(1, bf16)), __float_as_uint(0x1p-8f * widen16(less, bf16)));
}

// The values lie with their tokens last: a thread holds eight elements of four
// neighbouring tokens and writes a word for each element.
template <int D, bool BF16, int kThreads>
__device__ __forceinline__ void store_values(const AppendParams& p, int32_t page, int head, int a, int b, int64_t row,
                                             uint32_t* part)
{
    constexpr int PIECES = D / 8;
    const int P = 1 << p.b.page_bits;
    const uint16_t* src = p.v + row * p.v_stride + (int64_t)head * D;
    // Groups of four tokens with a new one; unit i is group g0 + i % groups, piece i / groups.
    const int g0 = a / 4, groups = (b + 3) / 4 - g0, count = groups * PIECES;
    uint32_t most = 0, less = 0;
    u32x4 kept[kValueUnits][4];
    auto look = [&](int i, u32x4 (&x)[4]) {
        const int off = 4 * (g0 + i % groups), c = 8 * (i / groups);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const bool mine = off + m >= a && off + m < b;
            x[m] = mine ? *reinterpret_cast<const u32x4*>(src + (off + m) * p.v_stride + c) : u32x4{0, 0, 0, 0};
        }
    };
    const bool keep = count <= kValueUnits * kThreads;
    if (keep) {
#pragma unroll
        for (int u = 0; u < kValueUnits; ++u) {
            const int i = threadIdx.x + u * kThreads;
            if (i < count) {
                look(i, kept[u]);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < 4; ++n) range16(kept[u][m][n], most, less);
            }
        }
    } else {
        for (int i = threadIdx.x; i < count; i += kThreads) {
            look(i, kept[0]);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 4; ++n) range16(kept[0][m][n], most, less);
        }
    }
    if (page < 0 || page >= p.b.pages) return;
    const int64_t at = (int64_t)page * p.heads + head;
    int8_t* dst = p.v_pages + (at << p.b.page_bits) * D;
    const OldScale old = a > 0 ? old_scale(p.v_scales[at]) : OldScale{0, 0};
    const uint32_t top = workgroup_max<kThreads>(max(range_of(most, less, BF16), old.bits), part);
    const bool finite = top < 0x7F800000u;
    const int e = exponent_of(top);
    if (threadIdx.x == 0) p.v_scales[at] = !finite ? __uint_as_float(0x7FC00000u) : top == 0 ? 0.f : power_of_two(e);
    const int d = old.bits && finite && e > old.e ? (e - old.e < 7 ? e - old.e : 7) : 0;
    if (d) {      // groups of old tokens only
        for (int i = threadIdx.x; i < g0 * D; i += kThreads) {
            uint32_t* w = reinterpret_cast<uint32_t*>(dst + (int64_t)(i / g0) * P) + i % g0;
            *w = shift_bytes(*w, d);
        }
    }
    auto store = [&](int i, const u32x4 (&x)[4]) {
        const int off = 4 * (g0 + i % groups), c = 8 * (i / groups);
        uint32_t* to = reinterpret_cast<uint32_t*>(dst + (int64_t)c * P + off);
        const bool whole = off >= a && off + 4 <= b;
        uint32_t fresh = 0, mine = 0;     // bytes that are new, and old ones of this sequence
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            fresh |= off + m >= a && off + m < b ? 255u << (8 * m) : 0u;
            mine |= off + m < a ? 255u << (8 * m) : 0u;
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            uint32_t w = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m) w |= (uint32_t)(quantize(element<BF16>(x[m], n), -e) & 255) << (8 * m);
            w = finite ? w : 0;
            uint32_t* word = to + n * (P / 4);
            if (whole) {
                *word = w;
                continue;
            }
            const uint32_t was = *word, moved = d ? shift_bytes(was, d) : was;
            *word = (w & fresh) | (moved & mine) | (was & ~(fresh | mine));
        }
    };
    if (keep) {
#pragma unroll
        for (int u = 0; u < kValueUnits; ++u)
            if ((int)threadIdx.x + u * kThreads < count) store(threadIdx.x + u * kThreads, kept[u]);
    } else {
        for (int i = threadIdx.x; i < count; i += kThreads) {
            look(i, kept[0]);
            store(i, kept[0]);
        }
    }
}

// The queries of one token (a wave each), rotated and rounded to their type
// once: to fp32 towards zero with the last bit holding whatever was cut off,
// then to nearest even.  (Past fp32's largest value that gives it, which is infinity
// in either type.)
__device__ __forceinline__ float round_to_odd(double x)
{
    const float f = (float)x;
    if ((double)f == x || !(fabs(x) < (double)__builtin_inff())) return f;
    uint32_t b = __float_as_uint(f);
    if (fabs((double)f) > fabs(x)) b -= 1;
    return __uint_as_float(b | 1u);
}

template <int D, bool BF16, bool NEAR>
__device__ __forceinline__ void turn_queries(const AppendParams& p, int64_t t)
{
    constexpr int UNITS = D / 16, EACH = 64 / UNITS;     // units of a head, heads of a wave at a time
    const int lane = threadIdx.x & 63, j = lane % UNITS;
    const Found f = find_sequence(p.b, t, [](int32_t t0, int32_t) { return (int64_t)t0; });
    const int64_t i = t - f.q.t0, position = (int64_t)f.q.length - f.q.n + i;
    if (i < 0 || i >= f.q.n || position < 0 || position >= ((int64_t)p.b.max_pages << p.b.page_bits)) return;
    int piece0, piece1;
    unit_of<NEAR>(j, p.rot, &piece0, &piece1);
    const uint16_t* src = p.q + t * p.q_stride;
    uint16_t* dst = p.q_out + t * p.q_out_stride;
    float4_t c[2], s[2];
    load_turn(p, position, j, c, s);
    constexpr int AHEAD = 4;
    for (int h0 = 0; h0 < p.q_heads; h0 += AHEAD * EACH) {
        u32x4 va[AHEAD], vb[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int h = h0 + u * EACH + lane / UNITS;
            if (h < p.q_heads) {
                va[u] = *reinterpret_cast<const u32x4*>(src + h * D + piece0);
                vb[u] = *reinterpret_cast<const u32x4*>(src + h * D + piece1);
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int h = h0 + u * EACH + lane / UNITS;
            if (h >= p.q_heads) continue;
            uint32_t out[16];
            turn<BF16, NEAR, false>(va[u], vb[u], c, s, 16 * j < p.rot,
                             [&](int n, double y) { out[n] = narrow16(round_to_odd(y), BF16); });
            u32x4 w[2];
#pragma unroll
            for (int m = 0; m < 8; ++m) w[m >> 2][m & 3] = out[2 * m] | out[2 * m + 1] << 16;
            *reinterpret_cast<u32x4*>(dst + h * D + piece0) = w[0];
            *reinterpret_cast<u32x4*>(dst + h * D + piece1) = w[1];
        }
    }
}

// (Workgroups of one wave or of four: see append_one_wave.)
template <int D, bool BF16, bool NEAR, int kThreads>
__global__ __launch_bounds__(kThreads) void mnb_append_kernel(AppendParams p)
{
    __shared__ uint32_t part[kThreads / 64];
    // Columns of workgroups: page slots (one row of the grid for the keys of each
    // head, one for its values), then the queries, four tokens a workgroup.
    const int kind = blockIdx.y;
    if (blockIdx.x >= (uint32_t)p.slots) {
        const int64_t id = (int64_t)(blockIdx.x - p.slots) * gridDim.y + kind;
        const int64_t t = id * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if (t < p.b.T) turn_queries<D, BF16, NEAR>(p, t);
        return;
    }
    const int64_t slot = blockIdx.x;
    const Found f = find_sequence(p.b, slot, [&](int32_t t0, int32_t i) { return slot_base(p, t0, i); });
    // Tokens before position 0 (a length shorter than its tokens) are passed over.
    const int64_t start = (int64_t)f.q.length - f.q.n, from = start < 0 ? 0 : start;
    const int64_t index = (from >> p.b.page_bits) + (slot - slot_base(p, f.q.t0, f.s));
    const int64_t first = index << p.b.page_bits;
    if (index < 0 || first >= f.q.length || index >= p.b.max_pages || f.q.n == 0) return;
    const int32_t page = p.b.table[(int64_t)f.s * p.b.max_pages + index];
    const int P = 1 << p.b.page_bits;
    const int a = from > first ? (int)(from - first) : 0;
    const int b = f.q.length - first < P ? (int)(f.q.length - first) : P;
    const int64_t row = f.q.t0 + (first - start);   // of position first; negative only where a > 0
    if (kind < p.heads) store_keys<D, BF16, NEAR, kThreads>(p, page, kind, first, a, b, row, part);
    else store_values<D, BF16, kThreads>(p, page, kind - p.heads, a, b, row, part);
}

template <int D, bool BF16, bool NEAR>
int queue(const AppendParams& p, int64_t tokens, hipStream_t stream)
{
    const int threads = p.narrow ? 64 : 256;
    const int64_t rows = 2 * p.heads, each = rows * (threads / 64);      // queries of a column: a token a wave
    const dim3 grid((unsigned)(p.slots + (p.q ? (tokens + each - 1) / each : 0)), (unsigned)rows);
    if (threads == 64) hipLaunchKernelGGL((mnb_append_kernel<D, BF16, NEAR, 64>), grid, dim3(64), 0, stream, p);
    else hipLaunchKernelGGL((mnb_append_kernel<D, BF16, NEAR, 256>), grid, dim3(256), 0, stream, p);
    return (int)hipGetLastError();
}

template <int D>
int queue(const AppendParams& p, const AppendArgs& a, hipStream_t s)
{
    const int64_t T = a.batch.tokens;
    if (a.bf16) return a.interleaved ? queue<D, true, true>(p, T, s) : queue<D, true, false>(p, T, s);
    return a.interleaved ? queue<D, false, true>(p, T, s) : queue<D, false, false>(p, T, s);
}

}  // namespace

int launch_append(const AppendArgs& a, void* stream)
{
    AppendParams p{};
    p.b = CacheBatch{a.batch.starts, a.batch.lengths, a.batch.page_table, (int32_t)a.batch.sequences,
                     (int32_t)a.batch.tokens, (int32_t)a.batch.max_pages, __builtin_ctzll((uint64_t)a.cache.page_size),
                     (int32_t)a.cache.pages};
    p.k = static_cast<const uint16_t*>(a.k);
    p.v = static_cast<const uint16_t*>(a.v);
    p.q = static_cast<const uint16_t*>(a.q);
    p.q_out = static_cast<uint16_t*>(a.q_out);
    p.cos = a.cos;
    p.sin = a.sin;
    p.k_pages = a.cache.k_pages;
    p.v_pages = a.cache.v_pages;
    p.k_scales = a.cache.k_scales;
    p.v_scales = a.cache.v_scales;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.q_stride = a.q_stride;
    p.q_out_stride = a.q_out_stride;
    p.heads = (int32_t)a.cache.kv_heads;
    p.q_heads = (int32_t)a.q_heads;
    p.rot = (int32_t)a.rot_dim;
    const int64_t T = a.batch.tokens;
    p.slots = (int32_t)append_slots(a.cache.page_size, T, a.batch.sequences);
    p.by_token = p.slots == T;
    p.narrow = append_one_wave(a.cache.page_size, T, a.batch.sequences, a.cache.kv_heads, a.cache.head_dim);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return a.cache.head_dim == 64 ? queue<64>(p, a, st) : a.cache.head_dim == 128 ? queue<128>(p, a, st) : queue<256>(p, a, st);
}

}  // namespace mnb
