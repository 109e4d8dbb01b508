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
// fp32 value rounded down is.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb.h"
#include "mnb_cache.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

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
    int32_t heads, q_heads, D, rot;
    int32_t slots;            // page slots of the grid
    int32_t by_token;         // slot of a sequence's first page: its first token, else see slot_base
    int32_t bf16, interleaved;
};

// A sequence of n tokens touches at most n pages, and at most floor((n - 1) /
// P) + 2.  Its slots start at its first token, or at floor(t0 / P) + 2 s, which
// leaves room for that many whatever the sequences before it hold.
__device__ __forceinline__ int64_t slot_base(const AppendParams& p, int32_t s)
{
    const int32_t t0 = clamp32(p.b.starts[s], 0, p.b.T);
    return p.by_token ? t0 : (int64_t)(t0 >> p.b.page_bits) + 2 * (int64_t)s;
}

// The fp32 value at or below x (the finite one next to it where x lies past
// fp32's range is never asked for: see not_finite).
__device__ __forceinline__ float round_down(double x)
{
    const float f = (float)x;
    const uint32_t b = __float_as_uint(f);
    const uint32_t lower = (b << 1) == 0 ? 0x80000001u : (b >> 31) ? b + 1 : b - 1;
    return (double)f > x ? __uint_as_float(lower) : f;
}

// Bits whose maximum over the page gives its exponent: those of |x|, less one
// step for negative x (-128 * 2^e still fits, 128 * 2^e does not), at least 1
// where x is not zero; 0x7F800000 and above where x is not finite.
__device__ __forceinline__ uint32_t range_bits(float x)
{
    const uint32_t b = __float_as_uint(x), m = b & 0x7FFFFFFFu;
    if (m >= 0x7F800000u) return 0x7F800000u;
    return (b >> 31) && m > 1 ? m - 1 : m;
}

__device__ __forceinline__ int exponent_of(uint32_t bits) { const int e = (int)(bits >> 23) - 133; return e < -126 ? -126 : e; }

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// floor(x / 2^e) of a value in range, with down = 2^-e.  (The product is exact
// unless it falls below fp32's range, where only its sign counts.)
__device__ __forceinline__ int quantize(float x, float down)
{
    const float y = x * down;
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
// where the unit lies in the first rot elements.  Piece 0 starts at element
// unit_first(), piece 1 at unit_second().
struct Unit {
    int first, second;
    bool turned;
};
__device__ __forceinline__ Unit unit_of(int j, int rot, int interleaved)
{
    const bool turned = 16 * j < rot;
    if (turned && !interleaved) return Unit{8 * j, rot / 2 + 8 * j, true};
    return Unit{16 * j, 16 * j + 8, turned};
}

__device__ __forceinline__ float element(const u32x4& a, int i, int bf16)
{
    const uint32_t w = a[i >> 1];
    return widen16(i & 1 ? w >> 16 : w & 0xFFFFu, bf16);
}

// The unit's values in 64 bits, pieces 0 and 1 after each other.
__device__ __forceinline__ void load_unit(const AppendParams& p, const uint16_t* src, int64_t position, int j,
                                          const Unit& u, double (&x)[16])
{
    const u32x4 a = *reinterpret_cast<const u32x4*>(src + u.first);
    const u32x4 b = *reinterpret_cast<const u32x4*>(src + u.second);
    if (!u.turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = element(a, i, p.bf16);
            x[8 + i] = element(b, i, p.bf16);
        }
        return;
    }
    const float4_t* cp = reinterpret_cast<const float4_t*>(p.cos + position * (p.rot / 2) + 8 * j);
    const float4_t* sp = reinterpret_cast<const float4_t*>(p.sin + position * (p.rot / 2) + 8 * j);
    const float4_t c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double c = i < 4 ? c0[i & 3] : c1[i & 3], s = i < 4 ? s0[i & 3] : s1[i & 3];
        if (p.interleaved) {       // pairs of neighbours: elements 2 i and 2 i + 1 of the sixteen
            const double e = element(i < 4 ? a : b, 2 * (i & 3), p.bf16), o = element(i < 4 ? a : b, 2 * (i & 3) + 1, p.bf16);
            x[2 * i] = e * c - o * s;
            x[2 * i + 1] = o * c + e * s;
        } else {
            const double e = element(a, i, p.bf16), o = element(b, i, p.bf16);
            x[i] = e * c - o * s;
            x[8 + i] = o * c + e * s;
        }
    }
}

// The largest of a workgroup's values, in every thread.
__device__ __forceinline__ uint32_t workgroup_max(uint32_t v, uint32_t* part)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
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
    int e = (int)(b >> 23) - 127;
    if (e < -126) e = -126;
    return OldScale{e + 133 < 255 ? (uint32_t)(e + 133) << 23 : 0x7F7FFFFFu, e};
}

// One page of one head: the tokens of positions first + a .. first + b - 1.
// tokens == the row of position first (rows follow each other).
__device__ __forceinline__ void store_keys(const AppendParams& p, int64_t page, int head, int64_t first, int a, int b,
                                           int64_t row, uint32_t* part)
{
    const int D = p.D, units = D / 16, count = (b - a) * units;
    const uint16_t* src = p.k + row * p.k_stride + (int64_t)head * D;
    float* scale = p.k_scales + page * p.heads + head;
    int8_t* dst = p.k_pages + ((page * p.heads + head) << p.b.page_bits) * D;
    const OldScale old = a > 0 ? old_scale(*scale) : OldScale{0, 0};
    uint32_t top = old.bits;
    double x[16];
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const int off = a + i / units, j = i % units;
        load_unit(p, src + off * p.k_stride, first + off, j, unit_of(j, p.rot, p.interleaved), x);
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const uint32_t r = range_bits(round_down(x[n]));
            top = r > top ? r : top;
        }
    }
    top = workgroup_max(top, part);
    const bool finite = top < 0x7F800000u;
    const int e = exponent_of(top);
    const float down = power_of_two(-e);
    if (threadIdx.x == 0) *scale = !finite ? __uint_as_float(0x7FC00000u) : top == 0 ? 0.f : power_of_two(e);
    if (old.bits && finite && e > old.e) {
        const int d = e - old.e < 7 ? e - old.e : 7;
        uint32_t* w = reinterpret_cast<uint32_t*>(dst);
        for (int i = threadIdx.x; i < a * D / 4; i += kThreads) w[i] = shift_bytes(w[i], d);
    }
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const int off = a + i / units, j = i % units;
        const Unit u = unit_of(j, p.rot, p.interleaved);
        load_unit(p, src + off * p.k_stride, first + off, j, u, x);
        uint32_t w[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            uint32_t r = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m) r |= (uint32_t)(quantize(round_down(x[4 * n + m]), down) & 255) << (8 * m);
            w[n] = finite ? r : 0;
        }
        *reinterpret_cast<u32x2*>(dst + off * D + u.first) = u32x2{w[0], w[1]};
        *reinterpret_cast<u32x2*>(dst + off * D + u.second) = u32x2{w[2], w[3]};
    }
}

// The values lie with their tokens last: a thread holds eight elements of four
// neighbouring tokens and writes a word for each element.
__device__ __forceinline__ void store_values(const AppendParams& p, int64_t page, int head, int a, int b, int64_t row,
                                             uint32_t* part)
{
    const int D = p.D, P = 1 << p.b.page_bits, pieces = D / 8;
    const uint16_t* src = p.v + row * p.v_stride + (int64_t)head * D;
    float* scale = p.v_scales + page * p.heads + head;
    int8_t* dst = p.v_pages + ((page * p.heads + head) << p.b.page_bits) * D;
    const OldScale old = a > 0 ? old_scale(*scale) : OldScale{0, 0};
    uint32_t top = old.bits;
    for (int i = threadIdx.x; i < (b - a) * pieces; i += kThreads) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(src + (a + i / pieces) * p.v_stride + 8 * (i % pieces));
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const uint32_t r = range_bits(element(x, n, p.bf16));
            top = r > top ? r : top;
        }
    }
    top = workgroup_max(top, part);
    const bool finite = top < 0x7F800000u;
    const int e = exponent_of(top);
    const float down = power_of_two(-e);
    if (threadIdx.x == 0) *scale = !finite ? __uint_as_float(0x7FC00000u) : top == 0 ? 0.f : power_of_two(e);
    const int d = old.bits && finite && e > old.e ? (e - old.e < 7 ? e - old.e : 7) : 0;
    // Groups of four tokens; those before the first new one only where they are shifted.
    const int g0 = d ? 0 : a / 4, g1 = (b + 3) / 4;
    for (int i = threadIdx.x; i < (g1 - g0) * pieces; i += kThreads) {
        const int off = 4 * (g0 + i % (g1 - g0)), c = 8 * (i / (g1 - g0));
        uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const bool mine = off + m >= a && off + m < b;
            if (!mine) continue;
            const u32x4 x = *reinterpret_cast<const u32x4*>(src + (off + m) * p.v_stride + c);
#pragma unroll
            for (int n = 0; n < 8; ++n)
                w[n] |= finite ? (uint32_t)(quantize(element(x, n, p.bf16), down) & 255) << (8 * m) : 0u;
        }
        uint32_t* to = reinterpret_cast<uint32_t*>(dst + (int64_t)c * P + off);
        const bool whole = off >= a && off + 4 <= b;
        uint32_t fresh = 0, kept = 0;     // bytes that are new, and old ones of this sequence
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (off + m >= a && off + m < b) fresh |= 255u << (8 * m);
            if (off + m < a) kept |= 255u << (8 * m);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            uint32_t* word = to + n * (P / 4);
            if (whole) {
                *word = w[n];
                continue;
            }
            const uint32_t was = *word;
            const uint32_t moved = d ? shift_bytes(was, d) : was;
            *word = (w[n] & fresh) | (moved & kept) | (was & ~(fresh | kept));
        }
    }
}

// The queries of one token (a wave each), rotated and rounded to their type
// once: to fp32 towards zero with the last bit holding whatever was cut off,
// then to nearest even.
__device__ __forceinline__ float round_to_odd(double x)
{
    const float f = (float)x;
    if ((double)f == x || !(fabs(x) < 3.0e38)) return f;
    uint32_t b = __float_as_uint(f);
    if (fabs((double)f) > fabs(x)) b -= 1;
    return __uint_as_float(b | 1u);
}

__device__ __forceinline__ void turn_queries(const AppendParams& p, int64_t t)
{
    const int lane = threadIdx.x & 63;
    const int32_t s = wave_search(p.b.S, t, [&](int32_t i) { return (int64_t)clamp32(p.b.starts[i], 0, p.b.T); });
    const Sequence q = sequence(p.b, s);
    const int64_t i = t - q.t0, position = (int64_t)q.length - q.n + i;
    if (i < 0 || i >= q.n || position < 0 || position >= ((int64_t)p.b.max_pages << p.b.page_bits)) return;
    const int units = p.D / 16;
    const uint16_t* src = p.q + t * p.q_stride;
    uint16_t* dst = p.q_out + t * p.q_out_stride;
    double x[16];
    for (int n = lane; n < p.q_heads * units; n += 64) {
        const int j = n % units;
        const int64_t at = (int64_t)(n / units) * p.D;
        const Unit u = unit_of(j, p.rot, p.interleaved);
        load_unit(p, src + at, position, j, u, x);
        u32x4 out[2];
#pragma unroll
        for (int m = 0; m < 8; ++m)
            out[m >> 2][m & 3] = (uint32_t)narrow16(round_to_odd(x[2 * m]), p.bf16) |
                                 (uint32_t)narrow16(round_to_odd(x[2 * m + 1]), p.bf16) << 16;
        *reinterpret_cast<u32x4*>(dst + at + u.first) = out[0];
        *reinterpret_cast<u32x4*>(dst + at + u.second) = out[1];
    }
}

__global__ __launch_bounds__(kThreads) void mnb_append_kernel(AppendParams p)
{
    __shared__ uint32_t part[kThreads / 64];
    // Columns of workgroups: page slots (one row of the grid for the keys of each
    // head, one for its values), then the queries, four tokens a workgroup.
    const int kind = blockIdx.y;
    if (blockIdx.x >= (uint32_t)p.slots) {
        const int64_t id = (int64_t)(blockIdx.x - p.slots) * gridDim.y + kind;
        const int64_t t = id * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if (t < p.b.T) turn_queries(p, t);
        return;
    }
    const int64_t slot = blockIdx.x;
    const int32_t s = wave_search(p.b.S, slot, [&](int32_t i) { return slot_base(p, i); });
    const Sequence q = sequence(p.b, s);
    // Tokens before position 0 (a length shorter than its tokens) are passed over.
    const int64_t start = (int64_t)q.length - q.n, from = start < 0 ? 0 : start;
    const int64_t index = (from >> p.b.page_bits) + (slot - slot_base(p, s));
    const int64_t first = index << p.b.page_bits;
    if (index < 0 || first >= q.length || index >= p.b.max_pages || q.n == 0) return;
    const int32_t page = p.b.table[(int64_t)s * p.b.max_pages + index];
    if (page < 0 || page >= p.b.pages) return;
    const int P = 1 << p.b.page_bits;
    const int a = from > first ? (int)(from - first) : 0;
    const int b = q.length - first < P ? (int)(q.length - first) : P;
    const int64_t row = q.t0 + (first - start);   // of position first; negative only where a > 0
    if (kind < p.heads) store_keys(p, page, kind, first, a, b, row, part);
    else store_values(p, page, kind - p.heads, a, b, row, part);
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
    p.D = (int32_t)a.cache.head_dim;
    p.rot = (int32_t)a.rot_dim;
    p.bf16 = a.bf16;
    p.interleaved = a.interleaved;
    const int64_t T = a.batch.tokens, loose = T / a.cache.page_size + 2 * a.batch.sequences;
    p.by_token = T <= loose;
    p.slots = (int32_t)(p.by_token ? T : loose);
    const int64_t rows = 2 * a.cache.kv_heads, waves = kThreads / 64;
    const int64_t columns = p.slots + (p.q ? (T + rows * waves - 1) / (rows * waves) : 0);
    hipLaunchKernelGGL(mnb_append_kernel, dim3((unsigned)columns, (unsigned)rows), dim3(kThreads), 0, static_cast<hipStream_t>(stream), p);
    return (int)hipGetLastError();
}

}  // namespace mnb
