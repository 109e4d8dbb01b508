// Causal attention of packed queries over the paged 8-bit cache on gfx950.
//
//   out[r] = sum_j softmax_j(scale * q[r] . k[j]) v[j],   j <= position of r
//
// with k[j][d] = (qk + 1/2) ks and v[j][d] = (qv + 1/2) vs, one scale per page
// and head.  The half steps leave the products: q . k = ks (q . qk + (sum of
// q) / 2), and the output gets vs / 2 times the sum of the weights.
//
// Few rows (the query heads that share a key head, times the tokens of a
// sequence): one pass over the cache, which HBM bounds.  Both products run on
// v_mfma_i32_16x16x64_i8 straight from the loads, with no conversion and no LDS:
//
// * scores: 16 keys (A) x 16 rows (B).  A row of q is held as a 23-bit integer
//   under a power of two of its own, in three 8-bit digits, so that the score's
//   integer part is exact but for what lies below 2^-22 of the row's largest
//   element.  Result lane (row, g) holds keys 4 g .. 4 g + 3 of a tile; the A
//   rows of tile t carry the keys 16 (r / 4) + 4 t + r % 4 of a unit of 64, so
//   that a lane ends with the sixteen keys 16 g .. 16 g + 15: just what the B
//   operand of the second product wants of it.
// * outputs: 16 elements (A: v with its tokens last) x 16 rows, 64 tokens deep.
//   The weights of a unit, largest 1 in each row, are held in 16 bits as two
//   digits: off by 2^-16 of the largest at most, as the 32-bit sums of the
//   products of two fp16 values would be off by 2^-12 of each.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb.h"
#include "mnb_cache.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr float kLowest = -3.0e38f;   // a running maximum before any key

struct AttentionParams {
    CacheBatch b;
    const uint16_t* q;
    uint16_t* out;
    const int8_t* k_pages;
    const int8_t* v_pages;
    const float* k_scales;
    const float* v_scales;
    float* part_o;            // [2 workgroups][16][D]: sums of split rows
    float* part_ml;           // [2 workgroups][16][2]: their maximum and weight
    int64_t q_stride, out_stride;
    int32_t heads, G;         // key heads, rows a token has for each
    int32_t bf16;
    int32_t slots;            // row tiles of the second launch's grid
    float scale_log2;         // scale * log2(e)
};

// The work of a sequence for one key head: its rows in tiles of 16, its keys in
// units of 64.
struct Work {
    int32_t tiles, units;
};
__device__ __forceinline__ Work work_of(const AttentionParams& p, const Sequence& q)
{
    const int64_t cap = (int64_t)p.b.max_pages << p.b.page_bits;
    const int64_t keys = q.length < cap ? q.length : cap;
    return Work{(int32_t)(((int64_t)q.n * p.G + 15) / 16), (int32_t)((keys + 63) / 64)};
}

__device__ __forceinline__ int64_t units_of(const AttentionParams& p, int32_t s)
{
    const Work w = work_of(p, sequence(p.b, s));
    return (int64_t)w.tiles * w.units * p.heads;
}

// Sum over the wave, in every lane.
__device__ __forceinline__ int64_t wave_sum(int64_t v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Units of every sequence, and of those before sequence s.
__device__ __forceinline__ void count_units(const AttentionParams& p, int32_t s, int64_t* all, int64_t* before)
{
    int64_t a = 0, b = 0;
    for (int32_t i = threadIdx.x & 63; i < p.b.S; i += 64) {
        const int64_t u = units_of(p, i);
        a += u;
        if (i < s) b += u;
    }
    *all = wave_sum(a);
    *before = wave_sum(b);
}

// The sequence that holds unit u of the batch, and the units before it.
__device__ __forceinline__ int32_t find_unit(const AttentionParams& p, int64_t u, int64_t* before)
{
    const int lane = threadIdx.x & 63;
    int64_t base = 0;
    for (int32_t s0 = 0; s0 < p.b.S; s0 += 64) {
        const int64_t mine = s0 + lane < p.b.S ? units_of(p, s0 + lane) : 0;
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const uint64_t past = __builtin_amdgcn_ballot_w64(base + upto > u);
        if (past) {
            const int l = __builtin_ctzll(past);
            *before = base + __shfl(upto - mine, l);
            return __builtin_amdgcn_readfirstlane(s0 + l);
        }
        base += __shfl(upto, 63);
    }
    *before = base;
    return p.b.S;
}

// Units of a workgroup: an even share, but no fewer than one for each wave.
__device__ __forceinline__ int64_t share_of(int64_t all, int64_t workgroups)
{
    const int64_t s = (all + workgroups - 1) / workgroups;
    return s < kWaves ? kWaves : s;
}

__device__ __forceinline__ float xor16_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

// A row's place: its token (of the sequence) and its head of q.
struct Row {
    int32_t token, head;
};
__device__ __forceinline__ Row row_of(const AttentionParams& p, int64_t row, int32_t h)
{
    const int32_t t = (int32_t)(row / p.G);
    return Row{t, h * p.G + (int32_t)(row - (int64_t)t * p.G)};
}

// Four bytes of the low digit (t mod 256, signed) or, from t + 128, of the high
// one: byte B of each of the four words.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d, bool high)
{
    const uint32_t lo = high ? 0x0C0C0501u : 0x0C0C0400u, hi = high ? 0x05010C0Cu : 0x04000C0Cu;
    return __builtin_amdgcn_perm(b, a, lo) | __builtin_amdgcn_perm(d, c, hi);
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void mnb_attention_rows_kernel(AttentionParams p)
{
    constexpr int KS = D / 64, DT = D / 16;
    __shared__ float lds_o[kWaves][16][D + 4];
    __shared__ float lds_m[kWaves][16], lds_l[kWaves][16];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t all, before;
    count_units(p, 0, &all, &before);
    const int64_t share = share_of(all, gridDim.x);
    int64_t u = (int64_t)blockIdx.x * share;
    const int64_t end = u + share < all ? u + share : all;
    if (u >= end) return;
    int32_t s = find_unit(p, u, &before);
    const int P = 1 << p.b.page_bits;
    for (; u < end; ) {
        // The segment: units c0 .. c1 - 1 of sequence s, head h, row tile rt.
        Sequence q = sequence(p.b, s);
        Work w = work_of(p, q);
        while (u - before >= (int64_t)w.tiles * w.units * p.heads) {   // on to the next sequence with work
            before += (int64_t)w.tiles * w.units * p.heads;
            if (++s >= p.b.S) return;
            q = sequence(p.b, s);
            w = work_of(p, q);
        }
        const int64_t in = u - before, pair = in / w.units;
        const int c0 = (int)(in - pair * w.units);
        const int c1 = end - u < w.units - c0 ? c0 + (int)(end - u) : w.units;
        const int32_t h = (int32_t)(pair / w.tiles), rt = (int32_t)(pair - (int64_t)h * w.tiles);
        const bool first_part = c0 > 0, whole = c0 == 0 && c1 == w.units;
        u += c1 - c0;

        // This lane's row.  Rows past the last one repeat it and are not stored.
        const int64_t rows = (int64_t)q.n * p.G, row0 = (int64_t)rt * 16;
        const int64_t my = row0 + r < rows ? row0 + r : rows - 1;
        const Row at = row_of(p, my, h);
        const int64_t position = (int64_t)q.length - q.n + at.token;
        const int64_t lowest = (int64_t)q.length - q.n + row_of(p, row0, h).token;   // of the tile's rows
        i32x4 qd[3][KS];
        float q_scale;
        int half;      // half the sum of the row's integers
        {
            const uint16_t* src = p.q + (q.t0 + at.token) * p.q_stride + (int64_t)at.head * D;
            u32x4 raw[KS][2];
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) raw[k][i] = *reinterpret_cast<const u32x4*>(src + 64 * k + 16 * g + 8 * i);
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max_u16x2(top, raw[k][i >> 2][i & 3] & 0x7FFF7FFFu);
            top = (top & 0xFFFFu) > (top >> 16) ? top & 0xFFFFu : top >> 16;
            uint32_t o = __shfl_xor(top, 16);
            top = o > top ? o : top;
            o = __shfl_xor(top, 32);
            top = o > top ? o : top;
            const bool finite = top < (p.bf16 ? 0x7F80u : 0x7C00u);
            // |x| < 2^ex; two steps of 2^(ex - 120) keep both factors in range.
            const float big = widen16(top, p.bf16);
            const int ex = finite && top ? ilogbf(big) + 1 : 0;
            int sum = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t d0 = 0, d1 = 0, d2 = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t pair2 = raw[k][i >> 1][(i & 1) * 2 + (j >> 1)];
                        const float x = widen16(j & 1 ? pair2 >> 16 : pair2 & 0xFFFFu, p.bf16);
                        int n = finite ? (int)rintf(ldexpf(x, 22 - ex)) : 0;
                        sum += n;
                        const int b0 = (int8_t)n;
                        n = (n - b0) >> 8;
                        const int b1 = (int8_t)n;
                        n = (n - b1) >> 8;
                        d0 |= (uint32_t)(b0 & 255) << (8 * j);
                        d1 |= (uint32_t)(b1 & 255) << (8 * j);
                        d2 |= (uint32_t)(n & 255) << (8 * j);
                    }
                    qd[0][k][i] = (int)d0;
                    qd[1][k][i] = (int)d1;
                    qd[2][k][i] = (int)d2;
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            half = sum >> 1;
            q_scale = finite ? ldexpf(p.scale_log2, ex - 22) : __uint_as_float(0x7FC00000u);
        }

        float4_t o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = float4_t{0.f, 0.f, 0.f, 0.f};
        float top = kLowest, weight = 0.f, halves = 0.f;   // weight, halves: this lane's keys only

        const int32_t* table = p.b.table + (int64_t)s * p.b.max_pages;
        for (int c = c0 + wave; c < c1; c += kWaves) {
            // Sixteen keys lie within a page.  Lane (r, g) loads keys of run r / 4
            // for the scores and holds run g afterwards.
            const int64_t key0 = (int64_t)c * 64;
            auto page_of = [&](int run, bool* good) {
                const int64_t index = (key0 + 16 * run) >> p.b.page_bits;
                const int32_t page = index < p.b.max_pages ? table[index] : -1;
                *good = page >= 0 && page < p.b.pages;
                return *good ? page : 0;
            };
            bool ok_k, ok_v;
            const int64_t page_k = page_of(r >> 2, &ok_k), page_v = page_of(g, &ok_v);
            const int8_t* kp = p.k_pages + (((page_k * p.heads + h) << p.b.page_bits) +
                                            ((key0 + 16 * (r >> 2) + (r & 3)) & (P - 1))) * D + 16 * g;
            i32x4 a[4][KS];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    a[t][k] = *reinterpret_cast<const i32x4*>(kp + 4 * t * D + 64 * k);
            const int8_t* vp = p.v_pages + ((page_v * p.heads + h) << p.b.page_bits) * D + (int64_t)r * P +
                               ((key0 + 16 * g) & (P - 1));
            i32x4 v[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d) v[d] = *reinterpret_cast<const i32x4*>(vp + (int64_t)16 * d * P);
            const int64_t run0 = key0 + 16 * g;
            // A run behind every row's position is not read into anything.
            const bool live = ok_v && run0 < q.length;
            const float ks = live ? p.k_scales[page_v * p.heads + h] : 0.f;
            const float vs = live ? fabsf(p.v_scales[page_v * p.heads + h]) : 0.f;

            float x[16];
            const float factor = q_scale * ks, bias = ok_v ? 0.f : -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                i32x4 c0v = i32x4{half, half, half, half}, c1v = i32x4{0, 0, 0, 0}, c2v = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    c0v = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[t][k], qd[0][k], c0v, 0, 0, 0);
                    c1v = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[t][k], qd[1][k], c1v, 0, 0, 0);
                    c2v = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[t][k], qd[2][k], c2v, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[4 * t + i] = fmaf(fmaf((float)((c2v[i] << 8) + c1v[i]), 256.f, (float)c0v[i]), factor, bias);
            }
            if (key0 + 63 > lowest)
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = run0 + j <= position ? x[j] : -__builtin_inff();

            float m_run = x[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) m_run = fmaxf(m_run, x[j]);
            const float m_unit = xor16_max(m_run);
            const float m_from = m_unit == -__builtin_inff() ? 0.f : m_unit;
            // The largest weight times value scale of the unit, which the 16-bit
            // weights are held against.
            const bool seen = m_run != -__builtin_inff();
            const float lvs = seen ? __log2f(vs) : -__builtin_inff();
            const float n_unit = xor16_max(m_run + lvs);
            const float n_from = n_unit == -__builtin_inff() ? 0.f : n_unit;
            const float c_run = seen ? exp2f(m_from + lvs - n_from) : 0.f;
            const float now = fmaxf(top, m_unit);
            const float keep = exp2f(top - now);
            const float f_weight = exp2f(m_unit - now);
            const float f_o = n_unit == -__builtin_inff() ? 0.f : exp2f(n_unit - now) * (1.f / 32512.f);
            top = now;
            float sum = 0.f;
            uint32_t lo[16], hi[16];
            const float step = 32512.f * c_run;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float e = __builtin_amdgcn_exp2f(x[j] - m_from);
                sum += e;
                lo[j] = __float_as_uint(fmaf(e, step, 12582912.f));
                hi[j] = __float_as_uint(fmaf(e, step, 12582912.f + 128.f));
            }
            weight = weight * keep + sum * f_weight;
            halves = halves * keep + sum * step * f_o;
            i32x4 b_lo, b_hi;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b_lo[i] = (int)pack_bytes(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3], false);
                b_hi[i] = (int)pack_bytes(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3], true);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const i32x4 zero = i32x4{0, 0, 0, 0};
                const i32x4 sh = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[d], b_hi, zero, 0, 0, 0);
                const i32x4 sl = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[d], b_lo, zero, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[d][i] = fmaf((float)((sh[i] << 8) + sl[i]), f_o, o[d][i] * keep);
            }
        }

        // The waves' sums meet in LDS.  Lane (r, g) holds elements 16 d + 4 g + i.
        weight += __shfl_xor(weight, 16);
        weight += __shfl_xor(weight, 32);
        halves += __shfl_xor(halves, 16);
        halves += __shfl_xor(halves, 32);
        if (g == 0) {
            lds_m[wave][r] = top;
            lds_l[wave][r] = weight;
        }
        __syncthreads();
        float m_all = kLowest;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) m_all = fmaxf(m_all, lds_m[i][r]);
        const float f = exp2f(top - m_all);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const float4_t y = (o[d] + 0.5f * halves) * f;
            *reinterpret_cast<float4_t*>(&lds_o[wave][r][16 * d + 4 * g]) = y;
        }
        __syncthreads();
        // Thread (row, part): D / 16 elements of a row.
        {
            const int row = threadIdx.x >> 4, e0 = (threadIdx.x & 15) * (D / 16);
            float m_row = kLowest, l_row = 0.f;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) m_row = fmaxf(m_row, lds_m[i][row]);
#pragma unroll
            for (int i = 0; i < kWaves; ++i) l_row += lds_l[i][row] * exp2f(lds_m[i][row] - m_row);
            float y[D / 16];
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                y[e] = lds_o[0][row][e0 + e];
#pragma unroll
                for (int i = 1; i < kWaves; ++i) y[e] += lds_o[i][row][e0 + e];
            }
            if (row0 + row < rows) {
                if (whole) {
                    const Row to = row_of(p, row0 + row, h);
                    uint16_t* dst = p.out + (q.t0 + to.token) * p.out_stride + (int64_t)to.head * D + e0;
                    const float inv = l_row == 0.f ? 0.f : 1.f / l_row;
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) dst[e] = narrow16(y[e] * inv, p.bf16);
                } else {
                    const int64_t slot = 2 * (int64_t)blockIdx.x + (first_part ? 0 : 1);
                    float* dst = p.part_o + (slot * 16 + row) * D + e0;
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) dst[e] = y[e];
                    if ((threadIdx.x & 15) == 0) {
                        p.part_ml[(slot * 16 + row) * 2] = m_row;
                        p.part_ml[(slot * 16 + row) * 2 + 1] = l_row;
                    }
                }
            }
        }
        __syncthreads();
    }
}

// Row tiles whose keys several workgroups shared: their sums, in the order of
// the keys.  Sequences without keys get rows of zeros.  Grid: (row tiles, heads).
template <int D>
__global__ __launch_bounds__(256) void mnb_attention_join_kernel(AttentionParams p, int32_t workgroups)
{
    const int64_t slot = blockIdx.x;
    const int32_t h = blockIdx.y;
    // A sequence's first slot: floor(t0 G / 16) + s leaves room for its tiles.
    auto base = [&](int32_t i) { return (int64_t)clamp32(p.b.starts[i], 0, p.b.T) * p.G / 16 + i; };
    const int32_t s = wave_search(p.b.S, slot, base);
    const Sequence q = sequence(p.b, s);
    const Work w = work_of(p, q);
    const int64_t rt = slot - base(s);
    if (rt < 0 || rt >= w.tiles) return;
    int64_t all, before;
    count_units(p, s, &all, &before);
    const int64_t share = share_of(all, workgroups);
    const int64_t u0 = before + ((int64_t)h * w.tiles + rt) * w.units, u1 = u0 + w.units;
    const int64_t w0 = u0 / share, w1 = w.units ? (u1 - 1) / share : w0;
    if (w.units && w0 == w1) return;     // stored by that workgroup
    const int row = threadIdx.x >> 4, e0 = (threadIdx.x & 15) * (D / 16);
    const int64_t rows = (int64_t)q.n * p.G, mine = rt * 16 + row;
    if (mine >= rows) return;
    float y[D / 16], m = kLowest, l = 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) y[e] = 0.f;
    if (w.units) {
        for (int64_t i = w0; i <= w1; ++i) {
            const int64_t at = (2 * i + (i == w0 && i * share <= u0 ? 1 : 0)) * 16 + row;
            const float m2 = p.part_ml[at * 2], l2 = p.part_ml[at * 2 + 1];
            const float now = fmaxf(m, m2), f1 = exp2f(m - now), f2 = exp2f(m2 - now);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) y[e] = y[e] * f1 + p.part_o[at * D + e0 + e] * f2;
            l = l * f1 + l2 * f2;
            m = now;
        }
    }
    const Row to = row_of(p, mine, h);
    uint16_t* dst = p.out + (q.t0 + to.token) * p.out_stride + (int64_t)to.head * D + e0;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) dst[e] = narrow16(y[e] * inv, p.bf16);
}

template <int D>
int queue(AttentionParams& p, int workgroups, hipStream_t stream)
{
    hipLaunchKernelGGL((mnb_attention_rows_kernel<D>), dim3((unsigned)workgroups), dim3(64 * kWaves), 0, stream, p);
    int e = (int)hipGetLastError();
    if (e != 0) return e;
    hipLaunchKernelGGL((mnb_attention_join_kernel<D>), dim3((unsigned)p.slots, (unsigned)p.heads), dim3(256), 0, stream,
                       p, workgroups);
    return (int)hipGetLastError();
}

}  // namespace

int launch_attention(const AttentionArgs& a, void* stream, int* launches)
{
    AttentionParams p{};
    p.b = CacheBatch{a.batch.starts, a.batch.lengths, a.batch.page_table, (int32_t)a.batch.sequences,
                     (int32_t)a.batch.tokens, (int32_t)a.batch.max_pages, __builtin_ctzll((uint64_t)a.cache.page_size),
                     (int32_t)a.cache.pages};
    p.q = static_cast<const uint16_t*>(a.q);
    p.out = static_cast<uint16_t*>(a.out);
    p.k_pages = a.cache.k_pages;
    p.v_pages = a.cache.v_pages;
    p.k_scales = a.cache.k_scales;
    p.v_scales = a.cache.v_scales;
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.heads = (int32_t)a.cache.kv_heads;
    p.G = (int32_t)(a.q_heads / a.cache.kv_heads);
    p.bf16 = a.bf16;
    p.scale_log2 = a.scale * 1.44269504088896340736f;
    const AttentionLayout lay = attention_layout(a.cache.head_dim);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.part_ml = reinterpret_cast<float*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + lay.o);
    p.slots = (int32_t)(a.batch.tokens * p.G / 16 + a.batch.sequences);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    *launches = 2;
    switch (a.cache.head_dim) {
    case 64: return queue<64>(p, lay.workgroups, s);
    case 128: return queue<128>(p, lay.workgroups, s);
    default: return queue<256>(p, lay.workgroups, s);
    }
}

}  // namespace mnb
