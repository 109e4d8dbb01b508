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
constexpr int kWorkgroups = kAttentionWorkgroups, kMostParts = kAttentionWorkgroups;
constexpr int kBegin = 4;
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
    float* tile_o;            // [slots of tiles][heads][splits][tile rows][D]
    float* tile_ml;           // the same without D, two each
    int64_t q_stride, out_stride;
    int32_t heads, G;         // key heads, rows a token has for each
    int32_t slots;            // row tiles of the joining launch's grid
    int32_t many;             // sequences of more rows than this go to the tiles
    int32_t tile_slots, splits;   // of the tiles' grid
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
    const int64_t keys = q.length < cap ? q.length : cap, rows = (int64_t)q.n * p.G;
    return Work{rows > p.many ? 0 : (int32_t)((rows + 15) / 16), (int32_t)((keys + 63) / 64)};
}

// The work of a row tile counts as its units and kBegin more, for its begin and
// end; a workgroup's share of the whole batch is cut by that count, kBegin first.
__device__ __forceinline__ int64_t count_of(const AttentionParams& p, const Work& w)
{
    return w.units ? (int64_t)w.tiles * (w.units + kBegin) * p.heads : 0;
}

__device__ __forceinline__ int64_t units_of(const AttentionParams& p, int32_t s)
{
    return count_of(p, work_of(p, sequence(p.b, s)));
}

// Sum over the wave, in every lane.
__device__ __forceinline__ int64_t wave_sum(int64_t v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int64_t wave_prefix(int64_t v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
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

// Units of a workgroup: an even share, but no fewer than one for each wave.
__device__ __forceinline__ int64_t share_of(int64_t all)
{
    const int64_t s = (all + kWorkgroups - 1) / kWorkgroups;
    return s < kWaves ? kWaves : s;
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The first unit of this workgroup, the units before its sequence, and the
// sequence (b.S: no work).
struct Start {
    int64_t share, all, unit, before;
    int32_t s;
};
__device__ __forceinline__ Start start_of(const AttentionParams& p)
{
    const int lane = threadIdx.x & 63;
    Start r;
    int64_t mine = lane < p.b.S ? units_of(p, lane) : 0, upto = wave_prefix(mine), base = 0;
    r.all = uniform64(__shfl(upto, 63));
    for (int32_t s0 = 64; s0 < p.b.S; s0 += 64) r.all += uniform64(wave_sum(s0 + lane < p.b.S ? units_of(p, s0 + lane) : 0));
    r.share = share_of(r.all);
    r.unit = (int64_t)blockIdx.x * r.share;
    r.before = 0;
    r.s = p.b.S;
    if (r.unit >= r.all) return r;
    for (int32_t s0 = 0; s0 < p.b.S; s0 += 64) {
        if (s0) {
            mine = s0 + lane < p.b.S ? units_of(p, s0 + lane) : 0;
            upto = wave_prefix(mine);
        }
        const uint64_t past = __builtin_amdgcn_ballot_w64(base + upto > r.unit);
        if (past) {
            const int l = __builtin_ctzll(past);
            r.before = uniform64(base + __shfl(upto - mine, l));
            r.s = uniform(s0 + l);
            return r;
        }
        base += uniform64(__shfl(upto, 63));
    }
    return r;
}

__device__ __forceinline__ float xor16_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

// A row's place: its token (of the sequence) and its head of q.  (A sequence
// has fewer than 2^20 * 64 rows.)
struct Row {
    int32_t token, head;
};
__device__ __forceinline__ Row row_of(const AttentionParams& p, uint32_t row, int32_t h)
{
    const uint32_t t = row / (uint32_t)p.G;
    return Row{(int32_t)t, (int32_t)(h * p.G + (row - t * p.G))};
}

// Byte B of each of four words.
template <int B>
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    constexpr uint32_t kLow = 0x0C0C0000u | (4u + B) << 8 | B, kHigh = (4u + B) << 24 | (uint32_t)B << 16 | 0x0C0Cu;
    return __builtin_amdgcn_perm(b, a, kLow) | __builtin_amdgcn_perm(d, c, kHigh);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }   // v_exp_f32: one step off at most
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kWaves, D <= 128 ? 2 : 1) void mnb_attention_rows_kernel(AttentionParams p)
{
    constexpr int KS = D / 64, DT = D / 16;
    __shared__ float lds_o[kWaves][16][D + 4];
    __shared__ float lds_m[kWaves][16], lds_l[kWaves][16];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Start start = start_of(p);
    int64_t u = start.unit, before = start.before;
    const int64_t end = u + start.share < start.all ? u + start.share : start.all;
    int32_t s = start.s;
    if (s >= p.b.S) return;
    const int P = 1 << p.b.page_bits;
    for (; u < end; ) {
        // The segment: units c0 .. c1 - 1 of sequence s, head h, row tile rt.
        Sequence q = uniform_sequence(p.b, s);
        Work w = work_of(p, q);
        while (u - before >= count_of(p, w)) {   // on to the next sequence with work
            before += count_of(p, w);
            if (++s >= p.b.S) return;
            q = uniform_sequence(p.b, s);
            w = work_of(p, q);
        }
        // (At most 2^2 tiles, 2^18 units and 2^8 heads.)
        const uint32_t in = (uint32_t)(u - before), each = (uint32_t)(w.units + kBegin), pair = in / each;
        const int from = (int)(in - pair * each) - kBegin, to = end - u < w.units - from ? from + (int)(end - u) : w.units;
        const int32_t h = (int32_t)(pair / (uint32_t)w.tiles), rt = (int32_t)(pair - h * w.tiles);
        u += to - from;
        const int c0 = from < 0 ? 0 : from, c1 = to;
        if (c1 <= c0) continue;
        const bool first_part = c0 > 0, whole = c0 == 0 && c1 == w.units;

        // This lane's row.  Rows past the last one repeat it and are not stored.
        const int32_t rows = q.n * p.G, row0 = rt * 16;
        const Row at = row_of(p, row0 + r < rows ? row0 + r : rows - 1, h);
        const int32_t position = q.length - q.n + at.token;
        const int32_t lowest = q.length - q.n + row_of(p, row0, h).token;   // of the tile's rows
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
            const bool finite = top < (BF16 ? 0x7F80u : 0x7C00u);
            // |x| < 2^ex, and n = rint(x 2^(22 - ex)) in the low bits of n + 1.5 * 2^23.
            // The three signed digits of n are the bytes of n + 0x808080, each with
            // its top bit turned.
            const int ex = (int)(__float_as_uint(widen16(top, BF16)) >> 23) - 126;
            const float pre = ex < -64 ? pow2(64) : 1.f, up = finite ? pow2((ex < -64 ? -42 : 22) - ex) : 0.f;
            uint32_t sum = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t pair2 = raw[k][i >> 1][(i & 1) * 2 + (j >> 1)];
                        const float x = widen16(j & 1 ? pair2 >> 16 : pair2 & 0xFFFFu, BF16);
                        const uint32_t n = __float_as_uint(fmaf(x * pre, up, 12582912.f)) - 0x4B400000u;
                        sum += n;
                        w[j] = n + 0x808080u;
                    }
                    qd[0][k][i] = (int)(pack_bytes<0>(w[0], w[1], w[2], w[3]) ^ 0x80808080u);
                    qd[1][k][i] = (int)(pack_bytes<1>(w[0], w[1], w[2], w[3]) ^ 0x80808080u);
                    qd[2][k][i] = (int)(pack_bytes<2>(w[0], w[1], w[2], w[3]) ^ 0x80808080u);
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            half = (int)sum >> 1;
            q_scale = finite ? p.scale_log2 * pow2(ex < -64 ? -64 : ex) * pow2(ex < -64 ? ex + 42 : -22)
                             : __uint_as_float(0x7FC00000u);
        }

        float4_t o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = float4_t{0.f, 0.f, 0.f, 0.f};
        float top = kLowest, weight = 0.f, halves = 0.f;   // weight, halves: this lane's keys only

        // Sixteen keys (a run) lie within a page.  Lane (r, g) loads keys of run r / 4
        // for the scores and holds run g afterwards.  The loads of a unit are
        // issued as the one before it lets go of their registers, its pages are
        // looked up one unit before that.
        const int32_t* table = p.b.table + (int64_t)s * p.b.max_pages;
        auto entry = [&](int c, int run) {
            const int32_t index = (c * 64 + 16 * run) >> p.b.page_bits;
            return index < p.b.max_pages ? table[index] : -1;
        };
        auto usable = [&](int32_t page) { return page >= 0 && page < p.b.pages; };
        i32x4 a[4][KS], v[DT];
        float ks, vs;
        bool ok;                 // run g lies in a usable page
        auto load_keys = [&](int c, int32_t page_k, int32_t page_v) {
            const int32_t key = c * 64 + 16 * (r >> 2) + (r & 3);
            const int8_t* kp = p.k_pages + ((((int64_t)(usable(page_k) ? page_k : 0) * p.heads + h) << p.b.page_bits) +
                                            (key & (P - 1))) * D + 16 * g;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    a[t][k] = *reinterpret_cast<const i32x4*>(kp + 4 * t * D + 64 * k);
            // The scales of a run behind the sequence's last token mean nothing; a page
            // of 64 tokens or more has one value scale for the whole unit.
            ok = usable(page_v);
            const int64_t at = (int64_t)(ok ? page_v : 0) * p.heads + h;
            const bool live = ok && c * 64 + 16 * g < q.length;
            ks = live ? p.k_scales[at] : 0.f;
            vs = live || (ok && P >= 64) ? p.v_scales[at] : 0.f;
        };
        auto load_values = [&](int c, int32_t page_v) {
            const int8_t* vp = p.v_pages + (((int64_t)(usable(page_v) ? page_v : 0) * p.heads + h) << p.b.page_bits) * D +
                               (int64_t)r * P + ((c * 64 + 16 * g) & (P - 1));
#pragma unroll
            for (int d = 0; d < DT; ++d) v[d] = *reinterpret_cast<const i32x4*>(vp + (int64_t)16 * d * P);
        };
        int c = c0 + wave;
        int32_t next_k = 0, next_v = 0;
        if (c < c1) {
            next_k = entry(c, r >> 2);
            next_v = entry(c, g);
            load_keys(c, next_k, next_v);
            load_values(c, next_v);
            if (c + kWaves < c1) {
                next_k = entry(c + kWaves, r >> 2);
                next_v = entry(c + kWaves, g);
            }
        }
        for (; c < c1; c += kWaves) {
            const bool more = c + kWaves < c1;
            const int32_t key0 = c * 64, run0 = key0 + 16 * g;
            const float v_scale = fabsf(vs);
            float x[16];
            const float factor = q_scale * ks, bias = ok ? 0.f : -__builtin_inff();
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
                if (t & 1) __builtin_amdgcn_sched_barrier(0);     // keeps the sums of few tiles live
            }
            if (more) load_keys(c + kWaves, next_k, next_v);
            __builtin_amdgcn_sched_barrier(0);
            if (key0 + 63 > lowest)
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = run0 + j <= position ? x[j] : -__builtin_inff();

            float m_run = x[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) m_run = fmaxf(m_run, x[j]);
            const float m_unit = xor16_max(m_run);
            const bool any = m_unit != -__builtin_inff();       // the row sees a key of the unit
            const float m_from = any ? m_unit : 0.f;
            const float now = fmaxf(top, m_unit);
            const float keep = exp2_fast(top - now), f_weight = exp2_fast(m_unit - now);
            top = now;
            // The weights are held against the unit's largest weight times value scale.
            float step = 32512.f, f_o;
            if (P >= 64) {
                f_o = any ? f_weight * v_scale * (1.f / 32512.f) : 0.f;
            } else {
                const bool seen = m_run != -__builtin_inff();
                const float lvs = seen ? __log2f(v_scale) : -__builtin_inff();
                const float n_unit = xor16_max(m_run + lvs);
                const bool some = n_unit != -__builtin_inff();
                step = seen && some ? 32512.f * exp2_fast(m_from + lvs - n_unit) : 0.f;
                f_o = some ? exp2_fast(n_unit - now) * (1.f / 32512.f) : 0.f;
            }
            // (A scale that is not finite has no largest: it goes into the sum.)
            float sum = m_run != -__builtin_inff() ? v_scale - v_scale : 0.f;
            uint32_t lo[16], hi[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float e = exp2_fast(x[j] - m_from);
                sum += e;
                lo[j] = __float_as_uint(fmaf(e, step, 12582912.f));
                hi[j] = __float_as_uint(fmaf(e, step, 12582912.f + 128.f));
            }
            weight = weight * keep + sum * f_weight;
            halves = halves * keep + sum * step * f_o;
            i32x4 b_lo, b_hi;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b_lo[i] = (int)pack_bytes<0>(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                b_hi[i] = (int)pack_bytes<1>(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
            }
            if (__builtin_amdgcn_ballot_w64(keep != 1.f))
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d] *= keep;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const i32x4 zero = i32x4{0, 0, 0, 0};
                const i32x4 sh = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[d], b_hi, zero, 0, 0, 0);
                const i32x4 sl = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[d], b_lo, zero, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[d][i] = fmaf((float)((sh[i] << 8) + sl[i]), f_o, o[d][i]);
                if (d & 1) __builtin_amdgcn_sched_barrier(0);
            }
            if (more) {
                load_values(c + kWaves, next_v);
                if (c + 2 * kWaves < c1) {
                    next_k = entry(c + 2 * kWaves, r >> 2);
                    next_v = entry(c + 2 * kWaves, g);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
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
        const float f = exp2_fast(top - m_all);
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
            for (int i = 0; i < kWaves; ++i) l_row += lds_l[i][row] * exp2_fast(lds_m[i][row] - m_row);
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
                    for (int e = 0; e < D / 16; ++e) dst[e] = narrow16(y[e] * inv, BF16);
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
// the keys.  Sequences without keys get rows of zeros.  Grid: (row tiles, heads,
// D / 64); a workgroup takes 64 elements of each of 16 rows.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void mnb_attention_join_kernel(AttentionParams p)
{
    __shared__ float factor[16][kMostParts + 1];
    __shared__ float inverse[16];
    __shared__ float4_t meet[256];
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
    const int64_t share = share_of(all);
    const int64_t u0 = before + ((int64_t)h * w.tiles + rt) * (w.units + kBegin) + kBegin, u1 = u0 + w.units;
    const int64_t w0 = divide(u0, share);
    const int parts = w.units ? (int)(divide(u1 - 1, share) - w0) + 1 : 0;
    if (parts == 1) return;              // stored by that workgroup
    const int rows = q.n * p.G - (int)rt * 16, count = rows < 16 ? rows : 16;
    auto part_of = [&](int i) { return (2 * (w0 + i) + (i == 0 ? 1 : 0)) * 16; };
    {
        const int row = threadIdx.x >> 4, j = threadIdx.x & 15;
        float m = kLowest, l = 0.f;
        if (row < count)
            for (int i = j; i < parts; i += 16) m = fmaxf(m, p.part_ml[(part_of(i) + row) * 2]);
#pragma unroll
        for (int d = 8; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
        if (row < count)
            for (int i = j; i < parts; i += 16) {
                const float f = exp2_fast(p.part_ml[(part_of(i) + row) * 2] - m);
                factor[row][i] = f;
                l += p.part_ml[(part_of(i) + row) * 2 + 1] * f;
            }
#pragma unroll
        for (int d = 8; d; d >>= 1) l += __shfl_xor(l, d);
        if (j == 0) inverse[row] = l == 0.f ? 0.f : 1.f / l;
    }
    __syncthreads();
    // Four elements of a row a thread; with few rows, groups of threads take every
    // so many of the parts.
    const int ways = count > 8 ? 1 : count > 4 ? 2 : count > 2 ? 4 : count > 1 ? 8 : 16, width = 256 / ways;
    const int way = threadIdx.x / width, row = (threadIdx.x % width) >> 4, e = (threadIdx.x & 15) * 4 + 64 * (int)blockIdx.z;
    float4_t y = float4_t{0.f, 0.f, 0.f, 0.f};
    if (row < count) {
#pragma unroll 4
        for (int i = way; i < parts; i += ways)
            y += *reinterpret_cast<const float4_t*>(p.part_o + (part_of(i) + row) * D + e) * factor[row][i];
    }
    meet[threadIdx.x] = y;
    __syncthreads();
    if (way == 0 && row < count) {
        for (int i = 1; i < ways; ++i) y += meet[threadIdx.x + i * width];
        y *= inverse[row];
        const Row to = row_of(p, (uint32_t)rt * 16 + row, h);
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (q.t0 + to.token) * p.out_stride + (int64_t)to.head * D + e);
        dst[0] = (uint32_t)narrow16(y[0], BF16) | (uint32_t)narrow16(y[1], BF16) << 16;
        dst[1] = (uint32_t)narrow16(y[2], BF16) | (uint32_t)narrow16(y[3], BF16) << 16;
    }
}

template <int D, bool BF16>
int queue(AttentionParams& p, hipStream_t stream)
{
    hipLaunchKernelGGL((mnb_attention_rows_kernel<D, BF16>), dim3(kWorkgroups), dim3(64 * kWaves), 0, stream, p);
    int e = (int)hipGetLastError();
    if (e != 0) return e;
    hipLaunchKernelGGL((mnb_attention_join_kernel<D, BF16>), dim3((unsigned)p.slots, (unsigned)p.heads, D / 64), dim3(256), 0,
                       stream, p);
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
    p.scale_log2 = a.scale * 1.44269504088896340736f;
    const AttentionLayout lay = attention_layout(a.cache.head_dim);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.part_ml = reinterpret_cast<float*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + lay.o);
    p.many = INT32_MAX;
    p.slots = (int32_t)(a.batch.tokens * p.G / 16 + a.batch.sequences);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    *launches = 2;
    switch (a.cache.head_dim) {
    case 64: return a.bf16 ? queue<64, true>(p, s) : queue<64, false>(p, s);
    case 128: return a.bf16 ? queue<128, true>(p, s) : queue<128, false>(p, s);
    default: return a.bf16 ? queue<256, true>(p, s) : queue<256, false>(p, s);
    }
}

}  // namespace mnb
