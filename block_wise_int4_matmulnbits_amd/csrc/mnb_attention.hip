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
//   digits: off by 1 / 65024 of the largest at most, where fp16 weights would be
//   off by 2^-11 of each.  (A third digit spills: heads of 128 102 -> 144 us in the
//   batch below, of 256 213 -> 367.)
//
// The batch's units are shared out evenly over a fixed number of workgroups, whose
// sums of the (at most two) row tiles that others share too are joined by a second
// launch, a workgroup for each border between two shares.  64 sequences of one token
// over 4000 keys, 32 heads on 8, read 5.7 / 5.1 / 4.9 TB/s with heads of 64 / 128 / 256
// (a plain read of as much 7.0); one token over 2049 keys takes 11 us, two launches of
// dependent loads.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "mnb.h"
#include "mnb_cache.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kWorkgroups = kAttentionWorkgroups;
constexpr int kBegin = kAttentionBegin;
constexpr int kGridTiles = 32768;     // tiles of a grid's y
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
    float* tile_o;            // [2 shares][tile rows][D]: sums of tiles that workgroups share
    float* tile_ml;           // [2 shares][tile rows][2]
    int64_t q_stride, out_stride;
    int32_t heads, G;         // key heads, rows a token has for each
    int32_t many;             // sequences of more rows than this go to the tiles
    int32_t tile_slots, shares;   // of the tiles' grid
    int32_t small;            // up to 64 sequences, whose work (but for the heads) fits 32 bits
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
    return (int64_t)w.tiles * (w.units + kBegin) * p.heads;
}
// The same without the heads, of this lane's sequence (p.small).
__device__ __forceinline__ int32_t small_count(const AttentionParams& p, const Sequences& all)
{
    const Work w = work_of(p, all.mine);
    return (int)(threadIdx.x & 63) < p.b.S ? w.tiles * (w.units + kBegin) : 0;
}

// Sum over the lanes up to this one, in the manner of wave_prefix32; and over all.
template <int kControl, int kRows>
__device__ __forceinline__ int64_t from_lane(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)v, kControl, kRows, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)(v >> 32), kControl, kRows, 0xF, false);
    return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int64_t wave_prefix(int64_t v)
{
    v += from_lane<0x111, 0xF>(v);
    v += from_lane<0x112, 0xF>(v);
    v += from_lane<0x114, 0xF>(v);
    v += from_lane<0x118, 0xF>(v);
    v += from_lane<0x142, 0xA>(v);
    v += from_lane<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ int64_t read_lane(int64_t v, int lane)
{
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int32_t)(v >> 32), lane) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int32_t)v, lane));
}
__device__ __forceinline__ int64_t wave_sum(int64_t v) { return read_lane(wave_prefix(v), 63); }

// The largest of the wave.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)v, 0x111, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)v, 0x112, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)v, 0x114, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)v, 0x118, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)v, 0x142, 0xA, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int32_t)v, 0x143, 0xC, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int32_t)v, 63);
}

// A count of every sequence, summed: lane l has an equal run of the sequences.  f(q,
// valid) counts sequence q (0 where it is not valid).
struct Counts {
    int64_t mine, upto, all;
    int32_t each;             // sequences of a lane
};
template <class F>
__device__ __forceinline__ Counts count_sequences(const CacheBatch& b, const Sequences& seqs, F f)
{
    const int32_t lane = threadIdx.x & 63;
    Counts c;
    c.each = (b.S + 63) >> 6;
    if (b.S <= 64) {
        c.mine = f(seqs.mine, lane < b.S);
    } else {
        c.mine = 0;
#pragma unroll 4
        for (int32_t i = 0; i < c.each; ++i) {
            const int32_t s = lane * c.each + i;
            c.mine += f(sequence(b, s < b.S ? s : b.S - 1), s < b.S);
        }
    }
    c.upto = wave_prefix(c.mine);
    c.all = read_lane(c.upto, 63);
    return c;
}

// The sequence that holds count `at`, and the count of those before it (s: b.S for none).
struct Holder {
    int64_t before;
    int32_t s;
    Sequence q;
};
template <class F>
__device__ __forceinline__ Holder find_holder(const CacheBatch& b, const Sequences& seqs, const Counts& c, int64_t at, F f)
{
    const int32_t lane = threadIdx.x & 63;
    Holder r{0, b.S, Sequence{0, 0, 0}};
    const uint64_t past = __builtin_amdgcn_ballot_w64(c.upto > at);
    if (!past) return r;
    const int32_t l = __builtin_ctzll(past);
    r.before = read_lane(c.upto - c.mine, l);
    if (b.S <= 64) {
        r.s = l;
        r.q = seqs.at(l);
        return r;
    }
    for (int32_t j = 0; j < c.each; j += 64) {
        const int32_t s = l * c.each + j + lane;
        const bool valid = j + lane < c.each && s < b.S;
        const Sequence q = sequence(b, valid ? s : b.S - 1);
        const int64_t mine = f(q, valid), upto = r.before + wave_prefix(mine);
        const uint64_t here = __builtin_amdgcn_ballot_w64(upto > at);
        if (here) {
            const int k = __builtin_ctzll(here);
            r.s = l * c.each + j + k;
            r.before = read_lane(upto - mine, k);
            r.q = Sequence{__builtin_amdgcn_readlane(q.t0, k), __builtin_amdgcn_readlane(q.n, k),
                           __builtin_amdgcn_readlane(q.length, k)};
            return r;
        }
        r.before = read_lane(upto, 63);
    }
    return r;
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

// Where share `number` begins: its first unit, the units before its sequence, and the
// sequence (b.S: no work).
struct Start {
    int64_t share, all, unit, before;
    int32_t s;
};
__device__ __forceinline__ Start start_of(const AttentionParams& p, const Sequences& seqs, int64_t number)
{
    Start r;
    r.before = 0;
    r.s = p.b.S;
    if (p.small) {
        const int32_t mine = small_count(p, seqs), upto = wave_prefix32(mine);
        r.all = (int64_t)__builtin_amdgcn_readlane(upto, 63) * p.heads;
        r.share = share_of(r.all);
        r.unit = number * r.share;
        if (r.unit >= r.all) return r;
        r.s = __builtin_ctzll(__builtin_amdgcn_ballot_w64((int64_t)upto * p.heads > r.unit));
        r.before = (int64_t)__builtin_amdgcn_readlane(upto - mine, r.s) * p.heads;
        return r;
    }
    auto count = [&](const Sequence& q, bool valid) { return valid ? count_of(p, work_of(p, q)) : 0; };
    const Counts c = count_sequences(p.b, seqs, count);
    r.all = c.all;
    r.share = share_of(r.all);
    r.unit = number * r.share;
    if (r.unit >= r.all) return r;
    const Holder at = find_holder(p.b, seqs, c, r.unit, count);
    r.before = at.before;
    r.s = at.s;
    return r;
}

// The larger of the lanes l and l ^ 32, and of the four lanes that share l % 16.
__device__ __forceinline__ float xor32_max(float v)
{
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
}
__device__ __forceinline__ float xor16_max(float v)
{
    const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return xor32_max(fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1])));
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

// The y-th tile of BR rows, counted from the last one, among the sequences of
// many rows (b.S: none).
struct Tile {
    int32_t s, rt;
    Sequence q;
};
__device__ __forceinline__ int32_t tiles_of(const AttentionParams& p, const Sequence& q, int BR)
{
    const int32_t rows = q.n * p.G;
    return rows > p.many ? (rows + BR - 1) / BR : 0;
}
__device__ __forceinline__ Tile tile_of(const AttentionParams& p, const Sequences& seqs, int32_t y, int BR)
{
    auto count = [&](const Sequence& q, bool valid) { return valid ? (int64_t)tiles_of(p, q, BR) : 0; };
    const Counts c = count_sequences(p.b, seqs, count);
    const int64_t v = c.all - 1 - y;
    Tile t{p.b.S, 0, Sequence{0, 0, 0}};
    if (v < 0 || y >= p.tile_slots) return t;
    const Holder at = find_holder(p.b, seqs, c, v, count);
    t.s = at.s;
    t.rt = (int32_t)(v - at.before);
    t.q = at.q;
    return t;
}

// The work of tiles (tiles_cut says when it is shared out).  Tile i of a sequence sees
// about start + (i + 1) BR / G keys, and counts as that and as kTileBegin units (64 keys)
// more; counts are in 1 / G of a key, so that those of the tiles before i have a closed
// form.
struct Count {
    int64_t first, tiles;     // of a tile but for its own rows; tiles of the sequence
    int32_t BR;
    __device__ __forceinline__ int64_t upto(int64_t i) const { return i * first + BR * (i * (i + 1) / 2); }
    __device__ __forceinline__ int64_t all() const { return upto(tiles); }
};
__device__ __forceinline__ Count count_tiles(const AttentionParams& p, const Sequence& q, int BR)
{
    const int32_t cap = p.b.max_pages << p.b.page_bits;
    return Count{(int64_t)p.G * (clamp32(q.length - q.n, 0, cap) + 64 * kTileBegin), tiles_of(p, q, BR), BR};
}

// Where a border between shares lies: sequence s, key head h, tile rt, and how far
// into its count (s: b.S where the batch ends before).  cut: false where whole tiles
// take no longer than shares.
struct Place {
    int64_t all, share, in;
    int32_t s, h, rt;
    bool cut;
    Sequence q;
    Count c;
};
__device__ __forceinline__ Place place_of(const AttentionParams& p, const Sequences& seqs, int64_t border, int BR)
{
    Place r;
    int64_t tiles = 0;
    uint32_t longest = 0;                 // count of a tile: 64 heads of 2^24 keys at most, and its own rows
    const Counts counts = count_sequences(p.b, seqs, [&](const Sequence& q, bool valid) {
        const Count c = count_tiles(p, q, BR);
        if (!valid || c.tiles == 0) return (int64_t)0;
        tiles += c.tiles;
        longest = max(longest, (uint32_t)(c.first + c.tiles * BR));
        return c.all() * p.heads;
    });
    tiles = wave_sum(tiles);
    longest = wave_max(longest);
    r.all = counts.all;
    r.share = uniform64(tile_share(divide(r.all + p.shares - 1, p.shares), p.G));
    r.cut = tiles_cut(r.all, tiles * p.heads, longest, p.G, p.shares, r.share, [](int64_t a, int64_t b) { return divide(a, b); });
    const int64_t at = border * r.share;
    r.s = p.b.S;
    r.h = r.rt = 0;
    r.in = 0;
    if (!r.cut || at >= r.all) return r;
    const Holder holder = find_holder(p.b, seqs, counts, at, [&](const Sequence& q, bool valid) {
        return valid ? count_tiles(p, q, BR).all() * p.heads : 0;
    });
    r.s = holder.s;
    r.q = holder.q;
    r.c = count_tiles(p, r.q, BR);
    r.in = at - holder.before;
    if (r.s >= p.b.S || r.in < 0) {       // (numbers of the batch that overflow)
        r.s = p.b.S;
        return r;
    }
    r.h = uniform((int32_t)divide(r.in, r.c.all()));
    r.in -= r.h * r.c.all();
    r.rt = wave_search((int32_t)r.c.tiles, r.in, [&](int32_t i) { return r.c.upto(i); });
    r.in -= r.c.upto(r.rt);
    return r;
}

// SMALL: pages of less than 64 tokens, several scales in a unit.
template <int D, bool BF16, bool SMALL>
__global__ __launch_bounds__(64 * kWaves, D <= 128 ? 2 : 1) void mnb_attention_rows_kernel(AttentionParams p)
{
    constexpr int KS = D / 64, DT = D / 16;
    // Pieces of a unit's keys and values that registers hold: all, or half, each one's
    // successor loaded as it is multiplied (heads of 256, all: spills, 64 sequences over
    // 4000 keys 289 -> 213 us; two waves a SIMD on half as many registers: 434).
    constexpr int KT = D <= 128 ? 4 : 2, VT = D <= 128 ? DT : DT / 2;
    __shared__ float lds_o[kWaves][16][D + 4];
    __shared__ float lds_m[kWaves][16], lds_l[kWaves][16];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Sequences seqs(p.b);
    const Start start = start_of(p, seqs, blockIdx.x);
    int64_t u = start.unit, before = start.before;
    const int64_t end = u + start.share < start.all ? u + start.share : start.all;
    int32_t s = start.s;
    if (s >= p.b.S) return;
    const int P = 1 << p.b.page_bits;
    for (; u < end; ) {
        // The segment: units c0 .. c1 - 1 of sequence s, head h, row tile rt.
        Sequence q = seqs.at(s);
        Work w = work_of(p, q);
        while (u - before >= count_of(p, w)) {   // on to the next sequence with work
            before += count_of(p, w);
            if (++s >= p.b.S) return;
            q = seqs.at(s);
            w = work_of(p, q);
        }
        const int64_t in = u - before, pair64 = divide(in, w.units + kBegin);
        const uint32_t pair = (uint32_t)pair64;      // tiles and heads: at most 2^22 and 2^8
        const int from = (int)(in - pair64 * (w.units + kBegin)) - kBegin, to = end - u < w.units - from ? from + (int)(end - u) : w.units;
        const int32_t h = (int32_t)(pair / (uint32_t)w.tiles), rt = (int32_t)(pair - h * w.tiles);
        u += to - from;
        const int c0 = from < 0 ? 0 : from, c1 = to < 0 ? 0 : to;
        if (c1 <= c0 && (w.units || from != -kBegin)) continue;      // (no keys at all: zeros)
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
            // (At least 2^-100: the factor of the scores stays a normal number.)
            const int ex = max((int)(__float_as_uint(widen16(top, BF16)) >> 23), 26) - 126;
            const float up = finite ? pow2(22 - ex) : 0.f;
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
                        const uint32_t n = __float_as_uint(fmaf(x, up, 12582912.f)) - 0x4B400000u;
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
            q_scale = finite ? p.scale_log2 * pow2(ex - 22) : __uint_as_float(0x7FC00000u);
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
        i32x4 a[KT][KS], v[VT];
        float ks, vs;
        bool ok;                 // run g lies in a usable page
        const int8_t *kp, *vp;   // the lane's part of the unit whose pieces are loaded next
        auto keys_at = [&](int c, int32_t page) {
            const int32_t key = c * 64 + 16 * (r >> 2) + (r & 3);
            kp = p.k_pages + ((((int64_t)(usable(page) ? page : 0) * p.heads + h) << p.b.page_bits) + (key & (P - 1))) * D + 16 * g;
        };
        auto load_keys = [&](int t) {
#pragma unroll
            for (int k = 0; k < KS; ++k) a[t % KT][k] = *reinterpret_cast<const i32x4*>(kp + 4 * t * D + 64 * k);
        };
        auto load_scales = [&](int c, int32_t page) {
            // The scales of a run behind the sequence's last token mean nothing; a page
            // of 64 tokens or more has one value scale for the whole unit.
            ok = usable(page);
            const int64_t at = (int64_t)(ok ? page : 0) * p.heads + h;
            const bool live = ok && c * 64 + 16 * g < q.length;
            ks = live ? p.k_scales[at] : 0.f;
            vs = live || (ok && !SMALL) ? p.v_scales[at] : 0.f;
        };
        auto values_at = [&](int c, int32_t page) {
            vp = p.v_pages + (((int64_t)(usable(page) ? page : 0) * p.heads + h) << p.b.page_bits) * D + (int64_t)r * P +
                 ((c * 64 + 16 * g) & (P - 1));
        };
        auto load_values = [&](int d) { v[d % VT] = *reinterpret_cast<const i32x4*>(vp + (int64_t)16 * d * P); };
        int c = c0 + wave;
        int32_t next_k = 0, next_v = 0;
        if (c < c1) {
            next_k = entry(c, r >> 2);
            next_v = entry(c, g);
            keys_at(c, next_k);
#pragma unroll
            for (int t = 0; t < KT; ++t) load_keys(t);
            load_scales(c, next_v);
            values_at(c, next_v);
#pragma unroll
            for (int d = 0; d < VT; ++d) load_values(d);
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
            const float factor = ok ? q_scale * ks : 0.f, bias = ok ? 0.f : -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                i32x4 c0v = i32x4{half, half, half, half}, c1v = i32x4{0, 0, 0, 0}, c2v = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    c0v = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[t % KT][k], qd[0][k], c0v, 0, 0, 0);
                    c1v = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[t % KT][k], qd[1][k], c1v, 0, 0, 0);
                    c2v = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[t % KT][k], qd[2][k], c2v, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[4 * t + i] = fmaf(fmaf((float)((c2v[i] << 8) + c1v[i]), 256.f, (float)c0v[i]), factor, bias);
                if (KT < 4) {
                    if (t + KT == 4 && more) keys_at(c + kWaves, next_k);
                    if (t + KT < 4 || more) load_keys((t + KT) % 4);
                }
                if (KT < 4 || (t & 1)) __builtin_amdgcn_sched_barrier(0);     // keeps the sums of few tiles live
            }
            if (more) {
                if (KT == 4) {
                    keys_at(c + kWaves, next_k);
#pragma unroll
                    for (int t = 0; t < 4; ++t) load_keys(t);
                }
                load_scales(c + kWaves, next_v);
            }
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
            // The weights are held against the unit's largest weight times value scale, which
            // stands 2^up above the unit's largest weight.  A run whose scale is more than
            // 2^64 above that (its scores lie as far below) has its exponentials taken from
            // where it would reach it, so that no factor overflows.
            float step = 32512.f, f_o, from = m_from;
            if constexpr (!SMALL) {
                f_o = any ? f_weight * v_scale : 0.f;
            } else {
                const bool seen = m_run != -__builtin_inff() && v_scale >= 0x1p-126f;     // (log2 takes no smaller ones)
                const float n_unit = xor16_max(seen ? m_run + __log2f(v_scale) : -__builtin_inff());
                const bool some = n_unit != -__builtin_inff();
                const float up = some ? n_unit - m_from : 0.f;
                const float over = (float)__builtin_amdgcn_frexp_expf(v_scale) - up;
                const bool far = seen && over > 64.f;
                from = far ? m_from - over : m_from;
                step = seen && some ? 32512.f * __builtin_amdgcn_frexp_mantf(v_scale) * (far ? 1.f : exp2_fast(over)) : 0.f;
                // (2^up by its exponent and the rest: it may lie below exp2's range.)
                const float whole_up = rintf(up);
                f_o = some ? ldexpf(exp2_fast(up - whole_up) * f_weight, (int)whole_up) : 0.f;
            }
            // (A scale that is not finite has no largest: it goes into the sum.)
            float sum = m_run != -__builtin_inff() ? v_scale - v_scale : 0.f;
            uint32_t lo[16], hi[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float e = exp2_fast(x[j] - from);
                sum += e;
                lo[j] = __float_as_uint(fmaf(e, step, 12582912.f));
                hi[j] = __float_as_uint(fmaf(e, step, 12582912.f + 128.f));
            }
            weight = weight * keep + sum * exp2_fast(from - m_from) * f_weight;
            halves = halves * keep + sum * step * (1.f / 32512.f) * f_o;
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
                const i32x4 sh = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[d % VT], b_hi, zero, 0, 0, 0);
                const i32x4 sl = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[d % VT], b_lo, zero, 0, 0, 0);
                // (1 / 32512 goes to the products: f_o may be next to fp32's smallest.)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[d][i] = fmaf((float)((sh[i] << 8) + sl[i]) * (1.f / 32512.f), f_o, o[d][i]);
                if (VT < DT) {
                    if (d + VT == DT && more) values_at(c + kWaves, next_v);
                    if (d + VT < DT || more) load_values((d + VT) % DT);
                }
                if (d & 1) __builtin_amdgcn_sched_barrier(0);
            }
            if (more) {
                if (VT == DT) {
                    values_at(c + kWaves, next_v);
#pragma unroll
                    for (int d = 0; d < DT; ++d) load_values(d);
                }
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

// Tiles of rows whose keys several workgroups shared: their sums, in the order of the
// keys.  The borders between shares that lie within a tile divide its rows among them,
// D / 4 threads a row; threads that few rows leave take every so many of the parts.
constexpr int kJoinThreads = 256, kJoinEach = 4;     // kJoinEach: workgroups of a border within a tile of many rows
template <int D>
struct Meet {
    float4_t y[kJoinThreads];
    float m[kJoinThreads * 4 / D], l[kJoinThreads * 4 / D];
};
template <int D, bool BF16, int BR>
__device__ __forceinline__ void join_parts(const AttentionParams& p, const float* ml, const float* o, int64_t w0, int parts,
                                           int worker, int workers, const Sequence& q, int32_t h, int32_t row0, Meet<D>& meet)
{
    constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
    const int rows = min(BR, q.n * p.G - row0);
    const int first = rows * worker / workers, count = rows * (worker + 1) / workers - first;
    int ways = GROUPS;
    while (ways > 1 && count > GROUPS / ways) ways >>= 1;
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES, way = group % ways;
    for (int i0 = 0; i0 < count; i0 += GROUPS / ways) {
        const int i = i0 + group / ways;
        const bool mine = i < count;
        const int in = first + (mine ? i : 0);
        float m = kLowest, l = 0.f;
        float4_t y = float4_t{0.f, 0.f, 0.f, 0.f};
        // K parts, all on their way before the first is added.
        auto add = [&](auto batch, int n0) {
            constexpr int K = decltype(batch)::value;
            float its[K], own[K];
            float4_t sums[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int n = n0 + k * ways < parts ? n0 + k * ways : parts - 1;
                const int64_t part = (2 * (w0 + n) + (n == 0 ? 1 : 0)) * BR + in;
                its[k] = ml[part * 2];
                own[k] = ml[part * 2 + 1];
                sums[k] = *reinterpret_cast<const float4_t*>(o + part * D + 4 * lane);
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (n0 + k * ways >= parts) own[k] = 0.f;
                const float now = own[k] == 0.f ? m : fmaxf(m, its[k]), keep = exp2_fast(m - now), f = exp2_fast(its[k] - now);
                m = now;
                l = l * keep + (own[k] == 0.f ? 0.f : own[k] * f);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = y[e] * keep + (own[k] == 0.f ? 0.f : sums[k][e] * f);   // 0: no sums stored
            }
        };
        int n0 = 0;
        for (; parts - n0 > 2 * ways; n0 += 8 * ways) add(std::integral_constant<int, 8>(), n0 + way);
        if (n0 < parts) add(std::integral_constant<int, 2>(), n0 + way);
        if (ways > 1) {
            if (lane == 0) {
                meet.m[group] = m;
                meet.l[group] = l;
            }
            meet.y[threadIdx.x] = y;
            __syncthreads();
            if (way == 0) {
                float m_all = m;
                for (int w = 1; w < ways; ++w) m_all = fmaxf(m_all, meet.m[group + w]);
                float f = exp2_fast(m - m_all);
                l *= f;
                y *= f;
                for (int w = 1; w < ways; ++w) {
                    f = exp2_fast(meet.m[group + w] - m_all);
                    l += meet.l[group + w] * f;
                    y += meet.y[threadIdx.x + w * LANES] * f;
                }
            }
            __syncthreads();
        }
        if (way == 0 && mine) {
            const Row to = row_of(p, row0 + in, h);
            const float by = l == 0.f ? 0.f : 1.f / l;
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (q.t0 + to.token) * p.out_stride + (int64_t)to.head * D + 4 * lane);
            dst[0] = (uint32_t)narrow16(y[0] * by, BF16) | (uint32_t)narrow16(y[1] * by, BF16) << 16;
            dst[1] = (uint32_t)narrow16(y[2] * by, BF16) | (uint32_t)narrow16(y[3] * by, BF16) << 16;
        }
    }
}

// Grid: the borders between the shares of few rows, then those of tiles.
template <int D, bool BF16>
__global__ __launch_bounds__(kJoinThreads) void mnb_attention_join_kernel(AttentionParams p)
{
    constexpr int BR = tile_rows(D);
    __shared__ Meet<D> meet;
    if ((int32_t)blockIdx.x < kWorkgroups - 1) {
        __shared__ Start start;
        __shared__ Sequence sequence_of_start;
        const int64_t border = (int64_t)blockIdx.x + 1;
        if (threadIdx.x < 64) {
            const Sequences seqs(p.b);
            const Start found = start_of(p, seqs, border);
            const Sequence its = found.s < p.b.S ? seqs.at(found.s) : Sequence{0, 0, 0};
            if (threadIdx.x == 0) {
                start = found;
                sequence_of_start = its;
            }
        }
        __syncthreads();
        const Start at = start;
        if (at.s >= p.b.S) return;
        const Sequence q = sequence_of_start;
        const Work w = work_of(p, q);
        const int64_t in = at.unit - at.before, per = w.units + kBegin, pair = divide(in, per);
        const int32_t h = (int32_t)((uint32_t)pair / (uint32_t)w.tiles), rt = (int32_t)(pair - (int64_t)h * w.tiles);
        // The shares w0 .. w1 of the row tile's keys.
        const int64_t u0 = at.unit - (in - pair * per) + kBegin, w0 = divide(u0, at.share);
        const int64_t w1 = divide(u0 + w.units - 1, at.share);
        if (border <= w0 || border > w1) return;
        if (in < 0 || w0 < 0 || h >= p.heads || w1 >= kWorkgroups) return;      // (numbers of the batch that overflow)
        join_parts<D, BF16, 16>(p, p.part_ml, p.part_o, w0, (int)(w1 - w0) + 1, (int)(border - w0) - 1, (int)(w1 - w0), q, h,
                                rt * 16, meet);
        return;
    }
    __shared__ Place place;
    const int32_t id = (int32_t)blockIdx.x - (kWorkgroups - 1);
    const int64_t border = id / kJoinEach + 1;
    if (border >= p.shares) return;
    if (threadIdx.x < 64) {
        const Place found = place_of(p, Sequences(p.b), border, BR);
        if (threadIdx.x == 0) place = found;
    }
    __syncthreads();
    const Place at = place;
    if (at.s >= p.b.S || at.in == 0) return;
    // The shares w0 .. w1 of the tile.
    const int64_t begin = border * at.share - at.in, w0 = divide(begin, at.share);
    const int64_t w1 = divide(begin + at.c.upto(at.rt + 1) - at.c.upto(at.rt) - 1, at.share);
    const int parts = (int)(w1 - w0) + 1;
    if (w0 < 0 || w0 + parts > p.shares || parts < 2) return;      // (numbers of the batch that overflow)
    join_parts<D, BF16, BR>(p, p.tile_ml, p.tile_o, w0, parts, (int)(border - w0 - 1) * kJoinEach + id % kJoinEach,
                            (parts - 1) * kJoinEach, at.q, at.h, at.rt * BR, meet);
}

// ---------------------------------------------------------------- many rows
//
// Tiles of 32 rows a wave, kTileWaves waves, over the keys in units of 64, the
// running maximum and sum in registers; matrix products and the exponentials
// share the time.  The workgroup stages a unit once for all its waves: integers
// as fp16 (q + 1/2 for the keys, (q + 1/2) r for the values; exact) in LDS, two
// units in turn, the next one's loads under way during the products.  Both
// products run on v_mfma_f32_32x32x16_f16:
//
// * scores: 32 keys (A) x 32 rows (B, in registers: fp16 as they are, bf16 under a
//   power of two of the row's own, exact but for what lies below 2^-39 of its
//   largest).  Result lane (row, half) holds keys 8 q + 4 half + j; row m of A
//   carries key 16 (q / 2) + 8 half + 4 (q % 2) + j for m = 8 q + 4 half + j, so that
//   a lane ends with eight neighbouring keys of each 16: the B operand of the
//   second product.
// * outputs: 32 elements (A) x 32 rows, 16 keys deep, the same order, so that a
//   lane stores eight neighbouring elements.  Weights in fp16 (2^-11 of each, which
//   goes into their sum as well): a second piece of them would double this product.
//
// Sixteen keys (a run), or a unit of pages of 64 and more, have one value scale, which
// stands as r times the sums' unit, r a power of two; the rest of the scale goes to the
// weights (not to their sum).  The unit changes, and the sums with it, only where r would leave
// 2^-10 .. 2^8, so that no weight times scale falls out of fp16's range, whatever
// the pages before it held, and pages of differing scales cost nothing.  A row's
// unit follows the keys that it sees: scales of later ones, which rows further down
// see, take nothing from it.
//
// A unit of a tile of 256 rows and heads of 128 takes 2.6 us on its compute unit, of which
// the products are 1.8 at the rate of a large fp16 library product: the exponentials and
// the conversion of the integers hide in part only, as the waves of a workgroup meet at
// a barrier every unit.  2.6 us is 836 TFLOP/s where all units have keys (one sequence of
// 16384); a prompt's short tiles end sooner than they begin.  Eight waves of 32 rows,
// because fewer rows convert the integers more often (four waves of 128 rows: the
// same time); heads of 256 have two waves to 32 rows, as the outputs of one would not
// fit its registers (458 -> 423 us for 512 tokens over 17000 keys).
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float16_t __attribute__((ext_vector_type(16)));

// What a unit's runs need: the factor of the scores, 0 or -infinity to add, and
// the units of the values.
template <int RUNS>
struct Runs {
    float ks[RUNS], bias[RUNS];
    uint32_t spoilt;          // runs with a scale that is not finite
    uint32_t valued;          // runs with a value scale above zero
    uint32_t fractions;       // runs whose value scale is no power of two
    int32_t ref;              // the unit of the first run's sums (bits), and the runs that have it
    uint32_t group;
};

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) { return f16_pair(lo, hi); }

// Sixteen integers to fp16: (q + 1/2) r.  1024 + (q + 128) has the byte in its low
// mantissa bits.
__device__ __forceinline__ void widen_bytes(i32x4 w, uint32_t r2, uint32_t half_r2, u32x4* out)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = (uint32_t)w[i] ^ 0x80808080u;
        const uint32_t a = hadd2(__builtin_amdgcn_perm(0x64646464u, u, 0x04010400u), 0xE480E480u);   // - 1152
        const uint32_t b = hadd2(__builtin_amdgcn_perm(0x64646464u, u, 0x04030402u), 0xE480E480u);
        out[i >> 1][(i & 1) * 2] = hfma2(a, r2, half_r2);
        out[i >> 1][(i & 1) * 2 + 1] = hfma2(b, r2, half_r2);
    }
}

template <int D, bool BF16, bool SMALL>
__global__ __launch_bounds__(64 * tile_waves(D), D == 64 ? 2 : 1) void mnb_attention_tile_kernel(AttentionParams p)
{
    constexpr int RUNS = SMALL ? 4 : 1;                    // of a unit that differ
    constexpr int NW = tile_waves(D), BR = tile_rows(D), THREADS = 64 * NW;
    constexpr int SHARE = 32 * NW / BR;                    // waves that share rows, an equal part of the output each
    constexpr int KQ = D / 16, DB = D / 32 / SHARE;
    constexpr int KROW = D + 8, VROW = 64 + 8;             // fp16; the rows of LDS start 4 banks apart
    constexpr int CHUNKS = 64 * D / 16 / THREADS;          // 16-byte pieces of the keys (and of the values) a thread
    extern __shared__ uint16_t tile_lds[];                 // [2][64][KROW], [2][D][VROW]
    uint16_t* const k_lds = tile_lds;
    uint16_t* const v_lds = tile_lds + 2 * 64 * KROW;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, hh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int part_of_row = wave % SHARE, elem0 = 32 * DB * part_of_row;
    const int32_t cap = p.b.max_pages << p.b.page_bits, P = 1 << p.b.page_bits;

    // A whole tile, counted from the last one, whose rows see the most keys; or those of
    // a share, the first and the last perhaps in part.
    Place at;
    int64_t left = 0;                                      // of the share
    const int32_t y = (int32_t)blockIdx.y + kGridTiles * (int32_t)blockIdx.z, number = y * p.heads + (int32_t)blockIdx.x;
    {
        const Sequences seqs(p.b);
        at.cut = false;
        if (p.shares) at = place_of(p, seqs, number, BR);
        if (at.cut) {
            if (number >= p.shares) return;
            left = at.all - number * at.share < at.share ? at.all - number * at.share : at.share;
        } else {
            const Tile t = tile_of(p, seqs, y, BR);
            at.s = t.s;
            at.h = blockIdx.x;
            at.rt = t.rt;
            at.q = t.q;
        }
    }
    if (at.s >= p.b.S) return;
    for (;;) {
    const int32_t s = at.s, h = at.h, row0 = at.rt * BR;
    const Sequence q = at.q;
    const int32_t rows = q.n * p.G, start = q.length - q.n;
    const int32_t wave0 = row0 + 32 * (wave / SHARE), mine = wave0 + r < rows ? wave0 + r : rows - 1;
    const Row me = row_of(p, mine, h);
    const int32_t position = start + me.token;
    // Positions of the tile's last row and of the wave's first and last one.
    const int32_t last = start + row_of(p, row0 + BR < rows ? row0 + BR - 1 : rows - 1, h).token;
    const int32_t lowest = start + row_of(p, wave0 < rows ? wave0 : rows - 1, h).token;
    const int32_t highest = start + row_of(p, wave0 + 31 < rows ? wave0 + 31 : rows - 1, h).token;
    const int32_t keys = last < 0 ? 0 : last + 1 < cap ? last + 1 : cap;
    const int32_t units = (keys + 63) / 64;
    int32_t c0 = 0, c1 = units;
    bool whole = true;
    int64_t slot = 0;
    if (at.cut) {
        const int64_t count = at.c.upto(at.rt + 1) - at.c.upto(at.rt), end = count - at.in < left ? count : at.in + left;
        whole = at.in == 0 && end == count;
        slot = 2 * (int64_t)number + (at.in ? 0 : 1);
        c0 = uniform((int32_t)divide(units * at.in, count));
        c1 = uniform((int32_t)divide(units * end, count));
        left -= end - at.in;
    }

    half8_t qv[KQ];
    float q_scale;
    bool q_finite;
    {
        const uint16_t* src = p.q + (q.t0 + me.token) * p.q_stride + (int64_t)me.head * D + 8 * hh;
        u32x4 raw[KQ];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KQ; ++k) raw[k] = *reinterpret_cast<const u32x4*>(src + 16 * k);
#pragma unroll
        for (int k = 0; k < KQ; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max_u16x2(top, raw[k][i] & 0x7FFF7FFFu);
        top = (top & 0xFFFFu) > (top >> 16) ? top & 0xFFFFu : top >> 16;
        const uint32_t o = __shfl_xor(top, 32);
        top = o > top ? o : top;
        const bool finite = top < (BF16 ? 0x7F80u : 0x7C00u);
        q_finite = finite;
        // The factor of the scores is kept positive: the scale's sign goes to the row.
        const float size = fabsf(p.scale_log2);
        const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        q_scale = size;
        if constexpr (BF16) {
            const int ex = max((int)(__float_as_uint(widen16(top, 1)) >> 23), 26) - 126;    // |x| < 2^ex, as above
            const float up = pow2(15 - ex);
            q_scale = finite ? size * pow2(ex - 15) : size;
#pragma unroll
            for (int k = 0; k < KQ; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    raw[k][i] = half_pair(bf16_lo(raw[k][i]) * up, bf16_hi(raw[k][i]) * up);
        }
        // (The products of a row that is not finite are done with zeros; it gets its NaN
        // at the end.)
#pragma unroll
        for (int k = 0; k < KQ; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[k][i] = finite ? raw[k][i] ^ sign : 0u;
            qv[k] = __builtin_bit_cast(half8_t, raw[k]);
        }
    }

    // Staging.  Piece i of a thread: key k_token of the unit, elements k_elem ..; and
    // element v_elem, run tid % 4.
    const int32_t* table = p.b.table + (int64_t)s * p.b.max_pages;
    auto entry = [&](int c) {            // lane: the page of run lane % 4 of unit c
        const int32_t index = (c * 64 + 16 * (lane & 3)) >> p.b.page_bits;
        return index < p.b.max_pages ? table[index] : -1;
    };
    auto usable = [&](int32_t page) { return page >= 0 && page < p.b.pages; };
    i32x4 raw_k[CHUNKS], raw_v[CHUNKS];
    float lane_ks, lane_vs;              // of run lane % 4
    bool lane_ok;
    auto load = [&](int c, int32_t page) {
        const int32_t safe = usable(page) ? page : 0;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int id = tid + i * THREADS, token = id / (D / 16), elem = 16 * (id % (D / 16));
            const int64_t pk = __shfl(safe, token >> 4);
            raw_k[i] = *reinterpret_cast<const i32x4*>(
                p.k_pages + (((pk * p.heads + h) << p.b.page_bits) + ((c * 64 + token) & (P - 1))) * D + elem);
            const int ve = id >> 2, run = id & 3;
            raw_v[i] = *reinterpret_cast<const i32x4*>(
                p.v_pages + (((int64_t)safe * p.heads + h) << p.b.page_bits) * D + (int64_t)ve * P +
                ((c * 64 + 16 * run) & (P - 1)));
        }
        lane_ok = usable(page);
        // Scales of a run behind the last key mean nothing.
        const bool live = lane_ok && (!SMALL || c * 64 + 16 * (lane & 3) < keys);
        const int64_t at_scale = (int64_t)safe * p.heads + h;
        lane_ks = live ? fabsf(p.k_scales[at_scale]) : 0.f;
        lane_vs = live ? fabsf(p.v_scales[at_scale]) : 0.f;
    };
    int32_t unit_bits = 0;               // bits of the unit of this row's sums; 0: no sums yet
    int32_t unit_of_all = 0;             // the same, where all rows of the wave have one
    int32_t staged = 0, peak = 0;        // bits of the unit to go on with and of the largest so far: alike in all waves
    Runs<RUNS> now;
    int32_t lane_ref;                    // of run lane % 4: bits of its sums' unit,
    float lane_r, lane_part;             // its value scale as a multiple of that, but for a fraction, and 1 / that
    auto settle = [&](Runs<RUNS>& n) {
        // The value scale is a power of two, vs, times a fraction from 1 to 2, which goes to
        // the weights (1 where append_kv_int8 stored it).  Powers of two by their bits.
        constexpr int32_t kOne = 0x3F800000, kStep = 1 << 23;
        const bool fine = lane_vs < __builtin_inff();      // false for NaN
        const int32_t bits = fine ? __float_as_uint(lane_vs) : 0, vs = bits & 0x7F800000;
        const bool spoilt = !(lane_ks < __builtin_inff()) || !fine, some = vs != 0;
        const float ks = spoilt ? 1.f : lane_ks, bias = lane_ok ? 0.f : -__builtin_inff();
        n.spoilt = (uint32_t)__builtin_amdgcn_ballot_w64(spoilt) & 15u;
        n.valued = (uint32_t)__builtin_amdgcn_ballot_w64(some) & 15u;
        n.fractions = (uint32_t)__builtin_amdgcn_ballot_w64(bits != vs) & 15u;
        lane_part = some && bits != vs ? __builtin_amdgcn_rcpf(__uint_as_float((bits & 0x007FFFFF) | kOne)) : 1.f;
        // A run whose scale is zero, or from 2^-10 to 2^8 of the sums' unit, keeps that
        // unit (128 times 2^8 is within fp16's range); another one has its own, but no less
        // than 2^-80 of the largest one of the keys up to it: so no sum grows by more than
        // that as its unit falls.  (Sums of a unit 2^80 larger have their last bit above what
        // they would lose.  Keys behind a run do not count: rows may not see them.)
        if (!staged && n.valued) staged = __builtin_amdgcn_readlane(vs, __builtin_ctz(n.valued));
        const int32_t base = staged ? staged : kOne;
        const bool near = !some || (uint32_t)vs - (uint32_t)base + 10u * kStep <= 18u * kStep;
        lane_ref = base;
        if (__builtin_amdgcn_ballot_w64(!near)) {
            const int32_t own = near ? base : vs;
            int32_t upto = peak;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t its = __builtin_amdgcn_readlane(own, i);
                upto = (lane & 3) > i ? max(upto, its) : upto;
                peak = max(peak, its);
            }
            lane_ref = max(own, upto - 80 * kStep);
            staged = __builtin_amdgcn_readlane(max(lane_ref, peak - 80 * kStep), 3);
        } else {
            peak = max(peak, staged);
        }
        lane_r = some ? __uint_as_float(max(vs - lane_ref + kOne, 0)) : 0.f;
        n.ref = __builtin_amdgcn_readlane(lane_ref, 0);
        n.group = (uint32_t)__builtin_amdgcn_ballot_w64(lane_ref == n.ref) & 15u;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            n.ks[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), i));
            n.bias[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(bias), i));
        }
    };
    auto store = [&](int buffer) {
        const uint32_t r2 = f16_pair(lane_r, lane_r), half_r2 = f16_pair(0.5f * lane_r, 0.5f * lane_r);
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int id = tid + i * THREADS, token = id / (D / 16), elem = 16 * (id % (D / 16));
            u32x4 w[2];
            widen_bytes(raw_k[i], 0x3C003C00u, 0x38003800u, w);      // 1, 1/2
            u32x4* to = reinterpret_cast<u32x4*>(k_lds + (buffer * 64 + token) * KROW + elem);
            to[0] = w[0];
            to[1] = w[1];
            widen_bytes(raw_v[i], r2, half_r2, w);
            to = reinterpret_cast<u32x4*>(v_lds + (buffer * D + (id >> 2)) * VROW + 16 * (id & 3));
            to[0] = w[0];
            to[1] = w[1];
        }
    };

    float16_t o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    float top = kLowest, weight = 0.f;
    // Row m of A: key (or element) order(m) of its 32.
    const int order = 16 * (r >> 4) + 8 * ((r >> 2) & 1) + 4 * ((r >> 3) & 1) + (r & 3);

    if (c0 < c1) {
        int32_t page = entry(c0);
        load(c0, page);
        page = c0 + 1 < c1 ? entry(c0 + 1) : 0;
        settle(now);
        store(0);
        __syncthreads();
        for (int c = c0; c < c1; ++c) {
            const int buffer = (c - c0) & 1;
            const bool more = c + 1 < c1;
            if (more) {
                load(c + 1, page);
                if (c + 2 < c1) page = entry(c + 2);
            }
            const int32_t key0 = c * 64;
            if (key0 <= highest) {
                // The pieces of A come two steps ahead of their products.
                float16_t x[2];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[b][i] = 0.f;
                const uint16_t* kl = k_lds + (buffer * 64 + order) * KROW + 8 * hh;
                half8_t ka[2][4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ka[0][k] = *reinterpret_cast<const half8_t*>(kl + 32 * (k & 1) * KROW + 16 * (k >> 1));
#pragma unroll
                for (int n = 0; n < KQ / 2; ++n) {
                    if (n + 1 < KQ / 2)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ka[(n + 1) & 1][k] = *reinterpret_cast<const half8_t*>(kl + 32 * (k & 1) * KROW +
                                                                                   32 * (n + 1) + 16 * (k >> 1));
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ka[n & 1][k], qv[2 * n + (k >> 1)], x[k & 1], 0, 0, 0);
                }
                // x[b][8 e + j]: key 32 b + 16 e + 8 hh + j, of run 2 b + e.
                if (key0 + 63 > lowest || now.spoilt) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float y = now.spoilt >> (2 * b + (i >> 3)) & 1 ? __uint_as_float(0x7FC00000u) : x[b][i];
                            x[b][i] = key0 + 32 * b + 16 * (i >> 3) + 8 * hh + (i & 7) <= position ? y : -__builtin_inff();
                        }
                }
                float factor[4], m = -__builtin_inff();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = q_scale * now.ks[e % RUNS];
                    factor[e] = f == 0.f ? 1e-37f : f;      // (a key that is not seen stands at -infinity)
                    float most = x[e >> 1][8 * (e & 1)];
#pragma unroll
                    for (int j = 1; j < 8; ++j) most = fmaxf(most, x[e >> 1][8 * (e & 1) + j]);
                    m = fmaxf(m, fmaf(most, factor[e], now.bias[e % RUNS]));
                }
                m = xor32_max(m);
                // The maximum is followed in steps of 2^6 at least: weights stay below
                // 2^6, and the sums are scaled again in few units.
                if (__builtin_amdgcn_ballot_w64(m > top + 6.f)) {
                    const float next = fmaxf(top, m), keep = exp2_fast(top - next);
                    top = next;
                    weight *= keep;
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[d] *= keep;
                }
                int from_v = (buffer * D + elem0 + order) * VROW + 8 * hh;
                auto values = [&](int e, half8_t (&f)[DB]) {
#pragma unroll
                    for (int d = 0; d < DB; ++d) f[d] = *reinterpret_cast<const half8_t*>(v_lds + from_v + 32 * d * VROW + 16 * e);
                };
                // (Their sum goes without the fraction of the scale.)
                auto weights = [&](int e, float from) {
                    u32x4 pairs;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = exp2_fast(fmaf(x[e >> 1][8 * (e & 1) + 2 * j], factor[e], from));
                        const float b = exp2_fast(fmaf(x[e >> 1][8 * (e & 1) + 2 * j + 1], factor[e], from));
                        pairs[j] = half_pair(a, b);
                        sum = dot2(pairs[j], 0x3C003C00u, sum);
                    }
                    weight = fmaf(sum, __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lane_part), e % RUNS)), weight);
                    return __builtin_bit_cast(half8_t, pairs);
                };
                // The runs of one unit of the sums at a time: all of them, but where their
                // scales lie far apart.
                uint32_t left = 15, group = now.group;
                int32_t ref = now.ref;
                for (;;) {
                    left &= ~group;
                    float from[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) from[e] = !SMALL || (group >> e & 1) ? now.bias[e % RUNS] - top : -__builtin_inff();
                    // A row's unit changes where it sees a value of the new one only.
                    const uint32_t valued = group & now.valued;
                    if (valued && ref != unit_of_all) {
                        const bool turns = unit_bits != ref && key0 + 16 * __builtin_ctz(valued) <= position;
                        const float by = turns && unit_bits ? __uint_as_float(unit_bits) / __uint_as_float(ref) : 1.f;
                        unit_bits = turns ? ref : unit_bits;
                        unit_of_all = __builtin_amdgcn_ballot_w64(unit_bits != ref) ? 0 : ref;
#pragma unroll
                        for (int d = 0; d < DB; ++d) o[d] *= by;
                    }
                    if (now.fractions)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            from[e] -= __log2f(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lane_part), e % RUNS)));
                    asm("" : "+v"(from_v));       // the loop's own loads: 16 pieces are too many to keep
                    half8_t va[2][DB];
                    values(0, va[0]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (e < 3) values(e + 1, va[(e + 1) & 1]);
                        const half8_t w = weights(e, from[e]);
#pragma unroll
                        for (int d = 0; d < DB; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(va[e & 1][d], w, o[d], 0, 0, 0);
                    }
                    if (!SMALL || !left) break;
                    ref = __builtin_amdgcn_readlane(lane_ref, __builtin_ctz(left));
                    group = (uint32_t)__builtin_amdgcn_ballot_w64(lane_ref == ref) & left;
                }
            }
            if (more) {
                settle(now);
                store(buffer ^ 1);
            }
            __syncthreads();
        }
    }

    const float unit = __uint_as_float(unit_bits);
    weight += __shfl_xor(weight, 32);
    if (!q_finite && weight > 0.f) weight = __uint_as_float(0x7FC00000u);
    // o[d][8 e + j]: element elem0 + 32 d + 16 e + 8 hh + j.
    if (wave0 + r < rows && whole) {
        const float by = weight == 0.f ? 0.f : 1.f / weight;      // (unit / weight may lie below fp32's range)
        uint16_t* dst = p.out + (q.t0 + me.token) * p.out_stride + (int64_t)me.head * D + elem0 + 8 * hh;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = (uint32_t)narrow16(o[d][8 * e + 2 * j] * by * unit, BF16) |
                           (uint32_t)narrow16(o[d][8 * e + 2 * j + 1] * by * unit, BF16) << 16;
                *reinterpret_cast<u32x4*>(dst + 32 * d + 16 * e) = w;
            }
    } else if (wave0 + r < rows) {
        const int64_t part = slot * BR + 32 * (wave / SHARE) + r;
        float* dst = p.tile_o + part * D + elem0 + 8 * hh;
        if (c0 < c1)
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<float4_t*>(dst + 32 * d + 16 * e + 4 * j) =
                            float4_t{o[d][8 * e + 4 * j] * unit, o[d][8 * e + 4 * j + 1] * unit,
                                     o[d][8 * e + 4 * j + 2] * unit, o[d][8 * e + 4 * j + 3] * unit};
        if (hh == 0 && part_of_row == 0) {
            p.tile_ml[part * 2] = top;
            p.tile_ml[part * 2 + 1] = weight;
        }
    }

    // On to the share's next tile.
    if (left <= 0) return;
    at.in = 0;
    if (++at.rt >= at.c.tiles) {
        at.rt = 0;
        if (++at.h >= p.heads) {
            at.h = 0;
            do {
                if (++at.s >= p.b.S) return;
                at.q = uniform_sequence(p.b, at.s);
                at.c = count_tiles(p, at.q, BR);
            } while (at.c.tiles == 0);
        }
    }
    }
}

template <int D, bool BF16>
int queue(const AttentionParams& p, const AttentionLayout& lay, hipStream_t stream, int* launches)
{
    // A workgroup for every tile, and for every share.
    const int rows = std::max(p.tile_slots, (p.shares + p.heads - 1) / p.heads);
    const dim3 tiles((unsigned)p.heads, (unsigned)std::min(rows, kGridTiles), (unsigned)((rows + kGridTiles - 1) / kGridTiles));
    if (p.tile_slots) {
        constexpr size_t lds = (size_t)4 * (64 * (D + 8) + D * 72);
        if (p.b.page_bits < 6)
            hipLaunchKernelGGL((mnb_attention_tile_kernel<D, BF16, true>), tiles, dim3(64 * tile_waves(D)), lds, stream, p);
        else
            hipLaunchKernelGGL((mnb_attention_tile_kernel<D, BF16, false>), tiles, dim3(64 * tile_waves(D)), lds, stream, p);
        const int e = (int)hipGetLastError();
        if (e != 0) return e;
        ++*launches;
    }
    if (p.b.page_bits < 6)
        hipLaunchKernelGGL((mnb_attention_rows_kernel<D, BF16, true>), dim3(kWorkgroups), dim3(64 * kWaves), 0, stream, p);
    else
        hipLaunchKernelGGL((mnb_attention_rows_kernel<D, BF16, false>), dim3(kWorkgroups), dim3(64 * kWaves), 0, stream, p);
    int e = (int)hipGetLastError();
    if (e != 0) return e;
    ++*launches;
    hipLaunchKernelGGL((mnb_attention_join_kernel<D, BF16>),
                       dim3((unsigned)(kWorkgroups - 1 + (p.shares ? (p.shares - 1) * kJoinEach : 0))), dim3(kJoinThreads), 0,
                       stream, p);
    e = (int)hipGetLastError();
    if (e == 0) ++*launches;
    return e;
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
    const AttentionLayout lay = attention_layout(a.batch.tokens, a.batch.sequences, a.q_heads, a.cache.kv_heads,
                                                a.cache.head_dim);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.part_ml = reinterpret_cast<float*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + lay.o);
    p.tile_ml = reinterpret_cast<float*>(ws + lay.tile_ml);
    p.tile_o = reinterpret_cast<float*>(ws + lay.tile_o);
    p.many = lay.many;
    // No sequence can have many rows where max_tokens says so.
    const bool few = a.max_tokens > 0 && a.max_tokens <= p.many / p.G;
    p.tile_slots = few ? 0 : lay.tile_slots;
    if (few) p.many = INT32_MAX;
    p.shares = few ? 0 : lay.shares;
    // Tiles of few rows: at most tokens G / 16 and one for each sequence, of 2^18 units.
    p.small = a.batch.sequences <= 64 && a.batch.tokens * p.G / 16 + a.batch.sequences < (1 << 12);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    *launches = 0;
    switch (a.cache.head_dim) {
    case 64: return a.bf16 ? queue<64, true>(p, lay, s, launches) : queue<64, false>(p, lay, s, launches);
    case 128: return a.bf16 ? queue<128, true>(p, lay, s, launches) : queue<128, false>(p, lay, s, launches);
    default: return a.bf16 ? queue<256, true>(p, lay, s, launches) : queue<256, false>(p, lay, s, launches);
    }
}

}  // namespace mnb
