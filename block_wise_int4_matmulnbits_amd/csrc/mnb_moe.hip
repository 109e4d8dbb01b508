// A mixture-of-experts layer of 4-bit weights for a few tokens (gfx950): two
// launches of narrow kernels (described here), or five of wide ones where the
// experts see eight tokens or more on average (moe_layout; further down).
//
//   out[t] = sum_j p[t][j] * Down_e( silu(Gate_e x[t]) * (Up_e x[t]) ),  e = ids[t][j]
//
// with W[n][k] = (q[n][k] - z[n][k/32]) * s[n][k/32] in every matrix.
//
// Rows.  The (token, slot) pairs are sorted by expert, and each expert's
// tokens are cut into batches of up to 4 RQ rows; a batch reads its expert's
// weights once for all of its rows.  Every workgroup of the first launch
// routes all tokens by itself (a few KB of logits, top_k rounds of one wave's
// maximum per token): that is cheaper than a launch of its own in front, whose
// result the others would wait for.  Workgroup 0 leaves the tables for the
// second launch.
//
// Products.  Both launches run on v_mfma_f32_4x4x4_16b_f16: lane (g, i) of a
// wave (g = lane / 4) holds one 32-weight block of column 4n + i of each of
// its column quads n, and on the A side row i of the same block's 32
// activations; eight chained MFMAs give the block's exact 4 x 4 products, one
// FMA per row applies the block's scale.  So the unpack, the zero point and the
// scale are paid once per lane and 32 weights for four rows (16x16x32
// products, a quarter block of every column per lane, pay them four times).
//
// Activations.  The products take fp16, whose exponents are fewer than bf16's:
// a bf16 token is multiplied by a power of two, which its sums take back.  Its
// largest element lands at 2^14 .. 2^15, so that elements down to 2^-31 of it
// are exact and those below lose at most 2^-39 of it.  (A power per block of 32
// would cost the first launch a product more per block, row and column: 20
// tokens, 2 of 8 of 4096, 14336: 244 us against 211.)
//
// Between the launches the activations h = silu(g) u lie in the workspace as
// fp16, scaled by a power of two per row and block of 32 (so that no h
// overflows and small ones keep their precision), in the order in which the
// second launch's lanes load them, 1 KB or less in one piece per load:
// [batch][row quad][16 blocks][piece of 8][block of 16][row][8], with as many
// rows as the quad has.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "mnb.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

constexpr int kMaxSlots = MNB_MOE_MAX_EXPERTS / 64;   // experts per lane of a routing wave
// First launch: 4 column waves by 2 slices of K, loads two steps ahead.  HBM sets
// the pace of its loop (5.8 TB/s, 64 KB in flight per CU): 12 waves or three or
// four steps ahead gained nothing, 16 waves (128 registers) spilled and cost
// 40%, 4 waves with 4 steps ahead 20%.
constexpr int kUpWaves = kMoeUpWaves, kUpRing = 2;
constexpr int kPadToken = 255;                        // a batch's unused rows

struct MoeParams {
    const uint16_t* x;
    const void* logits;
    const uint8_t *w1, *z1, *w2, *z2;
    const uint16_t *s1, *s2;
    uint16_t* out;
    int32_t* ids_out;
    float* probs_out;
    // Workspace (MoeLayout).
    int32_t* head;       // [0]: batches; [1 + t]: token t's logits hold NaN or +infinity
    int32_t* batch_e;    // expert of each batch, and its rows << 16
    int32_t* row_token;  // [batch][4 RQ]: token, -1 for unused rows
    float* row_p;        // its weight
    uint16_t* h;         // [batch][RQ], 128 * ceil16(I/32) each: see above
    float* hs;           // [batch][RQ][I/32][4]: powers of two
    // Workspace of the wide kernels.
    int32_t* pair_row;   // [T][top_k]: row of the batches, or -1
    uint16_t* xs;        // [T][H]: activations as fp16, in the unpack's order
    float* xe;           // [T]: the power of two taken out of them
    float* hf;           // [row][I]: silu(g) u
    uint16_t* hq;        // [row][I]: its fp16 form, in the unpack's order
    float* y;            // [row][H]: weighted outputs of the rows
    int32_t T, H, I, E, top_k;
    int32_t x_bf16, logits_dtype, renormalize, out_bf16;
    int32_t batch_cap;      // batches the workspace holds
    int32_t h_quad;         // elements of a row quad in h
    int32_t stage_blocks;   // first launch: blocks of K staged in LDS at a time
    uint32_t zero;          // always 0 (see vgpr_constant)
};

// Maximum and sum over a wave, the same in every lane (DPP: four row shifts,
// two row broadcasts; lane 63 ends with the result).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    auto mx = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = mx(v, dpp_u32<0x111, 0xF>(v));
    v = mx(v, dpp_u32<0x112, 0xF>(v));
    v = mx(v, dpp_u32<0x114, 0xF>(v));
    v = mx(v, dpp_u32<0x118, 0xF>(v));
    v = mx(v, dpp_u32<0x142, 0xA>(v));
    v = mx(v, dpp_u32<0x143, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float f)
{
    auto add = [](float a, uint32_t b) { return a + __uint_as_float(b); };
    f = add(f, dpp_u32<0x111, 0xF>(__float_as_uint(f)));
    f = add(f, dpp_u32<0x112, 0xF>(__float_as_uint(f)));
    f = add(f, dpp_u32<0x114, 0xF>(__float_as_uint(f)));
    f = add(f, dpp_u32<0x118, 0xF>(__float_as_uint(f)));
    f = add(f, dpp_u32<0x142, 0xA>(__float_as_uint(f)));
    f = add(f, dpp_u32<0x143, 0xC>(__float_as_uint(f)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), 63));
}

// The routing tables of a workgroup, in dynamic LDS.
struct Routing {
    uint64_t* mask;      // [E]: tokens that selected expert e
    float* p;            // [T][top_k]
    uint32_t* token4;    // [batch][RQ]: four rows' tokens
    uint16_t* first;     // [E]: first batch
    int16_t* sel;        // [T][top_k]: expert, or -1
    uint16_t* batch_e;   // [batch]
    __device__ uint8_t* token() const { return reinterpret_cast<uint8_t*>(token4); }   // [batch][4 RQ]
};
__device__ __forceinline__ Routing routing_tables(uint8_t* lds, int E, int pairs, int cap, int rq)
{
    Routing r;
    r.mask = reinterpret_cast<uint64_t*>(lds);
    r.p = reinterpret_cast<float*>(r.mask + E);
    r.token4 = reinterpret_cast<uint32_t*>(r.p + pairs);
    r.first = reinterpret_cast<uint16_t*>(r.token4 + cap * rq);
    r.sel = reinterpret_cast<int16_t*>(r.first + E);
    r.batch_e = reinterpret_cast<uint16_t*>(r.sel + pairs);
    return r;
}

// One wave routes token t; lane l holds experts l, 64 + l, ... (NS of them).
// Logits become 32-bit keys in the order of their values (-0 first becomes
// +0); 0 marks a selected or missing expert, and no key of -infinity or below
// is selected.  top_k rounds of a wave maximum: with a few experts per lane a
// round is some 25 instructions.
template <int NS>
__device__ __forceinline__ void route_token(const MoeParams& p, int t, const Routing& r)
{
    const int lane = threadIdx.x & 63;
    constexpr uint32_t kNegInf = 0x007FFFFFu;    // the key of -infinity
    const uint32_t size = p.logits_dtype == MNB_F32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t rL =
        make_rsrc_small(static_cast<const uint8_t*>(p.logits) + (int64_t)t * p.E * size, (uint32_t)p.E * size);
    uint32_t raw[NS], key[NS];
    if (size == 4) {
#pragma unroll
        for (int i = 0; i < NS; ++i) raw[i] = __builtin_amdgcn_raw_buffer_load_b32(rL, 4 * (64 * i + lane), 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) raw[i] = __builtin_amdgcn_raw_buffer_load_b16(rL, 2 * (64 * i + lane), 0, 0);
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const bool there = 64 * i + lane < p.E;
        const float l = size == 4 ? __uint_as_float(raw[i]) : widen16(raw[i], p.logits_dtype == MNB_BF16);
        bad |= there && !(l < __builtin_inff());
        const uint32_t b = __float_as_uint(l + 0.0f);
        key[i] = there ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0u;
    }
    bad = __any(bad);
    auto value = [](uint32_t k) { return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u)); };
    float peak = 0.f, mass = 0.f;
    int mine_e = -1;                             // lane j: slot j, and its logit's key
    uint32_t mine_key = 0;
    for (int j = 0; j < p.top_k && !bad; ++j) {
        uint32_t top = key[0];
#pragma unroll
        for (int i = 1; i < NS; ++i) top = key[i] > top ? key[i] : top;
        top = wave_max(top);
        if (top <= kNegInf) break;
        if (j == 0) {
            peak = value(top);
            if (!p.renormalize) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) m += key[i] > kNegInf ? expf(value(key[i]) - peak) : 0.f;
                mass = wave_sum(m);
            }
        }
        int e = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < NS; ++i) {           // the lowest expert of this value
            const uint64_t at = __ballot(key[i] == top);
            const int bit = __builtin_ctzll(at | (1ull << 63));
            const bool take = !found && at;
            e = take ? 64 * i + bit : e;
            key[i] = take && lane == bit ? 0u : key[i];
            found |= take;
        }
        mine_e = lane == j ? e : mine_e;
        mine_key = lane == j ? top : mine_key;
    }
    const float mine_w = mine_e < 0 ? 0.f : expf(value(mine_key) - peak);
    if (p.renormalize) mass = wave_sum(mine_w);
    if (lane < p.top_k) {
        const int s = t * p.top_k + lane;
        r.sel[s] = (int16_t)mine_e;
        r.p[s] = bad ? __uint_as_float(0x7FC00000u) : mine_e < 0 ? 0.f : mine_w / mass;
        if (mine_e >= 0)
            atomicOr(reinterpret_cast<unsigned long long*>(&r.mask[mine_e]), 1ull << t);
    }
}

// First batch of every expert, and the count of batches; lane l of a wave takes
// experts NS l .. NS l + NS - 1.  Every wave does this for itself.
template <int NS>
__device__ __forceinline__ int place_batches(const MoeParams& p, int rows, const Routing& r)
{
    const int lane = threadIdx.x & 63;
    int n[NS], sum = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = NS * lane + i;
        n[i] = e < p.E ? ((int)__popcll(r.mask[e]) + rows - 1) / rows : 0;
        sum += n[i];
    }
    uint32_t upto = (uint32_t)sum;               // inclusive sum over the lanes
    upto += dpp_u32<0x111, 0xF>(upto);
    upto += dpp_u32<0x112, 0xF>(upto);
    upto += dpp_u32<0x114, 0xF>(upto);
    upto += dpp_u32<0x118, 0xF>(upto);
    upto += dpp_u32<0x142, 0xA>(upto);
    upto += dpp_u32<0x143, 0xC>(upto);
    int first = (int)upto - sum;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = NS * lane + i;
        if (e < p.E) r.first[e] = (uint16_t)first;
        first += n[i];
    }
    return __builtin_amdgcn_readlane((int)upto, 63);
}

// All tokens, the batches in the order of the experts' numbers, and each
// batch's rows in the order of the tokens; the count of batches.  Workgroup 0
// writes the tables for the next launches and the caller's ids and weights.  `meanwhile` is run by
// the waves that have no token to route, before the routing is complete.
template <int RQ, typename F>
__device__ __forceinline__ int route(const MoeParams& p, const Routing& r, F meanwhile)
{
    const int tid = threadIdx.x, threads = blockDim.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), waves = threads >> 6;
    for (int e = tid; e < p.E; e += threads) r.mask[e] = 0;
    for (int i = tid; i < p.batch_cap * RQ; i += threads) r.token4[i] = 0xFFFFFFFFu;
    __syncthreads();
    for (int t = wv; t < p.T; t += waves) {
        if (p.E <= 64) route_token<1>(p, t, r);
        else if (p.E <= 128) route_token<2>(p, t, r);
        else route_token<kMaxSlots>(p, t, r);
    }
    meanwhile();
    __syncthreads();
    // (Every wave writes the same values of `first`, and reads its own.)
    const int batches = p.E <= 64 ? place_batches<1>(p, 4 * RQ, r) : place_batches<kMaxSlots>(p, 4 * RQ, r);
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    const bool tell = blockIdx.x == 0;
    const int pairs = p.T * p.top_k;
    for (int s = tid; s < pairs; s += threads) {
        const int e = r.sel[s], t = s / p.top_k;
        int row = -1;
        if (e >= 0) {
            const int rank = __popcll(r.mask[e] & ((1ull << t) - 1));
            const int b = r.first[e] + rank / (4 * RQ);
            row = b * 4 * RQ + rank % (4 * RQ);
            r.token()[row] = (uint8_t)t;
            if (rank % (4 * RQ) == 0) r.batch_e[b] = (uint16_t)e;
            if (tell) p.row_p[row] = r.p[s];
        }
        if (tell && p.pair_row) p.pair_row[s] = row;
        if (tell && p.ids_out) p.ids_out[s] = e;
        if (tell && p.probs_out) p.probs_out[s] = r.p[s];
    }
    __syncthreads();
    if (tell) {
        if (tid == 0) p.head[0] = batches;
        for (int t = tid; t < p.T; t += threads) p.head[1 + t] = __float_as_uint(r.p[t * p.top_k]) == 0x7FC00000u;
        for (int b = tid; b < batches; b += threads) {
            const int e = r.batch_e[b], left = __popcll(r.mask[e]) - (b - r.first[e]) * 4 * RQ;
            p.batch_e[b] = e | (left < 4 * RQ ? left : 4 * RQ) << 16;
        }
        for (int i = tid; i < batches * 4 * RQ; i += threads)
            p.row_token[i] = r.token()[i] == kPadToken ? -1 : r.token()[i];
    }
    return batches;
}

// Scales and zero points of a wave's step: 16 blocks (one per lane group) of
// 4 NC columns.  Lane l loads those of BPP = NC consecutive blocks of column
// l / (16 / NC): one load of scales and one of zero points per wave and step
// where a row's blocks come in whole groups of BPP and the arrays are aligned
// to them (VEC), in single loads otherwise.  They reach the lanes that need
// them through a wave-private piece of LDS (a 2-byte and a 1-byte load per
// lane, block and column took four times as many instructions as the weights
// themselves, and they, not HBM, set the pace: the first steps' loads alone
// took 5.7 us to issue at 16 waves per CU).
template <int NC, bool VEC>
struct StepScales {
    static constexpr int NSV = VEC ? (NC + 1) / 2 : NC, NZV = VEC ? 1 : (NC + 1) / 2;
    uint32_t s[NSV], z[NZV];
};
// Bytes of a wave's piece: [4 NC columns][16 fp16], then [4 NC columns][8].
template <int NC>
constexpr int kScaleBytes = 4 * NC * 40;

// so, zo: byte offsets of this lane's first block in rS and rZ (uniform part in
// ss, zs); blk: that block's number; nb: blocks of a row.  Loaded with the default
// cache policy: a wave takes 32 and 8 bytes of a line whose rest other waves
// and steps take.
template <int NC, bool VEC>
__device__ __forceinline__ void load_scales(StepScales<NC, VEC>& v, __amdgpu_buffer_rsrc_t rS, __amdgpu_buffer_rsrc_t rZ,
                                            uint32_t so, uint32_t zo, uint32_t ss, uint32_t zs, int blk, int nb)
{
    if constexpr (VEC) {
        const uint32_t s = blk < nb ? so : kOutOfRange, z = blk < nb ? zo : kOutOfRange;
        if constexpr (NC == 4) {
            const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(rS, s, ss, 0);
            v.s[0] = t[0];
            v.s[1] = t[1];
            v.z[0] = __builtin_amdgcn_raw_buffer_load_b16(rZ, z, zs, 0);
        } else {
            if constexpr (NC == 2) v.s[0] = __builtin_amdgcn_raw_buffer_load_b32(rS, s, ss, 0);
            else v.s[0] = __builtin_amdgcn_raw_buffer_load_b16(rS, s, ss, 0);
            v.z[0] = __builtin_amdgcn_raw_buffer_load_b8(rZ, z, zs, 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NC; ++i)
            v.s[i] = __builtin_amdgcn_raw_buffer_load_b16(rS, blk + i < nb ? so + 2 * i : kOutOfRange, ss, 0);
#pragma unroll
        for (int i = 0; i < (NC + 1) / 2; ++i)
            v.z[i] = __builtin_amdgcn_raw_buffer_load_b8(rZ, blk + 2 * i < nb ? zo + i : kOutOfRange, zs, 0);
    }
}

// Through LDS: s[n], z[n] become the scale and the zero-point byte of column
// 4 n + qi, block g.
template <int NC, bool VEC>
__device__ __forceinline__ void spread_scales(const StepScales<NC, VEC>& v, uint8_t* lds, uint32_t (&s)[NC],
                                              uint32_t (&z)[NC])
{
    const int lane = threadIdx.x & 63, qi = lane & 3, g = lane >> 2;
    const int c = lane / (16 / NC), part = lane % (16 / NC);
    uint8_t* const zl = lds + 4 * NC * 32;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    if constexpr (NC == 4) {
        const u32x2 t = VEC ? u32x2{v.s[0], v.s[1]}
                            : u32x2{v.s[0] | (v.s[VEC ? 0 : 1] << 16), v.s[VEC ? 0 : 2] | (v.s[VEC ? 0 : 3] << 16)};
        *reinterpret_cast<u32x2*>(lds + 32 * c + 8 * part) = t;
        *reinterpret_cast<uint16_t*>(zl + 8 * c + 2 * part) = (uint16_t)(VEC ? v.z[0] : v.z[0] | (v.z[VEC ? 0 : 1] << 8));
    } else if constexpr (NC == 2) {
        *reinterpret_cast<uint32_t*>(lds + 32 * c + 4 * part) = VEC ? v.s[0] : v.s[0] | (v.s[VEC ? 0 : 1] << 16);
        zl[8 * c + part] = (uint8_t)v.z[0];
    } else {
        *reinterpret_cast<uint16_t*>(lds + 32 * c + 2 * part) = (uint16_t)v.s[0];
        if (!(part & 1)) zl[8 * c + part / 2] = (uint8_t)v.z[0];
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        s[n] = *reinterpret_cast<const uint16_t*>(lds + 32 * (4 * n + qi) + 2 * g);
        z[n] = zl[8 * (4 * n + qi) + g / 2];
    }
}

// One lane's 32-weight blocks of NC column quads, times RQ row quads.
//   acc[n][rq][r] += s * sum_k a[4 rq + r][k] (q[k] - z)
// w: the packed block of column 4n + i; s, z: its scale (fp16 bits) and the
// byte of its zero point; act: the block's activations of row 4 rq + i (pairs in the
// unpack's order).  ROWSCALE: the rows' powers of two f[rq][r] are applied with s.
template <int NC, int RQ, bool ROWSCALE>
__device__ __forceinline__ void block_products(const u32x4 (&w)[NC], const uint32_t (&s)[NC], const uint32_t (&z)[NC],
                                               int zshift, uint32_t zdef, uint32_t magic, const u32x4 (&act)[RQ][4],
                                               const float4_t (&f)[RQ], float4_t (&acc)[NC][RQ])
{
    // Column quads taken together, so that four chains of MFMAs run at once.
    constexpr int NI = 4 / RQ < NC ? 4 / RQ : NC;
#pragma unroll
    for (int n0 = 0; n0 < NC; n0 += NI) {
        float4_t d4[NI][RQ];
        ZeroPoint zp[NI];
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            zp[n] = zero_point_pairs(((z[n0 + n] >> zshift) & 0xFu) | zdef);
#pragma unroll
            for (int rq = 0; rq < RQ; ++rq) d4[n][rq] = float4_t{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t pr[NI][4];
#pragma unroll
            for (int n = 0; n < NI; ++n) unpack_dword(w[n0 + n][d], zp[n], magic, pr[n]);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int n = 0; n < NI; ++n)
#pragma unroll
                    for (int rq = 0; rq < RQ; ++rq)
                        d4[n][rq] = __builtin_amdgcn_mfma_f32_4x4x4f16(
                            as_half4(act[rq][d][2 * hf], act[rq][d][2 * hf + 1]),
                            as_half4(pr[n][2 * hf], pr[n][2 * hf + 1]), d4[n][rq], 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const float sf = (float)__builtin_bit_cast(_Float16, (uint16_t)s[n0 + n]);
#pragma unroll
            for (int rq = 0; rq < RQ; ++rq)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[n0 + n][rq][r] = fmaf(d4[n][rq][r], ROWSCALE ? sf * f[rq][r] : sf, acc[n0 + n][rq][r]);
        }
    }
}

// The power of two that brings bf16 numbers, the largest of whose magnitudes has
// these bits, to at most 2^15 (`to`), and its inverse; 1 where an infinity or a
// NaN is among them.  (Rows below 2^-96 keep less than all their bits: their
// h lies below every number of bf16.)
struct Power {
    float to, back;
};
__device__ __forceinline__ Power fp16_power(uint32_t top)
{
    const int e = (int)(top >> 7) - 127 - 14, ex = top >= 0x7F80u ? 0 : e < -110 ? -110 : e;
    return Power{__uint_as_float((uint32_t)(127 - ex) << 23), __uint_as_float((uint32_t)(127 + ex) << 23)};
}
// Bits of the largest magnitude of eight bf16 numbers.
__device__ __forceinline__ uint32_t top_of_piece(u32x4 v)
{
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max_u16x2(m, v[d] & 0x7FFF7FFFu);
    return (m & 0xFFFFu) > (m >> 16) ? m & 0xFFFFu : m >> 16;
}
// Eight bf16 numbers times f as fp16 pairs in the unpack's order (f16_pairs).
__device__ __forceinline__ u32x4 scaled_pairs(u32x4 v, float f)
{
    const uint32_t x = v[0], y = v[1], z = v[2], w = v[3];
    return u32x4{f16_pair(bf16_lo(x) * f, bf16_lo(z) * f), f16_pair(bf16_hi(x) * f, bf16_hi(z) * f),
                 f16_pair(bf16_lo(y) * f, bf16_lo(w) * f), f16_pair(bf16_hi(y) * f, bf16_hi(w) * f)};
}

// First launch: routing, gate and up products, h.  A unit is one batch by 32
// columns of h; a workgroup takes a contiguous range of units.  Wave (cw, ks)
// owns columns 8 cw .. 8 cw + 7 of the unit (two gate quads and the two up
// quads of the same columns) and, of every 4 W blocks of K, the 16 from 16 ks.
// The rows' activations are staged in LDS as fp16 in the unpack's order, rows
// 16 bytes apart modulo 128 so that eight lanes' reads fall on distinct banks.
// BF16: each with its token's power of two.
template <int RQ, bool VEC, bool BF16>
__global__ __launch_bounds__(64 * kUpWaves) void mnb_moe_up_kernel(MoeParams p)
{
    constexpr int NC = 4, R = 4 * RQ, W = kUpWaves, P = kUpRing;
    constexpr int SB = 16 * (W / 4);                 // blocks of K of a step, 16 per slice
    __shared__ float part[2][W][NC * RQ * 16];
    __shared__ u32x2 scale_lds[W][kScaleBytes<NC> / 8];
    __shared__ float powers[R];                      // BF16: of the staged rows
    extern __shared__ u32x4 up_lds[];                // routing tables, then the stage
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), cw = wv & 3, ks = wv >> 2;
    const int qi = lane & 3, g = lane >> 2;
    const int nb = p.H / 32, zb = (nb + 1) / 2, hblocks = p.I / 32;
    const int row_pieces = 4 * p.stage_blocks + 1;   // 16-byte pieces of a staged row
    const uint32_t zdef = p.z1 ? 0u : 8u;
    const uint32_t magic = vgpr_constant(0x64006400u, p.zero);
    const int chunks = (nb + p.stage_blocks - 1) / p.stage_blocks;
    const bool all = p.T <= R;                       // every token staged once, rows by token
    const int pairs = p.T * p.top_k;
    const Routing rt = routing_tables(reinterpret_cast<uint8_t*>(up_lds), p.E, pairs, p.batch_cap, RQ);
    u32x4* const stage = up_lds + moe_routing_bytes(p.E, pairs, p.batch_cap, RQ) / 16;   // [rows][4 stage_blocks + 1]

    // Rows [0, n) of the stage from tokens tok(row), blocks [b0, b0 +
    // stage_blocks) of K, by the waves from wave0 on.  BF16: a row is the work of
    // one wave, or of several that each look for its largest element by
    // themselves, and is then read once more (against plain rounding to fp16: one
    // token, 8 of 64 of 2048, 768 17.2 us against 16.9; 16 tokens, 6 of 64 of 2048,
    // 1408 67.2 against 65.4); `fresh`: the rows' powers are not in LDS yet.
    auto fill = [&](int n, int b0, int wave0, bool fresh, auto tok) {
        const int per_row = 4 * p.stage_blocks;
        if constexpr (BF16) {
            const int nw = W - wave0, w = wv - wave0, wpr = n < nw ? nw / n : 1, groups = nw / wpr;
            const int part = w % wpr;
            for (int row = w / wpr < groups ? w / wpr : n; row < n; row += groups) {
                const int t = tok(row);
                const bool used = t != kPadToken;
                const __amdgpu_buffer_rsrc_t rX = make_rsrc_small(p.x + (int64_t)(used ? t : 0) * p.H, used ? 2 * (uint32_t)p.H : 0u);
                auto load = [&](uint32_t piece) { return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, 16 * piece, 0, 0)); };
                Power pw;
                if (fresh) {
                    uint32_t top = 0;
                    for (int pc = lane; pc < p.H / 8; pc += 64 * 8) {
                        u32x4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = load(pc + 64 * i);
#pragma unroll
                        for (int i = 0; i < 8; ++i) top = std::max(top, top_of_piece(v[i]));
                    }
                    pw = fp16_power(wave_max(top));
                    if (part == 0 && lane == 0) powers[row] = pw.back;
                } else {
                    pw.to = 1.f / powers[row];       // exact
                }
#pragma unroll 4
                for (int pc = 64 * part + lane; pc < per_row; pc += 64 * wpr)
                    stage[row * row_pieces + pc] = scaled_pairs(load(4 * b0 + pc), pw.to);
            }
        } else {
            const int tid0 = 64 * wave0;
            for (int i = tid - tid0; i < n * per_row; i += 64 * W - tid0) {
                const int row = i / per_row, pc = i - row * per_row, t = tok(row);
                u32x4 v = {0, 0, 0, 0};
                if (t != kPadToken && b0 + pc / 4 < nb)
                    v = *reinterpret_cast<const u32x4*>(p.x + (int64_t)t * p.H + 32 * b0 + 8 * pc);
                stage[row * row_pieces + pc] = f16_pairs(v, 0, 0);
            }
        }
    };
    const int batches = route<RQ>(p, rt, [&] {
        if (all && chunks == 1 && wv >= W / 4) fill(p.T, 0, W / 4, true, [](int row) { return row; });
    });

    const int64_t units = (int64_t)batches * hblocks;   // at most 2^21
    // As few units for every workgroup as the busiest one needs: HBM, not the
    // CUs, sets the pace, and what counts is that all end together (896 units
    // on 256 workgroups: 4 each on 224 of them against 3 or 4 on all: 32.3 ->
    // 31.5 us).
    const int per = (int)((units + gridDim.x - 1) / gridDim.x);
    const int u0 = std::min<int>((int)blockIdx.x * per, (int)units), u1 = std::min<int>(u0 + per, (int)units);
    const int steps = (nb + SB - 1) / SB;            // of a unit
    const int chunk_steps = p.stage_blocks / SB;

    struct Step {
        u32x4 w[NC];
        StepScales<NC, VEC> sz;
    };
    const uint32_t row_bytes = (uint32_t)p.H / 2;
    // This lane's weights: block 16 ks + g of every step, columns qi and 4 +
    // qi; its scales: blocks 16 ks + 4 (lane % 4) .. of column lane / 4 (gate
    // columns first, then up).
    const int wblk = 16 * ks + g, sblk = 16 * ks + 4 * (lane & 3);
    const uint32_t wo = (uint32_t)qi * row_bytes + 16 * (uint32_t)wblk;
    const uint32_t srow = (uint32_t)((lane >> 2) & 7) + (lane >> 5) * (uint32_t)p.I;
    const uint32_t so = 2 * (srow * (uint32_t)nb + (uint32_t)sblk), zo = srow * (uint32_t)zb + (uint32_t)sblk / 2;
    const uint32_t rows = (uint32_t)p.I + 8;         // from a wave's first gate row to its last up row
    // The loads run P steps ahead of use, across the units.
    int left = (u1 - u0) * steps, nbatch = u0 / hblocks, nhb = u0 - nbatch * hblocks, nstep = 0;
    auto next = [&](Step& st) {
        const bool live = left-- > 0;
        const int64_t e = live ? __builtin_amdgcn_readfirstlane(rt.batch_e[nbatch]) : 0;
        const int64_t row0 = e * 2 * p.I + (live ? 32 * nhb + 8 * cw : 0);
        const int end = live ? nb : 0;               // nothing behind the last unit
        const __amdgpu_buffer_rsrc_t rW = make_rsrc_small(p.w1 + row0 * row_bytes, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t rS = make_rsrc_small(p.s1 + row0 * nb, 2 * rows * (uint32_t)nb);
        const __amdgpu_buffer_rsrc_t rZ =
            make_rsrc_small(p.z1 ? p.z1 + row0 * zb : p.w1, p.z1 ? rows * (uint32_t)zb : 0u);
        const uint32_t at = SB * (uint32_t)nstep;
        const uint32_t v = wblk + (int)at < end ? wo : kOutOfRange;
        const uint32_t up = (uint32_t)p.I * row_bytes + 16 * at;
        const uint32_t v4 = wblk + (int)at < end ? wo + 4 * row_bytes : kOutOfRange;
        st.w[0] = __builtin_amdgcn_raw_buffer_load_b128(rW, v, 16 * at, kNontemporal);
        st.w[1] = __builtin_amdgcn_raw_buffer_load_b128(rW, v4, 16 * at, kNontemporal);
        st.w[2] = __builtin_amdgcn_raw_buffer_load_b128(rW, v, up, kNontemporal);
        st.w[3] = __builtin_amdgcn_raw_buffer_load_b128(rW, v4, up, kNontemporal);
        load_scales<NC, VEC>(st.sz, rS, rZ, so, zo, 2 * at, at / 2, sblk + (int)at, end);
        if (++nstep == steps) {
            nstep = 0;
            if (++nhb == hblocks) {
                nhb = 0;
                ++nbatch;
            }
        }
    };
    Step ring[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        next(ring[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    int staged = all && chunks == 1 ? -2 : -1;       // batch in the stage (-2: every token, -1: none)
    int buf = 0;
    float4_t acc[NC][RQ] = {};
    int b = u0 / hblocks, hb = u0 - b * hblocks, step = 0;   // the unit in work
    const float4_t no_f[RQ] = {};
    int todo = (u1 - u0) * steps;
    auto run = [&](Step& st) {
        if (staged != -2 && step % chunk_steps == 0 && (chunks > 1 || staged != b)) {
            __syncthreads();
            fill(R, SB * step, 0, staged != b, [&](int row) { return (int)rt.token()[b * R + row]; });
            __syncthreads();
            staged = b;
        }
        u32x4 act[RQ][4];
#pragma unroll
        for (int rq = 0; rq < RQ; ++rq) {
            int row = 4 * rq + qi;
            if (staged == -2) {
                const int t = rt.token()[b * R + row];
                row = t == kPadToken ? 0 : t;
            }
            const u32x4* src = stage + row * row_pieces + 4 * (SB * (step % chunk_steps) + 16 * ks + g);
#pragma unroll
            for (int pc = 0; pc < 4; ++pc) act[rq][pc] = src[pc];
        }
        uint32_t sc[NC], zc[NC];
        spread_scales<NC, VEC>(st.sz, reinterpret_cast<uint8_t*>(scale_lds[wv]), sc, zc);
        block_products<NC, RQ, false>(st.w, sc, zc, 4 * (g & 1), zdef, magic, act, no_f, acc);
        next(st);
        const bool live = todo-- > 0;
        if (++step < steps) return;
        step = 0;
        // Sums over the lane groups, then over the K slices in LDS.
        const int tr = quad_total_row(lane >> 4);
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int rq = 0; rq < RQ; ++rq) {
                const float t = quad_totals(acc[n][rq][0], acc[n][rq][1], acc[n][rq][2], acc[n][rq][3]);
                if ((lane & 12) == 0) part[buf][wv][(n * RQ + rq) * 16 + 4 * tr + qi] = t;
                acc[n][rq] = float4_t{0.f, 0.f, 0.f, 0.f};
            }
        __syncthreads();
        // Thread (row, c): column c of the unit, c = 8 cw + 4 n + qi.
        if (tid < 32 * R) {
            const int row = tid >> 5, c = tid & 31;
            const int at = ((c >> 2 & 1) * RQ + (row >> 2)) * 16 + 4 * (row & 3) + (c & 3);
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int k = 0; k < W / 4; ++k) {
                gate += part[buf][4 * k + (c >> 3)][at];
                up += part[buf][4 * k + (c >> 3)][at + 2 * RQ * 16];
            }
            const int token = rt.token()[b * R + row];
            if constexpr (BF16) {                    // (unused rows: any value)
                const float f = powers[staged != -2 ? row : token == kPadToken ? 0 : token];
                gate *= f;
                up *= f;
            }
            const float h = gate / (1.f + expf(-gate)) * up;
            uint32_t top = __float_as_uint(h) & 0x7FFFFFFFu;
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                const uint32_t o = __shfl_xor(top, d);
                top = o > top ? o : top;
            }
            // The block's largest to 2^13 .. 2^14 (left alone where it is 0
            // or not finite).
            int ex = (int)(top >> 23) - 127 - 13;
            ex = top == 0 || top >= 0x7F800000u ? 0 : ex < -110 ? -110 : ex;
            if (live && token != kPadToken) {
                const int64_t quad = (int64_t)b * RQ + (row >> 2);
                // Its rows: a prefix of the four (tokens are below 64, unused rows 255).
                const int rows = 4 - __popc(rt.token4[quad] & 0x80808080u);
                const int piece = ((hb & ~15) * 4 + (c >> 3) * 16 + (hb & 15)) * rows + (row & 3);
                const int pos = ((c & 3) << 1) | (c >> 2 & 1);   // the unpack's pair order
                p.h[quad * p.h_quad + piece * 8 + pos] = __builtin_bit_cast(uint16_t, (_Float16)ldexpf(h, -ex));
                if (c == 0) p.hs[(quad * hblocks + hb) * 4 + (row & 3)] = ldexpf(1.f, ex);
            }
        }
        buf ^= 1;
        if (todo > 0 && ++hb == hblocks) {
            hb = 0;
            ++b;
        }
    };
    // P steps at a time, without a way out between them (that would be, to the
    // compiler, a path from one slot of the ring round to itself, and it
    // would wait there for the loads of all the others): steps behind the
    // last one run on zeros.
    while (todo > 0) {
#pragma unroll
        for (int j = 0; j < P; ++j) run(ring[j]);
    }
}

// Second launch: down products and the weighted sum over experts.  A workgroup
// owns 4 NC columns of the output for every token.  Its items, one batch by 16
// blocks of K each, are dealt to its waves in contiguous runs; a wave adds
// each batch's products, weighted, to its own rows of y in LDS, and the
// waves' rows are added in wave order at the end.
template <int RQ, int NC, int W, bool VEC>
__global__ __launch_bounds__(64 * W) void mnb_moe_down_kernel(MoeParams p)
{
    constexpr int R = 4 * RQ, C = 4 * NC;
    __shared__ u32x2 scale_lds[W][kScaleBytes<NC> / 8];
    // y of each wave [W][T][C], then the tables: rows' weights and tokens and
    // the batches (expert | rows << 16), batch_cap of them.
    extern __shared__ float y_lds[];
    float* const row_p = y_lds + W * p.T * C;
    int* const row_token = reinterpret_cast<int*>(row_p + p.batch_cap * R);
    int* const batch = row_token + p.batch_cap * R;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int qi = lane & 3, g = lane >> 2;
    const int nb = p.I / 32, zb = (nb + 1) / 2, steps = (nb + 15) / 16;
    const uint32_t row_bytes = (uint32_t)p.I / 2;
    const uint32_t zdef = p.z2 ? 0u : 8u;
    const uint32_t magic = vgpr_constant(0x64006400u, p.zero);
    const int col0 = blockIdx.x * C;
    // The whole tables, in one round of loads with the count of batches (what
    // lies behind the last batch is not used).
    const int batches = p.head[0];
    for (int i = tid; i < p.batch_cap * R; i += 64 * W) {
        row_p[i] = p.row_p[i];
        row_token[i] = p.row_token[i];
    }
    for (int i = tid; i < p.batch_cap; i += 64 * W) batch[i] = p.batch_e[i];
    float* const y = y_lds + wv * p.T * C;
    for (int i = lane; i < p.T * C; i += 64) y[i] = 0.f;
    __syncthreads();
    const int items = batches * steps;   // at most 2^17
    const int i0 = (int)((int64_t)items * wv / W), i1 = (int)((int64_t)items * (wv + 1) / W);

    struct Step {
        u32x4 w[NC], a[RQ][4];
        StepScales<NC, VEC> sz;
        float4_t f[RQ];
    };
    const int scol = lane / (16 / NC), sblk = NC * (lane % (16 / NC));   // this lane's scales of a step
    const uint32_t so = 2 * ((uint32_t)scol * (uint32_t)nb + (uint32_t)sblk);
    const uint32_t zo = (uint32_t)scol * (uint32_t)zb + (uint32_t)sblk / 2;
    const uint32_t wo = (uint32_t)qi * row_bytes + 16 * (uint32_t)g;
    int nbatch = i0 / steps, nstep = i0 - nbatch * steps;
    auto next = [&](Step& st, bool live) {
        const int b = live ? nbatch : 0;
        const int entry = live ? __builtin_amdgcn_readfirstlane(batch[b]) : 0;
        const int64_t e = entry & 0xFFFF;
        const int rows = entry >> 16;
        const int blk = 16 * nstep + g;
        const bool in = live && blk < nb;
        const int64_t row0 = e * p.H + col0;
        const __amdgpu_buffer_rsrc_t rW = make_rsrc_small(p.w2 + row0 * row_bytes, C * row_bytes);
        const __amdgpu_buffer_rsrc_t rS = make_rsrc_small(p.s2 + row0 * nb, 2 * C * (uint32_t)nb);
        const __amdgpu_buffer_rsrc_t rZ =
            make_rsrc_small(p.z2 ? p.z2 + row0 * zb : p.w2, p.z2 ? C * (uint32_t)zb : 0u);
        const __amdgpu_buffer_rsrc_t rA =
            make_rsrc_small(p.h + (int64_t)b * RQ * p.h_quad, live ? 2 * RQ * (uint32_t)p.h_quad : 0u);
        const __amdgpu_buffer_rsrc_t rF = make_rsrc_small(p.hs + (int64_t)b * RQ * nb * 4, live ? RQ * (uint32_t)nb * 16 : 0u);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            st.w[n] = __builtin_amdgcn_raw_buffer_load_b128(rW, in ? wo + 4 * n * row_bytes : kOutOfRange,
                                                            256 * (uint32_t)nstep, kNontemporal);
        }
        load_scales<NC, VEC>(st.sz, rS, rZ, so, zo, 32 * (uint32_t)nstep, 8 * (uint32_t)nstep, 16 * nstep + sblk,
                             live ? nb : 0);
#pragma unroll
        for (int rq = 0; rq < RQ; ++rq) {
            // Unused rows load zeros.
            const int n4 = rows - 4 * rq < 4 ? rows - 4 * rq : 4;   // rows of the quad
            const bool used = in && qi < n4;
            const uint32_t at = (uint32_t)(rq * nb + blk);
            const uint32_t to = 2 * rq * (uint32_t)p.h_quad + 16 * ((64 * (uint32_t)nstep + g) * (uint32_t)n4 + qi);
#pragma unroll
            for (int pc = 0; pc < 4; ++pc)
                st.a[rq][pc] = __builtin_amdgcn_raw_buffer_load_b128(
                    rA, used ? to + 256 * pc * (uint32_t)n4 : kOutOfRange, 0, 0);
            st.f[rq] = __builtin_bit_cast(float4_t, __builtin_amdgcn_raw_buffer_load_b128(rF, in ? at * 16 : kOutOfRange, 0, 0));
        }
        if (++nstep == steps) {
            nstep = 0;
            ++nbatch;
        }
    };
    Step ring[2];
    next(ring[0], i0 < i1);
    next(ring[1], i0 + 1 < i1);
    int bt = i0 / steps;
    float4_t acc[NC][RQ] = {};
    auto run = [&](Step& st, int i) {
        uint32_t sc[NC], zc[NC];
        spread_scales<NC, VEC>(st.sz, reinterpret_cast<uint8_t*>(scale_lds[wv]), sc, zc);
        block_products<NC, RQ, true>(st.w, sc, zc, 4 * (g & 1), zdef, magic, st.a, st.f, acc);
        next(st, i + 2 < i1);
        if (i + 1 < i1 && (i + 1) % steps) return;
        // The batch ends for this wave: weighted rows to its y.
        const int tr = quad_total_row(lane >> 4);
#pragma unroll
        for (int rq = 0; rq < RQ; ++rq) {
            const int row = bt * R + 4 * rq + tr;
            const int t = row_token[row];
            const float w = row_p[row];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const float v = quad_totals(acc[n][rq][0], acc[n][rq][1], acc[n][rq][2], acc[n][rq][3]);
                if ((lane & 12) == 0 && t >= 0) y[t * C + 4 * n + qi] += w * v;
                acc[n][rq] = float4_t{0.f, 0.f, 0.f, 0.f};
            }
        }
        ++bt;
    };
    for (int i = i0; i < i1;) {   // ends right behind an item, as above
        run(ring[0], i);
        if (++i >= i1) break;
        run(ring[1], i);
        ++i;
    }
    __syncthreads();
    for (int i = tid; i < p.T * C; i += 64 * W) {
        float v = y_lds[i];
        for (int w = 1; w < W; ++w) v += y_lds[w * p.T * C + i];
        const int t = i / C;
        if (p.head[1 + t]) v = __uint_as_float(0x7FC00000u);
        p.out[(int64_t)t * p.H + col0 + i % C] = narrow16(v, p.out_bf16);
    }
}

// More rows per expert: the same layer on v_mfma_f32_16x16x32_f16, in five
// launches.  The 4x4x4 product's four rows per instruction make the matrix
// cores the bound from some eight rows on; here sixteen rows cost one
// 16-cycle product per 256 bytes of weights, and what bounds the loop is the
// unpacking.  Lane (j, g) supplies 8 k of column j and of row j and receives
// column j, rows 4 g .. 4 g + 3; one product spans one 32-weight block, whose
// scale is applied to its result, as above.
//
// A unit is one batch (16 RT rows of one expert) by 64 columns of weights: 32
// gate and the same 32 up columns, or 64 down columns.  The eight waves of a
// workgroup split K, and each takes all 64 columns of its part, so a row's
// activations are read once per unit, straight into registers in the
// product's order, and LDS holds only the waves' sums.  The activations h go
// through fp32 to fp16 with one power of two per row (scale_rows): with a
// scale per block, as in the narrow kernels, every product would need the
// scales of its four rows.
constexpr int kWideWaves = 8;

// Launch 1: the tables (workgroup 0; sixteen waves, each routes its tokens one
// after another) and x as fp16 in the unpack's order (a token for each of the
// others), bf16 with one power of two per token.
constexpr int kPrepareThreads = 1024;
template <int RT>
__global__ __launch_bounds__(kPrepareThreads) void mnb_moe_prepare_kernel(MoeParams p)
{
    extern __shared__ u32x4 prepare_lds[];
    if (blockIdx.x != 0) {
        __shared__ uint32_t tops[kPrepareThreads / 64];
        constexpr int P = MNB_MOE_MAX_WIDTH / 8 / kPrepareThreads;   // the whole token in registers
        const int t = blockIdx.x - 1, tid = threadIdx.x, pieces = p.H / 8;
        const u32x4* const x = reinterpret_cast<const u32x4*>(p.x + (int64_t)t * p.H);
        u32x4* const out = reinterpret_cast<u32x4*>(p.xs + (int64_t)t * p.H);
        u32x4 v[P];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            v[i] = tid + kPrepareThreads * i < pieces ? x[tid + kPrepareThreads * i] : u32x4{0, 0, 0, 0};
            top = std::max(top, top_of_piece(v[i]));
        }
        top = wave_max(top);
        if ((tid & 63) == 0) tops[tid >> 6] = top;
        __syncthreads();
        for (int w = 0; w < kPrepareThreads / 64; ++w) top = std::max(top, tops[w]);
        const Power pw = p.x_bf16 ? fp16_power(top) : Power{1.f, 1.f};
        if (tid == 0) p.xe[t] = pw.back;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (tid + kPrepareThreads * i < pieces)
                out[tid + kPrepareThreads * i] = p.x_bf16 ? scaled_pairs(v[i], pw.to) : f16_pairs(v[i], 0, 0);
        return;
    }
    const Routing rt = routing_tables(reinterpret_cast<uint8_t*>(prepare_lds), p.E, p.T * p.top_k, p.batch_cap, 4 * RT);
    route<4 * RT>(p, rt, [] {});
}

// Launches 2 (UP: x through gate and up to hf) and 4 (h through down to y).
template <int RT, bool UP, int VEC>
__global__ __launch_bounds__(64 * kWideWaves) void mnb_moe_wide_kernel(MoeParams p)
{
    constexpr int R = 16 * RT, CT = 4, W = kWideWaves;
    __shared__ float part[W][CT * RT * 4][64];
    __shared__ u32x4 scale_lds[W][64 * 20 / 16];    // of two steps: [64 columns][8 fp16], then [64][4]
    __shared__ float powers[UP ? MNB_MOE_MAX_TOKENS : 1];   // the tokens' (xe)
    // The tables, so that the loop reads none from memory (it would wait for
    // its own loads ahead): the batches, then each row's token (UP) or scale.
    extern __shared__ int wide_lds[];
    int* const batch = wide_lds;
    int* const row_info = batch + p.batch_cap;
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = UP ? p.H : p.I, N = UP ? p.I : p.H;
    const int nb = K / 32, zb = (nb + 1) / 2, tiles = (N + (UP ? 31 : 63)) / (UP ? 32 : 64);
    const uint8_t* const wq = UP ? p.w1 : p.w2;
    const uint16_t* const sq = UP ? p.s1 : p.s2;
    const uint8_t* const zq = UP ? p.z1 : p.z2;
    const uint32_t row_bytes = (uint32_t)K / 2, zdef = zq ? 0u : 0x88u;   // zero points of two blocks
    const uint32_t magic = vgpr_constant(0x64006400u, p.zero);
    const int64_t units = (int64_t)p.head[0] * tiles;
    for (int i = tid; i < p.batch_cap; i += 64 * W) batch[i] = p.batch_e[i];
    for (int i = tid; i < p.batch_cap * R; i += 64 * W) row_info[i] = UP ? p.row_token[i] : __float_as_int(p.hs[i]);
    if (UP && tid < p.T) powers[tid] = p.xe[tid];
    __syncthreads();
    const int per = (int)((units + gridDim.x - 1) / gridDim.x);
    const int u0 = std::min<int>((int)blockIdx.x * per, (int)units), u1 = std::min<int>(u0 + per, (int)units);
    // K in steps of four blocks; a wave takes two neighbours of every 16, whose
    // weights share 128-byte lines.
    const int quads = (nb + 3) / 4, steps = (quads + 2 * W - 1) / (2 * W) * 2;
    // Column of this lane's weights in tile ct, and of its scales: UP tiles 0
    // and 1 are gate columns, 2 and 3 the up columns of the same h.
    const uint32_t up = (uint32_t)p.I;
    const uint32_t scol = UP ? (uint32_t)(lane & 31) + (lane >> 5) * up : (uint32_t)lane;

    // Scales and zero points of this lane's column for two steps, eight
    // blocks, in as few loads as the rows' length and alignment allow: VEC
    // blocks at a time (every load touches 64 lines, one per column).
    struct Scales {
        uint32_t s[VEC > 1 ? 4 : 8], z[VEC == 8 ? 1 : VEC == 4 ? 2 : 4];
    };
    int left = (u1 - u0) * steps, nbatch = u0 / tiles, ntile = u0 - nbatch * tiles, nstep = 0;
    uint32_t wo[CT];                                 // this lane's weights
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
        wo[ct] = (UP ? (uint32_t)(16 * (ct & 1) + j) + (ct >> 1) * up : (uint32_t)(16 * ct + j)) * row_bytes + 16 * (uint32_t)g;
    const uint32_t so = 2 * scol * (uint32_t)nb, zo = scol * (uint32_t)zb;
    __amdgpu_buffer_rsrc_t rW, rS, rZ, rA;
    auto enter = [&] {                               // the unit (nbatch, ntile)
        const bool live = left > 0;
        const int64_t e = (live ? __builtin_amdgcn_readfirstlane(batch[nbatch]) : 0) & 0xFFFF;
        const int64_t row0 = e * (UP ? 2 : 1) * N + (live ? ntile * (UP ? 32 : 64) : 0);
        const uint32_t cols = !live ? 0u : UP ? up + 32u : (uint32_t)std::min<int>(64, N - ntile * 64);
        rW = make_rsrc_small(wq + row0 * row_bytes, cols * row_bytes);
        rS = make_rsrc_small(sq + row0 * nb, 2 * cols * (uint32_t)nb);
        rZ = make_rsrc_small(zq ? zq + row0 * zb : wq, zq ? cols * (uint32_t)zb : 0u);
    };
    auto quad_of = [&](int step) { return 2 * (wv + W * (step >> 1)) + (step & 1); };
    auto next = [&](u32x4 (&w)[CT], Scales* sz) {
        if (nstep == 0) enter();
        // Lane offsets stay; the step's is uniform.  Blocks past K load zeros
        // (whole steps of them where rows come in steps, VEC).
        const int quad = quad_of(nstep);
        const uint32_t at = 64 * (uint32_t)quad;
        const bool in = VEC > 1 ? 4 * quad < nb : 4 * quad + g < nb;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            w[ct] = __builtin_amdgcn_raw_buffer_load_b128(rW, in ? wo[ct] : kOutOfRange, at, 0);
        if (sz) {                                    // the first of two steps
            const uint32_t ss = 8 * (uint32_t)quad, zs = 2 * (uint32_t)quad;
            auto here = [&](uint32_t off, int blk) { return 4 * quad + blk < nb ? off : kOutOfRange; };
            if constexpr (VEC == 8) {
                const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(rS, here(so, 0), ss, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) sz->s[VEC > 1 ? i : 0] = t[i];
                sz->z[0] = __builtin_amdgcn_raw_buffer_load_b32(rZ, here(zo, 0), zs, 0);
            } else if constexpr (VEC == 4) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(rS, here(so + 8 * i, 4 * i), ss, 0);
                    sz->s[2 * i] = t[0];
                    sz->s[2 * i + 1] = t[1];
                    sz->z[VEC == 8 ? 0 : i] = __builtin_amdgcn_raw_buffer_load_b16(rZ, here(zo + 2 * i, 4 * i), zs, 0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sz->s[VEC > 1 ? 0 : i] = __builtin_amdgcn_raw_buffer_load_b16(rS, here(so + 2 * i, i), ss, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sz->z[VEC > 1 ? 0 : i] = __builtin_amdgcn_raw_buffer_load_b8(rZ, here(zo + i, 2 * i), zs, 0);
            }
        }
        --left;
        if (++nstep == steps) {
            nstep = 0;
            if (left > 0 && ++ntile == tiles) {
                ntile = 0;
                ++nbatch;
            }
        }
    };
    // Activations, one step ahead: blocks 2 ip, 2 ip + 1 of this lane's rows take
    // the place of the ones just used.  (They come from L2; two steps ahead the
    // kernel for 32 rows spilled, and the spills' reloads waited for the weights:
    // 64 tokens, 2 of 8 of 4096, 14336: 208 -> 189 us for launch 2.)
    uint32_t arow[RT];                               // this lane's rows, or kOutOfRange
    auto rows_of = [&](int b, bool live) {           // of batch b
        const int rows = live ? __builtin_amdgcn_readfirstlane(batch[b]) >> 16 : 0;
        rA = UP ? make_rsrc_small(p.xs, (uint32_t)p.T * (uint32_t)K * 2)
                : make_rsrc_small(p.hq + (int64_t)(live ? b : 0) * R * K, live ? (uint32_t)R * (uint32_t)K * 2 : 0u);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = 16 * rt + j;
            arow[rt] = r >= rows ? kOutOfRange
                                 : 16 * (uint32_t)g + 2 * (uint32_t)K * (uint32_t)(UP ? row_info[b * R + r] : r);
        }
    };
    u32x4 act[RT][4];
    auto next_rows = [&](int step, int ip) {
        const int quad = quad_of(step);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 2 * ip; i < 2 * ip + 2; ++i)
                act[rt][i] = __builtin_amdgcn_raw_buffer_load_b128(
                    rA, 4 * quad + (VEC > 1 ? 0 : i) < nb ? arow[rt] : kOutOfRange, 256 * (uint32_t)quad + 64 * i, 0);
    };

    float4_t acc[CT][RT] = {};
    int todo = (u1 - u0) * steps, step = 0, b = u0 / tiles, tile = u0 - b * tiles;
    u32x4 ring[2][CT];                               // weights, two steps ahead; steps of a unit are even
    Scales scales;
    next(ring[0], &scales);
    rows_of(b, todo > 0);
    next_rows(0, 0);
    next_rows(0, 1);
    __builtin_amdgcn_sched_barrier(0);
    next(ring[1], nullptr);
    __builtin_amdgcn_sched_barrier(0);

    uint8_t* const sl = reinterpret_cast<uint8_t*>(scale_lds[wv]);
    auto run = [&](u32x4 (&w)[CT], bool odd) {
        // The wave's scales and zero points of two steps, column by lane, to
        // the lanes of the column.
        if (!odd) {
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            u32x4 s8;
            uint32_t z8;
            if constexpr (VEC > 1) {
                s8 = u32x4{scales.s[0], scales.s[1], scales.s[2], scales.s[3]};
                z8 = VEC == 8 ? scales.z[0] : scales.z[0] | (scales.z[VEC == 8 ? 0 : 1] << 16);
            } else {
                for (int i = 0; i < 4; ++i) s8[i] = scales.s[VEC > 1 ? 0 : 2 * i] | (scales.s[VEC > 1 ? 0 : 2 * i + 1] << 16);
                z8 = scales.z[0] | (scales.z[VEC > 1 ? 0 : 1] << 8) | (scales.z[VEC > 1 ? 0 : 2] << 16) | (scales.z[VEC > 1 ? 0 : 3] << 24);
            }
            *reinterpret_cast<u32x4*>(sl + 16 * lane) = s8;
            *reinterpret_cast<uint32_t*>(sl + 1024 + 4 * lane) = z8;
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        }
        uint32_t d[CT][4];                           // d[ct][i]: dword g of block i
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            // (Kept whole until here: taken apart across the loop's end, the
            // loaded words would be copied there, and the copies would wait for
            // every load under way.)
            u32x4 v = w[ct];
            asm("" : "+v"(v));
#pragma unroll
            for (int i = 0; i < 4; ++i) d[ct][i] = v[i];
            transpose_rows(d[ct]);
        }
        const bool last = step + 1 == steps;
#pragma unroll
        for (int ip = 0; ip < 2; ++ip) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const uint32_t s2 = *reinterpret_cast<const uint32_t*>(sl + 16 * (16 * ct + j) + 8 * odd + 4 * ip);
                const uint32_t z2 = *(sl + 1024 + 4 * (16 * ct + j) + 2 * odd + ip) | zdef;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // The fields of zero_point_pairs: the zero point, plain and
                    // shifted by four, under the constants' upper bytes.
                    uint32_t pr[4];
                    const uint32_t lo = k ? z2 >> 4 : z2 & 0xFu, hi = k ? z2 & 0xF0u : z2 << 4;
                    const ZeroPoint zp{__builtin_amdgcn_perm(0xE4E4E4E4u, lo, 0x04000400u),
                                       __builtin_amdgcn_perm(0xD4D4D4D4u, hi, 0x04000400u)};
                    unpack_dword(d[ct][2 * ip + k], zp, magic, pr);
                    const half8_t bv = __builtin_bit_cast(half8_t, u32x4{pr[0], pr[1], pr[2], pr[3]});
                    const float sf = (float)__builtin_bit_cast(_Float16, (uint16_t)(k ? s2 >> 16 : s2));
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const float4_t zero = {0.f, 0.f, 0.f, 0.f};
                        const float4_t v = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            __builtin_bit_cast(half8_t, act[rt][2 * ip + k]), bv, zero, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[ct][rt][r] = fmaf(v[r], sf, acc[ct][rt][r]);
                    }
                }
            }
            if (ip == 0 && last) {
                const bool turn = tile + 1 == tiles;
                if (turn || todo == 1) rows_of(b + turn, todo > 1);
            }
            next_rows(last ? 0 : step + 1, ip);
        }
        const bool live = todo-- > 0;
        next(w, odd ? nullptr : &scales);
        if (++step < steps) return;
        step = 0;
        // The waves' sums, rows 16 rt + 4 g + r of column 16 ct + j.
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    part[wv][(ct * RT + rt) * 4 + r][lane] = acc[ct][rt][r];
                    acc[ct][rt][r] = 0.f;
                }
        __syncthreads();
        auto total = [&](int row, int c) {
            const float* at = &part[0][((c >> 4) * RT + (row >> 4)) * 4 + (row & 3)][16 * ((row >> 2) & 3) + (c & 15)];
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) v += at[w * CT * RT * 4 * 64];
            return v;
        };
        const int rows = batch[b] >> 16;
        if constexpr (UP) {
            for (int o = tid; o < 32 * rows && live; o += 64 * W) {
                const int row = o >> 5, c = o & 31;
                const float f = powers[row_info[b * R + row]], gate = total(row, c) * f, u = total(row, 32 + c) * f;
                p.hf[((int64_t)b * R + row) * N + 32 * tile + c] = gate / (1.f + expf(-gate)) * u;
            }
        } else {
            for (int o = tid; o < 64 * rows && live; o += 64 * W) {
                const int row = o >> 6, c = o & 63;
                if (64 * tile + c < N)
                    p.y[((int64_t)b * R + row) * N + 64 * tile + c] = total(row, c) * __int_as_float(row_info[b * R + row]);
            }
        }
        __syncthreads();                             // part is written again by the next unit
        if (todo > 0 && ++tile == tiles) {
            tile = 0;
            ++b;
        }
    };
    while (todo > 0) {
        run(ring[0], false);
        run(ring[1], true);
    }
}

// Launch 3: each row's h as fp16, its largest at 2^13 .. 2^14, in the unpack's
// order; hs: the power of two taken out, times the row's weight.
template <int RT>
__global__ __launch_bounds__(1024) void mnb_moe_scale_rows_kernel(MoeParams p)
{
    __shared__ uint32_t tops[16];
    const int row = blockIdx.x, tid = threadIdx.x;
    if (row >= p.head[0] * 16 * RT || p.row_token[row] < 0) return;
    const float4_t* const h = reinterpret_cast<const float4_t*>(p.hf + (int64_t)row * p.I);
    const int pieces = p.I / 8;
    constexpr int P = MNB_MOE_MAX_WIDTH / 8 / 1024;   // the whole row in registers
    float4_t v[P][2] = {};
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (tid + 1024 * i < pieces)
#pragma unroll
            for (int q = 0; q < 2; ++q) v[i][q] = h[2 * (tid + 1024 * i) + q];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t m = __float_as_uint(v[i][k >> 2][k & 3]) & 0x7FFFFFFFu;
            top = m > top ? m : top;
        }
    top = wave_max(top);
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
    for (int w = 0; w < 16; ++w) top = tops[w] > top ? tops[w] : top;
    int ex = (int)(top >> 23) - 127 - 13;
    ex = top == 0 || top >= 0x7F800000u ? 0 : ex < -110 ? -110 : ex;
    if (tid == 0) p.hs[row] = ldexpf(p.row_p[row], ex);
    u32x4* const out = reinterpret_cast<u32x4*>(p.hq + (int64_t)row * p.I);
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (tid + 1024 * i < pieces) {
            u32x4 o;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = f16_pair(ldexpf(v[i][0][k], -ex), ldexpf(v[i][1][k], -ex));
            out[tid + 1024 * i] = o;
        }
}

// Launch 5: each token's rows, in the order of its slots; four columns a thread.
__global__ __launch_bounds__(256) void mnb_moe_combine_kernel(MoeParams p)
{
    const int quads = p.H / 4;
    const int i = blockIdx.x * 256 + threadIdx.x;    // at most 2^20 of them
    if (i >= p.T * quads) return;
    const int t = i / quads, c = 4 * (i - t * quads);
    float4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.top_k; ++s) {
        const int row = p.pair_row[t * p.top_k + s];
        if (row >= 0) v += *reinterpret_cast<const float4_t*>(p.y + (int64_t)row * p.H + c);
    }
    const bool bad = p.head[1 + t];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        p.out[(int64_t)t * p.H + c + k] = narrow16(bad ? __uint_as_float(0x7FC00000u) : v[k], p.out_bf16);
}

hipError_t queue(const void* fn, const MoeParams& p, unsigned grid, int threads, size_t lds, hipStream_t s)
{
    MoeParams q = p;
    void* args[] = {&q};
    const hipError_t e = hipLaunchKernel(fn, dim3(grid), dim3((unsigned)threads), args, lds, s);
    return e != hipSuccess ? e : hipGetLastError();
}

template <int RQ>
hipError_t queue_up(const MoeParams& p, const MoeRoute& r, int cus, hipStream_t s)
{
    // Every token, where they are few and K is staged whole; else one batch.
    const int rows = p.T < 4 * RQ && p.H <= 32 * p.stage_blocks ? p.T : 4 * RQ;
    const size_t lds = moe_routing_bytes(p.E, p.T * p.top_k, p.batch_cap, RQ) + (size_t)rows * (4 * p.stage_blocks + 1) * 16;
    const int64_t units = (int64_t)p.T * p.top_k * (p.I / 32);
    const bool vec = r.up_vec > 1;
    const void* fn = p.x_bf16 ? (vec ? reinterpret_cast<const void*>(mnb_moe_up_kernel<RQ, true, true>)
                                     : reinterpret_cast<const void*>(mnb_moe_up_kernel<RQ, false, true>))
                              : (vec ? reinterpret_cast<const void*>(mnb_moe_up_kernel<RQ, true, false>)
                                     : reinterpret_cast<const void*>(mnb_moe_up_kernel<RQ, false, false>));
    return queue(fn, p, (unsigned)(units < cus ? units : cus), 64 * kUpWaves, lds, s);
}

template <int RQ, int NC, int W>
hipError_t queue_down(const MoeParams& p, const MoeRoute& r, hipStream_t s)
{
    const size_t lds = ((size_t)W * p.T * 4 * NC + (size_t)p.batch_cap * (8 * RQ + 1)) * 4;
    // (Of one quad a load brings one block either way.)
    const void* fn = r.down_vec == NC ? reinterpret_cast<const void*>(mnb_moe_down_kernel<RQ, NC, W, true>)
                                      : reinterpret_cast<const void*>(mnb_moe_down_kernel<RQ, NC, W, NC == 1>);
    return queue(fn, p, (unsigned)(p.H / (4 * NC)), 64 * W, lds, s);
}

template <int RT, bool UP>
const void* wide_kernel(int vec)
{
    return vec == 8   ? reinterpret_cast<const void*>(mnb_moe_wide_kernel<RT, UP, 8>)
           : vec == 4 ? reinterpret_cast<const void*>(mnb_moe_wide_kernel<RT, UP, 4>)
                      : reinterpret_cast<const void*>(mnb_moe_wide_kernel<RT, UP, 1>);
}

template <int RT>
hipError_t queue_wide(const MoeParams& p, const MoeRoute& r, int cus, int* launches, hipStream_t s)
{
    const int64_t rows = (int64_t)p.batch_cap * 16 * RT;
    const void* const prepare = reinterpret_cast<const void*>(mnb_moe_prepare_kernel<RT>);
    const void* const up = wide_kernel<RT, true>(r.up_vec);
    const void* const scale = reinterpret_cast<const void*>(mnb_moe_scale_rows_kernel<RT>);
    const void* const down = wide_kernel<RT, false>(r.down_vec);
    const void* const combine = reinterpret_cast<const void*>(mnb_moe_combine_kernel);
    const size_t tables = (size_t)p.batch_cap * (16 * RT + 1) * 4;
    struct Launch {
        const void* fn;
        int64_t grid;
        int threads;
        size_t lds;
    } const all[] = {{prepare, p.T + 1, kPrepareThreads, moe_routing_bytes(p.E, p.T * p.top_k, p.batch_cap, 4 * RT)},
                     {up, cus, 64 * kWideWaves, tables},
                     {scale, rows, 1024, 0},
                     {down, cus, 64 * kWideWaves, tables},
                     {combine, ((int64_t)p.T * p.H / 4 + 255) / 256, 256, 0}};
    for (const Launch& l : all) {
        const hipError_t e = queue(l.fn, p, (unsigned)l.grid, l.threads, l.lds, s);
        if (e != hipSuccess) return e;
        ++*launches;
    }
    return hipSuccess;
}

}  // namespace

int launch_moe(const MoeArgs& a, void* stream, int* launches)
{
    int cus = 0;
    int e = current_device_cus(&cus);
    if (e != 0) return e;
    const MoeLayout lay = moe_layout(a.T, a.w.hidden, a.w.inter, a.w.experts, a.top_k);
    const MoeRoute route = moe_route(a, lay, cus);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    MoeParams p{};
    p.x = static_cast<const uint16_t*>(a.x);
    p.logits = a.logits;
    p.w1 = a.w.gate_up;
    p.s1 = a.w.gate_up_scales;
    p.z1 = a.w.gate_up_zero_points;
    p.w2 = a.w.down;
    p.s2 = a.w.down_scales;
    p.z2 = a.w.down_zero_points;
    p.out = static_cast<uint16_t*>(a.out);
    p.ids_out = a.ids;
    p.probs_out = a.probs;
    p.head = reinterpret_cast<int32_t*>(ws);
    p.batch_e = reinterpret_cast<int32_t*>(ws + lay.batch_e);
    p.row_token = reinterpret_cast<int32_t*>(ws + lay.row_token);
    p.row_p = reinterpret_cast<float*>(ws + lay.row_p);
    p.hs = reinterpret_cast<float*>(ws + lay.hs);
    p.h = reinterpret_cast<uint16_t*>(ws + lay.h);
    p.pair_row = lay.wide ? reinterpret_cast<int32_t*>(ws + lay.pair_row) : nullptr;
    p.xs = reinterpret_cast<uint16_t*>(ws + lay.xs);
    p.xe = reinterpret_cast<float*>(ws + lay.xe);
    p.hf = reinterpret_cast<float*>(ws + lay.hf);
    p.hq = p.h;
    p.y = reinterpret_cast<float*>(ws + lay.y);
    p.T = a.T;
    p.H = (int32_t)a.w.hidden;
    p.I = (int32_t)a.w.inter;
    p.E = (int32_t)a.w.experts;
    p.top_k = a.top_k;
    p.x_bf16 = a.x_bf16;
    p.logits_dtype = a.logits_dtype;
    p.renormalize = a.renormalize;
    p.out_bf16 = a.out_bf16;
    p.zero = 0;
    p.batch_cap = lay.batches;
    p.h_quad = 128 * ((p.I / 32 + 15) / 16 * 16);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (lay.wide)
        return (int)(lay.wide == 1 ? queue_wide<1>(p, route, cus, launches, s) : queue_wide<2>(p, route, cus, launches, s));
    p.stage_blocks = route.stage_blocks;
    hipError_t he = lay.rq == 1 ? queue_up<1>(p, route, cus, s) : queue_up<2>(p, route, cus, s);
    if (he != hipSuccess) return (int)he;
    ++*launches;
    const int nc = route.down_quads;
    if (lay.rq == 1)
        he = nc == 4   ? queue_down<1, 4, 12>(p, route, s)
             : nc == 2 ? queue_down<1, 2, 16>(p, route, s)
                       : queue_down<1, 1, 16>(p, route, s);
    else
        he = nc == 4   ? queue_down<2, 4, 8>(p, route, s)
             : nc == 2 ? queue_down<2, 2, 8>(p, route, s)
                       : queue_down<2, 1, 8>(p, route, s);
    if (he == hipSuccess) ++*launches;
    return (int)he;
}

}  // namespace mnb
