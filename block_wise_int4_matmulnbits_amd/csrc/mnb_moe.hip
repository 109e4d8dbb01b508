// A mixture-of-experts layer of 4-bit weights for a few tokens (gfx950), in two
// launches.
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
// Between the launches the activations h = silu(g) u lie in the workspace as
// fp16, scaled by a power of two per row and block of 32 (so that no h
// overflows and small ones keep their precision), in the order in which the
// second launch's lanes load them: [batch][row quad][block][row of 4][32].
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

constexpr int kMaxPairs = MNB_MOE_MAX_TOKENS * MNB_MOE_MAX_TOP_K;
constexpr int kMaxSlots = MNB_MOE_MAX_EXPERTS / 64;   // experts per lane of a routing wave
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
    uint16_t* h;         // [batch][RQ][I/32][4][32]
    float* hs;           // [batch][RQ][I/32][4]: powers of two
    int32_t T, H, I, E, top_k;
    int32_t x_bf16, logits_dtype, renormalize, out_bf16;
    int32_t batch_cap;      // batches the workspace holds
    int32_t stage_blocks;   // first launch: blocks of K staged in LDS at a time
    uint32_t zero;          // always 0 (see vgpr_constant)
};

__device__ __forceinline__ float widen16(uint32_t bits, int bf16)
{
    return bf16 ? __uint_as_float(bits << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

__device__ __forceinline__ uint16_t narrow16(float v, int bf16)
{
    if (!bf16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

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

// The routing tables of a workgroup.
struct Routing {
    uint64_t mask[MNB_MOE_MAX_EXPERTS];          // tokens that selected expert e
    uint16_t first[MNB_MOE_MAX_EXPERTS];         // its first batch
    int16_t sel[kMaxPairs];                      // [t][top_k]: expert, or -1
    float p[kMaxPairs];
    uint16_t batch_e[kMaxPairs];
    uint8_t token[4 * kMaxPairs];                // [batch][4 RQ]
    int32_t batches;
};

// One wave routes token t.  Logits become 32-bit keys in the order of their
// values (-0 first becomes +0); 0 marks a selected or missing expert, and
// no key of -infinity or below is selected.
__device__ __forceinline__ void route_token(const MoeParams& p, int t, Routing& r)
{
    const int lane = threadIdx.x & 63;
    const int64_t base = (int64_t)t * p.E;
    constexpr uint32_t kNegInf = 0x007FFFFFu;    // the key of -infinity
    uint32_t key[kMaxSlots];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kMaxSlots; ++i) {
        const int e = 64 * i + lane;
        float l = -__builtin_inff();
        if (e < p.E)
            l = p.logits_dtype == MNB_F32 ? static_cast<const float*>(p.logits)[base + e]
                                          : widen16(static_cast<const uint16_t*>(p.logits)[base + e],
                                                    p.logits_dtype == MNB_BF16);
        bad |= !(l < __builtin_inff());
        const uint32_t b = __float_as_uint(l + 0.0f);
        key[i] = e < p.E ? b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u) : 0u;
    }
    bad = __any(bad);
    auto value = [](uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); };
    float peak = 0.f, mass = 0.f, mine_w = 0.f;
    int mine_e = -1;                             // lane j: slot j
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kMaxSlots; ++i) top = key[i] > top ? key[i] : top;
        top = wave_max(top);
        if (j == 0) {
            peak = value(top);
            if (!p.renormalize && !bad && top > kNegInf) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < kMaxSlots; ++i)
                    if (key[i] > kNegInf) m += __expf(value(key[i]) - peak);
                mass = wave_sum(m);
            }
        }
        if (bad || top <= kNegInf) break;
        int e = -1;
#pragma unroll
        for (int i = 0; i < kMaxSlots; ++i) {
            const uint64_t at = __ballot(key[i] == top);
            if (e < 0 && at) {
                e = 64 * i + __builtin_ctzll(at);
                if (lane == (e & 63)) key[i] = 0;
            }
        }
        const float w = __expf(value(top) - peak);
        if (p.renormalize) mass += w;
        if (lane == j) {
            mine_e = e;
            mine_w = w;
        }
    }
    if (lane < p.top_k) {
        const int s = t * p.top_k + lane;
        r.sel[s] = (int16_t)mine_e;
        r.p[s] = bad ? __uint_as_float(0x7FC00000u) : mine_e < 0 ? 0.f : mine_w / mass;
        if (mine_e >= 0)
            atomicOr(reinterpret_cast<unsigned long long*>(&r.mask[mine_e]), 1ull << t);
    }
}

// All tokens, the batches in the order of the experts' numbers, and each
// batch's rows in the order of the tokens.  Workgroup 0 writes the tables for
// the second launch and the caller's ids and weights.
template <int RQ>
__device__ void route(const MoeParams& p, Routing& r)
{
    const int tid = threadIdx.x, threads = blockDim.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), waves = threads >> 6, lane = tid & 63;
    for (int e = tid; e < p.E; e += threads) r.mask[e] = 0;
    __syncthreads();
    for (int t = wv; t < p.T; t += waves) route_token(p, t, r);
    __syncthreads();
    if (wv == 0) {
        // Lane l counts the batches of experts 8 l .. 8 l + 7.
        int n[kMaxSlots], sum = 0;
#pragma unroll
        for (int i = 0; i < kMaxSlots; ++i) {
            const int e = kMaxSlots * lane + i;
            n[i] = e < p.E ? ((int)__popcll(r.mask[e]) + 4 * RQ - 1) / (4 * RQ) : 0;
            sum += n[i];
        }
        int upto = sum;
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 63) r.batches = upto;
        upto -= sum;
#pragma unroll
        for (int i = 0; i < kMaxSlots; ++i) {
            const int e = kMaxSlots * lane + i;
            if (e < p.E) r.first[e] = (uint16_t)upto;
            upto += n[i];
        }
    }
    __syncthreads();
    const int batches = r.batches, pairs = p.T * p.top_k;
    for (int i = tid; i < batches * RQ; i += threads) reinterpret_cast<uint32_t*>(r.token)[i] = 0xFFFFFFFFu;
    __syncthreads();
    const bool tell = blockIdx.x == 0;
    for (int s = tid; s < pairs; s += threads) {
        const int e = r.sel[s], t = s / p.top_k;
        if (e >= 0) {
            const int rank = __popcll(r.mask[e] & ((1ull << t) - 1));
            const int b = r.first[e] + rank / (4 * RQ), row = b * 4 * RQ + rank % (4 * RQ);
            r.token[row] = (uint8_t)t;
            if (rank % (4 * RQ) == 0) r.batch_e[b] = (uint16_t)e;
            if (tell) p.row_p[row] = r.p[s];
        }
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
            p.row_token[i] = r.token[i] == kPadToken ? -1 : r.token[i];
    }
}

// One lane's 32-weight blocks of NC column quads, times RQ row quads.
//   acc[n][rq][r] += s * sum_k a[4 rq + r][k] (q[k] - z)
// w: the packed block of column 4n + i; s, z: its scale (fp16 bits) and the
// byte of its zero point; act: the block's activations of row 4 rq + i (pairs in the
// unpack's order).  ROWSCALE: acc[r] += s * f[rq][r] * ... with a scale per row.
template <int NC, int RQ, bool ROWSCALE>
__device__ __forceinline__ void block_products(const u32x4 (&w)[NC], const uint32_t (&s)[NC], const uint32_t (&z)[NC],
                                               int zshift, uint32_t zdef, uint32_t magic, const u32x4 (&act)[RQ][4],
                                               const float4_t (&f)[RQ], float4_t (&acc)[NC][RQ])
{
    // Column quads taken together, so that four chains of MFMAs run at once.
    constexpr int NI = RQ >= 4 ? 1 : 4 / RQ < NC ? 4 / RQ : NC;
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

// First launch: routing, gate and up products, h.  A unit is one batch by 32
// columns of h; a workgroup takes a contiguous range of units.  Wave (cw, ks)
// owns columns 8 cw .. 8 cw + 7 of the unit (two gate quads and the two up
// quads of the same columns) and, of every 4 W blocks of K, the 16 from 16 ks.
// The rows' activations are staged in LDS as fp16 in the unpack's order, rows
// 16 bytes apart modulo 128 so that eight lanes' reads fall on distinct banks.
template <int RQ, int W>
__global__ __launch_bounds__(64 * W) void mnb_moe_up_kernel(MoeParams p)
{
    constexpr int NC = 4, R = 4 * RQ;
    constexpr int SB = 16 * (W / 4);                 // blocks of K of a step, 16 per slice
    __shared__ Routing rt;
    __shared__ float part[2][W][NC * RQ * 16];
    extern __shared__ u32x4 stage[];                 // [rows][4 stage_blocks + 1]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), cw = wv & 3, ks = wv >> 2;
    const int qi = lane & 3, g = lane >> 2;
    const int nb = p.H / 32, zb = (nb + 1) / 2, hblocks = p.I / 32;
    const int row_pieces = 4 * p.stage_blocks + 1;   // 16-byte pieces of a staged row
    const uint32_t zdef = p.z1 ? 0u : 8u;
    const uint32_t magic = vgpr_constant(0x64006400u, p.zero);
    const int chunks = (nb + p.stage_blocks - 1) / p.stage_blocks;
    const bool all = p.T <= R;                       // every token staged once, rows by token

    // Rows [0, n) of the stage from tokens tok(row), blocks [b0, b0 + stage_blocks) of K.
    auto fill = [&](int n, int b0, auto tok) {
        const int per_row = 4 * p.stage_blocks;
        for (int i = tid; i < n * per_row; i += 64 * W) {
            const int row = i / per_row, pc = i - row * per_row, t = tok(row);
            u32x4 v = {0, 0, 0, 0};
            if (t != kPadToken && b0 + pc / 4 < nb)
                v = *reinterpret_cast<const u32x4*>(p.x + (int64_t)t * p.H + 32 * b0 + 8 * pc);
            stage[row * row_pieces + pc] = f16_pairs(v, p.x_bf16, 0);
        }
    };
    if (all && chunks == 1) fill(p.T, 0, [](int row) { return row; });
    route<RQ>(p, rt);

    const int batches = rt.batches;
    const int64_t units = (int64_t)batches * hblocks;   // at most 2^21
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    const int steps = (nb + SB - 1) / SB;            // of a unit
    const int chunk_steps = p.stage_blocks / SB;

    struct Step {
        u32x4 w[NC];
        uint32_t s[NC], z[NC];
    };
    const uint32_t row_bytes = (uint32_t)p.H / 2;
    // The loads run two steps ahead of use, across the units.
    int left = (u1 - u0) * steps, nbatch = u0 / hblocks, nhb = u0 - nbatch * hblocks, nstep = 0;
    auto next = [&](Step& st) {
        const bool live = left-- > 0;
        const int64_t e = live ? __builtin_amdgcn_readfirstlane(rt.batch_e[nbatch]) : 0;
        const int hb = live ? nhb : 0;
        const int blk = SB * nstep + 16 * ks + g;
        const bool in = live && blk < nb;
        if (++nstep == steps) {
            nstep = 0;
            if (++nhb == hblocks) {
                nhb = 0;
                ++nbatch;
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {       // gate, up
            const int64_t row0 = (e * 2 + half) * p.I + 32 * hb + 8 * cw;
            const __amdgpu_buffer_rsrc_t rW = make_rsrc_small(p.w1 + row0 * row_bytes, 8 * row_bytes);
            const __amdgpu_buffer_rsrc_t rS = make_rsrc_small(p.s1 + row0 * nb, 16 * (uint32_t)nb);
            const __amdgpu_buffer_rsrc_t rZ =
                make_rsrc_small(p.z1 ? p.z1 + row0 * zb : p.w1, p.z1 ? 8 * (uint32_t)zb : 0u);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint32_t c = (uint32_t)(4 * n + qi);
                st.w[2 * half + n] = __builtin_amdgcn_raw_buffer_load_b128(
                    rW, in ? c * row_bytes + 16 * (uint32_t)blk : kOutOfRange, 0, kNontemporal);
                st.s[2 * half + n] = __builtin_amdgcn_raw_buffer_load_b16(
                    rS, in ? 2 * (c * (uint32_t)nb + (uint32_t)blk) : kOutOfRange, 0, kNontemporal);
                st.z[2 * half + n] = __builtin_amdgcn_raw_buffer_load_b8(
                    rZ, in ? c * (uint32_t)zb + (uint32_t)blk / 2 : kOutOfRange, 0, kNontemporal);
            }
        }
    };

    Step ring[2];
    next(ring[0]);
    next(ring[1]);
    int staged = all && chunks == 1 ? -2 : -1;       // batch in the stage (-2: every token, -1: none)
    int buf = 0;
    float4_t acc[NC][RQ] = {};
    int b = u0 / hblocks, hb = u0 - b * hblocks, step = 0;   // the unit in work
    const float4_t no_f[RQ] = {};
    auto run = [&](Step& st) {
        if (staged != -2 && step % chunk_steps == 0 && (chunks > 1 || staged != b)) {
            __syncthreads();
            fill(R, SB * step, [&](int row) { return (int)rt.token[b * R + row]; });
            __syncthreads();
            staged = b;
        }
        u32x4 act[RQ][4];
#pragma unroll
        for (int rq = 0; rq < RQ; ++rq) {
            int row = 4 * rq + qi;
            if (staged == -2) {
                const int t = rt.token[b * R + row];
                row = t == kPadToken ? 0 : t;
            }
            const u32x4* src = stage + row * row_pieces + 4 * (SB * (step % chunk_steps) + 16 * ks + g);
#pragma unroll
            for (int pc = 0; pc < 4; ++pc) act[rq][pc] = src[pc];
        }
        block_products<NC, RQ, false>(st.w, st.s, st.z, 4 * (g & 1), zdef, magic, act, no_f, acc);
        next(st);
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
            const float h = gate / (1.f + __expf(-gate)) * up;
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
            if (rt.token[b * R + row] != kPadToken) {
                const int64_t at_h = (((int64_t)b * RQ + (row >> 2)) * hblocks + hb) * 4 + (row & 3);
                const int pos = (c & ~7) | ((c & 3) << 1) | (c >> 2 & 1);   // the unpack's pair order
                p.h[at_h * 32 + pos] = __builtin_bit_cast(uint16_t, (_Float16)ldexpf(h, -ex));
                if (c == 0) p.hs[at_h] = ldexpf(1.f, ex);
            }
        }
        buf ^= 1;
        if (++hb == hblocks) {
            hb = 0;
            ++b;
        }
    };
    const int total = (u1 - u0) * steps;
    for (int i = 0; i < total; i += 2) {
        run(ring[0]);
        if (i + 1 < total) run(ring[1]);
    }
}

// Second launch: down products and the weighted sum over experts.  A workgroup
// owns 4 NC columns of the output for every token.  Its items, one batch by 16
// blocks of K each, are dealt to its waves in contiguous runs; a wave adds
// each batch's products, weighted, to its own rows of y in LDS, and the
// waves' rows are added in wave order at the end.
template <int RQ, int NC, int W>
__global__ __launch_bounds__(64 * W) void mnb_moe_down_kernel(MoeParams p)
{
    constexpr int R = 4 * RQ, C = 4 * NC;
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
        uint32_t s[NC], z[NC];
        float4_t f[RQ];
    };
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
            make_rsrc_small(p.h + (int64_t)b * RQ * nb * 128, live ? RQ * (uint32_t)nb * 256 : 0u);
        const __amdgpu_buffer_rsrc_t rF = make_rsrc_small(p.hs + (int64_t)b * RQ * nb * 4, live ? RQ * (uint32_t)nb * 16 : 0u);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const uint32_t c = (uint32_t)(4 * n + qi);
            st.w[n] = __builtin_amdgcn_raw_buffer_load_b128(rW, in ? c * row_bytes + 16 * (uint32_t)blk : kOutOfRange, 0,
                                                            kNontemporal);
            st.s[n] = __builtin_amdgcn_raw_buffer_load_b16(
                rS, in ? 2 * (c * (uint32_t)nb + (uint32_t)blk) : kOutOfRange, 0, kNontemporal);
            st.z[n] = __builtin_amdgcn_raw_buffer_load_b8(rZ, in ? c * (uint32_t)zb + (uint32_t)blk / 2 : kOutOfRange, 0,
                                                          kNontemporal);
        }
#pragma unroll
        for (int rq = 0; rq < RQ; ++rq) {
            // Unused rows load zeros.
            const bool used = in && 4 * rq + qi < rows;
            const uint32_t at = (uint32_t)(rq * nb + blk);
#pragma unroll
            for (int pc = 0; pc < 4; ++pc)
                st.a[rq][pc] = __builtin_amdgcn_raw_buffer_load_b128(
                    rA, used ? at * 256 + 64 * (uint32_t)qi + 16 * pc : kOutOfRange, 0, 0);
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
        block_products<NC, RQ, true>(st.w, st.s, st.z, 4 * (g & 1), zdef, magic, st.a, st.f, acc);
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
    for (int i = i0; i < i1; i += 2) {
        run(ring[0], i);
        if (i + 1 < i1) run(ring[1], i + 1);
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

template <int RQ, int W>
hipError_t queue_up(const MoeParams& p, int cus, hipStream_t s)
{
    const size_t lds = (size_t)4 * RQ * (4 * p.stage_blocks + 1) * 16;
    const void* fn = reinterpret_cast<const void*>(mnb_moe_up_kernel<RQ, W>);
    hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    const int64_t most = (int64_t)p.T * p.top_k * (p.I / 32);
    const unsigned grid = (unsigned)(most < cus ? most : cus);
    MoeParams q = p;
    void* args[] = {&q};
    return hipLaunchKernel(fn, dim3(grid), dim3(64 * W), args, lds, s);
}

template <int RQ, int NC, int W>
hipError_t queue_down(const MoeParams& p, hipStream_t s)
{
    const size_t lds = ((size_t)W * p.T * 4 * NC + (size_t)p.batch_cap * (8 * RQ + 1)) * 4;
    const void* fn = reinterpret_cast<const void*>(mnb_moe_down_kernel<RQ, NC, W>);
    hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    MoeParams q = p;
    void* args[] = {&q};
    return hipLaunchKernel(fn, dim3((unsigned)(p.H / (4 * NC))), dim3(64 * W), args, lds, s);
}

}  // namespace

int launch_moe(const MoeArgs& a, void* stream, int* launches)
{
    int cus = 0;
    int e = current_device_cus(&cus);
    if (e != 0) return e;
    const MoeLayout lay = moe_layout(a.T, a.w.hidden, a.w.inter, a.w.experts, a.top_k);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    MoeParams p;
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
    // The first launch stages whole rows where they fit, else spans of K.
    const int blocks = (p.H / 32 + 63) / 64 * 64, most = lay.rq == 1 ? 512 : 192;
    p.stage_blocks = blocks < most ? blocks : most;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t he = lay.rq == 1 ? queue_up<1, 16>(p, cus, s) : queue_up<2, 8>(p, cus, s);
    if (he != hipSuccess) return (int)he;
    ++*launches;
    // Columns of a workgroup: as few as fill the device.
    const int nc = p.H / 16 >= cus ? 4 : p.H / 8 >= cus ? 2 : 1;
    if (lay.rq == 1)
        he = nc == 4 ? queue_down<1, 4, 12>(p, s) : nc == 2 ? queue_down<1, 2, 16>(p, s) : queue_down<1, 1, 16>(p, s);
    else
        he = nc == 4 ? queue_down<2, 4, 8>(p, s) : nc == 2 ? queue_down<2, 2, 8>(p, s) : queue_down<2, 1, 8>(p, s);
    if (he == hipSuccess) ++*launches;
    return (int)he;
}

}  // namespace mnb
