// 8-bit products on gfx950: rows of activations quantised to int8 with one
// scale per row, and their product with int8 weights on the integer matrix
// cores.
//
//   scale[r] = max|a[r]| / 127,   q[r][k] = rint(127 a[r][k] / max|a[r]|)
//   y[r][n]  = (sum_k q[r][k] w[n][k]) * a_scale[r] * b_scale[n] + bias[n]
//
// The sum over k is exact: int32 products, at most 2^31 / 2^14 of them.  So
// the order in which it runs never shows in the result, and every split of K
// over lanes and waves gives the same bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mnb.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Quantising a row: L threads hold it in P pieces of eight elements each
// (rows longer than 8 L P are walked in such chunks and read twice), the row's
// largest magnitude is found on the bit patterns (for fp16 and bf16 alike the
// absolute value's bits are in the order of the values, infinities and NaN
// above every finite one), and the pieces are rounded.
//
// The integer is the exact quotient 127 a / max rounded to nearest even.
// t = a * fl(127 / max) is off by at most 127 * 2^-23 < 2^-16, so rint(t) is
// that integer wherever t is further than 2^-15 from a half-integer; the few
// other elements take the division.  There 127 a is exact in fp32, and no
// quotient but an exact tie comes closer to a half-integer than 2^-21 of it
// (both sides have at most 18 significant bits), so the fp32 quotient rounds
// to the same integer.  Rows whose largest magnitude lies outside 2^-100 ..
// 2^100, where 127 / max or 127 a leave fp32, are first scaled by a power of
// two (exact: what that flushes is far below half a step).
struct QuantizeParams {
    const uint16_t* A;   // [m][K]
    int8_t* q;           // [m][K]
    float* scales;       // [m]
    int64_t m, K;
    int32_t a_bf16;
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// What quantising needs of a row.
struct RowScale {
    float top, inv, scale;   // largest magnitude (normalised), 127 / top, the row's scale
    int shift;               // elements are multiplied by 2^shift first
    bool zero;               // zeros, or a value that is not finite: q = 0
};

__device__ __forceinline__ RowScale row_scale(uint32_t top_bits, int bf16)
{
    RowScale r;
    const float amax = widen16(top_bits, bf16);
    const bool finite = top_bits < (bf16 ? 0x7F80u : 0x7C00u);
    r.scale = finite ? amax / 127.0f : __uint_as_float(0x7FC00000u);
    r.zero = !finite || top_bits == 0;
    const int e = r.zero ? 0 : ilogbf(amax);
    r.shift = e < -100 || e > 100 ? -e : 0;
    r.top = r.zero ? 1.f : ldexpf(amax, r.shift);
    r.inv = 127.0f / r.top;
    return r;
}

// Two elements (the halves of w) to int8 in bytes 0 and 1 of the result.
__device__ __forceinline__ uint32_t quantize_pair(uint32_t w, const RowScale& r, int bf16)
{
    constexpr float kRound = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer in the low bits
    float x[2] = {widen16(w & 0xFFFFu, bf16), widen16(w >> 16, bf16)};
    if (r.shift)
        for (int i = 0; i < 2; ++i) x[i] = ldexpf(x[i], r.shift);
    float s[2], far = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float t = x[i] * r.inv;
        s[i] = t + kRound;
        far = fmaxf(far, fabsf(t - (s[i] - kRound)));
    }
    if (far > 0.5f - 0x1p-15f)
#pragma unroll
        for (int i = 0; i < 2; ++i) s[i] = rintf(127.0f * x[i] / r.top) + kRound;
    return r.zero ? 0u : __builtin_amdgcn_perm(__float_as_uint(s[1]), __float_as_uint(s[0]), 0x0C0C0400u);
}

__device__ __forceinline__ u32x2 quantize_piece(u32x4 v, const RowScale& r, int bf16)
{
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = quantize_pair(v[i], r, bf16);
    return u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)};
}

template <int L, int P>
__global__ __launch_bounds__(L < 256 ? 256 : L) void mnb_quantize_rows_kernel(QuantizeParams p)
{
    constexpr int ROWS = L < 256 ? 256 / L : 1;   // rows of a workgroup
    constexpr int W = L / 64;                     // waves of a row
    __shared__ uint32_t part[L < 256 ? 4 : W];
    const int tid = threadIdx.x % L;
    const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / L;
    const bool mine = r < p.m;
    const u32x4* src = reinterpret_cast<const u32x4*>(p.A + (mine ? r * p.K : 0));
    const int64_t pieces = mine ? p.K / 8 : 0;    // K is a multiple of 16
    u32x4 v[P];
    uint32_t top2 = 0;
    for (int64_t c = 0; c < pieces || c == 0; c += L * P) {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = c + L * i + tid < pieces ? src[c + L * i + tid] : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) top2 = max_u16x2(top2, v[i][d] & 0x7FFF7FFFu);
    }
    uint32_t top = (top2 & 0xFFFFu) > (top2 >> 16) ? top2 & 0xFFFFu : top2 >> 16;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = __shfl_xor(top, d);
        top = o > top ? o : top;
    }
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) top = part[w] > top ? part[w] : top;
    }
    if (!mine) return;
    const RowScale rs = row_scale(top, p.a_bf16);
    if (tid == 0) p.scales[r] = rs.scale;
    u32x2* dst = reinterpret_cast<u32x2*>(p.q + r * p.K);
    const bool again = pieces > L * P;            // the registers hold the last chunk only
    for (int64_t c = 0; c < pieces; c += L * P) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t k = c + L * i + tid;
            if (k < pieces) dst[k] = quantize_piece(again ? src[k] : v[i], rs, p.a_bf16);
        }
    }
}

template <int L, int P>
void queue_quantize(const QuantizeParams& p, hipStream_t stream)
{
    constexpr int ROWS = L < 256 ? 256 / L : 1;
    hipLaunchKernelGGL((mnb_quantize_rows_kernel<L, P>), dim3((unsigned)((p.m + ROWS - 1) / ROWS)),
                       dim3(L < 256 ? 256 : L), 0, stream, p);
}

struct Int8Params {
    const int8_t* A;        // [M][K]
    const uint16_t* A16;    // the rows as fp16 or bf16, quantised by the kernel
    const float* a_scales;  // [M]
    const int8_t* B;        // [N][K]
    const float* b_scales;  // [N]
    const float* bias;      // [N] or null
    uint16_t* out;          // [M][N]
    int64_t M, N;
    int32_t K;
    int32_t a_bf16, out_bf16;
};

// The result of one output from its exact sum.  (The FMA is spelled out: the
// kernels must give the same bits.)
__device__ __forceinline__ uint16_t finish(int sum, float a_scale, float b_scale, float bias, int out_bf16)
{
    return narrow16(fmaf((float)sum * b_scale, a_scale, bias), out_bf16);
}

// Few rows (m <= 16, K <= 16384): one pass over the weights, which HBM bounds.
//
// A workgroup keeps the rows in LDS and walks its tiles of 16 columns.  Its
// waves split K: wave w takes every W-th 128 bytes of it, NU of them, whose
// weights it loads one tile ahead (16 KB to 256 KB under way per workgroup).
// v_mfma_i32_16x16x64_i8: lane (j, g) supplies 16 k of row j and of column j.  The
// waves' sums of a tile meet in LDS.  FUSE: the rows come as fp16 or bf16 and
// the workgroup quantises them itself, which spares a launch.
//
// LDS: rows [M][K + 16] (lanes j read rows 16 bytes apart modulo 128), then the
// sums of two tiles [2][W][64] x 16 bytes.
template <int NU, bool FUSE>
__global__ __launch_bounds__(1024) void mnb_int8_rows_kernel(Int8Params p)
{
    extern __shared__ u32x4 rows_lds_buf[];
    __shared__ float row_scales[16];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), threads = (int)blockDim.x, W = threads >> 6;
    const int M = (int)p.M;
    const uint32_t K = (uint32_t)p.K, stride = K + 16;
    char* const rows = reinterpret_cast<char*>(rows_lds_buf);
    i32x4* const part = reinterpret_cast<i32x4*>(rows + (uint32_t)M * stride);   // [2][W][64]

    // This workgroup's tiles: as few for each as the busiest one needs.
    const int tiles = (int)((p.N + 15) / 16), per = (tiles + (int)gridDim.x - 1) / (int)gridDim.x;
    const int t0 = (int)blockIdx.x * per < tiles ? (int)blockIdx.x * per : tiles;
    const int t1 = t0 + per < tiles ? t0 + per : tiles;

    u32x4 b[NU][2];
    // Piece (u, d) of a tile: 16 bytes of column j from 128 (wv + W u) + 64 d + 16 g.
    auto offset = [&](int u, int d) { return 128u * (uint32_t)(wv + W * u) + 64u * d + 16u * (uint32_t)g; };
    auto issue = [&](int t, int u) {
        const int64_t c0 = (int64_t)t * 16, left = p.N - c0;
        const uint32_t cols = t >= t1 ? 0u : left < 16 ? (uint32_t)left : 16u;
        const __amdgpu_buffer_rsrc_t rB = make_rsrc_small(p.B + (t < t1 ? c0 * K : 0), cols * K);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const uint32_t k = offset(u, d);
            b[u][d] = __builtin_amdgcn_raw_buffer_load_b128(rB, k < K ? (uint32_t)j * K + k : kOutOfRange, 0, kNontemporal);
        }
    };
#pragma unroll
    for (int u = 0; u < NU; ++u) issue(t0, u);

    if constexpr (FUSE) {
        // Each row is one wave's, or with more waves than rows that of WR
        // waves.  A lane holds eight pieces of eight elements; what a row has
        // beyond that is read again.
        const int pieces = (int)K / 8;
        u32x4 v[8];
        auto load = [&](int r, int at, int step) {
            const __amdgpu_buffer_rsrc_t rA = make_rsrc_small(p.A16 + (int64_t)r * K, 2 * K);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __builtin_amdgcn_raw_buffer_load_b128(rA, 16 * (uint32_t)(at + i * step), 0, 0);
        };
        auto largest = [&](int r, int first, int step) {
            uint32_t top2 = 0;
            for (int at = first; at < pieces; at += 8 * step) {
                load(r, at, step);
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int d = 0; d < 4; ++d) top2 = max_u16x2(top2, v[i][d] & 0x7FFF7FFFu);
            }
            uint32_t top = (top2 & 0xFFFFu) > (top2 >> 16) ? top2 & 0xFFFFu : top2 >> 16;
#pragma unroll
            for (int d = 32; d; d >>= 1) {
                const uint32_t o = __shfl_xor(top, d);
                top = o > top ? o : top;
            }
            return top;
        };
        auto store = [&](int r, uint32_t top, int first, int step) {
            const RowScale rs = row_scale(top, p.a_bf16);
            if (first == 0) row_scales[r] = rs.scale;
            for (int at = first; at < pieces; at += 8 * step) {
                if (pieces > 8 * step) load(r, at, step);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int k = at + i * step;
                    if (k < pieces)
                        *reinterpret_cast<u32x2*>(rows + (uint32_t)r * stride + 8 * k) = quantize_piece(v[i], rs, p.a_bf16);
                }
            }
        };
        if (M >= W) {
            for (int r = wv; r < M; r += W) store(r, largest(r, lane, 64), lane, 64);
        } else {
            const int WR = W / M, r = wv / WR, first = (wv - r * WR) * 64 + lane, step = 64 * WR;
            uint32_t* const tops = reinterpret_cast<uint32_t*>(part);   // [row][WR]
            const uint32_t mine = r < M ? largest(r, first, step) : 0u;
            if (lane == 0 && r < M) tops[wv] = mine;
            __syncthreads();
            if (r < M) {
                uint32_t top = 0;
                for (int w = 0; w < WR; ++w) top = tops[r * WR + w] > top ? tops[r * WR + w] : top;
                store(r, top, first, step);
            }
        }
    } else {
        const int pieces = (int)K / 16;
        for (int i = tid; i < M * pieces; i += threads) {
            const int r = i / pieces;
            *reinterpret_cast<u32x4*>(rows + 16 * (uint32_t)(i + r)) = *reinterpret_cast<const u32x4*>(p.A + 16 * (int64_t)i);
        }
    }
    __syncthreads();

    // Lanes of rows past M read row 0; their results are not used.
    const char* const mine = rows + (j < M ? (uint32_t)j * stride : 0u);
    for (int t = t0; t < t1; ++t) {
        i32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < NU; ++u) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                // (Past K the weights are zeros, and the row's bytes anything.)
                const uint32_t k = offset(u, d);
                const i32x4 a = *reinterpret_cast<const i32x4*>(mine + (k < K ? k : 0u));
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, __builtin_bit_cast(i32x4, b[u][d]), acc, 0, 0, 0);
            }
            issue(t + 1, u);
        }
        // Lane (j, g) holds rows 4 g .. 4 g + 3 of column j.
        i32x4* const now = part + (t & 1) * W * 64;
        if (4 * g < M) now[wv * 64 + lane] = acc;
        __syncthreads();
        // Output (row, column) by thread: the waves' sums.
        const int* const sums = reinterpret_cast<const int*>(now);
        for (int o = tid; o < 16 * M; o += threads) {
            const int row = o >> 4, c = o & 15;
            const int at = ((row >> 2) * 16 + c) * 4 + (row & 3);
            int sum = 0;
            for (int w = 0; w < W; ++w) sum += sums[w * 256 + at];
            const int64_t col = (int64_t)t * 16 + c;
            if (col < p.N)
                p.out[row * p.N + col] = finish(sum, FUSE ? row_scales[row] : p.a_scales[row], p.b_scales[col],
                                                p.bias ? p.bias[col] : 0.f, p.out_bf16);
        }
    }
}

// Sixteen bytes per lane from global memory straight into LDS (lane l to lds +
// 16 l).  Written as assembly because the compiler makes every LDS read that
// follows the builtin wait for the transfer; here the caller waits, once per
// stage (turn_over).  It has no result registers, and M0, which it sets, is
// read by nothing else in these kernels (the compiler reserves it).
__device__ __forceinline__ void load_to_lds(i32x4 rsrc, uint32_t voffset, uint32_t soffset, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(voffset), "s"(rsrc), "s"(soffset), "s"(lds) : "memory");
}

__device__ __forceinline__ i32x4 rsrc_words(const void* base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)(uintptr_t)base;
    return i32x4{(int)(uint32_t)b, (int)(uint32_t)((b >> 32) & 0xFFFFu), (int)bytes, kRsrcWord3};
}

// Sixteen bytes at any even address (rows of an odd number of columns).
struct __attribute__((packed, aligned(2))) Loose16 {
    u32x4 v;
};

// A workgroup tile of BM rows by BN columns: WM x WN waves of (BM / WM) x (BN /
// WN) each, and KS such sets that split each stage's K.  A stage is KB (64 or
// 128) bytes of every row and column for each set, NS of them in LDS.  Rows lie
// KB bytes apart, 16-byte piece c of row r in slot c ^ swizzle(r), so that the
// eight rows that one LDS access of a fragment covers lie in distinct banks.
template <int BM, int BN, int WM, int WN, int KS, int NS, int KB>
__global__ __launch_bounds__(64 * WM * WN * KS) void mnb_int8_tile_kernel(Int8Params p)
{
    constexpr int W = WM * WN * KS, RT = BM / WM / 32, CT = BN / WN / 32;
    constexpr int LR = KB / 16, RR = 64 / LR;                        // lanes of a row, rows of a transfer
    constexpr int PA = BM * KS / RR / W, PB = BN * KS / RR / W;      // transfers of a wave and stage
    static_assert(PA * RR * W == BM * KS && PB * RR * W == BN * KS, "whole transfers per wave");
    constexpr uint32_t kStage = (BM + BN) * KS * KB;
    static_assert((KS - 1) * WM * WN * RT * CT * 4096u + WM * WN * 32 * (2 * BN / WN + 16) <= NS * kStage,
                  "partial sums and turned rows fit the stages");
    auto swizzle = [](int r) { return KB == 128 ? r & 7 : (r >> 1) & 3; };
    extern __shared__ u32x4 tile_lds[];
    __shared__ float scale_lds[BN], bias_lds[BN];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 31, h = lane >> 5;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = wv / (WM * WN), wm = wv / WN % WM, wn = wv % WN;
    const uint32_t K = (uint32_t)p.K;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)tile_lds;

    // Consecutive tiles share their columns; each of the 8 dies (workgroups
    // are dealt to them in turn) gets a contiguous run of tiles, so that its
    // L2 holds few columns at a time.
    const int tiles_m = (int)((p.M + BM - 1) / BM);
    const int64_t tiles = (int64_t)gridDim.x, share = tiles / 8, extra = tiles % 8;
    const int64_t die = blockIdx.x & 7, in_die = blockIdx.x >> 3;
    const int64_t tile = die * share + (die < extra ? die : extra) + in_die;
    const int64_t r0 = tile % tiles_m * BM, c0 = tile / tiles_m * BN;
    const int rows = (int)(p.M - r0 < BM ? p.M - r0 : BM), cols = (int)(p.N - c0 < BN ? p.N - c0 : BN);
    const i32x4 rA = rsrc_words(p.A + r0 * K, (uint32_t)rows * K), rB = rsrc_words(p.B + c0 * K, (uint32_t)cols * K);

    for (int c = tid; c < BN; c += 64 * W) {
        scale_lds[c] = c < cols ? p.b_scales[c0 + c] : 0.f;
        bias_lds[c] = c < cols && p.bias ? p.bias[c0 + c] : 0.f;
    }

    // This lane's part of the wave's transfers: one slot of one of RR rows;
    // rows past the last repeat it (their results are not stored).
    const uint32_t piece = 16u * (uint32_t)((lane % LR) ^ swizzle(lane / LR));
    uint32_t oa[PA], ob[PB];
#pragma unroll
    for (int i = 0; i < PA; ++i) {
        const int q = (wv * PA + i) * RR, r = q % BM + lane / LR;
        oa[i] = (uint32_t)(r < rows ? r : rows - 1) * K + KB * (q / BM) + piece;
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
        const int q = (wv * PB + i) * RR, r = q % BN + lane / LR;
        ob[i] = (uint32_t)(r < cols ? r : cols - 1) * K + KB * (q / BN) + piece;
    }
    const int stages = (int)((K + KB * KS - 1) / (KB * KS));
    // Transfers [i0, i1) of the wave's PER of stage st.
    constexpr int PER = PA + PB, V = KB / 32;
    auto fetch = [&](int st, int i0, int i1) {
        const uint32_t k0 = KB * KS * (uint32_t)st, base = lds0 + (uint32_t)(st % NS) * kStage;
#pragma unroll
        for (int i = 0; i < PA; ++i) {
            const int q = (wv * PA + i) * RR;
            if (i >= i0 && i < i1)
                load_to_lds(rA, k0 + KB * (q / BM) + piece < K ? oa[i] : kOutOfRange, k0, base + KB * q);
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int q = (wv * PB + i) * RR;
            if (PA + i >= i0 && PA + i < i1)
                load_to_lds(rB, k0 + KB * (q / BN) + piece < K ? ob[i] : kOutOfRange, k0, base + KB * (BM * KS + q));
        }
    };

    typedef int i32x16 __attribute__((ext_vector_type(16)));
    i32x16 acc[RT][CT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[rt][ct][q] = 0;

    // Fragment v (32 of a stage's k): piece 2 v + h of row j of each tile.
    const char* const lds = reinterpret_cast<const char*>(tile_lds);
    const uint32_t fa = KB * (uint32_t)(ks * BM + wm * (BM / WM) + j);
    const uint32_t fb = KB * (uint32_t)(BM * KS + ks * BN + wn * (BN / WN) + j);
    auto read = [&](int st, int v, i32x4 (&a)[RT], i32x4 (&b)[CT]) {
        const char* const base = lds + (uint32_t)(st % NS) * kStage + 16u * (uint32_t)((2 * v + h) ^ swizzle(j));
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) b[ct] = *reinterpret_cast<const i32x4*>(base + fb + 32 * KB * ct);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) a[rt] = *reinterpret_cast<const i32x4*>(base + fa + 32 * KB * rt);
    };
    // Each of a stage's V fragments multiplies while the next one's operands
    // are read.  Stage st + 1 is waited for, and its first operands are read,
    // before the last products of stage st, which cover that: this wave's
    // transfers of it are complete (later ones may be under way) and its
    // reads of stage st too, then every wave's.  From there on stage st + NS
    // takes the place of stage st, a part of its transfers with each
    // fragment: all at once they hold up the waves, which issue in order
    // behind them (256 x 128 on 2048 x 14336 x 4096: 121 -> 115 us; without any
    // transfers 96, with the products alone 85).
    // (Stages past K transfer zeros.)
    i32x4 a[2][RT], b[2][CT];
    auto turn_over = [&](int st) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                     ::"i"((NS - 3) * PER + PER * (V - 1) / V) : "memory");
        read(st + 1, 0, a[0], b[0]);
    };
    static_assert(NS >= 3, "a stage's transfers are issued over the length of one");
#pragma unroll
    for (int st = 0; st < NS - 2; ++st) fetch(st, 0, PER);
    fetch(NS - 2, 0, PER * (V - 1) / V);
    turn_over(-1);
    fetch(NS - 2, PER * (V - 1) / V, PER);
    for (int st = 0; st < stages; ++st) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (v + 1 < V) read(st, v + 1, a[(v + 1) & 1], b[(v + 1) & 1]);
            else turn_over(st);
            fetch(st + NS - 1, PER * v / V, PER * (v + 1) / V);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    acc[rt][ct] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[v & 1][ct], a[v & 1][rt], acc[rt][ct], 0, 0, 0);
        }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

    if constexpr (KS > 1) {
        // Sets 1 .. KS - 1 leave their sums in LDS; set 0 adds them.
        i32x16* const part = reinterpret_cast<i32x16*>(tile_lds);
        auto at = [&](int k, int rt, int ct) { return ((((k - 1) * WM * WN + wm * WN + wn) * RT + rt) * CT + ct) * 64 + lane; };
        if (ks > 0) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) part[at(ks, rt, ct)] = acc[rt][ct];
        }
        __syncthreads();
        if (ks > 0) return;
#pragma unroll
        for (int k = 1; k < KS; ++k)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) acc[rt][ct] += part[at(k, rt, ct)];
    }

    // The weights are the product's first operand, so element q of lane (j,
    // h) is row j, column (q % 4) + 4 h + 8 (q / 4): four neighbours of one row
    // at a time.  A wave turns each 32 rows of its part through LDS into whole
    // 16-byte pieces of rows (one 2-byte store per element had cost the 256 x
    // 128 tile 10 us).
    constexpr int CW = BN / WN, kPitch = 2 * CW + 16;   // bytes of a turned row
    char* const turn = reinterpret_cast<char*>(tile_lds) + (KS - 1) * WM * WN * RT * CT * 4096 + (wm * WN + wn) * 32 * kPitch;
    const int wc = wn * CW, width = cols - wc < CW ? cols - wc : CW;   // the wave's columns
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int wr = wm * (BM / WM) + 32 * rt;
        const float as = p.a_scales[r0 + (wr + j < rows ? wr + j : rows - 1)];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
                const int c = 32 * ct + 8 * q4 + 4 * h;
                const float4_t bs = *reinterpret_cast<const float4_t*>(&scale_lds[wc + c]);
                const float4_t bias = *reinterpret_cast<const float4_t*>(&bias_lds[wc + c]);
                uint32_t o[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    o[i] = finish(acc[rt][ct][4 * q4 + 2 * i], as, bs[2 * i], bias[2 * i], p.out_bf16) |
                           (uint32_t)finish(acc[rt][ct][4 * q4 + 2 * i + 1], as, bs[2 * i + 1], bias[2 * i + 1], p.out_bf16) << 16;
                *reinterpret_cast<u32x2*>(turn + j * kPitch + 2 * c) = u32x2{o[0], o[1]};
            }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        constexpr int LPR = CW / 8;                     // lanes of a row
#pragma unroll
        for (int i = 0; i < 32 * LPR / 64; ++i) {
            const int r = i * (64 / LPR) + lane / LPR, c = lane % LPR * 8;
            if (wr + r >= rows || c >= width) continue;
            uint16_t* const out = p.out + (r0 + wr + r) * p.N + c0 + wc + c;
            const uint16_t* const from = reinterpret_cast<const uint16_t*>(turn + r * kPitch + 2 * c);
            if (c + 8 <= width) {
                reinterpret_cast<Loose16*>(out)->v = *reinterpret_cast<const u32x4*>(from);
            } else {
                for (int k = 0; k < width - c; ++k) out[k] = from[k];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    }
}

typedef void (*Int8Fn)(Int8Params);

template <bool FUSE>
Int8Fn rows_kernel(int nu)
{
    switch (nu) {
    case 1: return mnb_int8_rows_kernel<1, FUSE>;
    case 2: return mnb_int8_rows_kernel<2, FUSE>;
    case 3: return mnb_int8_rows_kernel<3, FUSE>;
    case 4: return mnb_int8_rows_kernel<4, FUSE>;
    case 5: return mnb_int8_rows_kernel<5, FUSE>;
    case 6: return mnb_int8_rows_kernel<6, FUSE>;
    case 7: return mnb_int8_rows_kernel<7, FUSE>;
    default: return mnb_int8_rows_kernel<8, FUSE>;
    }
}

hipError_t queue(Int8Fn fn, const Int8Params& p, int64_t grid, int threads, size_t lds, hipStream_t s)
{
    Int8Params q = p;
    void* args[] = {&q};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)grid), dim3((unsigned)threads),
                                         args, lds, s);
    return e != hipSuccess ? e : hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int KS, int NS, int KB>
hipError_t queue_tile(const Int8Params& p, hipStream_t s)
{
    const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
    return queue(mnb_int8_tile_kernel<BM, BN, WM, WN, KS, NS, KB>, p, tiles, 64 * WM * WN * KS,
                 (size_t)NS * (BM + BN) * KS * KB, s);
}

}  // namespace

int launch_quantize_rows(const void* A, int a_bf16, int64_t m, int64_t K, int8_t* q, float* scales, void* stream)
{
    const QuantizeParams p{static_cast<const uint16_t*>(A), q, scales, m, K, a_bf16};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (quantize_variant(m, K)) {
    case 0: queue_quantize<64, 1>(p, s); break;
    case 1: queue_quantize<256, 1>(p, s); break;
    case 2: queue_quantize<256, 8>(p, s); break;
    case 3: queue_quantize<1024, 1>(p, s); break;
    default: queue_quantize<1024, 4>(p, s); break;
    }
    return (int)hipGetLastError();
}

int launch_int8(const Int8Args& a, void* stream, int* launches)
{
    int cus = 0;
    int e = current_device_cus(&cus);
    if (e != 0) return e;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const Int8Route route = int8_route(a.a_dtype, a.m, a.K, a.N, cus);
    Int8Params p{};
    p.A = static_cast<const int8_t*>(a.A);
    p.A16 = static_cast<const uint16_t*>(a.A);
    p.a_scales = a.a_scales;
    p.a_bf16 = a.a_dtype == MNB_BF16;
    if (a.a_dtype != MNB_I8 && !route.fused) {
        int8_t* q = static_cast<int8_t*>(a.ws);
        float* scales = reinterpret_cast<float*>(q + a.m * a.K);
        e = launch_quantize_rows(a.A, p.a_bf16, a.m, a.K, q, scales, stream);
        if (e != 0) return e;
        ++*launches;
        p.A = q;
        p.a_scales = scales;
    }
    p.B = a.B;
    p.b_scales = a.b_scales;
    p.bias = a.bias;
    p.out = static_cast<uint16_t*>(a.out);
    p.M = a.m;
    p.N = a.N;
    p.K = (int32_t)a.K;
    p.out_bf16 = a.out_bf16;
    hipError_t he;
    if (route.tile < 0) {
        he = queue(route.fused ? rows_kernel<true>(route.nu) : rows_kernel<false>(route.nu), p, route.workgroups,
                   64 * route.waves, int8_rows_lds(a.m, a.K, route.waves), s);
    } else {
        switch (route.tile) {
        case 0: he = queue_tile<256, 256, 2, 4, 1, 4, 64>(p, s); break;
        case 1: he = queue_tile<256, 128, 4, 2, 1, 3, 128>(p, s); break;
        case 2: he = queue_tile<128, 128, 2, 4, 1, 4, 128>(p, s); break;
        case 3: he = queue_tile<128, 64, 2, 2, 2, 3, 128>(p, s); break;
        case 4: he = queue_tile<64, 64, 2, 2, 2, 3, 128>(p, s); break;
        case 5: he = queue_tile<64, 32, 2, 1, 4, 3, 128>(p, s); break;
        default: he = queue_tile<32, 32, 1, 1, 4, 4, 128>(p, s); break;
        }
    }
    if (he == hipSuccess) ++*launches;
    return (int)he;
}

}  // namespace mnb
