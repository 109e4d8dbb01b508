// Low-rank adapters of many requests at once, beside a shared projection, on
// gfx950.
//
//   out[r] = base[r] + s[a] B[a] (A[a] x[r]),   a = ids[r]   (out[r] = base[r] without one)
//
// Two launches.  The first multiplies tiles of rows with the A of every adapter
// that one of them uses, K split over workgroups, and leaves fp32 sums per row
// and slice.  The second adds the slices in order, splits the sums into two
// 16-bit pieces (together they keep 16 bits of a bf16 operand's sum and 21 of
// an fp16 one's), multiplies with the rows of B and adds the base, rounding
// once.  Both run on v_mfma_f32_16x16x32_{f16,bf16} straight from the loads.
// HBM bounds both: x, the used adapters, base and out are read or written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8_t __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;

struct LoraParams {
    const uint16_t* x;        // [m][K]
    const int32_t* ids;       // [m]
    const uint16_t* A;        // [adapters][R][K]
    const uint16_t* B;        // [adapters][N][R]
    const float* scaling;     // [adapters] or null
    const uint16_t* base;     // [m][N] rows of base_stride, or null
    uint16_t* out;
    float* t;                 // [splits][m][R]
    int64_t m, x_stride, base_stride, out_stride;
    int32_t K, N, R, adapters, splits;
    int32_t k_slice;          // K of a slice: a multiple of 32 * kWaves
    int32_t out_bf16;
};

template <bool BF16>
__device__ __forceinline__ float4_t mfma(u32x4 a, u32x4 b, float4_t c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8_t, a), __builtin_bit_cast(bhalf8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// The adapter of a row of this tile, -1 for none (or a number that is none).
template <int RT>
__device__ __forceinline__ int32_t tile_id(const LoraParams& p, int64_t row0)
{
    const int64_t r = row0 + (threadIdx.x & 63);
    if ((int)(threadIdx.x & 63) >= RT || r >= p.m) return -1;
    const int32_t a = p.ids[r];
    return a >= 0 && a < p.adapters ? a : -1;
}

// Rows to rank: a workgroup takes RT = 16 NRT rows, one slice of K and, of the
// adapters that its rows use, every gridDim.z-th; its waves split the slice.
// RKT tiles of 16 ranks at a time.
template <bool BF16, int NRT, int RKT>
__global__ __launch_bounds__(64 * kWaves) void mnb_lora_down_kernel(LoraParams p)
{
    constexpr int RT = 16 * NRT;
    __shared__ float4_t part[kWaves - 1][NRT * RKT][64];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row0 = (int64_t)blockIdx.x * RT;
    const int32_t id = tile_id<RT>(p, row0);
    uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0);
    const int32_t k0 = (int32_t)blockIdx.y * p.k_slice, k1 = k0 + p.k_slice < p.K ? k0 + p.k_slice : p.K;
    const uint16_t* xr[NRT];
#pragma unroll
    for (int n = 0; n < NRT; ++n) {
        const int64_t row = row0 + 16 * n + r < p.m ? row0 + 16 * n + r : p.m - 1;
        xr[n] = p.x + row * p.x_stride + 8 * g;
    }
    for (int j = 0; left; ++j) {
        const int32_t a = __shfl(id, __builtin_ctzll(left));
        const uint64_t mine = __builtin_amdgcn_ballot_w64(id == a);
        left &= ~mine;
        if (j % gridDim.z != blockIdx.z) continue;
        for (int c0 = 0; c0 < p.R; c0 += 16 * RKT) {
            const uint16_t* ar[RKT];
#pragma unroll
            for (int c = 0; c < RKT; ++c) {
                const int rank = c0 + 16 * c + r < p.R ? c0 + 16 * c + r : p.R - 1;
                ar[c] = p.A + ((int64_t)a * p.R + rank) * p.K + 8 * g;
            }
            float4_t acc[NRT][RKT];
#pragma unroll
            for (int n = 0; n < NRT; ++n)
#pragma unroll
                for (int c = 0; c < RKT; ++c) acc[n][c] = float4_t{0.f, 0.f, 0.f, 0.f};
            for (int k = k0 + 32 * wave; k < k1; k += 32 * kWaves) {
                u32x4 av[RKT], xv[NRT];
                const bool in = k + 8 * g < k1;      // K is a multiple of 8
                const u32x4 zero = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < RKT; ++c) av[c] = in ? *reinterpret_cast<const u32x4*>(ar[c] + k) : zero;
#pragma unroll
                for (int n = 0; n < NRT; ++n) xv[n] = in ? *reinterpret_cast<const u32x4*>(xr[n] + k) : zero;
#pragma unroll
                for (int n = 0; n < NRT; ++n)
#pragma unroll
                    for (int c = 0; c < RKT; ++c) acc[n][c] = mfma<BF16>(av[c], xv[n], acc[n][c]);
            }
            if (wave) {
#pragma unroll
                for (int n = 0; n < NRT; ++n)
#pragma unroll
                    for (int c = 0; c < RKT; ++c) part[wave - 1][n * RKT + c][lane] = acc[n][c];
            }
            __syncthreads();
            if (!wave) {
#pragma unroll
                for (int n = 0; n < NRT; ++n) {
                    if (!((mine >> (16 * n + r)) & 1)) continue;
                    float* dst = p.t + ((int64_t)blockIdx.y * p.m + row0 + 16 * n + r) * p.R;
#pragma unroll
                    for (int c = 0; c < RKT; ++c) {
                        float4_t sum = acc[n][c];
#pragma unroll
                        for (int w = 0; w < kWaves - 1; ++w) sum += part[w][n * RKT + c][lane];
                        const int rank = c0 + 16 * c + 4 * g;
                        if (rank < p.R) *reinterpret_cast<float4_t*>(dst + rank) = sum;   // R is a multiple of 8
                    }
                }
            }
            __syncthreads();
        }
    }
}

// Rank to columns: a workgroup takes RT rows and 256 columns, 64 a wave.  The
// rows' sums are scaled, split and kept in LDS.  fp16: under a power of two of
// the row's own, so that they neither overflow nor fall below fp16's range.
template <bool BF16, int NRT>
__global__ __launch_bounds__(64 * kWaves) void mnb_lora_up_kernel(LoraParams p)
{
    constexpr int RT = 16 * NRT;
    extern __shared__ uint16_t t_lds[];          // [2][RT][R32 + 8]
    __shared__ float t_unit[RT];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row0 = (int64_t)blockIdx.y * RT;
    const int R32 = (p.R + 31) / 32 * 32, stride = R32 + 8;
    const int32_t id = tile_id<RT>(p, row0);
    // Each row by 16 neighbouring threads.
    for (int i = threadIdx.x >> 4; i < RT; i += 64 * kWaves / 16) {
        const int32_t a = __shfl(id, i);         // RT <= 64: the lane that holds row i
        const int64_t row = row0 + i;
        const float s = a >= 0 ? (p.scaling ? p.scaling[a] : 1.f) : 0.f;
        float top = 0.f;
        auto value = [&](int c) {
            if (a < 0 || c >= p.R) return 0.f;
            float sum = 0.f;
            for (int n = 0; n < p.splits; ++n) sum += p.t[((int64_t)n * p.m + row) * p.R + c];
            return sum * s;
        };
        float unit = 1.f, down = 1.f;
        if constexpr (!BF16) {
            for (int c = threadIdx.x & 15; c < R32; c += 16) top = fmaxf(top, fabsf(value(c)));
#pragma unroll
            for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
            // A sum that is not finite spoils its row through fp16 as it is.
            const int e = top > 0.f && top < __builtin_inff() ? ilogbf(top) : 0;
            const int e2 = e < -126 ? -126 : e > 126 ? 126 : e;
            unit = ldexpf(1.f, e2);
            down = ldexpf(1.f, -e2);
        }
        for (int c = threadIdx.x & 15; c < R32; c += 16) {
            const float v = value(c) * down;
            const uint16_t hi = narrow16(v, BF16);
            t_lds[i * stride + c] = hi;
            const float rest = v - widen16(hi, BF16);
            t_lds[(RT + i) * stride + c] = narrow16(rest, BF16);
        }
        if ((threadIdx.x & 15) == 0) t_unit[i] = unit;
    }
    __syncthreads();
    // Row j of tile t of A carries column 16 (j / 4) + 4 t + j % 4, so that lane
    // (r, g) ends with columns 16 g .. 16 g + 15 of row r.
    const int32_t n0 = (int32_t)blockIdx.x * 256 + 64 * wave;
    if (n0 >= p.N) return;
    float4_t acc[NRT][4];
#pragma unroll
    for (int n = 0; n < NRT; ++n)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[n][t] = float4_t{0.f, 0.f, 0.f, 0.f};
    uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0);
    const u32x4 zero = u32x4{0, 0, 0, 0};
    while (left) {
        const int32_t a = __shfl(id, __builtin_ctzll(left));
        const uint64_t mine = __builtin_amdgcn_ballot_w64(id == a);
        left &= ~mine;
        const uint16_t* br[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            int32_t col = n0 + 16 * (r >> 2) + 4 * t + (r & 3);
            if (col >= p.N) col = p.N - 1;
            br[t] = p.B + ((int64_t)a * p.N + col) * p.R + 8 * g;
        }
        for (int k = 0; k < p.R; k += 32) {
            u32x4 bv[4];
            const bool in = k + 8 * g < p.R;
#pragma unroll
            for (int t = 0; t < 4; ++t) bv[t] = in ? *reinterpret_cast<const u32x4*>(br[t] + k) : zero;
#pragma unroll
            for (int n = 0; n < NRT; ++n) {
                if (!((mine >> (16 * n)) & 0xFFFF)) continue;
                const bool own = (mine >> (16 * n + r)) & 1;
                const u32x4 hi = own ? *reinterpret_cast<const u32x4*>(t_lds + (16 * n + r) * stride + k + 8 * g) : zero;
                const u32x4 lo = own ? *reinterpret_cast<const u32x4*>(t_lds + (RT + 16 * n + r) * stride + k + 8 * g) : zero;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    acc[n][t] = mfma<BF16>(bv[t], hi, acc[n][t]);
                    acc[n][t] = mfma<BF16>(bv[t], lo, acc[n][t]);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NRT; ++n) {
        const int64_t row = row0 + 16 * n + r;
        if (row >= p.m) continue;
        const float unit = t_unit[16 * n + r];
        const int32_t col = n0 + 16 * g;
        const uint16_t* src = p.base ? p.base + row * p.base_stride + col : nullptr;
        uint16_t* dst = p.out + row * p.out_stride + col;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (col + i >= p.N) break;
            const float b = src ? widen16(src[i], p.out_bf16) : 0.f;
            dst[i] = narrow16(fmaf(acc[n][i >> 2][i & 3], unit, b), p.out_bf16);
        }
    }
}

template <bool BF16, int NRT, int RKT>
int queue_down(const LoraParams& p, unsigned ways, hipStream_t s)
{
    hipLaunchKernelGGL((mnb_lora_down_kernel<BF16, NRT, RKT>),
                       dim3((unsigned)((p.m + 16 * NRT - 1) / (16 * NRT)), (unsigned)p.splits, ways), dim3(64 * kWaves), 0, s, p);
    return (int)hipGetLastError();
}

template <bool BF16, int NRT>
int queue(const LoraParams& p, unsigned ways, hipStream_t s)
{
    const int e = p.R <= 16 ? queue_down<BF16, NRT, 1>(p, ways, s)
                : p.R <= 32 ? queue_down<BF16, NRT, 2>(p, ways, s) : queue_down<BF16, NRT, 4>(p, ways, s);
    if (e != 0) return e;
    const size_t lds = (size_t)2 * 16 * NRT * ((p.R + 31) / 32 * 32 + 8) * 2;
    hipLaunchKernelGGL((mnb_lora_up_kernel<BF16, NRT>),
                       dim3((unsigned)((p.N + 255) / 256), (unsigned)((p.m + 16 * NRT - 1) / (16 * NRT))),
                       dim3(64 * kWaves), lds, s, p);
    return (int)hipGetLastError();
}

}  // namespace

int launch_lora(const LoraArgs& a, void* stream, int* launches)
{
    const LoraLayout lay = lora_layout(a.m, a.K, a.R);
    LoraParams p{};
    p.x = static_cast<const uint16_t*>(a.x);
    p.ids = a.ids;
    p.A = static_cast<const uint16_t*>(a.A);
    p.B = static_cast<const uint16_t*>(a.B);
    p.scaling = a.scaling;
    p.base = static_cast<const uint16_t*>(a.base);
    p.out = static_cast<uint16_t*>(a.out);
    p.t = static_cast<float*>(a.ws);
    p.m = a.m;
    p.x_stride = a.x_stride;
    p.base_stride = a.base_stride;
    p.out_stride = a.out_stride;
    p.K = (int32_t)a.K;
    p.N = (int32_t)a.N;
    p.R = (int32_t)a.R;
    p.adapters = (int32_t)a.adapters;
    p.splits = lay.splits;
    p.k_slice = lay.k_slice;
    p.out_bf16 = a.out_bf16;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    *launches = 2;
    if (lay.row_tiles == 1) {
        const unsigned ways = (unsigned)(a.adapters < 1 ? 1 : a.adapters < 16 ? a.adapters : 16);
        return a.bf16 ? queue<true, 1>(p, ways, s) : queue<false, 1>(p, ways, s);
    }
    if (lay.row_tiles == 2) return a.bf16 ? queue<true, 2>(p, 1, s) : queue<false, 2>(p, 1, s);
    return a.bf16 ? queue<true, 4>(p, 1, s) : queue<false, 4>(p, 1, s);
}

}  // namespace mnb
