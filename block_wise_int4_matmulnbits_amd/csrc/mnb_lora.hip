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
// HBM bounds both where there are many rows: x, base and out are read or written once
// (4091 rows, 14336 -> 40 -> 4097: 179 MB in 87 us), and the used adapters once for each
// tile of rows (64 rows of 32 adapters, 4096 -> 64 -> 28672: 125 MB in 38 to 45 us).  One
// row is bound by the two launches (9 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8_t __attribute__((ext_vector_type(8)));

constexpr int kDownWaves = 4;

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
    int32_t k_slice;          // K of a slice: a multiple of 32 * kDownWaves
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

// The adapters of a tile one after another, by their first row; rows: a bit each.
struct Adapters {
    uint64_t left;
    int32_t id;               // of this lane's row
    __device__ __forceinline__ int32_t next(uint64_t* rows)
    {
        const int32_t a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        *rows = __builtin_amdgcn_ballot_w64(id == a);
        left &= ~*rows;
        return a;
    }
};

// Rows to rank: a workgroup takes RT = 16 NRT rows, one slice of K and, of the
// adapters that its rows use, every gridDim.z-th; its waves split the slice, two
// steps of 32 in flight.  RKT tiles of 16 ranks at a time.
template <bool BF16, int NRT, int RKT>
__global__ __launch_bounds__(64 * kDownWaves) void mnb_lora_down_kernel(LoraParams p)
{
    constexpr int RT = 16 * NRT, STEP = 32 * kDownWaves;
    __shared__ float4_t part[kDownWaves - 1][NRT * RKT][64];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row0 = (int64_t)blockIdx.x * RT;
    Adapters list;
    list.id = tile_id<RT>(p, row0);
    list.left = __builtin_amdgcn_ballot_w64(list.id >= 0);
    const int32_t k0 = (int32_t)blockIdx.y * p.k_slice, k1 = k0 + p.k_slice < p.K ? k0 + p.k_slice : p.K;
    const uint16_t* xr[NRT];
#pragma unroll
    for (int n = 0; n < NRT; ++n) {
        const int64_t row = row0 + 16 * n + r < p.m ? row0 + 16 * n + r : p.m - 1;
        xr[n] = p.x + row * p.x_stride + 8 * g;
    }
    for (uint32_t j = 0; list.left; ++j) {
        uint64_t mine;
        const int32_t a = list.next(&mine);
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
            const u32x4 zero = u32x4{0, 0, 0, 0};
            u32x4 av[2][RKT], xv[2][NRT];
            auto load = [&](int k, u32x4 (&a2)[RKT], u32x4 (&x2)[NRT]) {
                const bool in = k + 8 * g < k1;              // K is a multiple of 8
#pragma unroll
                for (int n = 0; n < NRT; ++n)
                    x2[n] = in && ((mine >> (16 * n)) & 0xFFFF) ? *reinterpret_cast<const u32x4*>(xr[n] + k) : zero;
#pragma unroll
                for (int c = 0; c < RKT; ++c) a2[c] = in ? *reinterpret_cast<const u32x4*>(ar[c] + k) : zero;
            };
            auto multiply = [&](const u32x4 (&a2)[RKT], const u32x4 (&x2)[NRT]) {
#pragma unroll
                for (int n = 0; n < NRT; ++n)
                    if ((mine >> (16 * n)) & 0xFFFF)
#pragma unroll
                        for (int c = 0; c < RKT; ++c) acc[n][c] = mfma<BF16>(a2[c], x2[n], acc[n][c]);
            };
            int k = k0 + 32 * wave;
            load(k, av[0], xv[0]);
            load(k + STEP, av[1], xv[1]);
            for (; k < k1; k += 2 * STEP) {
                multiply(av[0], xv[0]);
                load(k + 2 * STEP, av[0], xv[0]);
                __builtin_amdgcn_sched_barrier(0);
                multiply(av[1], xv[1]);
                load(k + 3 * STEP, av[1], xv[1]);
                __builtin_amdgcn_sched_barrier(0);
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
                        for (int w = 0; w < kDownWaves - 1; ++w) sum += part[w][n * RKT + c][lane];
                        const int rank = c0 + 16 * c + 4 * g;
                        if (rank < p.R) *reinterpret_cast<float4_t*>(dst + rank) = sum;   // R is a multiple of 8
                    }
                }
            }
            __syncthreads();
        }
    }
}

// Eight bytes at any even address, and whole words.  Sixteen bytes that begin within a
// word take far longer, so a lane of sixteen columns moves whole words and shifts them
// (4091 rows, 512 -> 40 -> 4097 columns: 57 -> 43 us; 4098 columns, which need no
// shift, 39 both ways).
struct __attribute__((packed, aligned(2))) Loose8 {
    uint32_t v[2];
};
struct __attribute__((packed, aligned(4))) Words4 {
    uint32_t v[4];
};
struct __attribute__((packed, aligned(4))) Words3 {
    uint32_t v[3];
};

// The pairs of two words' four elements that begin at the first (shift 0) or second (16).
__device__ __forceinline__ uint32_t shifted(uint32_t hi, uint32_t lo, uint32_t shift) { return __builtin_amdgcn_alignbit(hi, lo, shift); }

// C = 4 CT columns of a row's base, none of them behind the last one; the buffer is
// what lies from first to last.
template <int CT>
__device__ __forceinline__ void load_base(const uint16_t* src, const uint16_t* first, const uint16_t* last,
                                          uint32_t (&b)[2 * CT])
{
    constexpr int C = 4 * CT;
    if constexpr (CT == 1) {
        const Loose8 t = *reinterpret_cast<const Loose8*>(src);
        b[0] = t.v[0];
        b[1] = t.v[1];
    } else {
        // The words that hold these columns: one more where the first begins within one.
        const bool odd = (uintptr_t)src & 2;
        if (odd && (src == first || src + C == last)) {      // a word that is in the buffer in half
#pragma unroll
            for (int i = 0; i < 2 * CT; ++i) b[i] = (uint32_t)src[2 * i] | (uint32_t)src[2 * i + 1] << 16;
            return;
        }
        const Words4* from = reinterpret_cast<const Words4*>((uintptr_t)src & ~(uintptr_t)3);
        uint32_t w[2 * CT + 1];
#pragma unroll
        for (int i = 0; i < CT / 2; ++i) {
            const Words4 t = from[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[4 * i + e] = t.v[e];
        }
        if (!__builtin_amdgcn_ballot_w64(odd)) {
#pragma unroll
            for (int i = 0; i < 2 * CT; ++i) b[i] = w[i];
            return;
        }
        w[2 * CT] = reinterpret_cast<const uint32_t*>(from)[odd ? 2 * CT : 2 * CT - 1];
#pragma unroll
        for (int i = 0; i < 2 * CT; ++i) b[i] = shifted(w[i + 1], w[i], odd ? 16 : 0);
    }
}

// base + acc * unit, of a row's 4 CT columns from col (the wave's lanes 16 apart hold
// neighbours of one row; every lane comes here).
template <int CT>
__device__ __forceinline__ void finish(const LoraParams& p, int64_t row, int32_t col, const uint32_t (&b)[2 * CT],
                                       const float4_t (&acc)[CT], float unit)
{
    constexpr int C = 4 * CT;
    const int g = (threadIdx.x & 63) >> 4;
    uint32_t w[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
        const float lo = fmaf(acc[i >> 1][2 * (i & 1)], unit, widen16(b[i] & 0xFFFFu, p.out_bf16));
        const float hi = fmaf(acc[i >> 1][2 * (i & 1) + 1], unit, widen16(b[i] >> 16, p.out_bf16));
        w[i] = (uint32_t)narrow16(lo, p.out_bf16) | (uint32_t)narrow16(hi, p.out_bf16) << 16;
    }
    uint16_t* dst = p.out + row * p.out_stride + col;
    const bool odd = (uintptr_t)dst & 2;
    uint32_t before = 0;
    if (CT > 1 && __builtin_amdgcn_ballot_w64(odd)) before = __shfl_up(w[C / 2 - 1], 16);
    if (row >= p.m || col >= p.N) return;
    if (col + C <= p.N) {
        if constexpr (CT == 1) {
            *reinterpret_cast<Loose8*>(dst) = Loose8{{w[0], w[1]}};
        } else if (!odd) {
#pragma unroll
            for (int i = 0; i < CT / 2; ++i)
                reinterpret_cast<Words4*>(dst)[i] = Words4{{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]}};
        } else {
            // Whole words: the first begins with the left neighbour's last column, and this
            // one's last column goes to the right neighbour, where there is one.
            uint32_t v[C / 2];
#pragma unroll
            for (int i = 0; i < C / 2; ++i) v[i] = shifted(w[i], i ? w[i - 1] : before, 16);
            if (g == 0) {
                dst[0] = (uint16_t)w[0];
                *reinterpret_cast<Words3*>(dst + 1) = Words3{{v[1], v[2], v[3]}};
            } else {
                *reinterpret_cast<Words4*>(dst - 1) = Words4{{v[0], v[1], v[2], v[3]}};
            }
#pragma unroll
            for (int i = 1; i < CT / 2; ++i)
                *reinterpret_cast<Words4*>(dst - 1 + 8 * i) = Words4{{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}};
            if (g == 3 || col + 2 * C > p.N) dst[C - 1] = (uint16_t)(w[C / 2 - 1] >> 16);
        }
        return;
    }
    const uint16_t* src = p.base ? p.base + row * p.base_stride + col : nullptr;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (col + i < p.N)
            dst[i] = narrow16(fmaf(acc[i >> 2][i & 3], unit, src ? widen16(src[i], p.out_bf16) : 0.f), p.out_bf16);
    }
}

// Rank to columns: a workgroup of W waves takes RT rows and 16 CT columns a wave.
// The rows' sums are added over the slices, scaled, split and kept in LDS.  fp16:
// under a power of two of the row's own, so that they neither overflow nor fall
// below fp16's range.  The pieces of B, an adapter's 64 ranks at a time, come
// up to three ahead of their products.
template <bool BF16, int NRT, int CT, int W>
__global__ __launch_bounds__(64 * W) void mnb_lora_up_kernel(LoraParams p)
{
    constexpr int RT = 16 * NRT, AHEAD = CT == 1 ? 3 : 1;
    extern __shared__ uint16_t t_lds[];          // [2][RT][R64 + 8]
    __shared__ float t_unit[RT];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row0 = (int64_t)blockIdx.y * RT;
    const int R64 = (p.R + 63) / 64 * 64, stride = R64 + 8;
    Adapters list;
    list.id = tile_id<RT>(p, row0);
    list.left = __builtin_amdgcn_ballot_w64(list.id >= 0);
    // Row j of tile t of A carries column CT * 4 * (j / 4) + 4 t + j % 4, so that lane
    // (r, g) ends with 4 CT neighbouring columns of row r.
    const int32_t n0 = ((int32_t)blockIdx.x * W + wave) * 16 * CT;
    const int32_t chunks = R64 / 64;
    struct Item {
        u32x4 b[2][CT];
        uint64_t rows;
    };
    int32_t a = 0, chunk = chunks;               // of the last item fetched
    uint64_t rows = 0;
    const u32x4 zero = u32x4{0, 0, 0, 0};
    auto fetch = [&](Item& it) {                 // the next item; rows 0: no more
        if (++chunk >= chunks) {
            chunk = 0;
            rows = 0;
            if (list.left) a = list.next(&rows);
        }
        it.rows = rows;
        if (!rows || n0 >= p.N) {
            it.rows = 0;
            return;
        }
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            int32_t col = n0 + 4 * CT * (r >> 2) + 4 * t + (r & 3);
            if (col >= p.N) col = p.N - 1;
            const uint16_t* src = p.B + ((int64_t)a * p.N + col) * p.R + 64 * chunk + 8 * g;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                it.b[k][t] = 64 * chunk + 32 * k + 8 * g < p.R ? *reinterpret_cast<const u32x4*>(src + 32 * k) : zero;
        }
    };
    Item items[AHEAD + 1];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(items[i]);

    // The base of this lane's columns; with few rows and many adapters, behind their
    // weights.
    const int32_t mine0 = n0 + 4 * CT * g;
    const bool whole = mine0 + 4 * CT <= p.N;
    uint32_t base[NRT][2 * CT];
    auto read_base = [&] {
#pragma unroll
        for (int n = 0; n < NRT; ++n) {
#pragma unroll
            for (int i = 0; i < 2 * CT; ++i) base[n][i] = 0;
            if (p.base && whole && row0 + 16 * n + r < p.m)
                load_base<CT>(p.base + (row0 + 16 * n + r) * p.base_stride + mine0, p.base,
                              p.base + (p.m - 1) * p.base_stride + p.N, base[n]);
        }
    };
    if (CT > 1) read_base();

    // Each row by 16 neighbouring threads, four ranks a time: at most 256 ranks.
    for (int i = threadIdx.x >> 4; i < RT; i += 4 * W) {
        const int32_t own = __shfl(list.id, i);  // the lane that holds row i
        const float s = own >= 0 ? (p.scaling ? p.scaling[own] : 1.f) : 0.f;
        const float* src = p.t + (row0 + i) * p.R;
        float4_t v[4];
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int rank = 64 * c + 4 * (threadIdx.x & 15);
            v[c] = float4_t{0.f, 0.f, 0.f, 0.f};
            if (own >= 0 && rank < p.R) {
#pragma unroll 8
                for (int n = 0; n < p.splits; ++n) v[c] += *reinterpret_cast<const float4_t*>(src + (int64_t)n * p.m * p.R + rank);
                v[c] *= s;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(v[c][e]));
        }
        float unit = 1.f, down = 1.f;
        if constexpr (!BF16) {
#pragma unroll
            for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
            // A sum that is not finite spoils its row through fp16 as it is.
            const int e = top > 0.f && top < __builtin_inff() ? ilogbf(top) : 0;
            const int e2 = e < -126 ? -126 : e > 126 ? 126 : e;
            unit = ldexpf(1.f, e2);
            down = ldexpf(1.f, -e2);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int rank = 64 * c + 4 * (threadIdx.x & 15);
            if (rank >= R64) continue;
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = v[c][2 * e] * down, y = v[c][2 * e + 1] * down;
                const uint16_t xh = narrow16(x, BF16), yh = narrow16(y, BF16);
                hi[e] = (uint32_t)xh | (uint32_t)yh << 16;
                lo[e] = (uint32_t)narrow16(x - widen16(xh, BF16), BF16) |
                        (uint32_t)narrow16(y - widen16(yh, BF16), BF16) << 16;
            }
            uint32_t* to = reinterpret_cast<uint32_t*>(t_lds + i * stride + rank);
            to[0] = hi[0];
            to[1] = hi[1];
            to = reinterpret_cast<uint32_t*>(t_lds + (RT + i) * stride + rank);
            to[0] = lo[0];
            to[1] = lo[1];
        }
        if ((threadIdx.x & 15) == 0) t_unit[i] = unit;
    }
    __syncthreads();
    if (n0 >= p.N) return;
    float4_t acc[NRT][CT];
#pragma unroll
    for (int n = 0; n < NRT; ++n)
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[n][t] = float4_t{0.f, 0.f, 0.f, 0.f};
    int at = 0;                                  // chunk of the item in hand
    auto multiply = [&](const Item& it) {
#pragma unroll
        for (int n = 0; n < NRT; ++n) {
            if (!((it.rows >> (16 * n)) & 0xFFFF)) continue;
            // Rows of other adapters keep their sums (0 times a weight that is not finite
            // would not).
            const bool own = (it.rows >> (16 * n + r)) & 1;
            float4_t sum[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) sum[t] = acc[n][t];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (64 * at + 32 * k >= p.R) continue;
                const int from = (16 * n + r) * stride + 64 * at + 32 * k + 8 * g;
                const u32x4 hi = *reinterpret_cast<const u32x4*>(t_lds + from);
                const u32x4 lo = *reinterpret_cast<const u32x4*>(t_lds + RT * stride + from);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    sum[t] = mfma<BF16>(it.b[k][t], hi, sum[t]);
                    sum[t] = mfma<BF16>(it.b[k][t], lo, sum[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][t][i] = own ? sum[t][i] : acc[n][t][i];
        }
        at = at + 1 < chunks ? at + 1 : 0;
    };
    bool more = true;
    while (more) {
#pragma unroll
        for (int i = 0; i <= AHEAD; ++i) {
            if (!more) continue;
            more = items[i].rows != 0;
            if (!more) continue;
            fetch(items[(i + AHEAD) % (AHEAD + 1)]);
            multiply(items[i]);
        }
    }
    if (CT == 1) read_base();
#pragma unroll
    for (int n = 0; n < NRT; ++n) {
        finish<CT>(p, row0 + 16 * n + r, mine0, base[n], acc[n], t_unit[16 * n + r]);
    }
}

template <bool BF16, int NRT, int RKT>
int queue_down(const LoraParams& p, unsigned ways, hipStream_t s)
{
    hipLaunchKernelGGL((mnb_lora_down_kernel<BF16, NRT, RKT>),
                       dim3((unsigned)((p.m + 16 * NRT - 1) / (16 * NRT)), (unsigned)p.splits, ways), dim3(64 * kDownWaves), 0, s, p);
    return (int)hipGetLastError();
}

template <bool BF16, int NRT, int CT, int W>
int queue_up(const LoraParams& p, hipStream_t s)
{
    constexpr int COLS = 16 * CT * W;
    const size_t lds = (size_t)2 * 16 * NRT * ((p.R + 63) / 64 * 64 + 8) * 2;
    hipLaunchKernelGGL((mnb_lora_up_kernel<BF16, NRT, CT, W>),
                       dim3((unsigned)((p.N + COLS - 1) / COLS), (unsigned)((p.m + 16 * NRT - 1) / (16 * NRT))),
                       dim3(64 * W), lds, s, p);
    return (int)hipGetLastError();
}

template <bool BF16, int NRT>
int queue_down(const LoraParams& p, unsigned ways, hipStream_t s)
{
    return p.R <= 16 ? queue_down<BF16, NRT, 1>(p, ways, s) : p.R <= 32 ? queue_down<BF16, NRT, 2>(p, ways, s)
         : p.R <= 48 ? queue_down<BF16, NRT, 3>(p, ways, s) : queue_down<BF16, NRT, 4>(p, ways, s);
}

template <bool BF16>
int queue(const LoraParams& p, const LoraLayout& lay, hipStream_t s)
{
    const unsigned ways = (unsigned)lay.ways;
    const int e = lay.down_tiles == 1 ? queue_down<BF16, 1>(p, ways, s) : lay.down_tiles == 2 ? queue_down<BF16, 2>(p, ways, s)
                                      : queue_down<BF16, 4>(p, ways, s);
    if (e != 0) return e;
    if (lay.up_tiles == 1) return lay.wide ? queue_up<BF16, 1, 4, 8>(p, s) : queue_up<BF16, 1, 1, 4>(p, s);
    if (lay.up_tiles == 4) return queue_up<BF16, 4, 1, 4>(p, s);
    return lay.wide ? queue_up<BF16, 2, 4, 8>(p, s) : queue_up<BF16, 2, 1, 4>(p, s);
}

}  // namespace

int launch_lora(const LoraArgs& a, void* stream, int* launches)
{
    const LoraLayout lay = lora_layout(a.m, a.K, a.N, a.R, a.adapters);
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
    return a.bf16 ? queue<true>(p, lay, s) : queue<false>(p, lay, s);
}

}  // namespace mnb
