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

#include "mnb.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// fp16 or bf16 bits as fp32 (exact).
__device__ __forceinline__ float widen16(uint32_t bits, int bf16)
{
    return bf16 ? __uint_as_float(bits << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

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

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

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

// fp32 -> fp16 or bf16 bits (RNE).
__device__ __forceinline__ uint16_t narrow16(float v, int bf16)
{
    if (!bf16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

struct Int8Params {
    const int8_t* A;        // [M][K]
    const float* a_scales;  // [M]
    const int8_t* B;        // [N][K]
    const float* b_scales;  // [N]
    const float* bias;      // [N] or null
    uint16_t* out;          // [M][N]
    int64_t M, N;
    int32_t K;
    int32_t out_bf16;
};

// A wave owns 16 rows by 16 columns.  v_mfma_i32_16x16x64_i8: lane (j, g)
// supplies 16 k of row j and of column j and receives column j, rows 4 g ..
// 4 g + 3.
__global__ __launch_bounds__(256) void mnb_int8_kernel(Int8Params p)
{
    const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
    const int64_t tiles_n = (p.N + 15) / 16, tiles = tiles_n * ((p.M + 15) / 16);
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tiles; t += (int64_t)gridDim.x * 4) {
        const int64_t r0 = t / tiles_n * 16, c0 = t % tiles_n * 16;
        const int64_t rows = p.M - r0 < 16 ? p.M - r0 : 16, cols = p.N - c0 < 16 ? p.N - c0 : 16;
        const __amdgpu_buffer_rsrc_t rA = make_rsrc(p.A + r0 * p.K, (uint64_t)rows * p.K);
        const __amdgpu_buffer_rsrc_t rB = make_rsrc(p.B + c0 * p.K, (uint64_t)cols * p.K);
        i32x4 acc = {0, 0, 0, 0};
        for (int k = 16 * g; k - 16 * g < p.K; k += 64) {
            const uint32_t off = k < p.K ? (uint32_t)j * p.K + k : kOutOfRange;
            const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(rA, off, 0, 0);
            const u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(rB, off, 0, 0);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b),
                                                        acc, 0, 0, 0);
        }
        if (j < cols)
            for (int i = 0; i < 4; ++i) {
                const int64_t r = r0 + 4 * g + i;
                if (r >= p.M) continue;
                float v = (float)acc[i] * p.b_scales[c0 + j] * p.a_scales[r];
                if (p.bias) v += p.bias[c0 + j];
                p.out[r * p.N + c0 + j] = narrow16(v, p.out_bf16);
            }
    }
}

}  // namespace

int launch_quantize_rows(const void* A, int a_bf16, int64_t m, int64_t K, int8_t* q, float* scales, void* stream)
{
    const QuantizeParams p{static_cast<const uint16_t*>(A), q, scales, m, K, a_bf16};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    // Threads per row: where the rows fill the device, as few as hold the row
    // in eight pieces each; few rows are spread over one workgroup each.
    const bool many = m >= 1024;
    if (K <= (many ? 4096 : 512)) {
        if (K <= 512) queue_quantize<64, 1>(p, s);
        else queue_quantize<64, 8>(p, s);
    } else if (K <= (many ? 16384 : 2048)) {
        if (K <= 2048) queue_quantize<256, 1>(p, s);
        else queue_quantize<256, 8>(p, s);
    } else if (K <= 8192) {
        queue_quantize<1024, 1>(p, s);
    } else {
        queue_quantize<1024, 4>(p, s);
    }
    return (int)hipGetLastError();
}

int launch_int8(const Int8Args& a, void* stream, int* launches)
{
    Int8Params p;
    p.A = static_cast<const int8_t*>(a.A);
    p.a_scales = a.a_scales;
    if (a.a_dtype != MNB_I8) {
        int8_t* q = static_cast<int8_t*>(a.ws);
        float* scales = reinterpret_cast<float*>(q + a.m * a.K);
        const int e = launch_quantize_rows(a.A, a.a_dtype == MNB_BF16, a.m, a.K, q, scales, stream);
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
    const int64_t tiles = ((a.m + 15) / 16) * ((a.N + 15) / 16), wgs = (tiles + 3) / 4;
    hipLaunchKernelGGL(mnb_int8_kernel, dim3((unsigned)(wgs < 65536 ? wgs : 65536)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), p);
    const int e = (int)hipGetLastError();
    if (e == 0) ++*launches;
    return e;
}

}  // namespace mnb
