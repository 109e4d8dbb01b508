// A mixture-of-experts layer of 4-bit weights for a few tokens (gfx950).
//
//   out[t] = sum_j p[t][j] * Down_e( silu(Gate_e x[t]) * (Up_e x[t]) ),  e = ids[t][j]
//
// with W[n][k] = (q[n][k] - z[n][k/32]) * s[n][k/32] in every matrix.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb.h"
#include "mnb_device.h"
#include "mnb_internal.h"

namespace mnb {
namespace {

__device__ __forceinline__ float widen16(uint32_t bits, int bf16)
{
    return bf16 ? __uint_as_float(bits << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

__device__ __forceinline__ uint16_t narrow16(float v, int bf16)
{
    if (!bf16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

struct MoeParams {
    const uint16_t* x;
    const void* logits;
    const uint8_t *w1, *z1, *w2, *z2;
    const uint16_t *s1, *s2;
    uint16_t* out;
    int32_t* ids_out;
    float* probs_out;
    int32_t* ids;      // workspace: [T][top_k]
    float* probs;      // [T][top_k]
    float* h;          // [T][top_k][I]
    int32_t T, H, I, E, top_k;
    int32_t x_bf16, logits_dtype, renormalize, out_bf16;
};

__device__ __forceinline__ float logit_at(const MoeParams& p, int64_t i)
{
    if (p.logits_dtype == MNB_F32) return static_cast<const float*>(p.logits)[i];
    return widen16(static_cast<const uint16_t*>(p.logits)[i], p.logits_dtype == MNB_BF16);
}

// One thread per token.
__global__ void mnb_moe_route_kernel(MoeParams p)
{
    const int t = threadIdx.x;
    if (t >= p.T) return;
    const int64_t base = (int64_t)t * p.E;
    const float ninf = -__builtin_inff();
    float peak = ninf;
    bool bad = false;
    for (int e = 0; e < p.E; ++e) {
        const float l = logit_at(p, base + e);
        if (!(l < __builtin_inff())) bad = true;   // NaN or +infinity
        peak = fmaxf(peak, l);
    }
    float mass = 0.f;
    float last = __builtin_inff();
    int last_e = -1;
    for (int j = 0; j < p.top_k; ++j) {
        // The largest (logit, -number) below the last one.
        float best = ninf;
        int be = -1;
        if (!bad)
            for (int e = 0; e < p.E; ++e) {
                const float l = logit_at(p, base + e);
                const bool after = l < last || (l == last && e > last_e);
                if (after && l > best) {
                    best = l;
                    be = e;
                }
            }
        const float w = be < 0 ? 0.f : __expf(best - peak);
        p.ids[t * p.top_k + j] = be;
        p.probs[t * p.top_k + j] = w;
        mass += w;
        last = best;
        last_e = be;
    }
    if (!p.renormalize) {
        mass = 0.f;
        for (int e = 0; e < p.E; ++e) mass += __expf(logit_at(p, base + e) - peak);
    }
    for (int j = 0; j < p.top_k; ++j) {
        const int i = t * p.top_k + j;
        const float w = bad ? __builtin_nanf("") : p.ids[i] < 0 ? 0.f : p.probs[i] / mass;
        p.probs[i] = w;
        if (p.ids_out) p.ids_out[i] = p.ids[i];
        if (p.probs_out) p.probs_out[i] = w;
    }
}

// Dot product of row n of a packed matrix with a vector of fp16-rounded
// activations, over the wave's lanes (block by block).
template <typename F>
__device__ __forceinline__ float row_dot(const uint8_t* w, const uint16_t* s, const uint8_t* z, int64_t n, int K, F act)
{
    const int nb = K / 32, zb = (nb + 1) / 2;
    float acc = 0.f;
    for (int b = threadIdx.x & 63; b < nb; b += 64) {
        const float scale = (float)__builtin_bit_cast(_Float16, s[n * nb + b]);
        const int zero = z ? (z[n * zb + b / 2] >> (4 * (b & 1))) & 15 : 8;
        float part = 0.f;
        for (int i = 0; i < 32; ++i) {
            const int q = (w[n * (K / 2) + 16 * b + i / 2] >> (4 * (i & 1))) & 15;
            part += (float)(q - zero) * act(32 * b + i);
        }
        acc += part * scale;
    }
    for (int d = 32; d; d >>= 1) acc += __shfl_xor(acc, d);
    return acc;
}

// One wave per (token, slot, column of the intermediate activations).
__global__ __launch_bounds__(64) void mnb_moe_up_kernel(MoeParams p)
{
    const int64_t n = (int64_t)p.T * p.top_k * p.I;
    for (int64_t u = blockIdx.x; u < n; u += gridDim.x) {
        const int64_t pair = u / p.I, i = u - pair * p.I, t = pair / p.top_k;
        const int e = p.ids[pair];
        if (e < 0) continue;
        auto act = [&](int k) { return (float)(_Float16)widen16(p.x[t * p.H + k], p.x_bf16); };
        const int64_t row = (int64_t)e * 2 * p.I + i;
        const float gate = row_dot(p.w1, p.s1, p.z1, row, p.H, act);
        const float up = row_dot(p.w1, p.s1, p.z1, row + p.I, p.H, act);
        if (threadIdx.x == 0) p.h[pair * p.I + i] = gate / (1.f + __expf(-gate)) * up;
    }
}

// One wave per (token, output column).
__global__ __launch_bounds__(64) void mnb_moe_down_kernel(MoeParams p)
{
    const int64_t n = (int64_t)p.T * p.H;
    for (int64_t u = blockIdx.x; u < n; u += gridDim.x) {
        const int64_t t = u / p.H, c = u - t * p.H;
        float y = 0.f;
        for (int j = 0; j < p.top_k; ++j) {
            const int64_t pair = t * p.top_k + j;
            const int e = p.ids[pair];
            if (e < 0) {
                y += p.probs[pair];   // 0, or NaN where the logits were not finite
                continue;
            }
            auto act = [&](int k) { return p.h[pair * p.I + k]; };
            y += p.probs[pair] * row_dot(p.w2, p.s2, p.z2, (int64_t)e * p.H + c, p.I, act);
        }
        if (threadIdx.x == 0) p.out[u] = narrow16(y, p.out_bf16);
    }
}

}  // namespace

int launch_moe(const MoeArgs& a, void* stream, int* launches)
{
    const int64_t pairs = (int64_t)a.T * a.top_k;
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
    p.ids = static_cast<int32_t*>(a.ws);
    p.probs = reinterpret_cast<float*>(p.ids + pairs);
    p.h = p.probs + pairs;
    p.T = a.T;
    p.H = (int32_t)a.w.hidden;
    p.I = (int32_t)a.w.inter;
    p.E = (int32_t)a.w.experts;
    p.top_k = a.top_k;
    p.x_bf16 = a.x_bf16;
    p.logits_dtype = a.logits_dtype;
    p.renormalize = a.renormalize;
    p.out_bf16 = a.out_bf16;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    auto grid = [](int64_t n) { return dim3((unsigned)(n < (1 << 20) ? n : (1 << 20))); };
    hipLaunchKernelGGL(mnb_moe_route_kernel, dim3(1), dim3(64), 0, s, p);
    hipLaunchKernelGGL(mnb_moe_up_kernel, grid(pairs * p.I), dim3(64), 0, s, p);
    hipLaunchKernelGGL(mnb_moe_down_kernel, grid((int64_t)p.T * p.H), dim3(64), 0, s, p);
    const int e = (int)hipGetLastError();
    if (e == 0) *launches += 3;
    return e;
}

}  // namespace mnb
