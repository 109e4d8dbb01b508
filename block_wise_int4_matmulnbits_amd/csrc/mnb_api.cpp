// Host front end of libmnb: argument validation, launch planning, counters
// and status strings.  Plain C++ (no HIP headers): everything here runs, and
// is tested, without a GPU.  The kernels and their launch live in
// mnb_gemv.hip.
#include <algorithm>
#include <cmath>
#include <atomic>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "mnb.h"
#include "mnb_internal.h"

namespace {

std::atomic<uint64_t> g_calls{0}, g_launches{0}, g_f16{0}, g_bf16{0}, g_rows{0};
thread_local int t_last_hip_error = 0;

// Register budget: M rows x blocks_per_lane blocks of activations stay in
// VGPRs (16 per block and row), at most 8 such blocks per lane.
int max_blocks_per_lane(int64_t m) { return m == 1 ? 8 : m == 2 ? 4 : m <= 4 ? 2 : 1; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t pow2_ceil(int64_t x)
{
    int64_t p = 1;
    while (p < x) p <<= 1;
    return p;
}

bool is_pow2_in(int64_t x, int64_t lo, int64_t hi)
{
    return x >= lo && x <= hi && (x & (x - 1)) == 0;
}

bool overlaps(const void* a, int64_t an, const void* b, int64_t bn)
{
    if (!a || !b || an <= 0 || bn <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)bn && b0 < a0 + (uintptr_t)an;
}

// Nominal resident waves per CU, used to size the grid when the occupancy of
// the chosen kernel variant is not known (host-only planning).
constexpr int kTargetWavesPerCu = 16;
constexpr int kMaxKSplits = 64;   // K slices over workgroups (engine 2)
// Largest workspace a default plan uses (K split over workgroups).
constexpr size_t kMaxSplitWorkspaceBytes = MNB_MAX_SPLIT_WORKSPACE;

int validate(const void* A, int a_dtype, int64_t m, int64_t K, int64_t N,
             const uint8_t* Bpacked, const uint16_t* scales,
             const uint8_t* zero_points, int block, void* out, int out_dtype)
{
    if (m < 0 || m > MNB_MAX_ROWS) return MNB_ERR_M_RANGE;
    if (K < 0 || N < 0 || K > MNB_MAX_K || N > INT32_MAX) return MNB_ERR_SHAPE;
    if (block != 32) return MNB_ERR_BLOCK;
    if (K % 32 != 0) return MNB_ERR_SHAPE;
    if ((a_dtype != MNB_F16 && a_dtype != MNB_BF16) ||
        (out_dtype != MNB_F16 && out_dtype != MNB_BF16))
        return MNB_ERR_DTYPE;
    if (m == 0 || N == 0) return MNB_OK;
    if (!out) return MNB_ERR_NULL;
    if (K > 0 && (!A || !Bpacked || !scales)) return MNB_ERR_NULL;
    if (((uintptr_t)A & 15) || ((uintptr_t)Bpacked & 15) ||
        ((uintptr_t)scales & 1) || ((uintptr_t)out & 1))
        return MNB_ERR_ALIGN;
    const int64_t nb = K / 32;
    const int64_t out_bytes = m * N * 2;
    if (overlaps(out, out_bytes, A, m * K * 2) ||
        overlaps(out, out_bytes, Bpacked, N * (K / 2)) ||
        overlaps(out, out_bytes, scales, N * nb * 2) ||
        overlaps(out, out_bytes, zero_points, N * ((nb + 1) / 2)))
        return MNB_ERR_ALIAS;
    return MNB_OK;
}

// MNB_LOG set to anything but "0" in the environment (read once): each call
// that reaches its launches prints its shape and plan to stderr, one line.
bool log_enabled()
{
    static const bool on = [] {
        const char* v = getenv("MNB_LOG");
        return v && *v && !(v[0] == '0' && v[1] == 0);
    }();
    return on;
}

void log_plan(int64_t m, int64_t K, int64_t N, int a_dtype, int out_dtype, const mnb_plan& p, bool explicit_plan,
              bool fixed_scratch)
{
    const int64_t step = p.engine == 2 ? m : MNB_MAX_M;
    const int64_t launches = (m + step - 1) / step * (p.k_splits > 1 ? 2 : 1);
    fprintf(stderr,
            "mnb: m=%lld K=%lld N=%lld a=%s out=%s %s plan: engine=%d lanes_per_col=%d blocks_per_lane=%d "
            "cols_per_tile=%d waves_per_wg=%d row_tiles=%d k_splits=%d a_via_lds=%d b_layout=%d interleave=%d "
            "workgroups=%d threads_per_wg=%d k_chunks=%d launches=%lld%s\n",
            (long long)m, (long long)K, (long long)N, a_dtype == MNB_BF16 ? "bf16" : "f16",
            out_dtype == MNB_BF16 ? "bf16" : "f16", explicit_plan ? "explicit" : "default", p.engine,
            p.lanes_per_col, p.blocks_per_lane, p.cols_per_tile, p.waves_per_wg, p.row_tiles, p.k_splits,
            p.a_via_lds, p.b_layout, p.interleave, p.workgroups, p.threads_per_wg, p.k_chunks,
            (long long)launches, fixed_scratch ? " fixed-scratch" : "");
}

constexpr int kNoDevice = 100;   // hipErrorNoDevice: a build without the kernels

const char* dtype_name(int dtype)
{
    static const char* const names[] = {"f16", "bf16", "f32", "i8"};
    return names[dtype];
}

// A buffer of a call; null or empty ones overlap nothing.
struct Span {
    const void* p;
    int64_t bytes;
};

// Whether a written buffer overlaps an input or another written buffer.
bool aliased(const Span* in, int n_in, const Span* wr, int n_wr)
{
    for (int i = 0; i < n_wr; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlaps(wr[i].p, wr[i].bytes, in[j].p, in[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(wr[i].p, wr[i].bytes, wr[j].p, wr[j].bytes)) return true;
    }
    return false;
}

// The end of a call that queued `launches` kernels with status e (a hipError_t).
int finish_launches(int e, int launches)
{
    g_launches.fetch_add((uint64_t)launches, std::memory_order_relaxed);
    if (e != 0) {
        t_last_hip_error = e;
        return MNB_ERR_HIP;
    }
    g_calls.fetch_add(1, std::memory_order_relaxed);
    return MNB_OK;
}

// Rows of a buffer: `rows` of `width` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t rows, width, stride;
};

Span span_of(const Rows& r) { return Span{r.p, r.rows > 0 ? (r.rows - 1) * r.stride + r.width : 0}; }

// Whether two sets of rows share a byte.  Rows of one stride may lie between
// each other (parts of one buffer); others must not overlap as a whole.
bool rows_overlap(const Rows& a, const Rows& b)
{
    const Span x = span_of(a), y = span_of(b);
    if (!overlaps(x.p, x.bytes, y.p, y.bytes)) return false;
    if (a.stride != b.stride || a.stride <= 0) return true;
    int64_t d = ((int64_t)((uintptr_t)b.p - (uintptr_t)a.p)) % a.stride;
    if (d < 0) d += a.stride;
    return d < a.width || d + b.width > a.stride;
}

int check_kv(const mnb_kv_cache& c, const mnb_kv_batch& b)
{
    if (b.tokens < 0 || b.tokens > MNB_MAX_ROWS) return MNB_ERR_M_RANGE;
    if (c.pages < 0 || c.pages > INT32_MAX || !is_pow2_in(c.page_size, 16, 256) || c.kv_heads < 1 ||
        c.kv_heads > MNB_KV_MAX_HEADS || !is_pow2_in(c.head_dim, 64, 256) || b.sequences < 0 ||
        b.sequences > MNB_KV_MAX_SEQUENCES || b.max_pages < 0 || b.max_pages > MNB_KV_MAX_LENGTH / c.page_size)
        return MNB_ERR_SHAPE;
    return MNB_OK;
}

int check_kv_pointers(const mnb_kv_cache& c, const mnb_kv_batch& b)
{
    if (!b.starts || !b.lengths || (b.max_pages > 0 && !b.page_table)) return MNB_ERR_NULL;
    if (c.pages > 0 && (!c.k_pages || !c.v_pages || !c.k_scales || !c.v_scales)) return MNB_ERR_NULL;
    if (((uintptr_t)b.starts & 3) || ((uintptr_t)b.lengths & 3) || ((uintptr_t)b.page_table & 3) ||
        ((uintptr_t)c.k_pages & 15) || ((uintptr_t)c.v_pages & 15) || ((uintptr_t)c.k_scales & 3) ||
        ((uintptr_t)c.v_scales & 3))
        return MNB_ERR_ALIGN;
    return MNB_OK;
}

// Whether q_heads query heads can share kv_heads key heads.
bool good_group(int64_t q_heads, int64_t kv_heads)
{
    return q_heads > 0 && q_heads % kv_heads == 0 && q_heads / kv_heads <= MNB_KV_MAX_GROUP;
}

// A strided operand [tokens][heads][D]: its row stride in elements.
bool bad_stride(int64_t stride, int64_t heads, int64_t D, int64_t tokens)
{
    return tokens > 1 && (stride < heads * D || stride % 8 || stride > ((int64_t)1 << 40));
}

int check_lora_shape(int64_t m, int64_t K, int64_t N, int64_t rank, int64_t adapters)
{
    if (m < 0 || m > MNB_MAX_ROWS) return MNB_ERR_M_RANGE;
    if (K < 0 || K % 16 || K > MNB_MAX_K || N < 0 || N > MNB_MAX_N_INT8 || rank < 8 || rank % 8 ||
        rank > MNB_LORA_MAX_RANK || adapters < 0 || adapters > MNB_LORA_MAX_ADAPTERS)
        return MNB_ERR_SHAPE;
    return MNB_OK;
}

int check_int8_shape(int a_dtype, int64_t m, int64_t K, int64_t N)
{
    if (m < 0 || m > MNB_MAX_ROWS) return MNB_ERR_M_RANGE;
    if (K < 0 || N < 0 || K % 16 || K > MNB_MAX_K_INT8 || N > MNB_MAX_N_INT8) return MNB_ERR_SHAPE;
    if (a_dtype != MNB_F16 && a_dtype != MNB_BF16 && a_dtype != MNB_I8) return MNB_ERR_DTYPE;
    return MNB_OK;
}

int check_moe_shape(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int top_k)
{
    if (tokens < 0 || tokens > MNB_MOE_MAX_TOKENS) return MNB_ERR_M_RANGE;
    if (hidden < 32 || hidden % 32 || hidden > MNB_MOE_MAX_WIDTH || inter < 32 || inter % 32 ||
        inter > MNB_MOE_MAX_WIDTH || experts < 1 || experts > MNB_MOE_MAX_EXPERTS || top_k < 1 ||
        top_k > MNB_MOE_MAX_TOP_K || top_k > experts)
        return MNB_ERR_SHAPE;
    return MNB_OK;
}

int run(const void* A, int a_dtype, int64_t m, int64_t K, int64_t N,
        const uint8_t* Bpacked, const uint16_t* scales, const uint8_t* zero_points,
        int block, void* out, int out_dtype, void* stream, const mnb_plan* explicit_plan,
        bool fixed_scratch = false)
{
    int st = validate(A, a_dtype, m, K, N, Bpacked, scales, zero_points, block, out,
                      out_dtype);
    if (st != MNB_OK) return st;
    if (m == 0 || N == 0) {
        g_calls.fetch_add(1, std::memory_order_relaxed);
        return MNB_OK;
    }
    mnb_plan plan;
    if (explicit_plan) {
        plan = *explicit_plan;
        if (mnb_plan_check(m, K, N, &plan) != MNB_OK) return MNB_ERR_PLAN;
    } else {
        int cus = 0;
        int e = mnb::current_device_cus(&cus);
        if (e != 0) {
            t_last_hip_error = e;
            return MNB_ERR_HIP;
        }
        // Plan once with a nominal occupancy to pick the kernel variant, then
        // again with that variant's measured occupancy for the grid.
        st = mnb_plan_default(m, K, N, cus, 0, &plan);
        if (st != MNB_OK) return st;
        const int per_cu = mnb::workgroups_per_cu(plan.engine == 2 ? m : std::min<int64_t>(m, MNB_MAX_M), K, N, plan);
        if (per_cu > 0) {
            st = mnb_plan_default(m, K, N, cus, per_cu, &plan);
            if (st != MNB_OK) return st;
        }
    }
    if (log_enabled()) log_plan(m, K, N, a_dtype, out_dtype, plan, explicit_plan != nullptr, fixed_scratch);
    // One launch (two with K split over workgroups: the tiles, then the sum
    // of their slices), or for a decode plan with more than MNB_MAX_M rows
    // one launch per MNB_MAX_M rows (rows are independent in those kernels).
    const int64_t step = plan.engine == 2 ? m : MNB_MAX_M;
    const size_t a_row = (size_t)K * 2, out_row = (size_t)N * 2;
    const int per_launch = plan.k_splits > 1 ? 2 : 1;
    void* ws = nullptr;
    bool held = false;   // the per-stream workspace is held until the launches are queued
    const size_t ws_bytes = mnb::workspace_bytes(m, N, plan);
    if (ws_bytes && fixed_scratch) {
        if (ws_bytes > mnb::kScratchBytes) return MNB_ERR_WORKSPACE;
        int e = mnb::scratch_address(&ws);
        if (e != 0) {
            t_last_hip_error = e;
            return MNB_ERR_HIP;
        }
    } else if (ws_bytes) {
        int e = mnb::workspace_acquire(ws_bytes, stream, &ws);
        if (e != 0) {
            t_last_hip_error = e;
            return MNB_ERR_HIP;
        }
        held = true;
    }
    int64_t launched = 0, batched = 0;
    for (int64_t r0 = 0; r0 < m; r0 += step) {
        const int64_t mc = std::min<int64_t>(step, m - r0);
        mnb::GemvArgs args{static_cast<const uint8_t*>(A) + r0 * a_row, Bpacked, scales, zero_points,
                           static_cast<uint8_t*>(out) + r0 * out_row, mc, K, N,
                           a_dtype == MNB_BF16, out_dtype == MNB_BF16, ws};
        int e = mnb::launch_gemv(args, plan, stream);
        if (e != 0) {
            t_last_hip_error = e;
            g_launches.fetch_add((uint64_t)launched, std::memory_order_relaxed);
            if (held) mnb::workspace_release();
            return MNB_ERR_HIP;
        }
        launched += per_launch;
        if (mc > 1) ++batched;
    }
    if (held) mnb::workspace_release();
    g_calls.fetch_add(1, std::memory_order_relaxed);
    g_launches.fetch_add((uint64_t)launched, std::memory_order_relaxed);
    if (out_dtype == MNB_BF16) g_bf16.fetch_add((uint64_t)(m * N), std::memory_order_relaxed);
    else g_f16.fetch_add((uint64_t)(m * N), std::memory_order_relaxed);
    g_rows.fetch_add((uint64_t)batched, std::memory_order_relaxed);
    return MNB_OK;
}

}  // namespace

namespace mnb {

size_t workspace_bytes(int64_t m, int64_t N, const mnb_plan& plan)
{
    return plan.engine == 2 && plan.k_splits > 1 ? (size_t)plan.k_splits * (size_t)m * (size_t)N * 4 : 0;
}

int64_t gemv_lds_bytes(int64_t m, int64_t N, const mnb_plan& plan, int32_t* tcap)
{
    *tcap = 0;
    if (plan.engine != 0 || plan.lanes_per_col < 64) return 0;
    if (plan.lanes_per_col == 64)   // activations shared by the workgroup's waves
        return plan.k_chunks == 1 ? m * plan.blocks_per_lane * 256 * 16 : 0;
    const int64_t nw = plan.lanes_per_col / 64;
    const int64_t nv = (int64_t)plan.cols_per_tile * m;
    const int64_t g = plan.workgroups < 1 ? 1 : plan.workgroups;
    // Most tiles any group gets: dealt round-robin, or a contiguous range of
    // at most ceil(N / g) columns.
    const int64_t tiles = plan.interleave ? ceil_div(N, plan.cols_per_tile * g)
                                          : ceil_div(ceil_div(N, g), plan.cols_per_tile);
    const int64_t t = tiles < 1 ? 1 : tiles;
    if (t * nw * nv * 4 <= kDeferLdsBytes) {
        *tcap = (int32_t)t;
        return t * nw * nv * 4;
    }
    return 2 * nw * nv * 4;
}

}  // namespace mnb

namespace {

// Prefill tilings of engine 2 (row tiles, columns, waves, K splits over
// workgroups) and their fitted cost in microseconds on gfx950:
//   t0 + a*k*(R-1) + g*(R-1) + d*k + h*W + u*U
// with k the thousands of K per workgroup (K / splits), R = ceil(tiles /
// CUs) rounds of tiles over the compute units (a split multiplies the
// tiles), W the MB of weights (with scales and zero points) per CU and U the
// MB of fp32 partial sums per CU that a split writes and its second launch
// reads.  a and g price the rounds after the first, d and t0 the first (a CU
// with one tile runs it faster than two that share it), h the weights that
// stream from HBM when few row tiles share them, u the partial sums.
struct Tiling {
    int32_t rt, cols, waves, splits;
    double t0, a, g, d, h, u;
};
constexpr Tiling kTilings[] = {
    {1, 16, 4, 1, 3.8610, 1.3850, 1.9342, 1.8901, 0.0000, 0.0000},   // 16 columns on a 32-column tile, K split over the waves
    {1, 16, 8, 1, 5.8870, 2.0036, 1.9578, 1.7275, 0.0000, 0.0000},
    {1, 32, 4, 1, 4.9887, 1.4723, 2.3993, 1.9066, 3.2569, 0.0000},   // K split over the four waves
    {1, 64, 2, 1, 1.0704, 2.2076, 1.7534, 5.4974, 10.5770, 0.0000},
    {1, 128, 4, 1, 1.3403, 4.3963, 2.3819, 5.5898, 13.0526, 0.0000},
    {2, 128, 4, 1, 3.5663, 5.8118, 2.3400, 6.0021, 6.7267, 0.0000},
    {4, 128, 4, 1, 4.8855, 12.3022, 3.1521, 11.2704, 0.0000, 0.0000},
    {1, 256, 8, 1, 0.0000, 9.4388, 3.2051, 8.9528, 34.2933, 0.0000},
    {2, 256, 8, 1, 1.2841, 12.2381, 4.1168, 10.2565, 24.1162, 0.0000},
    {4, 256, 8, 1, 3.7579, 17.8627, 7.8076, 14.5888, 8.0399, 0.0000},
    {8, 256, 8, 1, 7.1312, 33.1356, 0.0000, 24.0315, 10.5656, 0.0000},   // 256 x 256, weights through LDS
    {1, 128, 4, 2, 5.6571, 3.8579, 0.0000, 4.8528, 7.4596, 198.7183},   // K split over 2..16 workgroups, a second launch adds the slices
    {1, 128, 4, 4, 6.4293, 3.9396, 0.0000, 4.4597, 10.4470, 161.6987},
    {1, 128, 4, 8, 5.9191, 3.4284, 1.3289, 5.3852, 9.2180, 115.3103},
    {1, 128, 4, 16, 6.7797, 1.6008, 1.9160, 4.2164, 17.8949, 115.9995},
    {2, 128, 4, 2, 6.1070, 4.2767, 0.0000, 5.9467, 2.2971, 197.8420},
    {2, 128, 4, 4, 7.1911, 5.1908, 0.0000, 5.7611, 3.9607, 124.0901},
    {2, 128, 4, 8, 7.1840, 4.8146, 0.7588, 6.3397, 3.3817, 110.2482},
    {2, 128, 4, 16, 7.5359, 2.1214, 2.8233, 6.5482, 0.0000, 122.8116},
    {4, 128, 4, 2, 6.8219, 11.1767, 0.0000, 11.0433, 3.0875, 190.7041},
    {4, 128, 4, 4, 8.1219, 11.8653, 0.1360, 10.4706, 12.1705, 145.6724},
    {4, 128, 4, 8, 7.4293, 10.2051, 5.1548, 12.0446, 8.9930, 111.4425},
    {4, 128, 4, 16, 9.2655, 7.5497, 8.0509, 11.1810, 0.0000, 104.2306},
    {1, 256, 8, 2, 3.7288, 7.2387, 0.0000, 8.5014, 23.7040, 193.0096},
    {1, 256, 8, 4, 5.5982, 7.9531, 0.0000, 8.4352, 15.2034, 128.6234},
    {1, 256, 8, 8, 6.1386, 9.1381, 0.0000, 8.8607, 17.0575, 79.5319},
    {1, 256, 8, 16, 7.3761, 7.1060, 2.1161, 7.8029, 18.2416, 59.4031},
    {2, 256, 8, 2, 4.8553, 11.6227, 0.0000, 10.3156, 13.5775, 182.9153},
    {2, 256, 8, 4, 6.4314, 11.4627, 0.0000, 10.2646, 8.3824, 133.9338},
    {2, 256, 8, 8, 6.2573, 12.3964, 0.3921, 10.7960, 14.1889, 108.8004},
    {2, 256, 8, 16, 7.6852, 8.0358, 5.4080, 9.0132, 20.0183, 85.1982},
};
// The decode plan per launch of r <= 8 rows: a part that grows with K (the
// activation staging and the per-wave work of each workgroup) and a part
// linear in the weight MB (with scales and zero points) at a rate per row,
//   exp(c0) * (K / 4096)^c1 + MB * (c2 + c3 * r / 8),
// and no less than 3 us, about what one launch takes however small.  (A
// power law in N, as first fitted, ran 15-20% below the launches on 151936
// columns, where the time is linear in the weights.)
constexpr double kDecode[4] = {1.6501, 0.1652, 0.1290, 0.0767};
constexpr double kBytesPerWeight = 0.578;   // 4 bits, and a 2-byte scale and a 4-bit zero point per 32
constexpr double kDecodeLaunchUs = 3.0;

int64_t prefill_tiles(const Tiling& t, int64_t m, int64_t N)
{
    const int64_t rows = t.rt == 8 ? 256 : 32 * (int64_t)t.rt;
    return ceil_div(m, rows) * ceil_div(N, t.cols) * t.splits;
}

double tiling_cost(const Tiling& t, int64_t m, int64_t K, int64_t N, int num_cus)
{
    const double R = (double)ceil_div(prefill_tiles(t, m, N), num_cus);
    const double k = (double)K / t.splits / 1e3;
    const double w = (double)N * (double)K * kBytesPerWeight / num_cus / 1e6;
    const double ws = t.splits > 1 ? (double)t.splits * (double)m * (double)N * 4 / num_cus / 1e6 : 0.0;
    return t.t0 + t.a * k * (R - 1) + t.g * (R - 1) + t.d * k + t.h * w + t.u * ws;
}

double decode_cost(int64_t m, int64_t K, int64_t N)
{
    const double mb = (double)N * (double)K * kBytesPerWeight / 1e6;
    auto one = [&](int64_t r) {
        const double t = std::exp(kDecode[0]) * std::pow((double)K / 4096, kDecode[1]) +
                         mb * (kDecode[2] + kDecode[3] * (double)r / 8);
        return t > kDecodeLaunchUs ? t : kDecodeLaunchUs;
    };
    const int64_t full = m / MNB_MAX_M, rem = m % MNB_MAX_M;
    return (double)full * one(MNB_MAX_M) + (rem ? one(rem) : 0.0);
}

struct PrefillChoice {
    Tiling t;
    bool decode;
};

// The cheapest plan by the model among the tilings the plan check accepts
// for (m, K, N) and, with `decode`, the decode plan; ties go to the earlier
// tiling.
PrefillChoice cheapest_prefill(int64_t m, int64_t K, int64_t N, int num_cus, bool decode = true)
{
    PrefillChoice best{kTilings[0], decode};
    double best_cost = decode ? decode_cost(m, K, N) : HUGE_VAL;
    for (const Tiling& t : kTilings) {
        mnb_plan q{};
        q.engine = 2;
        q.row_tiles = t.rt;
        q.cols_per_tile = t.cols;
        q.waves_per_wg = t.waves;
        q.k_splits = t.splits;
        q.workgroups = 1;
        if (mnb_plan_check(m, K, N, &q) != MNB_OK) continue;
        // A K split is there to fill the device: only while its tiles fit
        // in less than four rounds over the CUs, within the workspace bound.
        if (t.splits > 1 && (prefill_tiles(t, m, N) >= 4 * (int64_t)num_cus ||
                             mnb::workspace_bytes(m, N, q) > kMaxSplitWorkspaceBytes))
            continue;
        const double c = tiling_cost(t, m, K, N, num_cus);
        if (c < best_cost) {
            best_cost = c;
            best = PrefillChoice{t, false};
        }
    }
    return best;
}

// The prefill plan of tiling t: one resident generation of workgroups, at
// most one per tile.
int prefill_plan(const Tiling& t, int64_t m, int64_t K, int64_t N, int num_cus, int wgs_per_cu, mnb_plan* plan)
{
    const int64_t per_cu = wgs_per_cu > 0 ? wgs_per_cu : 1;
    const int64_t tiles = prefill_tiles(t, m, N);
    int64_t wgs = per_cu * num_cus;
    if (wgs > tiles) wgs = tiles;
    plan->engine = 2;
    plan->row_tiles = t.rt;
    plan->cols_per_tile = t.cols;
    plan->waves_per_wg = t.waves;
    plan->k_splits = t.splits;
    plan->workgroups = (int32_t)(wgs < 1 ? 1 : wgs);
    return mnb_plan_check(m, K, N, plan) == MNB_OK ? MNB_OK : MNB_ERR_PLAN;
}

}  // namespace

namespace mnb {

size_t int8_workspace_bytes(int a_dtype, int64_t m, int64_t K, int64_t)
{
    if (a_dtype == MNB_I8 || int8_fused(a_dtype, m, K)) return 0;
    return (size_t)(m * K) + (size_t)(m * 4);   // rows (a multiple of 16 bytes), then scales
}

int quantize_variant(int64_t m, int64_t K)
{
    // Rows that fill the device take no more waves than hold them, few rows are
    // spread wide (us, 64 x 1, 256 x 1, 256 x 8, 1024 x 1, 1024 x 4): 4096 rows of 512
    // 4.2, 6.2, 9.4, 17.1, 20.9; of 2048 10.0, 8.8, 11.6, 18.3, 21.9; of 8192 34.3,
    // 25.8, 20.1, 26.7, 30.4; 2048 rows of 16384 50.3, 27.8, 22.1, 26.2, 23.8, of
    // 32768 101, 59, 61, 50, 38.5; 16 rows of 2048 5.6, 3.3, 3.5, 3.3, 3.6; of 8192
    // 15.1, 5.9, 4.8, 3.8, 4.2; of 16384 28.3, 9.2, 6.5, 4.8, 4.7.  At 512 rows of 4096
    // (10.5, 5.0, 5.0, 4.8, 5.6) and 1024 (11.2, 6.3, 6.5, 7.5, 8.5) the order turns.
    const bool many = m >= 1024;
    if (K <= 512) return 0;
    if (K <= (many ? 4096 : 2048)) return 1;
    if (many && K <= 16384) return 2;
    return K <= 8192 ? 3 : 4;
}

// The tile with the least time: rounds of one tile per CU, each a fixed part
// (filling the stages, the epilogue) and one that grows with K, us and us per
// 1024 of K.  Fitted to the seven tiles' times on 72 shapes (m = 17 .. 2048; K
// x N = 4096 x 4096, 4096 x 28672, 14336 x 4096, 4112 x 5999, 1024 x 8192, 8192 x
// 1024); its choice is 0.2% slower than the fastest tile on average, at most
// 4%.  256 x 256 against 256 x 128 on 2048 x
// 4096 x 28672: 258 and 275 us, on 2048 x 14336 x 4096: 154 and 116; 32 x 32
// against 64 x 64 on 32 x 14336 x 4096: 21 and 38, on 256 x 4096 x 4096: 20 and 10.
struct Int8TileCost {
    int bm, bn;
    double fixed, per_k;
};
constexpr Int8TileCost kInt8Tiles[] = {{256, 256, 8.0, 13.4}, {256, 128, 8.0, 7.2}, {128, 128, 4.5, 4.4},
                                       {128, 64, 5.5, 2.85},  {64, 64, 5.0, 2.33},  {64, 32, 4.8, 1.42},
                                       {32, 32, 4.5, 0.98}};

int int8_cheapest_tile(int64_t m, int64_t K, int64_t N, int cus)
{
    int best = 0;
    double least = 0;
    for (int t = 0; t < (int)(sizeof(kInt8Tiles) / sizeof(kInt8Tiles[0])); ++t) {
        const Int8TileCost& c = kInt8Tiles[t];
        const int64_t tiles = ((m + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn), rounds = (tiles + cus - 1) / cus;
        const double us = (double)rounds * (c.fixed + c.per_k * (double)K / 1024);
        // (A grid holds 2^32 threads; the largest tile fits for every N there is.)
        if (t == 0 || (tiles < (1 << 23) && us < least)) {
            best = t;
            least = us;
        }
    }
    return best;
}

Int8Route int8_route(int a_dtype, int64_t m, int64_t K, int64_t N, int cus)
{
    Int8Route r{};
    r.fused = int8_fused(a_dtype, m, K);
    if (m > 16 || K > kInt8RowsK || int8_rows_lds(m, K, 16) > kInt8RowsLds) {
        r.tile = int8_cheapest_tile(m, K, N, cus);
        return r;
    }
    r.tile = -1;
    // Sixteen waves, or eight in two workgroups a CU where both fit LDS:
    // with K <= 2048, where sixteen would have one unit each under way
    // (us, eight against sixteen: 2048 x 28672, 4 rows 14.8 and 16.1; 2048 x
    // 151936, one row 60.4 and 75.4), and up to 4096 with so many columns that
    // an odd tile does not count (4096 x 151936 111 and 119, but with 16 rows 117
    // and 111; 4096 x 28672 25.9 and 24.6; 8192 x 28672 47.0 and 42.2).
    const int64_t units = std::max<int64_t>((K + 127) / 128, 1), tiles = (N + 15) / 16;
    const bool eight = 2 * int8_rows_lds(m, K, 8) <= kInt8RowsLds &&
                       ((units <= 16 && tiles > cus) || (units <= 32 && tiles > 16 * (int64_t)cus));
    const int64_t w = std::min<int64_t>(eight ? 8 : 16, units);
    r.nu = (int)((units + w - 1) / w);
    r.waves = (int)((units + r.nu - 1) / r.nu);
    r.workgroups = std::min(tiles, (r.waves <= 8 ? 2 : 1) * (int64_t)cus);
    return r;
}

MoeLayout moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int top_k)
{
    const int64_t pairs = T * top_k;
    MoeLayout l{};
    // The kernels and the rows of a batch, by the tokens an expert sees on
    // average (us, narrow with 8 rows against wide with 16 and with 32): 6 tokens
    // (24 tokens, 2 of 8 experts of 4096, 14336) 218 against 237 and 262; 8 (32
    // tokens) 269 against 253 and 279, (64 tokens, 8 of 64 of 2048, 768) 98 against
    // 100 and 119; 16 (64 tokens, 2 of 8) 451 against 354 and 295, (64 tokens, 8 of
    // 32 of 2048, 768) 89 against 85 and 76; 32 (64 tokens, 2 of 4 of 4096, 4096) 145
    // against 102 and 88.  Narrow with 4 rows against 8 (2 of 8 of 4096, 14336):
    // 3 tokens for an expert 156 against 171, 4 214 against 199, 5 228 against 200.
    // (Kernel times; three more launches cost the wide form about 5 us besides.)
    l.wide = pairs > 12 * E ? 2 : pairs >= 8 * E ? 1 : 0;
    l.rq = l.wide ? 4 * l.wide : pairs > 4 * E ? 2 : 1;
    // Every expert has at most one batch that is not full.
    const int64_t rows = 4 * l.rq;
    int64_t batches = std::min(pairs, E) + pairs / rows;
    if (batches > pairs) batches = pairs;
    l.batches = (int)batches;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at = (at + (size_t)bytes + 255) & ~(size_t)255;
        return here;
    };
    take((1 + T) * 4);
    l.batch_e = take(batches * 4);
    l.row_token = take(batches * rows * 4);
    l.row_p = take(batches * rows * 4);
    if (l.wide) {
        l.hs = take(batches * rows * 4);
        l.h = take(batches * rows * I * 2);
        l.pair_row = take(pairs * 4);
        l.xs = take(T * H * 2);
        l.xe = take(T * 4);
        l.hf = take(batches * rows * I * 4);
        l.y = take(batches * rows * H * 4);
    } else {
        l.hs = take(batches * rows * (I / 32) * 4);
        l.h = take(batches * rows * ((I / 32 + 15) / 16 * 512) * 2);   // blocks of I in groups of 16
    }
    l.bytes = at;
    return l;
}

MoeRoute moe_route(const MoeArgs& a, const MoeLayout& l, int cus)
{
    const mnb_moe_weights& w = a.w;
    // Whether a matrix's scales and zero points can be loaded for `blocks`
    // consecutive blocks at a time.
    auto vec_ok = [](int64_t K, const uint16_t* scales, const uint8_t* zp, int blocks) {
        return (K / 32) % blocks == 0 && ((uintptr_t)scales & (2 * blocks - 1)) == 0 &&
               (blocks < 4 || ((uintptr_t)zp & (blocks / 2 - 1)) == 0);
    };
    MoeRoute r{};
    if (l.wide) {
        auto vec = [&](int64_t K, const uint16_t* s, const uint8_t* z) { return vec_ok(K, s, z, 8) ? 8 : vec_ok(K, s, z, 4) ? 4 : 1; };
        r.up_vec = vec(w.hidden, w.gate_up_scales, w.gate_up_zero_points);
        r.down_vec = vec(w.inter, w.down_scales, w.down_zero_points);
        return r;
    }
    r.up_vec = vec_ok(w.hidden, w.gate_up_scales, w.gate_up_zero_points, 4) ? 4 : 1;
    // The first launch stages whole rows where they fit, else spans of K.
    const int blocks = (int)(w.hidden / 32 + 31) / 32 * 32, rows = 4 * l.rq;
    const int64_t lds = kMoeLds - (int64_t)moe_up_static_lds(l.rq) -
                        moe_routing_bytes((int)w.experts, a.T * a.top_k, l.batches, l.rq);
    const int most = (int)(lds / (rows * 16) - 1) / 4 / 32 * 32;
    r.stage_blocks = std::min(blocks, most);
    // Columns of a workgroup of the second: as many (16, 8, 4) as leave one for
    // every CU (us of this launch with 4, 8 and 16): 2 of 8 experts of 4096,
    // 14336, 1 token 36, 25, 19; 8 of 64 of 2048, 768, 4 tokens 17.6, 11.8, 15.9;
    // 8 of 32 of 1024, 512, 4 tokens 6.9, 7.8, 8.9.
    r.down_quads = w.hidden / 16 >= cus ? 4 : w.hidden / 8 >= cus ? 2 : 1;
    r.down_vec = vec_ok(w.inter, w.down_scales, w.down_zero_points, r.down_quads) ? r.down_quads : 1;
    return r;
}

}  // namespace mnb

namespace mnb {

AttentionLayout attention_layout(int64_t tokens, int64_t sequences, int64_t q_heads, int64_t kv_heads, int64_t head_dim)
{
    AttentionLayout l;
    const size_t parts = 2 * (size_t)kAttentionWorkgroups, D = (size_t)head_dim;
    l.o = parts * 16 * 2 * 4;
    l.tile_ml = l.o + parts * 16 * D * 4;
    const int64_t rows = tokens * (q_heads / kv_heads), tile = tile_rows(head_dim);
    // Full tiles, and one more for each sequence that can have many rows.
    l.many = attention_many_rows(tokens, q_heads, head_dim);
    l.tile_slots = rows > l.many ? (int)(rows / tile + std::min<int64_t>(sequences, rows / (l.many + 1))) : 0;
    // From five rounds of them on, whole tiles leave too little idle for shares to pay.
    const int64_t shares = tile_shares(head_dim);
    l.shares = l.tile_slots && (rows / tile + 1) * kv_heads < 5 * shares ? (int)shares : 0;
    const size_t each = 2 * (size_t)l.shares * (size_t)tile;
    l.tile_o = l.tile_ml + each * 2 * 4;
    l.bytes = l.tile_o + each * D * 4;
    return l;
}

LoraLayout lora_layout(int64_t m, int64_t K, int64_t N, int64_t R, int64_t adapters)
{
    LoraLayout l;
    // 64 columns a wave, or 16 where that leaves half of the compute units empty: 512 rows x
    // 6144 columns 17.6 us wide, 23.8 narrow; 64 rows x 14336, 32 adapters 71.2, 32.9; 33 rows
    // x 32768, 32 adapters (128 workgroups) 71.4, 39.0, x 36864, 8 adapters 16.9, 19.5.
    l.wide = ceil_div(N, 512) * ceil_div(m, m <= 16 ? 16 : 32) > 128;
    // Narrow: tiles of 32 rows, or of 64 where those, counted by their rows, are more than
    // two workgroups a compute unit and an adapter would be read for one after another (64
    // rows, 32 adapters, rank 64: x 16384 33.2 us with 32, 40.4 with 64; x 20480 53.4, 41.9;
    // 40 rows x 20480 33.9, 38.2, x 28672 41.7, 39.1).  Against the times of all three over
    // 160 shapes: 2.4% above the fastest on average (tests/data/kv_rules_gfx950.json).
    l.up_tiles = m <= 16 ? 1 : !l.wide && R <= 128 && m * ceil_div(N, 64) > 32 * 512 ? 4 : 2;
    // The first launch: 512 rows, 14336 -> 16 15.8 us with 32, 17.9 with 64; 1024 rows of 8
    // adapters, 4096 -> 64 50.7 with 32, 44.7 with 64.
    l.down_tiles = m <= 16 ? 1 : m < 1024 || R > 128 ? 2 : 4;
    const int64_t rows = 16 * l.down_tiles, tiles = ceil_div(m, rows);
    // Workgroups of 256 or more of K each; slices cost the second launch their sums.
    const int64_t splits = std::min<int64_t>(ceil_div(kLoraDownWorkgroups, tiles), std::min<int64_t>(m <= 16 ? 16 : 8, std::max<int64_t>(1, K / 256)));
    const int64_t slice = ceil_div(ceil_div(K, splits), 128) * 128;
    l.k_slice = (int)std::max<int64_t>(128, slice);
    l.splits = (int)std::max<int64_t>(1, ceil_div(K, l.k_slice));
    // Rows may have an adapter each: workgroups that share a tile's adapters (64 rows of
    // 32 adapters, rank 64: one workgroup 188 us, these 33); those that get none end at
    // once (4096 rows in runs of 500: 90 us with or without them).
    l.ways = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(adapters, std::min(m, rows)), kLoraDownWorkgroups / (tiles * l.splits)));
    l.bytes = (size_t)l.splits * (size_t)m * (size_t)R * 4;
    return l;
}

}  // namespace mnb

extern "C" {

int mnb_plan_check(int64_t m, int64_t K, int64_t N, mnb_plan* plan)
{
    if (!plan || m < 1 || m > MNB_MAX_ROWS || K < 0 || K % 32 || N < 0) return MNB_ERR_PLAN;
    if (plan->workgroups < 1) return MNB_ERR_PLAN;
    if (plan->b_layout != MNB_LAYOUT_NATURAL &&
        !(plan->b_layout == MNB_LAYOUT_EVEN_ODD && (plan->engine == 0 || plan->engine == 3)))
        return MNB_ERR_PLAN;
    if (plan->a_via_lds != 0 && (plan->a_via_lds != 1 || plan->engine != 3)) return MNB_ERR_PLAN;
    const int64_t nb = K / 32;
    if (plan->engine == 2) {
        const bool shape_ok =
            plan->row_tiles == 8 ? (plan->waves_per_wg == 8 && plan->cols_per_tile == 256)
                                 : ((plan->row_tiles == 1 && ((plan->cols_per_tile == 32 && plan->waves_per_wg == 4) ||
                                                              (plan->cols_per_tile == 16 &&
                                                               (plan->waves_per_wg == 4 || plan->waves_per_wg == 8)))) ||
                                    (plan->waves_per_wg == 2 && plan->cols_per_tile == 64) ||
                                    (plan->waves_per_wg == 4 && is_pow2_in(plan->cols_per_tile, 128, 256)) ||
                                    (plan->waves_per_wg == 8 && plan->cols_per_tile == 256));
        if (!is_pow2_in(plan->row_tiles, 1, 8) || !shape_ok ||
            (uint64_t)64 * plan->row_tiles * (uint64_t)K > mnb::kPrefillRowBlockBytes)
            return MNB_ERR_PLAN;
        // K split over workgroups: at least one 128-wide step per slice, not
        // for the LDS-staged 256 x 256 tiles, a workspace below 2^31 floats
        // per slice plane, and fewer than 2^31 tiles (the kernel's slice
        // arithmetic is 32-bit).
        if (plan->k_splits < 0 || plan->k_splits > kMaxKSplits) return MNB_ERR_PLAN;
        if (plan->k_splits > 1 &&
            (plan->row_tiles == 8 || plan->k_splits > ceil_div(nb, 4) || m * N > (int64_t)INT32_MAX ||
             ceil_div(m, 32 * (int64_t)plan->row_tiles) * ceil_div(N, (int64_t)plan->cols_per_tile) *
                     plan->k_splits > (int64_t)INT32_MAX))
            return MNB_ERR_PLAN;
        plan->threads_per_wg = 64 * plan->waves_per_wg;
        plan->k_chunks = (int32_t)ceil_div(nb, 4);   // 128-wide steps of K
        return MNB_OK;
    }
    if (plan->k_splits > 1) return MNB_ERR_PLAN;
    // Decode engines: a launch serves at most MNB_MAX_M rows; more rows run
    // as launches of MNB_MAX_M rows (the last one fewer) under this plan, so
    // the plan must fit MNB_MAX_M rows.
    if (m > MNB_MAX_M) m = MNB_MAX_M;
    if (plan->engine == 3) {
        // 4x4x4 MFMA kernel: the workgroup's 16 * waves lane groups cover K
        // in one pass, blocks_per_lane blocks each; 4 or 8 columns per tile.
        const int64_t w = plan->waves_per_wg, bpl = plan->blocks_per_lane;
        if (w < 1 || w > 8 || !is_pow2_in(bpl, 1, 4) ||
            (plan->cols_per_tile != 4 && plan->cols_per_tile != 8))
            return MNB_ERR_PLAN;
        if (16 * w * bpl < nb) return MNB_ERR_PLAN;
        if (m > 4 && bpl * (plan->cols_per_tile / 4) > 4) return MNB_ERR_PLAN;   // registers
        plan->threads_per_wg = (int32_t)(64 * w);
        plan->k_chunks = 1;
        return MNB_OK;
    }
    if (plan->engine != 0) return MNB_ERR_PLAN;
    const int64_t lpc = plan->lanes_per_col;
    const int64_t bpl = plan->blocks_per_lane;
    const int64_t nc = plan->cols_per_tile;
    const bool inwave = is_pow2_in(lpc, 16, 64);
    const bool xwave = lpc % 64 == 0 && lpc >= 128 && lpc <= 512;
    if (!inwave && !xwave) return MNB_ERR_PLAN;
    if (!is_pow2_in(bpl, 1, 8) || m * bpl > 8) return MNB_ERR_PLAN;
    if (!is_pow2_in(nc, 1, 8) || nc * bpl > 8 || nc * m > 32) return MNB_ERR_PLAN;
    if (plan->interleave != 0 && plan->interleave != 1) return MNB_ERR_PLAN;
    plan->threads_per_wg = inwave ? 256 : (int32_t)lpc;
    const int64_t chunks = nb == 0 ? 1 : ceil_div(nb, lpc * bpl);
    if (chunks > INT32_MAX) return MNB_ERR_PLAN;
    plan->k_chunks = (int32_t)chunks;
    return MNB_OK;
}

int mnb_plan_default(int64_t m, int64_t K, int64_t N, int num_cus, int wgs_per_cu,
                     mnb_plan* plan)
{
    if (!plan) return MNB_ERR_NULL;
    if (m < 1 || m > MNB_MAX_ROWS) return MNB_ERR_M_RANGE;
    if (K < 0 || K % 32 || K > MNB_MAX_K || N < 1 || N > INT32_MAX) return MNB_ERR_SHAPE;
    if (num_cus < 1) num_cus = 1;
    *plan = mnb_plan{};

    if (m > MNB_MAX_M) {
        // Prefill: every tiling of the prefill kernel that the plan check
        // accepts (with K split over workgroups where that fills the
        // device), and the 8-row decode plan run once per 8 rows, priced by
        // a cost model fitted to timings on gfx950 (256 CUs, bf16 in and
        // out, 64 shapes from 9 x 2048 x 8192 to 4096 x 4096 x 28672 and
        // 640 x 4096 x 151936; plan_tune.py measures and fits it).  On
        // those shapes the cheapest modelled plan runs 0.37% slower than
        // the fastest measured one on average (6.9% at most, where a split
        // the model ranks second would have won), and 11.9% faster on
        // average than the fastest plan without a K split (never more than
        // 2.7% slower: a choice between unsplit tilings).
        const PrefillChoice c = cheapest_prefill(m, K, N, num_cus);
        if (c.decode) return mnb_plan_default(MNB_MAX_M, K, N, num_cus, wgs_per_cu, plan);
        return prefill_plan(c.t, m, K, N, num_cus, wgs_per_cu, plan);
    }
    const int64_t nb = K / 32;
    const int64_t bmax = max_blocks_per_lane(m);

    // Two or more rows with K within one pass of a workgroup (8 waves x 16
    // lane groups x 4 blocks): the 4x4x4 MFMA kernel, whose dot products do
    // not grow the VALU work with m (against the lane split below, bf16:
    // lm_head m = 2 82.9 -> 69.7 us, m = 8 104 -> 90.6; gate_up m = 8 70.4 ->
    // 26.9, m = 3 25.4 -> 20.0; down m = 8 26.1 -> 18.5, m = 3 15.6 -> 12.9;
    // the 6144-column shape gains at m = 8 and loses up to 1 us at m <= 3).
    // Lane split, a function of (m, K) only (the exceptions below): the
    // fewest blocks per lane group that
    // cover K with at most four waves, else eight waves, of which the kernel
    // gives the fewest that need them four blocks per lane group and the
    // rest three (K = 14336: four of each, against seven waves of four,
    // interleaved A/B, us: m = 2 11.0 -> 10.4, m = 4 11.7 -> 11.3, m = 6
    // 14.8 -> 13.8, m = 8 15.2 -> 14.1; 10240 x 4096 m = 4 10.3 -> 9.5,
    // 12288 x 8192 m = 8 19.8 -> 18.2).  Four columns per tile.
    // Grid: whole workgroups per CU, about 12 * K/4096 tiles (column quads)
    // each, within one resident generation and at least two tiles each (the
    // tile loop runs in pairs).  Every workgroup stages all of K's
    // activations, so fewer, longer-lived workgroups win until the CUs run
    // short of waves (at one or two rows, two workgroups per CU at least,
    // below).  On a sweep of 50 shapes (m = 2..8, K = 2048..14336, N =
    // 4096..151936, bf16): 0.30% above the fastest grid on average, 6.1% at
    // most (10 * K/4096, fitted on an earlier sweep, gave 0.63% and 8.2% on
    // this one: 2048 x 28672 at six and eight rows took six workgroups per
    // CU where five are 8% faster; 14 * K/4096 and above put 4096 x 14336
    // at three rows on one workgroup per CU, 22% slower).
    // Activations through LDS from three rows up where K or N exceeds 8192
    // (interleaved A/B, same bits, us: down projection m = 3 12.5 -> 11.5,
    // m = 4 13.6 -> 11.9, m = 7 17.5 -> 15.4, m = 8 18.3 -> 15.7; gate_up
    // m = 4 18.7 -> 17.0, m = 8 24.3 -> 22.3; lm_head m = 3 -2.0%, m = 6
    // -1.7%); at 8192 x 8192, 4096 x 6144 and 4096 x 4096 it was 2-4.5%
    // slower, and at m = 2, where half of the lanes' own loads read nothing,
    // 0-4% slower.
    if (m >= 2 && nb >= 1 && nb <= 512) {
        // Up to four rows, at least two blocks per lane group where that
        // still leaves two waves: K = 2048 runs two waves of two blocks
        // instead of four of one (m = 2: 8.2 -> 7.1 us at N = 14336, 11.9 ->
        // 10.4 at 28672, 40.3 -> 34.8 at 151936, 5.8 -> 5.2 at 8192; m = 4
        // 8-13% faster from N = 14336 up, 3% slower at 8192).  From five
        // rows it lost at N = 8192 (m = 8: 7.3 -> 8.2 us), so there the
        // four waves of one stay.  A function of (m, K), like the rest of
        // the lane split.
        int64_t bpl3 = nb >= 64 && m <= 4 ? 2 : 1;
        while (bpl3 < 4 && ceil_div(nb, 16 * bpl3) > 4) bpl3 *= 2;
        // Three waves of four blocks (4096 < K <= 6144) leave one SIMD of
        // each workgroup idle: five or six waves of two instead (5120 x
        // 4096 m = 4 / 6 / 8 7.4 / 9.4 / 9.9 -> 7.0 / 8.4 / 9.3 us; 6144 x
        // 4096 m = 2 / 8 7.6 / 10.5 -> 7.0 / 9.8, 6144 x 14336 m = 6 / 8
        // 19.4 / 19.8 -> 18.4 / 18.5; at 28672 columns 0.5-2.6% slower).
        if (bpl3 == 4 && ceil_div(nb, 64) == 3) bpl3 = 2;
        int64_t w3 = ceil_div(nb, 16 * bpl3);
        if (w3 > 4 && bpl3 == 4) w3 = 8;   // two waves per SIMD; the kernel gives some three blocks per lane group
        const int64_t tiles3 = ceil_div(N, 4);
        const int64_t per_cu3 = wgs_per_cu > 0 ? wgs_per_cu : (w3 >= 4 ? 2 : 4);
        const double per_wg = 12.0 * (double)K / 4096.0;
        int64_t c3 = (int64_t)std::ceil((double)tiles3 / (double)num_cus / per_wg);
        // Two-wave workgroups of two blocks: whole multiples of four per CU
        // (eight waves), about 16 column quads each (K = 2048: four per CU
        // within 1% of the fastest grid up to N = 28672, eight at 151936,
        // where four are 4.5% slower; three or six per CU ran 10-15% slower
        // than four).
        if (w3 == 2 && bpl3 == 2)
            c3 = 4 * std::max<int64_t>(1, std::llround((double)tiles3 / ((double)num_cus * 64.0)));
        // With twelve or more column quads per CU, at least two workgroups
        // per CU where one would leave the CU fewer than six waves (three
        // waves of four blocks at 5120 and 6144 x 14336, m = 4 / 6 / 8: 16.1
        // / 19.1 / 19.2 -> 14.1 / 17.4 / 17.8 us and 16.8 / 20.2 / 20.3 ->
        // 15.2 / 19.4 / 19.8; four waves at 8192 x 14336 m = 4 18.4 -> 18.2,
        // m = 6 and 8 1% slower; six waves of two at 6144 x 14336 ran 1-7%
        // faster at one per CU).
        if (tiles3 >= 12 * num_cus && c3 < 2 && w3 < 6) c3 = 2;
        // One or two rows stage their activations with the lanes' own loads,
        // half of which read nothing: two workgroups per CU at least (4096 x
        // 4096 m = 2 5.72 -> 5.22 us, 8192 x 8192 12.0 -> 11.1).
        if (m <= 2 && c3 < 2) c3 = 2;
        if (c3 < 1) c3 = 1;
        if (c3 > per_cu3) c3 = per_cu3;
        int64_t wgs3 = c3 * num_cus;
        if (wgs3 > ceil_div(tiles3, 2)) wgs3 = ceil_div(tiles3, 2);
        plan->engine = 3;
        plan->waves_per_wg = (int32_t)w3;
        plan->blocks_per_lane = (int32_t)bpl3;
        plan->cols_per_tile = 4;
        plan->a_via_lds = m >= 3 && (K > 8192 || N > 8192);
        plan->workgroups = (int32_t)(wgs3 < 1 ? 1 : wgs3);
        return mnb_plan_check(m, K, N, plan) == MNB_OK ? MNB_OK : MNB_ERR_PLAN;
    }

    // 1. Lane split -- a function of (m, K) only, so the fp32 summation order
    //    of a column never depends on N or on the device (column shards of
    //    one matrix give the bits of the whole).
    //    m = 1: two blocks per lane, so a 4096-long K is one wave per column.
    //    m > 1: one block per lane (activation VGPRs grow with m), whole waves
    //    per column up to 8, then K chunks.
    const int64_t bpl_pref = m == 1 ? 2 : 1;
    int64_t lpc, bpl;
    if (ceil_div(nb, bpl_pref) <= 64) {
        lpc = pow2_ceil(ceil_div(nb, bpl_pref));
        if (lpc < 16) lpc = 16;
        bpl = pow2_ceil(nb == 0 ? 1 : ceil_div(nb, lpc));
    } else {
        lpc = 64 * ceil_div(ceil_div(nb, bpl_pref), 64);
        if (lpc > 512) lpc = 512;
        bpl = pow2_ceil(ceil_div(nb, lpc));
        if (bpl > bmax) bpl = bmax;
    }

    // Two or more rows whose K the lane split cannot cover in one pass (eight
    // waves of one to four blocks per lane, as registers allow: K > 16384 at
    // five to eight rows, K > 32768 at three or four): the chunked passes
    // take one tile at a time and reload the activations per chunk (K =
    // 28672, N = 4096, m = 8: 178 us against 26 at m = 4), so the prefill
    // tiles run instead, K split over workgroups, priced by the prefill cost
    // model (that shape 31.8 us; 28672 x 8192 m = 8 345 -> 52.4, 20480 x 8192
    // 320 -> 44.4, 65536 x 4096 342 -> 59.2).  Whether this happens depends
    // on (m, K) only; which tiling runs then depends on N and the CUs, as
    // for m > 8.
    if (m >= 2 && nb > 0 && ceil_div(nb, lpc * bpl) > 1)
        return prefill_plan(cheapest_prefill(m, K, N, num_cus, false).t, m, K, N, num_cus, wgs_per_cu, plan);

    // 2. Column tile: two columns per lane group in a wave; one column per
    //    multi-wave group, whose waves then keep the next column's loads in
    //    flight (measured on the down-projection shape).
    int64_t nc = lpc <= 64 ? (bpl >= 4 ? 1 : 2) : 1;
    while (nc > 1 && (nc * bpl > 8 || nc * m > 32)) nc /= 2;

    // 3. Grid.  Tiles are dealt round-robin, so all lane groups sweep the
    //    weights as one front.  In-wave groups: about five tiles per group,
    //    in whole rounds of the CU count, between half and three times one
    //    resident generation of workgroups (measured best on the lm_head
    //    and gate_up shapes).  Multi-wave groups: whole workgroups per CU,
    //    about eight waves per CU (more tiles per workgroup share its
    //    activation fetch).  Measured at m = 1 on 11 shapes with K from 6144
    //    to 28672 against half a resident generation (2.5 four-wave
    //    workgroups per CU, which leaves the CUs uneven): the down projection
    //    10.39 -> 9.57 us, 8192 x 14336 14.52 -> 13.69, 16384 x 16384 29.32
    //    -> 26.28; best or within 1% of the best count on eight of the 11,
    //    4.7% from it on the other three.
    const bool inwave = lpc <= 64;
    const int64_t gpw = inwave ? 256 / lpc : 1;
    const int64_t waves_per_wg = inwave ? 4 : lpc / 64;
    const int64_t per_cu = wgs_per_cu > 0 ? wgs_per_cu
                                          : (kTargetWavesPerCu + waves_per_wg - 1) / waves_per_wg;
    const int64_t resident = per_cu * num_cus;
    // Too few columns to give half a resident generation one tile per lane
    // group: one column per tile doubles the groups at work (the 4096-column
    // shape: 4.56 -> 4.36 us).
    while (inwave && nc > 1 && ceil_div(ceil_div(N, nc), gpw) < resident / 2) nc /= 2;
    const int64_t tiles = ceil_div(N, nc);
    int64_t wgs = resident / 2 > num_cus ? resident / 2 : num_cus;
    if (!inwave) {
        int64_t c = (8 + waves_per_wg / 2) / waves_per_wg;   // ~8 waves per CU
        if (c > per_cu) c = per_cu;
        if (c < 1) c = 1;
        wgs = c * num_cus;
    }
    if (inwave) {
        wgs = num_cus * ceil_div(ceil_div(tiles, 5 * gpw), num_cus);   // whole rounds of CUs
        const int64_t lo = resident / 2 > 0 ? resident / 2 : 1;
        if (wgs < lo) wgs = lo;
        if (wgs > 3 * resident) wgs = 3 * resident;
        // One tile per lane group fits in one resident generation: take it.
        if (ceil_div(tiles, gpw) <= resident) wgs = ceil_div(tiles, gpw);
    }
    if (!inwave) {
        // Multi-wave groups: enough workgroups that every wave's partial sums
        // of all of a group's tiles fit the deferred-sum LDS.
        const int64_t slot = waves_per_wg * nc * m * 4;
        const int64_t tmax = mnb::kDeferLdsBytes / slot;
        const int64_t need = ceil_div(tiles, tmax < 1 ? 1 : tmax);
        if (wgs < need) wgs = need;
    }
    if (wgs > ceil_div(tiles, gpw)) wgs = ceil_div(tiles, gpw);

    plan->engine = 0;
    plan->lanes_per_col = (int32_t)lpc;
    plan->blocks_per_lane = (int32_t)bpl;
    plan->cols_per_tile = (int32_t)nc;
    plan->waves_per_wg = 0;
    plan->workgroups = (int32_t)(wgs < 1 ? 1 : wgs);
    plan->interleave = 1;
    return mnb_plan_check(m, K, N, plan) == MNB_OK ? MNB_OK : MNB_ERR_PLAN;
}

int matmul_nbits(const void* A, int a_dtype, int64_t m, int64_t K, int64_t N,
                 const uint8_t* Bpacked, const uint16_t* scales,
                 const uint8_t* zero_points, int block, void* out, int out_dtype,
                 void* stream)
{
    return run(A, a_dtype, m, K, N, Bpacked, scales, zero_points, block, out, out_dtype,
               stream, nullptr);
}

int matmul_nbits_noalloc(const void* A, int a_dtype, int64_t m, int64_t K, int64_t N,
                         const uint8_t* Bpacked, const uint16_t* scales,
                         const uint8_t* zero_points, int block, void* out, int out_dtype,
                         void* stream)
{
    return run(A, a_dtype, m, K, N, Bpacked, scales, zero_points, block, out, out_dtype,
               stream, nullptr, true);
}

int matmul_nbits_planned(const void* A, int a_dtype, int64_t m, int64_t K, int64_t N,
                         const uint8_t* Bpacked, const uint16_t* scales,
                         const uint8_t* zero_points, int block, void* out, int out_dtype,
                         void* stream, const mnb_plan* plan)
{
    if (!plan) return MNB_ERR_NULL;
    return run(A, a_dtype, m, K, N, Bpacked, scales, zero_points, block, out, out_dtype,
               stream, plan);
}

int mnb_repack_weights(const uint8_t* src, int src_layout, uint8_t* dst, int dst_layout,
                       int64_t N, int64_t K, void* stream)
{
    auto known = [](int l) { return l == MNB_LAYOUT_NATURAL || l == MNB_LAYOUT_EVEN_ODD; };
    if (!known(src_layout) || !known(dst_layout)) return MNB_ERR_LAYOUT;
    if (K < 0 || N < 0 || K % 32 || K > MNB_MAX_K || N > INT32_MAX) return MNB_ERR_SHAPE;
    const int64_t bytes = N * (K / 2);
    if (bytes == 0) return MNB_OK;
    if (!src || !dst) return MNB_ERR_NULL;
    if (((uintptr_t)src & 15) || ((uintptr_t)dst & 15)) return MNB_ERR_ALIGN;
    if (dst != src && overlaps(src, bytes, dst, bytes)) return MNB_ERR_ALIAS;
    const int e = mnb::launch_repack(src, src_layout, dst, dst_layout, bytes / 4, stream);
    if (e != 0) {
        t_last_hip_error = e;
        return MNB_ERR_HIP;
    }
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return MNB_OK;
}

int quantize_rows_int8(const void* A, int a_dtype, int64_t m, int64_t K, int8_t* q, float* scales, void* stream)
{
    if (m < 0 || m > MNB_MAX_ROWS) return MNB_ERR_M_RANGE;
    if (K < 0 || K % 16 || K > MNB_MAX_K) return MNB_ERR_SHAPE;
    if (a_dtype != MNB_F16 && a_dtype != MNB_BF16) return MNB_ERR_DTYPE;
    if (m == 0) return finish_launches(0, 0);
    if (!scales || (K > 0 && (!A || !q))) return MNB_ERR_NULL;
    if (((uintptr_t)A & 15) || ((uintptr_t)q & 15) || ((uintptr_t)scales & 3)) return MNB_ERR_ALIGN;
    const Span in[] = {{A, m * K * 2}}, wr[] = {{q, m * K}, {scales, m * 4}};
    if (aliased(in, 1, wr, 2)) return MNB_ERR_ALIAS;
    if (log_enabled())
        fprintf(stderr, "mnb: quantize_rows_int8 m=%lld K=%lld a=%s launches=1\n", (long long)m, (long long)K,
                dtype_name(a_dtype));
    if (!mnb::launch_quantize_rows) return finish_launches(kNoDevice, 0);
    const int e = mnb::launch_quantize_rows(A, a_dtype == MNB_BF16, m, K, q, scales, stream);
    return finish_launches(e, 1);
}

size_t mnb_int8_workspace(int a_dtype, int64_t m, int64_t K, int64_t N)
{
    if (check_int8_shape(a_dtype, m, K, N) != MNB_OK || m == 0 || N == 0) return 0;
    return mnb::int8_workspace_bytes(a_dtype, m, K, N);
}

int matmul_int8(const void* A, int a_dtype, const float* a_scales, int64_t m, int64_t K, int64_t N,
                const int8_t* B, const float* b_scales, const float* bias, void* out, int out_dtype,
                void* workspace, size_t workspace_bytes, void* stream)
{
    int st = check_int8_shape(a_dtype, m, K, N);
    if (st != MNB_OK) return st;
    if (out_dtype != MNB_F16 && out_dtype != MNB_BF16) return MNB_ERR_DTYPE;
    if (m == 0 || N == 0) return finish_launches(0, 0);
    const bool rows8 = a_dtype == MNB_I8;
    if (!out || !b_scales || (K > 0 && (!A || !B)) || (rows8 && !a_scales)) return MNB_ERR_NULL;
    if (((uintptr_t)A & 15) || ((uintptr_t)B & 15) || ((uintptr_t)a_scales & 3) || ((uintptr_t)b_scales & 3) ||
        ((uintptr_t)bias & 3) || ((uintptr_t)out & 1) || ((uintptr_t)workspace & 15))
        return MNB_ERR_ALIGN;
    const size_t need = mnb::int8_workspace_bytes(a_dtype, m, K, N);
    if (need && !workspace) return MNB_ERR_NULL;
    if (need > workspace_bytes) return MNB_ERR_WORKSPACE;
    const Span in[] = {{A, m * K * (rows8 ? 1 : 2)}, {rows8 ? a_scales : nullptr, m * 4}, {B, N * K},
                       {b_scales, N * 4}, {bias, N * 4}};
    const Span wr[] = {{out, m * N * 2}, {workspace, (int64_t)need}};
    if (aliased(in, 5, wr, 2)) return MNB_ERR_ALIAS;
    if (!mnb::launch_int8) return finish_launches(kNoDevice, 0);
    const mnb::Int8Args args{A, a_scales, B, b_scales, bias, out, m, K, N, a_dtype, out_dtype == MNB_BF16, workspace};
    int launches = 0;
    const int e = mnb::launch_int8(args, stream, &launches);
    if (log_enabled())
        fprintf(stderr, "mnb: matmul_int8 m=%lld K=%lld N=%lld a=%s out=%s bias=%d launches=%d\n", (long long)m,
                (long long)K, (long long)N, dtype_name(a_dtype), dtype_name(out_dtype), bias != nullptr, launches);
    return finish_launches(e, launches);
}

size_t mnb_moe_workspace(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int top_k)
{
    if (check_moe_shape(tokens, hidden, inter, experts, top_k) != MNB_OK || tokens == 0) return 0;
    return mnb::moe_layout(tokens, hidden, inter, experts, top_k).bytes;
}

int moe_nbits(const void* x, int x_dtype, int64_t tokens, const void* router_logits, int logits_dtype, int top_k,
              int renormalize, const mnb_moe_weights* weights, void* out, int out_dtype, int32_t* expert_ids,
              float* expert_weights, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!weights) return MNB_ERR_NULL;
    const mnb_moe_weights& w = *weights;
    int st = check_moe_shape(tokens, w.hidden, w.inter, w.experts, top_k);
    if (st != MNB_OK) return st;
    if (w.block != 32) return MNB_ERR_BLOCK;
    if ((x_dtype != MNB_F16 && x_dtype != MNB_BF16) || (out_dtype != MNB_F16 && out_dtype != MNB_BF16) ||
        (logits_dtype != MNB_F32 && logits_dtype != MNB_F16 && logits_dtype != MNB_BF16))
        return MNB_ERR_DTYPE;
    if (tokens == 0) return finish_launches(0, 0);
    if (!x || !router_logits || !w.gate_up || !w.gate_up_scales || !w.down || !w.down_scales || !out || !workspace)
        return MNB_ERR_NULL;
    const int64_t lsize = logits_dtype == MNB_F32 ? 4 : 2;
    if (((uintptr_t)x & 15) || ((uintptr_t)router_logits & (lsize - 1)) || ((uintptr_t)w.gate_up & 15) ||
        ((uintptr_t)w.gate_up_scales & 1) || ((uintptr_t)w.down & 15) || ((uintptr_t)w.down_scales & 1) ||
        ((uintptr_t)out & 1) || ((uintptr_t)expert_ids & 3) || ((uintptr_t)expert_weights & 3) ||
        ((uintptr_t)workspace & 15))
        return MNB_ERR_ALIGN;
    const size_t need = mnb::moe_layout(tokens, w.hidden, w.inter, w.experts, top_k).bytes;
    if (need > workspace_bytes) return MNB_ERR_WORKSPACE;
    const int64_t E = w.experts, H = w.hidden, I = w.inter, hb = H / 32, ib = I / 32;
    const Span in[] = {{x, tokens * H * 2}, {router_logits, tokens * E * lsize},
                       {w.gate_up, E * I * H}, {w.gate_up_scales, E * 2 * I * hb * 2},
                       {w.gate_up_zero_points, E * 2 * I * ((hb + 1) / 2)},
                       {w.down, E * H * (I / 2)}, {w.down_scales, E * H * ib * 2},
                       {w.down_zero_points, E * H * ((ib + 1) / 2)}};
    const Span wr[] = {{out, tokens * H * 2}, {expert_ids, tokens * top_k * 4}, {expert_weights, tokens * top_k * 4},
                       {workspace, (int64_t)need}};
    if (aliased(in, 8, wr, 4)) return MNB_ERR_ALIAS;
    if (!mnb::launch_moe) return finish_launches(kNoDevice, 0);
    const mnb::MoeArgs args{x, router_logits, w, out, expert_ids, expert_weights, (int32_t)tokens, top_k,
                            x_dtype == MNB_BF16, logits_dtype, renormalize != 0, out_dtype == MNB_BF16, workspace};
    int launches = 0;
    const int e = mnb::launch_moe(args, stream, &launches);
    if (log_enabled())
        fprintf(stderr, "mnb: moe_nbits tokens=%lld hidden=%lld inter=%lld experts=%lld top_k=%d x=%s logits=%s "
                "out=%s launches=%d\n", (long long)tokens, (long long)H, (long long)I, (long long)E, top_k,
                dtype_name(x_dtype), dtype_name(logits_dtype), dtype_name(out_dtype), launches);
    return finish_launches(e, launches);
}

int append_kv_int8(const mnb_kv_cache* cache, const mnb_kv_batch* batch, int dtype, const void* k, int64_t k_stride,
                   const void* v, int64_t v_stride, const void* q, int64_t q_stride, void* q_out,
                   int64_t q_out_stride, int64_t q_heads, const float* cos, const float* sin, int64_t rot_dim,
                   int64_t table_rows, int interleaved, void* stream)
{
    if (!cache || !batch) return MNB_ERR_NULL;
    const mnb_kv_cache& c = *cache;
    const mnb_kv_batch& b = *batch;
    int st = check_kv(c, b);
    if (st != MNB_OK) return st;
    const int64_t H = c.kv_heads, D = c.head_dim, P = c.page_size, T = b.tokens;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 || q_heads < 0 || q_heads > MNB_KV_MAX_HEADS * MNB_KV_MAX_GROUP ||
        (rot_dim > 0 && table_rows < b.max_pages * P) || bad_stride(k_stride, H, D, T) ||
        bad_stride(v_stride, H, D, T) || (q_heads && (bad_stride(q_stride, q_heads, D, T) ||
                                                      bad_stride(q_out_stride, q_heads, D, T))))
        return MNB_ERR_SHAPE;
    if (dtype != MNB_F16 && dtype != MNB_BF16) return MNB_ERR_DTYPE;
    if (T == 0 || b.sequences == 0 || b.max_pages == 0) return finish_launches(0, 0);
    st = check_kv_pointers(c, b);
    if (st == MNB_ERR_NULL || !k || !v || (q_heads > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr) ||
        (rot_dim > 0 && (!cos || !sin)))
        return MNB_ERR_NULL;
    if (st != MNB_OK || ((uintptr_t)k & 15) || ((uintptr_t)v & 15) || ((uintptr_t)q & 15) || ((uintptr_t)q_out & 15) ||
        (rot_dim > 0 && (((uintptr_t)cos & 15) || ((uintptr_t)sin & 15))))
        return MNB_ERR_ALIGN;
    const Rows kr{k, T, H * D * 2, k_stride * 2}, vr{v, T, H * D * 2, v_stride * 2},
        qr{q, T, q_heads * D * 2, q_stride * 2}, qo{q_out, T, q_heads * D * 2, q_out_stride * 2};
    const Span tables = {rot_dim ? cos : nullptr, table_rows * (rot_dim / 2) * 4},
               tables2 = {rot_dim ? sin : nullptr, table_rows * (rot_dim / 2) * 4};
    const Span in[] = {span_of(kr), span_of(vr), span_of(qr), tables, tables2, {b.starts, (b.sequences + 1) * 4},
                       {b.lengths, b.sequences * 4}, {b.page_table, b.sequences * b.max_pages * 4}};
    const int64_t each = c.pages * H;
    const Span wr[] = {{c.k_pages, each * P * D}, {c.v_pages, each * P * D}, {c.k_scales, each * 4},
                       {c.v_scales, each * 4}};
    const Span qw[] = {span_of(qo)};
    if (aliased(in, 8, wr, 4) || aliased(in + 3, 5, qw, 1) || aliased(wr, 4, qw, 1)) return MNB_ERR_ALIAS;
    const bool in_place = q && q_out == q && (T == 1 || q_out_stride == q_stride);
    if (q && (rows_overlap(qo, kr) || rows_overlap(qo, vr) || (!in_place && rows_overlap(qo, qr)))) return MNB_ERR_ALIAS;
    if (log_enabled())
        fprintf(stderr, "mnb: append_kv_int8 sequences=%lld tokens=%lld heads=%lld q_heads=%lld dim=%lld page=%lld "
                "rot=%lld type=%s launches=1\n", (long long)b.sequences, (long long)T, (long long)H,
                (long long)q_heads, (long long)D, (long long)P, (long long)rot_dim, dtype_name(dtype));
    if (!mnb::launch_append) return finish_launches(kNoDevice, 0);
    const mnb::AppendArgs args{c, b, k, v, q, q_out, k_stride, v_stride, q_stride, q_out_stride, q_heads, rot_dim,
                               cos, sin, dtype == MNB_BF16, interleaved != 0};
    return finish_launches(mnb::launch_append(args, stream), 1);
}

size_t mnb_attention_workspace(int64_t tokens, int64_t sequences, int64_t q_heads, int64_t kv_heads, int64_t head_dim)
{
    const mnb_kv_cache c{0, 16, kv_heads, head_dim, nullptr, nullptr, nullptr, nullptr};
    const mnb_kv_batch b{sequences, tokens, 0, nullptr, nullptr, nullptr};
    if (check_kv(c, b) != MNB_OK || !good_group(q_heads, kv_heads) || tokens == 0 || sequences == 0) return 0;
    return mnb::attention_layout(tokens, sequences, q_heads, kv_heads, head_dim).bytes;
}

int attention_int8(const mnb_kv_cache* cache, const mnb_kv_batch* batch, int dtype, const void* q, int64_t q_stride,
                   int64_t q_heads, float scale, void* out, int64_t out_stride, int64_t max_tokens, void* workspace,
                   size_t workspace_bytes, void* stream)
{
    if (!cache || !batch) return MNB_ERR_NULL;
    const mnb_kv_cache& c = *cache;
    const mnb_kv_batch& b = *batch;
    int st = check_kv(c, b);
    if (st != MNB_OK) return st;
    const int64_t H = c.kv_heads, D = c.head_dim, P = c.page_size, T = b.tokens;
    if (!good_group(q_heads, H) || bad_stride(q_stride, q_heads, D, T) || bad_stride(out_stride, q_heads, D, T) ||
        max_tokens < 0 || !std::isfinite(scale))
        return MNB_ERR_SHAPE;
    if (dtype != MNB_F16 && dtype != MNB_BF16) return MNB_ERR_DTYPE;
    if (T == 0 || b.sequences == 0) return finish_launches(0, 0);
    st = check_kv_pointers(c, b);
    if (st == MNB_ERR_NULL || !q || !out || !workspace) return MNB_ERR_NULL;
    if (st != MNB_OK || ((uintptr_t)q & 15) || ((uintptr_t)out & 15) || ((uintptr_t)workspace & 15))
        return MNB_ERR_ALIGN;
    const size_t need = mnb::attention_layout(T, b.sequences, q_heads, H, D).bytes;
    if (need > workspace_bytes) return MNB_ERR_WORKSPACE;
    const int64_t each = c.pages * H;
    const Rows qr{q, T, q_heads * D * 2, q_stride * 2}, orow{out, T, q_heads * D * 2, out_stride * 2};
    const Span in[] = {{c.k_pages, each * P * D}, {c.v_pages, each * P * D}, {c.k_scales, each * 4},
                       {c.v_scales, each * 4}, {b.starts, (b.sequences + 1) * 4}, {b.lengths, b.sequences * 4},
                       {b.page_table, b.sequences * b.max_pages * 4}};
    const Span wr[] = {span_of(orow), {workspace, (int64_t)need}}, qs[] = {span_of(qr)};
    if (aliased(in, 7, wr, 2) || aliased(qs, 1, wr + 1, 1) || rows_overlap(orow, qr)) return MNB_ERR_ALIAS;
    if (!mnb::launch_attention) return finish_launches(kNoDevice, 0);
    mnb_kv_batch seen = b;
    if (c.pages == 0) seen.max_pages = 0;      // no token stands anywhere: nothing of the cache is read
    const mnb::AttentionArgs args{c, seen, q, out, q_stride, out_stride, q_heads, max_tokens, scale, dtype == MNB_BF16,
                                  workspace};
    int launches = 0;
    const int e = mnb::launch_attention(args, stream, &launches);
    if (log_enabled())
        fprintf(stderr, "mnb: attention_int8 sequences=%lld tokens=%lld heads=%lld q_heads=%lld dim=%lld page=%lld "
                "type=%s launches=%d\n", (long long)b.sequences, (long long)T, (long long)H, (long long)q_heads,
                (long long)D, (long long)P, dtype_name(dtype), launches);
    return finish_launches(e, launches);
}

size_t mnb_lora_workspace(int64_t m, int64_t K, int64_t N, int64_t rank, int64_t adapters)
{
    if (check_lora_shape(m, K, N, rank, adapters) != MNB_OK || m == 0 || N == 0) return 0;
    return mnb::lora_layout(m, K, N, rank, adapters).bytes;
}

int matmul_lora(const void* x, int x_dtype, int64_t x_stride, int64_t m, int64_t K, int64_t N, int64_t rank,
                int64_t adapters, const int32_t* ids, const void* A, const void* B, const float* scaling,
                const void* base, int64_t base_stride, void* out, int64_t out_stride, int out_dtype, void* workspace,
                size_t workspace_bytes, void* stream)
{
    int st = check_lora_shape(m, K, N, rank, adapters);
    if (st != MNB_OK) return st;
    const int64_t most = (int64_t)1 << 40;
    if (K == 0) x_stride = 0;      // rows of nothing, wherever they are said to be
    if (m > 1 && (x_stride < K || x_stride % 8 || x_stride > most || out_stride < N || out_stride > most ||
                  (base && (base_stride < N || base_stride > most))))
        return MNB_ERR_SHAPE;
    if ((x_dtype != MNB_F16 && x_dtype != MNB_BF16) || (out_dtype != MNB_F16 && out_dtype != MNB_BF16))
        return MNB_ERR_DTYPE;
    if (m == 0 || N == 0) return finish_launches(0, 0);
    if (!out || !ids || !workspace || (adapters > 0 && (!B || (K > 0 && (!x || !A))))) return MNB_ERR_NULL;
    if (((uintptr_t)x & 15) || ((uintptr_t)A & 15) || ((uintptr_t)B & 15) || ((uintptr_t)ids & 3) ||
        ((uintptr_t)scaling & 3) || ((uintptr_t)base & 1) || ((uintptr_t)out & 1) || ((uintptr_t)workspace & 15))
        return MNB_ERR_ALIGN;
    const size_t need = mnb::lora_layout(m, K, N, rank, adapters).bytes;
    if (need > workspace_bytes) return MNB_ERR_WORKSPACE;
    const Rows xr{x, m, K * 2, x_stride * 2}, br{base, m, N * 2, base_stride * 2}, orow{out, m, N * 2, out_stride * 2};
    const Span in[] = {{ids, m * 4}, {A, adapters * rank * K * 2}, {B, adapters * N * rank * 2}, {scaling, adapters * 4},
                       span_of(xr), span_of(br)};
    const Span wr[] = {span_of(orow), {workspace, (int64_t)need}};
    const bool in_place = base == out && (m == 1 || base_stride == out_stride);
    if (aliased(in, 4, wr, 2) || aliased(in + 4, 2, wr + 1, 1) || rows_overlap(orow, xr) ||
        (base && !in_place && rows_overlap(orow, br)))
        return MNB_ERR_ALIAS;
    if (!mnb::launch_lora) return finish_launches(kNoDevice, 0);
    const mnb::LoraArgs args{x, ids, A, B, scaling, base, out, x_stride, base_stride, out_stride, m, K, N, rank,
                             adapters, x_dtype == MNB_BF16, out_dtype == MNB_BF16, workspace};
    int launches = 0;
    const int e = mnb::launch_lora(args, stream, &launches);
    if (log_enabled())
        fprintf(stderr, "mnb: matmul_lora m=%lld K=%lld N=%lld rank=%lld adapters=%lld x=%s out=%s launches=%d\n",
                (long long)m, (long long)K, (long long)N, (long long)rank, (long long)adapters, dtype_name(x_dtype),
                dtype_name(out_dtype), launches);
    return finish_launches(e, launches);
}

void mnb_counters_get(mnb_counters* out)
{
    if (!out) return;
    out->calls = g_calls.load();
    out->launches = g_launches.load();
    out->elements_f16 = g_f16.load();
    out->elements_bf16_direct = g_bf16.load();
    out->row_batched_launches = g_rows.load();
}

void mnb_counters_reset(void)
{
    g_calls = 0;
    g_launches = 0;
    g_f16 = 0;
    g_bf16 = 0;
    g_rows = 0;
}

int mnb_get_kernel_info(int64_t m, int64_t K, const mnb_plan* plan, mnb_kernel_info* info)
{
    if (!plan || !info) return MNB_ERR_NULL;
    mnb_plan p = *plan;
    if (p.workgroups < 1) p.workgroups = 1;
    if (mnb_plan_check(m, K, 1, &p) != MNB_OK) return MNB_ERR_PLAN;
    int e = mnb::kernel_info(p.engine == 2 ? m : std::min<int64_t>(m, MNB_MAX_M), K, p, info);
    if (e == -1) return MNB_ERR_PLAN;
    if (e != 0) {
        t_last_hip_error = e;
        return MNB_ERR_HIP;
    }
    return MNB_OK;
}

const char* mnb_status_string(int status)
{
    switch (status) {
    case MNB_OK: return "ok";
    case MNB_ERR_NULL: return "a required pointer is NULL";
    case MNB_ERR_SHAPE: return "bad shape (matmul_nbits: K must be a non-negative multiple of 32, N >= 0, within limits)";
    case MNB_ERR_BLOCK: return "block size must be 32";
    case MNB_ERR_DTYPE: return "an element type the call does not take (matmul_nbits: MNB_F16 or MNB_BF16)";
    case MNB_ERR_ALIGN: return "a buffer is not aligned (matmul_nbits: A and Bpacked to 16 bytes, scales and out to 2)";
    case MNB_ERR_M_RANGE: return "m (or the tokens of a batch) must be in [0, MNB_MAX_ROWS], tokens of the expert layer in [0, MNB_MOE_MAX_TOKENS]";
    case MNB_ERR_HIP: return "HIP runtime error (see mnb_last_hip_error)";
    case MNB_ERR_ALIAS: return "a written buffer overlaps an input or another written buffer";
    case MNB_ERR_PLAN: return "launch plan not supported";
    case MNB_ERR_LAYOUT: return "unknown weight layout";
    case MNB_ERR_WORKSPACE: return "the call needs more workspace than it was given (matmul_nbits_noalloc: than its fixed buffer holds)";
    }
    return "unknown status";
}

int mnb_last_hip_error(void) { return t_last_hip_error; }

int mnb_abi_version(void) { return MNB_ABI_VERSION; }

}  // extern "C"
