// Internal interface between the host front end (mnb_api.cpp, plain C++)
// and the HIP side (mnb_gemv.hip and the other .hip files).  Not installed; not part of the C ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "mnb.h"

namespace mnb {

struct GemvArgs {
    const void* A;
    const uint8_t* B;
    const uint16_t* scales;
    const uint8_t* zp;      // may be null: every zero point is 8
    void* out;
    int64_t m, K, N;
    int a_bf16, out_bf16;
    void* ws;               // device workspace of workspace_bytes(), or null
};

// Queue one GEMV launch.  `plan` has passed mnb_plan_check.  Returns the
// hipError_t of the launch (0 on success).  Dispatches on plan.engine.
int launch_gemv(const GemvArgs& args, const mnb_plan& plan, void* stream);

// The 4x4x4 MFMA kernel (engine 3), mnb_gemv_mfma4.hip: W waves per
// workgroup whose 16 W lane groups cover K in one pass (16 W * blocks_per_lane
// >= K/32), cols_per_tile = 4 or 8.  With plan.a_via_lds, dynamic LDS of 4160
// bytes per wave, through which the activations reach their lanes.
int launch_mfma4(const GemvArgs& args, const mnb_plan& plan, void* stream);
int mfma4_workgroups_per_cu(int64_t m, int64_t K, const mnb_plan& plan);
int mfma4_kernel_info(int64_t m, int64_t K, const mnb_plan& plan, mnb_kernel_info* info);

// The prefill kernel (engine 2), mnb_gemm_mfma.hip: a workgroup of 4 or 8
// waves owns 32 * row_tiles rows by cols_per_tile columns (4 waves: 128 or
// 256 columns, 32 or 64 per wave; 8 waves: 256 columns, 32 per wave).
// A workgroup's activation rows (32 * row_tiles rows of K fp16) are
// addressed with 32-bit buffer offsets: 64 * row_tiles * K must stay within
// this many bytes.
constexpr uint64_t kPrefillRowBlockBytes = 0xFFFFFFF0u;
// With plan.k_splits > 1 the workgroups each take one of k_splits slices of
// K and leave fp32 partial sums in args.ws; a second launch adds them in
// slice order and stores the narrowed result.
int launch_gemm(const GemvArgs& args, const mnb_plan& plan, void* stream);
int gemm_workgroups_per_cu(const mnb_plan& plan);
int gemm_kernel_info(const mnb_plan& plan, mnb_kernel_info* info);
size_t gemm_lds_bytes(const mnb_plan& plan);

// Weight-layout conversion (mnb_layout.hip): `words` 32-bit words of packed
// weights from src_layout to dst_layout.  Returns a hipError_t.
int launch_repack(const uint8_t* src, int src_layout, uint8_t* dst, int dst_layout, int64_t words,
                  void* stream);

// Device workspace a launch under `plan` needs for m x N outputs: the fp32
// partial sums of a K split over workgroups (k_splits x m x N x 4 bytes),
// else 0.  Host-only arithmetic (mnb_api.cpp).
size_t workspace_bytes(int64_t m, int64_t N, const mnb_plan& plan);

// The library's workspace for launches on `stream` (a buffer per device and
// stream, kept for the process and grown with hipMalloc when a call needs
// more): on success (0) the buffer is held until workspace_release(), which
// must follow once the launches that use it are queued; otherwise a
// hipError_t and nothing is held.
int workspace_acquire(size_t bytes, void* stream, void** ptr);
void workspace_release();

// The fixed workspace of matmul_nbits_noalloc: a file-scope device array of
// kScratchBytes in mnb_gemv.hip, one per device for the life of the process.
// Its device address on the current device, looked up (hipGetSymbolAddress)
// on the first call per device.  Returns a hipError_t.
constexpr size_t kScratchBytes = MNB_MAX_SPLIT_WORKSPACE;
int scratch_address(void** ptr);

// Compute units of the current device.  Returns a hipError_t.
int current_device_cus(int* num_cus);

// Occupancy-limited workgroups per CU of kernel `fn` at a block size and
// dynamic LDS size (0 if the query fails).  Cached per (device, kernel,
// threads, LDS).
int occupancy(const void* fn, int threads, size_t lds);

// Occupancy-limited workgroups per CU for the kernel a plan selects, with
// the LDS it needs for N columns (0 if the query fails).
int workgroups_per_cu(int64_t m, int64_t K, int64_t N, const mnb_plan& plan);

// Dynamic LDS of a lane-split launch (engine 0) over N columns.  Multi-wave
// groups keep every wave's partial sums of all their tiles in LDS and sum
// them over waves once, at the end (*tcap = tiles per group), when that
// fits kDeferLdsBytes; otherwise they sum after each tile through two
// slots (*tcap = 0).  One-wave groups with K in one pass stage the
// workgroup's activations (m * blocks_per_lane * 4 KB); groups inside a
// wave need none.  Host-only.
constexpr int64_t kDeferLdsBytes = 48 * 1024;
int64_t gemv_lds_bytes(int64_t m, int64_t N, const mnb_plan& plan, int32_t* tcap);

// Code-object facts of the variant (m, K and the plan select it).  Returns a hipError_t, or -1 when no
// variant matches.
int kernel_info(int64_t m, int64_t K, const mnb_plan& plan, mnb_kernel_info* info);

// The launchers below are weak: a build of the front end alone (the host-only
// builds of the tests) links without them, and its calls report that no
// device is present.
#define MNB_WEAK __attribute__((weak))

// 8-bit products (mnb_int8.hip).  Arguments have passed the front end's
// checks; m, N > 0.  Each returns a hipError_t and, in *launches, the kernels
// it queued.
struct Int8Args {
    const void* A;           // [m][K], a_dtype
    const float* a_scales;   // [m] with MNB_I8 rows
    const int8_t* B;         // [N][K]
    const float* b_scales;   // [N]
    const float* bias;       // [N] or null
    void* out;               // [m][N]
    int64_t m, K, N;
    int a_dtype, out_bf16;
    void* ws;                // int8_workspace_bytes()
};
int launch_quantize_rows(const void* A, int a_bf16, int64_t m, int64_t K, int8_t* q, float* scales, void* stream)
    MNB_WEAK;
int launch_int8(const Int8Args& args, void* stream, int* launches) MNB_WEAK;

// Threads of a row and pieces of each when rows are quantised: 64 x 1, 256 x 1,
// 256 x 8, 1024 x 1 or 1024 x 4.  Host-only arithmetic (mnb_api.cpp).
int quantize_variant(int64_t m, int64_t K);

// The kernel for few rows takes up to 16 of them where they fit its LDS with
// the sums of its (at most 16) waves, and K up to 16 waves of eight 128-byte
// units.
constexpr int64_t kInt8RowsK = 16 * 8 * 128;
constexpr size_t kInt8RowsLds = 160 * 1024 - 128;
// Whether it also quantises fp16 or bf16 rows itself, in one launch: every
// workgroup then reads all of them.  One launch against two (us of kernels; a
// launch more costs 2 or 3 us besides): 4096 x 4096 with 1 row 8.6 against 2.5 +
// 6.4, with 8 rows 11.1 against 3.4 + 7.2, with 16 12.4 against 3.4 + 7.7; 14336
// x 4096 with 1 row 21.5 against 4.1 + 15.6, with 4 rows 23.9 against 4.1 + 16.3.
constexpr int64_t kInt8FusedElements = 32768;
static_assert(kInt8FusedElements + 16 * 16 + 16 * 2048 <= kInt8RowsLds, "fused rows always go to the kernel for few rows");
inline size_t int8_rows_lds(int64_t m, int64_t K, int waves) { return (size_t)(m * (K + 16)) + (size_t)waves * 2048; }
inline bool int8_fused(int a_dtype, int64_t m, int64_t K)
{
    return a_dtype != MNB_I8 && m <= 16 && K <= kInt8RowsK && m * K <= kInt8FusedElements;
}

// The kernel of an 8-bit product on a device of `cus` compute units.
// Host-only arithmetic (mnb_api.cpp).
struct Int8Route {
    int tile;             // number of the tile (launch_int8), or -1: few rows
    int waves, nu;        // few rows: waves, and 128-byte units of K of each
    int64_t workgroups;   // few rows
    bool fused;           // the kernel quantises the rows itself
};
Int8Route int8_route(int a_dtype, int64_t m, int64_t K, int64_t N, int cus);

// Workspace of an 8-bit product: the quantised rows and their scales where the
// rows come as fp16 or bf16.  Host-only arithmetic (mnb_api.cpp).
size_t int8_workspace_bytes(int a_dtype, int64_t m, int64_t K, int64_t N);

// The expert layer (mnb_moe.hip).
struct MoeArgs {
    const void* x;           // [T][H]
    const void* logits;      // [T][E]
    mnb_moe_weights w;
    void* out;               // [T][H]
    int32_t* ids;            // [T][top_k] or null
    float* probs;            // [T][top_k] or null
    int32_t T, top_k;
    int x_bf16, logits_dtype, renormalize, out_bf16;
    void* ws;                // moe_layout().bytes
};
int launch_moe(const MoeArgs& args, void* stream, int* launches) MNB_WEAK;

// Layout of the expert layer's workspace (byte offsets; the head, the count
// of batches and a word per token, comes first) and the row quads of a batch.
// Host-only arithmetic (mnb_api.cpp).
struct MoeLayout {
    int wide;                // 0: the narrow kernels; 1, 2: the wide ones with 16 or 32 rows
    int rq, batches;         // row quads of a batch; the most batches there can be
    size_t batch_e, row_token, row_p, hs, h, pair_row, xs, xe, hf, y, bytes;
};
MoeLayout moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int top_k);

// LDS of a workgroup, of the first narrow launch that the kernel declares (two
// units' partial sums, the waves' scales, the rows' powers of two), and of the
// routing tables.
constexpr int64_t kMoeLds = 160 * 1024;
constexpr int kMoeUpWaves = 8;
constexpr uint32_t moe_up_static_lds(int rq) { return 2 * kMoeUpWaves * 64 * rq * 4 + kMoeUpWaves * 640 + 16 * rq; }
constexpr uint32_t moe_routing_bytes(int E, int pairs, int cap, int rq)
{
    return (uint32_t)(8 * E + 4 * pairs + 4 * cap * rq + 2 * E + 2 * pairs + 2 * cap + 15) & ~15u;
}

// The variants of its kernels on a device of `cus` compute units.  Host-only
// arithmetic (mnb_api.cpp).
struct MoeRoute {
    int up_vec, down_vec;   // blocks whose scales one load brings
    int stage_blocks;       // narrow: blocks of K staged in LDS at a time
    int down_quads;         // narrow: column quads of a workgroup of the second launch
};
MoeRoute moe_route(const MoeArgs& args, const MoeLayout& layout, int cus);

}  // namespace mnb
