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

// The paged 8-bit cache: appending (mnb_append.hip) and attention over it
// (mnb_attention.hip).  Arguments have passed the front end's checks; tokens,
// sequences, max_pages > 0.
struct AppendArgs {
    mnb_kv_cache cache;
    mnb_kv_batch batch;
    const void* k;
    const void* v;
    const void* q;           // or null
    void* q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride, q_heads, rot_dim;
    const float* cos;
    const float* sin;
    int bf16, interleaved;
};
int launch_append(const AppendArgs& args, void* stream) MNB_WEAK;

// Page slots of the appending grid: a token touches one page, a sequence of n tokens
// at most floor((n - 1) / P) + 2 (slot_base in mnb_append.hip).
constexpr int64_t append_slots(int64_t page_size, int64_t tokens, int64_t sequences)
{
    const int64_t loose = tokens / page_size + 2 * sequences;
    return tokens <= loose ? tokens : loose;
}

// Workgroups of one wave, or of four.  One where a page gets 16 tokens or fewer on
// average, whose few units would leave the other waves none; and where there are
// enough workgroups for two rounds of waves and a wave holds what a page gets (4096
// elements) between its two looks at it.  8 heads of 128, one / four waves: 64
// sequences of one token 7.7 / 9.7 us, 200 of 32 on pages of 64 34 / 44, 4 of 1800 43 /
// 37, one of 64 16.0 / 7.0.  Against the times of both over 341 batches: 0.6% above the
// faster on average (tests/data/kv_rules_gfx950.json).
constexpr bool append_one_wave(int64_t page_size, int64_t tokens, int64_t sequences, int64_t heads, int64_t head_dim)
{
    const int64_t each = tokens / sequences < page_size ? tokens / sequences : page_size;
    return page_size <= 16 || tokens <= 16 * sequences ||
           (append_slots(page_size, tokens, sequences) * 2 * heads >= 1024 && each * head_dim <= 4096);
}

struct AttentionArgs {
    mnb_kv_cache cache;
    mnb_kv_batch batch;
    const void* q;
    void* out;
    int64_t q_stride, out_stride, q_heads, max_tokens;
    float scale;
    int bf16;
    void* ws;                // attention_layout().bytes
};
int launch_attention(const AttentionArgs& args, void* stream, int* launches) MNB_WEAK;

// Sequences of more rows (tokens times query heads of a key head) than this go to
// tiles of tile_rows() rows, the others to a fixed number of workgroups.  The tiles'
// workgroups take long to begin and end; the others read the keys once for every 16
// rows.  (8 heads of 128, one sequence of 256 rows over 1024 / 8192 / 32768 keys: 16 /
// 36 / 102 us against tiles' 29 / 38 / 70, of 128 rows 13 / 26 / 61 against 27 / 34 /
// 65; 16 sequences of 96 rows 48 / 242 / 904 against 55 / 205 / 785.  Heads of 256, one
// sequence over 1024 / 8192 keys: 96 rows 16 / 52 against 39 / 43, 256 rows 31 / 81
// against 45 / 62.)
constexpr int attention_many_rows(int64_t tokens, int64_t q_heads, int64_t head_dim)
{
    return tokens * q_heads > 2048 ? 64 : head_dim <= 128 ? 256 : 128;
}
constexpr int kAttentionWorkgroups = 512;     // (256 / 512 / 1024: 64 sequences over 1000 keys 29 / 27 / 34 us, one over 131072 48 / 49 / 54)
// Units that a row tile's begin and end count as in a share.  (2 / 4 / 8: one token over
// 2049 keys 13.0 / 10.5 / 10.5 us, 7 sequences over 999 10.7 / 12.4 / 12.5; 11.3 / 3.8 / 5.3%
// above the fastest of seven on average over 30 batches.)
constexpr int kAttentionBegin = 4;
constexpr int tile_waves(int64_t head_dim) { return head_dim >= 128 ? 8 : 4; }
constexpr int tile_rows(int64_t head_dim) { return head_dim == 128 ? 256 : 128; }
constexpr int tile_shares(int64_t head_dim) { return head_dim == 64 ? 512 : 256; }   // workgroups that run at a time

// Few tiles of many rows are cut into equal shares of the whole batch's work, a
// workgroup each, unless whole tiles take no longer (32 heads on 8 of 128: 512 tokens over
// 17000 keys whole 685 us, cut 207; 5000 over 20000 2109, 1868; 300 over their own 22, 33;
// 4096 over their own 190, 224).  all: their work, in 1 / G of a key; longest: a tile's.
// Whole tiles take rounds of them where all are about as long; else the longest first,
// and short ones behind them.  Units that a tile's begin and end count as, that a share has
// at least, that the second tile of a share and the joining launch cost more than whole
// tiles do:
constexpr int kTileBegin = 4, kTileLeast = 2, kTileMore = 4, kTileJoin = 10;
constexpr int64_t tile_share(int64_t share, int64_t G) { return share < 64 * G * kTileLeast ? 64 * G * kTileLeast : share; }
template <class Divide>
constexpr bool tiles_cut(int64_t all, int64_t tiles, int64_t longest, int64_t G, int64_t shares, int64_t share, Divide divide)
{
    const int64_t mixed = divide(all, shares) + (longest >> 3);
    const int64_t whole = 2 * longest * tiles <= 3 * all ? divide(tiles + shares - 1, shares) * longest
                          : longest > mixed              ? longest
                                                         : mixed;
    return whole > share + 64 * G * kTileMore + divide(64 * G * kTileJoin * all, share * shares);
}

// The attention's workspace.  Few rows: for each workgroup the sums of two row
// tiles that it shares with others, behind their maxima and weights.  Many: the
// tiles there can be; where they are few, the workgroups that may share them (else
// 0) and the same sums of two tiles for each.  Host-only arithmetic (mnb_api.cpp).
struct AttentionLayout {
    int many, tile_slots, shares;
    size_t o, tile_ml, tile_o, bytes;
};
AttentionLayout attention_layout(int64_t tokens, int64_t sequences, int64_t q_heads, int64_t kv_heads, int64_t head_dim);

// Low-rank adapters (mnb_lora.hip).  Arguments have passed the front end's
// checks; m, N > 0.
struct LoraArgs {
    const void* x;           // [m][K]
    const int32_t* ids;      // [m]
    const void* A;           // [adapters][R][K]
    const void* B;           // [adapters][N][R]
    const float* scaling;    // [adapters] or null
    const void* base;        // [m][N] or null
    void* out;               // [m][N]
    int64_t x_stride, base_stride, out_stride, m, K, N, R, adapters;
    int bf16, out_bf16;
    void* ws;                // lora_layout().bytes
};
int launch_lora(const LoraArgs& args, void* stream, int* launches) MNB_WEAK;

// Row tiles of 16 of a workgroup, slices of K of the first launch and their
// length, workgroups that share the adapters of a tile in it, whether the second
// launch takes 64 columns a wave (or 16), and the workspace that holds the
// slices' sums.  Host-only arithmetic (mnb_api.cpp).
struct LoraLayout {
    int down_tiles, up_tiles;    // of 16 rows, a workgroup's
    int splits, k_slice, ways;
    bool wide;
    size_t bytes;
};
// Workgroups that the first launch is divided into, two a compute unit.  (Half as many
// 0.2%, these 1.0%, twice as many 1.0% above the fastest on average over 24 shapes.)
constexpr int kLoraDownWorkgroups = 512;
LoraLayout lora_layout(int64_t m, int64_t K, int64_t N, int64_t R, int64_t adapters);

}  // namespace mnb
