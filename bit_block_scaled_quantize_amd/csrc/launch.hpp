// Internal host interface between the C-ABI layer (nvfp4_api.hip) and the
// kernel translation units.  Arguments are already validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace nvfp4 {

enum { kLayoutRow = 0, kLayoutCol = 1, kLayoutRowCol = 2, kLayout2D = 3 };

// MX element formats (nvfp4_mx_elem).
enum { kMxE4M3 = 0, kMxE2M1 = 1 };

// Upper bound on the per-workgroup partial maxima of one amax pass; the
// quantize workspace holds exactly these floats, and every quantize
// workgroup reduces them in its prologue.
constexpr int64_t kMaxPartials = 512;
constexpr size_t kQuantWorkspaceBytes = (size_t)kMaxPartials * sizeof(float);

struct QOut {
    uint8_t* codes;
    uint8_t* scales;
    float* ts;
};

hipError_t launch_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ld,
                           int layout, bool sr, uint64_t seed, bool rht, uint64_t hseed,
                           const float* amax_in, float* amax_out, const QOut* out, float* ws,
                           hipStream_t s);

// COL_1D re-quantization of a row-blocked NVFP4 tensor (rows x cols, both
// multiples of 16); out is cols x rows.
hipError_t launch_requantize(const uint8_t* icodes, const uint8_t* iscales, const float* its,
                             int64_t rows, int64_t cols, bool sr, uint64_t seed, bool rht,
                             uint64_t hseed, const float* amax_in, float* amax_out, const QOut* out,
                             float* ws, hipStream_t s);

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, const float* ts,
                             int64_t rows, int64_t cols, bool scale_2d, void* y, bool bf16,
                             int64_t ld, hipStream_t s);

// One GEMM operand as the kernels see it.
struct Operand {
    const uint8_t* codes;   // rows x K/2
    const uint8_t* scales;  // 1D: rows x K/16; 2D: rows/16 x K/16
    const float* ts;        // tensor scale(s)
    int scale_2d;
};

// C (M x N, ldc) = A * B^T; c_bf16 selects the output type.  swiglu: N = 2F,
// C (M x F, BF16) = gate * sigmoid(gate) * up with gate = columns [0, F) and
// up = columns [F, 2F) of A * B^T.
hipError_t launch_gemm(const Operand& A, const Operand& B, int64_t M, int64_t N, int64_t K,
                       void* C, bool c_bf16, int64_t ldc, bool swiglu, void* ws, size_t ws_bytes,
                       hipStream_t s);

// Split of a plain GEMM's last round of tiles along K (workspace for the
// parts' accumulators: `bytes`; split 1: none).  The tiles after t_main, a
// round that would leave compute units idle, are each computed in `split`
// parts by otherwise idle units and summed in part order by a second kernel.
struct GemmSplit {
    int64_t t_main;
    int split;
    int64_t bytes;
};
constexpr int64_t kMaxTailSplit = 8;
GemmSplit gemm_split_plan(int64_t M, int64_t N, int64_t K, bool swiglu, int cus);
// Compute units of the current device.
hipError_t device_cus(int& cus);

// Grouped GEMM over G groups (see nvfp4_grouped_gemm).  n_per_group = rows of
// one group's weight matrix; swiglu halves the output width.
hipError_t launch_grouped_gemm(int G, const Operand& A, const int64_t* offsets, int64_t total_rows,
                               const Operand& B, int64_t n_per_group, int64_t K, void* C,
                               bool c_bf16, int64_t ldc, bool swiglu, float* amax_out,
                               hipStream_t s);

// MX quantization (layout kLayoutRow or kLayoutCol; the block dimension is a
// multiple of 32) into codes / E8M0 scales of the output orientation.
hipError_t launch_mx_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ld, int layout,
                              int elem, bool sr, uint64_t seed, uint8_t* codes, uint8_t* scales,
                              hipStream_t s);

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int elem, int64_t rows,
                                int64_t cols, void* y, bool bf16, int64_t ld, hipStream_t s);

// C (M x N, ldc) = A * B^T for MX operands of one element format; K % 64 == 0.
// exact: every product exact and binary32 accumulation (BF16 matrix cores on
// exactly rescaled elements) instead of the scaled matrix cores.
hipError_t launch_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                          const uint8_t* b_scales, int elem, int64_t M, int64_t N, int64_t K, void* C,
                          bool c_bf16, int64_t ldc, bool exact, void* ws, size_t ws_bytes, hipStream_t s);
// The MX GEMM's split plan (full-line kernels: K % 1024 == 0).
GemmSplit mx_gemm_split_plan(int64_t M, int64_t N, int64_t K, double tile_us, int cus);
// A lone last-round tile's time per 1024 K for this element format and accumulation mode, in µs.
double mx_split_tile_us(int elem, bool exact);

// Workgroups that one launch can hold in a dimension of its grid: the runtime
// takes more than 2^32 - 1 threads without an error, and runs what is left of
// their number in 32 bits.
constexpr int64_t max_blocks(int threads) { return 0xFFFFFFFFll / threads; }

// RMS norm (see nvfp4_rmsnorm); cols in [1, kMaxNormCols], codes NULL for no
// MX output.
constexpr int64_t kMaxNormCols = 32768;
struct RmsNorm {
    const void* x;
    const void* residual;
    const void* weight;
    bool bf16, w_bf16;
    int64_t rows, cols, ldx, ldr, ldh, ldy;
    float eps;
    void* h;
    void* y;
    uint8_t* codes;
    uint8_t* scales;
    int elem;
    float* rstd;
};
hipError_t launch_rmsnorm(const RmsNorm& n, hipStream_t s);

struct RmsNormBackward {
    const void* dy;
    const void* h;
    const void* dh;
    const float* rstd;
    const void* weight;
    bool bf16, w_bf16;
    int64_t rows, cols, lddy, ldh, lddh, lddx;
    void* dx;
    float* dweight;
    float* ws;  // rmsnorm_backward_workspace_floats
};
int64_t rmsnorm_backward_workspace_floats(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_backward(const RmsNormBackward& n, hipStream_t s);

// Expert routing (see nvfp4_route).
constexpr int kMaxExperts = 2048, kMaxTopK = 16, kMaxRouteGroups = 64;
struct RouteShape {
    int experts, groups, group_size, top_groups, top_k;
    int lane_shift;  // a group lies on 2^lane_shift lanes; set by the launcher
    bool group_top2;
};
struct RouteArgs {
    const void* logits;
    bool bf16;
    int64_t tokens, ld;
    const float* bias;
    RouteShape shape;
    bool sigmoid, renorm;
    int* ids;
    float* weights;
    int64_t* offsets;  // NULL: no dispatch plan (order and position unused)
    int* order;
    int* position;
    uint8_t* counts;  // route_workspace_bytes
    int64_t span;      // tokens of a workgroup; set by the launcher, as group is
    int group;         // spans of a workgroup of the second step
};
bool route_shape_fits(int experts, int groups);
size_t route_workspace_bytes(int64_t tokens, int experts);
hipError_t launch_route(RouteArgs a, hipStream_t s);

struct RouteBackward {
    const float* dweights;
    const void* logits;
    const int* ids;
    const float* dscores;  // nullable
    void* dlogits;
    int64_t tokens, ld, ldds, lddl;
    int experts, top_k;
    bool sigmoid, renorm;
};
hipError_t launch_route_backward(const RouteBackward& a, bool bf16, hipStream_t s);

// Products of a few rows with 4-bit weights (see nvfp4_gemv, nvfp4_mx_gemv and
// nvfp4_expert_gemv).
constexpr int64_t kMaxGemvRows = 1024;
constexpr int kMaxGemvAssignments = 1024;
// Rows of a matrix at most: one grid holds 256 threads (of so many tiles, the
// most) for each 32 of them.
constexpr int64_t kMaxGemvCols = ((int64_t)1 << 29) - 32;
static_assert(kMaxGemvCols == 32 * max_blocks(256));
struct GemvArgs {
    const void* x;
    int64_t m, ldx;
    const uint8_t* codes;
    const uint8_t* scales;
    const float* ts;  // NULL: 1
    int64_t N, K;     // one matrix
    void* y;
    int64_t ldy;
    // the routed form (ids NULL: none): assignment i = token * top_k + place
    const int* ids;
    int assignments, top_k, experts;
    bool x_per_assignment;
    bool x_bf16, y_bf16, scale_2d, mx;
    int rows;  // of x at a time; set by the launcher
};
hipError_t launch_gemv(const GemvArgs& p, bool swiglu, hipStream_t s);
// weights NULL: a row of y for each assignment; else their weighted sums, by
// way of ws (assignments x output columns floats).
hipError_t launch_expert_gemv(GemvArgs p, bool swiglu, const float* weights, float* ws, hipStream_t s);

// The paged 4-bit key/value cache (see nvfp4_kv_cache) and the plan of a call
// (nvfp4_kv_plan).
struct KvCache {
    uint8_t* k_codes;
    uint8_t* k_scales;
    uint8_t* v_codes;
    uint8_t* v_scales;
    const float* k_scale;  // NULL: MX
    const float* v_scale;
    int pages, heads, dim;
    bool mx;
};
struct KvPlan {
    const int* table;
    int64_t ld_table;
    const int* lengths;
    const int* offsets;  // NULL: one row a sequence
    int width, page_shift, seqs, rows;
};
// Rows x heads of dim elements each, strides in elements.
struct KvRows {
    const void* data;
    int64_t row, head;
};
constexpr int64_t kMaxKvSeqs = 65536;
// Rows x heads of q of one call (its workgroups, at most one for 64 of them and
// one for 128, then fit a grid).
constexpr int64_t kMaxKvQueries = (int64_t)1 << 28;
struct KvAppend {
    KvCache cache;
    KvPlan plan;
    KvRows k, v, q;
    struct { void* data; int64_t row, head; } q_out;
    int q_heads;  // 0: no q
    bool bf16, interleaved;
    const float* rope;
    int64_t rope_ld;
    int rope_rows, rot;  // no rotation: INT32_MAX, 0
    int rows_each, chunks_each;  // of a wave; set by the launcher
};
hipError_t launch_kv_append(KvAppend p, hipStream_t s);
struct KvGather {
    KvCache cache;
    KvPlan plan;
    KvRows k, v;
    bool bf16;
    int rows_each, chunks_each;  // of a wave; set by the launcher
};
hipError_t launch_kv_gather(KvGather p, hipStream_t s);

// Attention over the cache (see nvfp4_kv_attention).
struct KvAttention {
    KvCache cache;
    KvPlan plan;
    KvRows q;
    struct { void* data; int64_t row, head; } out;
    float* lse;  // nullable, rows x q_heads
    int q_heads, group;
    int window;  // 0: none
    float scale;
    bool bf16;
    float* ws;
    int64_t blocks;  // of many rows, in all kv heads, and the most parts that each
    int splits;      // one's keys are split into; set by the launcher, as
    float* pre_ws;   // their part of ws
};
size_t kv_attention_workspace_bytes(int64_t rows, int64_t seqs, int q_heads, int kv_heads, int dim, bool bf16);
hipError_t launch_kv_attention(const KvAttention& p, hipStream_t s);

}  // namespace nvfp4
