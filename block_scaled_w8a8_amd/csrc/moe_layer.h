// Launchers of the mixture-of-experts layer around the grouped GEMM (csrc/route.hip,
// csrc/moe_rows.hip, csrc/checkpoint.hip). Not part of the public C-ABI (include/bfq.h).
#pragma once
#include "bfq_internal.h"

namespace bfq {

// Experts a token may have, and tokens a call may have: a pair is a lane of a wave, a grid dimension
// holds fewer than 2^32 threads (at most 256 a token), and a pair's number (below 2^28) fits an int32.
constexpr int kMoeMaxTopk = 64;
constexpr int64_t kMoeMaxTokens = int64_t(1) << 22;
constexpr int64_t kMoeMaxK = int64_t(1) << 23;
// Groups of experts that the router may choose among: a lane each.
constexpr int kRouteMaxGroups = 64;
// Added to the sum that a token's weights are divided by.
constexpr float kRouteEps = 1e-20f;

struct RouteArgs {
    const void* logits;      // [T][E] of otype
    int otype;               // O_BF16 / O_FP16 / O_FP32, the gradient's too
    const float* bias;       // [E] or NULL
    int64_t T;
    int E, topk, sigmoid, groups, topk_groups, renorm;
    float weight_scale;
    int32_t* ids;            // [T][topk], read by the gradient
    float* weights;          // [T][topk]
    const float* d_weights;  // backward
    void* d_logits;          // backward
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_bwd(const RouteArgs& a, hipStream_t stream);

size_t moe_sort_workspace_bytes(int64_t pairs, int E);
hipError_t launch_moe_sort(const int32_t* ids, int64_t pairs, int E, int32_t* offsets,
                           int32_t* sorted, int32_t* pair_rows, int32_t* counts,
                           hipStream_t stream);

// Where the row of pair q = t * topk + j is: pair_rows[q] if that is in [0, R), or q itself unless
// its id is outside [0, E); else the pair has none.
struct PairPlaces {
    const int32_t* pair_rows;
    const int32_t* ids;
    int E, topk;
    int64_t R;
};

// Codes that are written: codes and scales of `rows` rows.
struct CodesOut {
    void* q;
    float* scales;
    int64_t stride_m, stride_g;   // of a row and of a group (packed: word row)
    int qtype, ue8m0, packed;
    float eps;
};

struct DispatchArgs {
    const void* x;           // [T][K] bf16, or codes
    const float* x_scales;   // of codes
    int64_t xs_stride_m, xs_stride_g;
    int64_t T, K;
    PairPlaces at;
    void* rows;              // [R][K] bf16 or NULL
    CodesOut out;            // [R][K]
};
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream);
hipError_t launch_dispatch_codes(const DispatchArgs& a, hipStream_t stream);

struct CombineArgs {
    const void* rows;        // [R][K] of rows_type
    int rows_type;           // O_BF16 / O_FP16 / O_FP32
    const float* weights;    // [T][topk] or NULL
    PairPlaces at;
    const void* base;        // [T][K] of out_type, or NULL
    void* out;               // [T][K]
    int out_type;
    void* ckpt;              // [R][K] codes or NULL
    float* ckpt_scales;      // [R][K/128]
    int ckpt_type;
    float ckpt_eps;
    int64_t T, K;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream);

// Types of the rows that the combine's gradient reads.
enum RowKind { R_NONE = 0, R_BF16 = 1, R_FP16 = 2, R_FP32 = 3, R_FP8 = 4, R_INT8 = 5 };
struct CombineBwdArgs {
    const void* dout;        // [T][K] bf16 / fp32
    int dout_f32;
    const float* weights;    // [T][topk] or NULL
    const void* rows;        // [R][K] of row_kind
    const float* rows_scales;   // [R][K/128] of codes
    int row_kind;
    PairPlaces at;
    void* d_rows;            // [R][K] bf16 or NULL
    CodesOut out;
    float* d_weights;        // [T][topk] or NULL
    int64_t T, K;
};
hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t stream);

struct CheckpointArgs {
    const void* pre;         // [M][2F] bf16 (forward)
    const void* dh;          // [M][F] bf16 (backward)
    void* ckpt;              // [M][2F] codes (backward: read)
    float* ckpt_scales;      // [M][2F/128]
    int ckpt_type;
    float ckpt_eps;
    void* h;                 // [M][F] bf16 or NULL
    void* dpre;              // [M][2F] bf16 or NULL (backward)
    CodesOut out;            // of h [M][F], backward of (dg, du) [M][2F]
    const int32_t* live;     // rows that exist, or NULL: all
    int64_t M, F;
    float c1, c3;            // the activation's constants (gated_activation)
};
hipError_t launch_checkpoint(const CheckpointArgs& a, hipStream_t stream);
hipError_t launch_checkpoint_bwd(const CheckpointArgs& a, hipStream_t stream);

}  // namespace bfq
