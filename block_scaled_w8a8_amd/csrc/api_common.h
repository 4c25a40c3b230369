// What the C-ABI entry points share: status reporting and the checks of arguments that recur.
#pragma once
#include <string>

#include "bfq_internal.h"

namespace bfq {

// Sets the thread's detail string (bfq_last_error) and returns s.
bfq_status fail(bfq_status s, const std::string& msg);
bool batch_invariant();

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// Largest output count (M * N, grouped: T * topk * N) the GEMMs take: 2^40 elements, far past
// any device memory, keeps split-K workspace sizes (256 splits of fp32) and the reduce
// kernel's one-dimensional grid within range.
constexpr int64_t kMaxOutputs = int64_t(1) << 40;

// a * b >= kMaxOutputs for positive a, b, without overflow
inline bool too_many_outputs(int64_t a, int64_t b) {
    return a > 0 && b > 0 && a > (kMaxOutputs - 1) / b;
}

constexpr int64_t kNumCUs = 256;   // MI355X: 8 XCDs x 32 CUs

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int qtype_of(bfq_dtype d) { return d == BFQ_E4M3FN ? Q_FP8 : Q_INT8; }

inline int otype_of(bfq_dtype d) { return d == BFQ_BF16 ? O_BF16 : d == BFQ_FP16 ? O_FP16 : O_FP32; }

inline bool wlayout_ok(bfq_weight_layout w) { return w == BFQ_W_ROW_MAJOR || w == BFQ_W_PACKED16; }

inline bool sfmt_ok(bfq_scale_format f) { return f == BFQ_SCALE_FP32 || f == BFQ_SCALE_UE8M0; }

// Rows of the kernels with a workgroup of 256 threads a row: a grid dimension holds fewer than 2^32
// threads. (The norm step takes more threads a row, and a launch for each slice of rows that fits.)
constexpr int64_t kMaxRows = (int64_t(1) << 24) - 4;
constexpr int64_t kMaxScaleLd = int64_t(1) << 40;

// Strides of quantizer output scales over M tokens and G groups (layout, leading dimension).
inline bfq_status out_scale_strides(bfq_scale_layout layout, int64_t ld, int64_t M,
                                    int64_t G, bfq_scale_format fmt, bool per_token, int64_t* sm,
                                    int64_t* sg, int* packed) {
    if (ld > kMaxScaleLd) return fail(BFQ_ERR_SHAPE, "scale_ld must be at most 2^40");
    *packed = 0;
    if (layout == BFQ_SCALES_ROW_MAJOR) {
        if (ld < G) return fail(BFQ_ERR_SHAPE, "row-major scale_ld must be >= the groups of a token");
        *sm = ld; *sg = 1;
    } else if (layout == BFQ_SCALES_COL_MAJOR) {
        if (ld < M) return fail(BFQ_ERR_SHAPE, "column-major scale_ld must be >= M");
        *sm = 1; *sg = ld;
    } else if (layout == BFQ_SCALES_PACKED_UE8M0) {
        if (fmt != BFQ_SCALE_UE8M0 || per_token)
            return fail(BFQ_ERR_ARG, "packed scale words need UE8M0 scales of 1x128 groups");
        if (ld < (M + 3) / 4 * 4)
            return fail(BFQ_ERR_SHAPE, "packed scale_ld must be >= M rounded up to a multiple of 4");
        *sm = 1; *sg = ld; *packed = 1;
    } else {
        return fail(BFQ_ERR_ARG, "unknown scale layout");
    }
    return BFQ_OK;
}

inline bool eps_ok(float e) { return e > 0.0f && e <= 3.0e38f; }

}  // namespace bfq
