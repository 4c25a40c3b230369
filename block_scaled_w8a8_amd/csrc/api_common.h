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

}  // namespace bfq
