// C-ABI entry points of the mixture-of-experts layer around the grouped GEMM (include/bfq.h): the
// router, the sort and the dispatch, the combine, the 8-bit checkpoint of a gated product, and their
// gradients. Arguments are validated before any launch, as in api.cpp.
#include "api_common.h"
#include "moe_layer.h"

using namespace bfq;

namespace {

bool float_type(bfq_dtype d) { return d == BFQ_BF16 || d == BFQ_FP16 || d == BFQ_FP32; }
bool code_type(bfq_dtype d) { return d == BFQ_E4M3FN || d == BFQ_INT8; }

bfq_status launched(hipError_t e) { return e == hipSuccess ? BFQ_OK : fail(BFQ_ERR_HIP, hipGetErrorString(e)); }

// Output codes of R rows of N columns (q non-NULL): formats, strides.
bfq_status check_codes(void* q, bfq_dtype q_dtype, float* scales, bfq_scale_layout layout, int64_t ld,
                       float eps, bfq_scale_format fmt, int64_t R, int64_t N, CodesOut* o) {
    if (!code_type(q_dtype)) return fail(BFQ_ERR_DTYPE, "q_dtype must be BFQ_E4M3FN or BFQ_INT8");
    if (N % 128 != 0) return fail(BFQ_ERR_SHAPE, "codes need a multiple of 128 columns");
    if (!eps_ok(eps)) return fail(BFQ_ERR_ARG, "q_eps must be positive and finite");
    if (!sfmt_ok(fmt)) return fail(BFQ_ERR_ARG, "unknown scale format");
    const bfq_status s = out_scale_strides(layout, ld, R, N / 128, fmt, false, &o->stride_m, &o->stride_g, &o->packed);
    if (s != BFQ_OK) return s;
    o->q = q;
    o->scales = scales;
    o->qtype = qtype_of(q_dtype);
    o->ue8m0 = fmt == BFQ_SCALE_UE8M0;
    o->eps = eps;
    return BFQ_OK;
}

// An empty batch still writes the zero words of rows R .. round_up(R, 4) - 1.
bool only_padding(const CodesOut& o, int64_t T, int64_t R) { return T == 0 && o.packed && o.scales && R % 4 != 0; }

bfq_status check_tokens(int64_t T, int32_t topk, int64_t K, int64_t R) {
    if (T < 0 || T >= kMoeMaxTokens) return fail(BFQ_ERR_SHAPE, "need 0 <= T < 2^22");
    if (topk < 1 || topk > kMoeMaxTopk) return fail(BFQ_ERR_SHAPE, "need 1 <= topk <= 64");
    if (K <= 0 || K % 8 != 0 || K > kMoeMaxK)
        return fail(BFQ_ERR_SHAPE, "K must be a positive multiple of 8, at most 2^23");
    if (R < 0 || R > 0x7FFFFFFF) return fail(BFQ_ERR_SHAPE, "need 0 <= R < 2^31 rows");
    return BFQ_OK;
}

// Where the pairs' rows are, for the combine and its gradient.
bfq_status check_places(const int32_t* pair_rows, const int32_t* topk_ids, int32_t E, int64_t T, int32_t topk,
                        int64_t R, PairPlaces* at) {
    if (pair_rows && topk_ids) return fail(BFQ_ERR_ARG, "pair_rows says which pairs exist: topk_ids must be NULL");
    if (topk_ids && E < 1) return fail(BFQ_ERR_SHAPE, "topk_ids need E >= 1");
    // of an empty batch the places are an empty tensor, NULL: both orders are the same there
    if (!pair_rows && T != 0 && R != T * topk) return fail(BFQ_ERR_SHAPE, "rows in pair order: R must be T * topk");
    if (!aligned(pair_rows, 4) || !aligned(topk_ids, 4)) return fail(BFQ_ERR_ALIGN, "int32 buffers must be 4-byte aligned");
    *at = PairPlaces{pair_rows, topk_ids, E, topk, R};
    return BFQ_OK;
}

bfq_status check_route(const void* logits, bfq_dtype dt, int64_t T, int32_t E, int32_t topk, bfq_score score,
                       float weight_scale, const void* ids, const void* w) {
    if (T != 0 && (!logits || !ids || !w)) return fail(BFQ_ERR_NULL, "logits, topk_ids and the weights must be non-NULL");
    if (!float_type(dt)) return fail(BFQ_ERR_DTYPE, "logits must be BF16, FP16 or FP32");
    if (score != BFQ_SCORE_SOFTMAX && score != BFQ_SCORE_SIGMOID) return fail(BFQ_ERR_ARG, "unknown score function");
    if (!(weight_scale >= -3.0e38f && weight_scale <= 3.0e38f)) return fail(BFQ_ERR_ARG, "weight_scale must be finite");
    if (T < 0 || T >= kMoeMaxTokens || E < 1 || E > kMoeMaxExperts || topk < 1 || topk > E || topk > kMoeMaxTopk)
        return fail(BFQ_ERR_SHAPE, "need 0 <= T < 2^22, 1 <= E <= 1023 and 1 <= topk <= min(E, 64)");
    if (!aligned(logits, dt == BFQ_FP32 ? 4 : 2) || !aligned(ids, 4) || !aligned(w, 4))
        return fail(BFQ_ERR_ALIGN, "logits must be aligned to their type, ids and weights to 4 bytes");
    return BFQ_OK;
}

RouteArgs route_args(const void* logits, bfq_dtype dt, int64_t T, int32_t E, int32_t topk, bfq_score score,
                     int32_t renorm, float weight_scale) {
    RouteArgs a{};
    a.logits = logits;
    a.otype = otype_of(dt);
    a.T = T;
    a.E = E;
    a.topk = topk;
    a.sigmoid = score == BFQ_SCORE_SIGMOID;
    a.groups = a.topk_groups = 1;
    a.renorm = renorm != 0;
    a.weight_scale = weight_scale;
    return a;
}

}  // namespace

extern "C" {

bfq_status bfq_moe_route(const void* logits, bfq_dtype logits_dtype, const float* bias, int64_t T, int32_t E,
                         int32_t topk, bfq_score score, int32_t n_groups, int32_t topk_groups, int32_t renorm,
                         float weight_scale, int32_t* topk_ids, float* topk_weights, void* stream) {
    const bfq_status s = check_route(logits, logits_dtype, T, E, topk, score, weight_scale, topk_ids, topk_weights);
    if (s != BFQ_OK) return s;
    if (n_groups < 1 || n_groups > kRouteMaxGroups || E % n_groups != 0 || topk_groups < 1 ||
        topk_groups > n_groups || (int64_t)topk_groups * (E / n_groups) < topk)
        return fail(BFQ_ERR_SHAPE, "need 1 <= topk_groups <= n_groups <= 64, E a multiple of n_groups, and topk "
                                   "experts in topk_groups of them");
    if (!aligned(bias, 4)) return fail(BFQ_ERR_ALIGN, "bias must be 4-byte aligned");
    if (T == 0) return BFQ_OK;
    RouteArgs a = route_args(logits, logits_dtype, T, E, topk, score, renorm, weight_scale);
    a.bias = bias;
    a.groups = n_groups;
    a.topk_groups = topk_groups;
    a.ids = topk_ids;
    a.weights = topk_weights;
    return launched(launch_route(a, (hipStream_t)stream));
}

bfq_status bfq_moe_route_backward(const void* logits, bfq_dtype logits_dtype, const int32_t* topk_ids,
                                  const float* d_weights, int64_t T, int32_t E, int32_t topk, bfq_score score,
                                  int32_t renorm, float weight_scale, void* d_logits, void* stream) {
    const bfq_status s = check_route(logits, logits_dtype, T, E, topk, score, weight_scale, topk_ids, d_weights);
    if (s != BFQ_OK) return s;
    if (T != 0 && !d_logits) return fail(BFQ_ERR_NULL, "d_logits must be non-NULL");
    if (!aligned(d_logits, logits_dtype == BFQ_FP32 ? 4 : 2)) return fail(BFQ_ERR_ALIGN, "d_logits must be aligned to its type");
    if (T == 0) return BFQ_OK;
    RouteArgs a = route_args(logits, logits_dtype, T, E, topk, score, renorm, weight_scale);
    a.ids = const_cast<int32_t*>(topk_ids);
    a.d_weights = d_weights;
    a.d_logits = d_logits;
    return launched(launch_route_bwd(a, (hipStream_t)stream));
}

size_t bfq_moe_sort_workspace_bytes(int64_t T, int32_t topk, int32_t E) {
    if (T <= 0 || topk <= 0 || E <= 0 || E > kMoeMaxExperts || T > 0x7FFFFFFF / topk) return 0;
    return moe_sort_workspace_bytes(T * topk, E);
}

bfq_status bfq_moe_sort(const int32_t* topk_ids, int64_t T, int32_t topk, int32_t E, int32_t* expert_offsets,
                        int32_t* sorted_pairs, int32_t* pair_rows, void* workspace, size_t workspace_bytes,
                        void* stream) {
    if (!expert_offsets || (T > 0 && (!topk_ids || !sorted_pairs || !pair_rows)))
        return fail(BFQ_ERR_NULL, "topk_ids, expert_offsets, sorted_pairs and pair_rows must be non-NULL");
    if (T < 0 || topk < 1 || E < 1 || E > kMoeMaxExperts)
        return fail(BFQ_ERR_SHAPE, "need T >= 0, topk >= 1 and 1 <= E <= 1023");
    if (T > 0x7FFFFFFF / topk) return fail(BFQ_ERR_SHAPE, "T * topk must be below 2^31");
    if (!aligned(topk_ids, 4) || !aligned(expert_offsets, 4) || !aligned(sorted_pairs, 4) || !aligned(pair_rows, 4) ||
        !aligned(workspace, 4))
        return fail(BFQ_ERR_ALIGN, "int32 buffers must be 4-byte aligned");
    const size_t need = T > 0 ? moe_sort_workspace_bytes(T * topk, E) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(BFQ_ERR_WORKSPACE, "workspace of " + std::to_string(need) + " bytes required");
    return launched(launch_moe_sort(topk_ids, T * topk, E, expert_offsets, sorted_pairs, pair_rows,
                                    static_cast<int32_t*>(workspace), (hipStream_t)stream));
}

bfq_status bfq_moe_dispatch(const void* x, bfq_dtype x_dtype, const float* x_scales, bfq_scale_layout x_layout,
                            int64_t x_scale_ld, const int32_t* pair_rows, void* rows, void* q, bfq_dtype q_dtype,
                            float* scales, bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                            bfq_scale_format scale_fmt, int64_t T, int32_t topk, int64_t K, int64_t R,
                            void* stream) {
    const bool some = T != 0 && R != 0;                  // a row to write; else its tensors may be NULL
    if (T != 0 && (!x || !pair_rows)) return fail(BFQ_ERR_NULL, "x and pair_rows must be non-NULL");
    if (some && !rows && !q) return fail(BFQ_ERR_NULL, "one of rows and q must be non-NULL");
    if (some && (q != nullptr) != (scales != nullptr))
        return fail(BFQ_ERR_NULL, "q and scales must both be given or both be NULL");
    const bool copy = code_type(x_dtype);
    if (!copy && x_dtype != BFQ_BF16) return fail(BFQ_ERR_DTYPE, "x must be BF16, or codes E4M3FN or INT8");
    if (some && copy && (!q || !x_scales || rows))
        return fail(BFQ_ERR_NULL, "codes are dispatched as codes: x_scales, q and scales non-NULL, rows NULL");
    if (T != 0 && !copy && x_scales) return fail(BFQ_ERR_NULL, "bf16 rows have no x_scales");
    bfq_status s = check_tokens(T, topk, K, R);
    if (s != BFQ_OK) return s;
    if (!aligned(x, 16) || !aligned(rows, 16) || !aligned(q, 16) || !aligned(scales, 4) || !aligned(x_scales, 4) ||
        !aligned(pair_rows, 4))
        return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned, scales and pair_rows 4-byte");
    DispatchArgs a{};
    if (q) {
        s = check_codes(q, q_dtype, scales, layout, scale_ld, q_eps, scale_fmt, R, K, &a.out);
        if (s != BFQ_OK) return s;
    }
    if (copy && q) {
        if (q_dtype != x_dtype) return fail(BFQ_ERR_DTYPE, "q_dtype must be x_dtype: the codes are copied");
        if ((x_layout == BFQ_SCALES_PACKED_UE8M0) != (layout == BFQ_SCALES_PACKED_UE8M0))
            return fail(BFQ_ERR_ARG, "packed scale words are copied as such: both layouts packed, or neither");
        if (x_layout == BFQ_SCALES_ROW_MAJOR || x_layout == BFQ_SCALES_COL_MAJOR) {
            const bool row = x_layout == BFQ_SCALES_ROW_MAJOR;
            if (x_scale_ld < (row ? K / 128 : T) || x_scale_ld > kMaxScaleLd)
                return fail(BFQ_ERR_SHAPE, "x_scale_ld must be >= K / 128 (row-major) or T (column-major)");
            a.xs_stride_m = row ? x_scale_ld : 1;
            a.xs_stride_g = row ? 1 : x_scale_ld;
        } else if (x_layout == BFQ_SCALES_PACKED_UE8M0) {
            if (x_scale_ld < T || x_scale_ld > kMaxScaleLd) return fail(BFQ_ERR_SHAPE, "packed x_scale_ld must be >= T");
            a.xs_stride_m = 1;
            a.xs_stride_g = x_scale_ld;
        } else {
            return fail(BFQ_ERR_ARG, "unknown scale layout");
        }
    }
    if (!some && !only_padding(a.out, T, R)) return BFQ_OK;
    a.x = x;
    a.x_scales = copy ? x_scales : nullptr;
    a.T = T;
    a.K = K;
    a.at = PairPlaces{pair_rows, nullptr, 0, topk, R};
    a.rows = rows;
    return launched(q ? launch_dispatch_codes(a, (hipStream_t)stream) : launch_dispatch(a, (hipStream_t)stream));
}

bfq_status bfq_moe_combine(const void* rows, bfq_dtype rows_dtype, const float* weights, const int32_t* pair_rows,
                           const int32_t* topk_ids, int32_t E, const void* base, void* out, bfq_dtype out_dtype,
                           void* ckpt, bfq_dtype ckpt_dtype, float* ckpt_scales, float q_eps, int64_t T,
                           int32_t topk, int64_t K, int64_t R, void* stream) {
    if (T != 0 && ((!rows && R != 0) || !out)) return fail(BFQ_ERR_NULL, "rows and out must be non-NULL");
    if (T != 0 && R != 0 && (ckpt != nullptr) != (ckpt_scales != nullptr))
        return fail(BFQ_ERR_NULL, "ckpt and ckpt_scales must both be given or both be NULL");
    if (!float_type(rows_dtype) || !float_type(out_dtype))
        return fail(BFQ_ERR_DTYPE, "rows and out must be BF16, FP16 or FP32");
    bfq_status s = check_tokens(T, topk, K, R);
    if (s != BFQ_OK) return s;
    CombineArgs a{};
    s = check_places(pair_rows, topk_ids, E, T, topk, R, &a.at);
    if (s != BFQ_OK) return s;
    if (ckpt) {
        if (!code_type(ckpt_dtype)) return fail(BFQ_ERR_DTYPE, "ckpt_dtype must be BFQ_E4M3FN or BFQ_INT8");
        if (K % 128 != 0) return fail(BFQ_ERR_SHAPE, "codes need a multiple of 128 columns");
        if (!eps_ok(q_eps)) return fail(BFQ_ERR_ARG, "q_eps must be positive and finite");
    }
    if (!aligned(rows, 16) || !aligned(base, 16) || !aligned(out, 16) || !aligned(ckpt, 16) ||
        !aligned(ckpt_scales, 4) || !aligned(weights, 4))
        return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned, weights and scales 4-byte");
    if (T == 0) return BFQ_OK;
    a.rows = rows;
    a.rows_type = otype_of(rows_dtype);
    a.weights = weights;
    a.base = base;
    a.out = out;
    a.out_type = otype_of(out_dtype);
    a.ckpt = ckpt;
    a.ckpt_scales = ckpt_scales;
    a.ckpt_type = qtype_of(ckpt_dtype);
    a.ckpt_eps = q_eps;
    a.T = T;
    a.K = K;
    return launched(launch_combine(a, (hipStream_t)stream));
}

bfq_status bfq_moe_combine_backward(const void* dout, bfq_dtype dout_dtype, const float* weights, const void* rows,
                                    bfq_dtype rows_dtype, const float* rows_scales, const int32_t* pair_rows,
                                    const int32_t* topk_ids, int32_t E, void* d_rows, void* q, bfq_dtype q_dtype,
                                    float* scales, bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                                    bfq_scale_format scale_fmt, float* d_weights, int64_t T, int32_t topk,
                                    int64_t K, int64_t R, void* stream) {
    if (T != 0 && !dout) return fail(BFQ_ERR_NULL, "dout must be non-NULL");
    const bool some = T != 0 && R != 0;                  // a row to read or write; else its tensors may be NULL
    if (some && !d_rows && !q && !d_weights) return fail(BFQ_ERR_NULL, "one of d_rows, q and d_weights must be non-NULL");
    if (some && (q != nullptr) != (scales != nullptr))
        return fail(BFQ_ERR_NULL, "q and scales must both be given or both be NULL");
    if (some && (rows != nullptr) != (d_weights != nullptr))
        return fail(BFQ_ERR_NULL, "d_weights needs rows, and rows are read for it only");
    if (dout_dtype != BFQ_BF16 && dout_dtype != BFQ_FP32) return fail(BFQ_ERR_DTYPE, "dout must be BF16 or FP32");
    CombineBwdArgs a{};
    if (rows) {
        if (!float_type(rows_dtype) && !code_type(rows_dtype))
            return fail(BFQ_ERR_DTYPE, "rows must be BF16, FP16, FP32, or codes E4M3FN or INT8");
        if (some && code_type(rows_dtype) != (rows_scales != nullptr))
            return fail(BFQ_ERR_NULL, "rows_scales go with rows of codes");
        a.row_kind = rows_dtype == BFQ_BF16 ? R_BF16 : rows_dtype == BFQ_FP16 ? R_FP16 : rows_dtype == BFQ_FP32 ? R_FP32
                   : rows_dtype == BFQ_E4M3FN ? R_FP8 : R_INT8;
    }
    bfq_status s = check_tokens(T, topk, K, R);
    if (s != BFQ_OK) return s;
    if (rows && code_type(rows_dtype) && K % 128 != 0) return fail(BFQ_ERR_SHAPE, "codes need a multiple of 128 columns");
    s = check_places(pair_rows, topk_ids, E, T, topk, R, &a.at);
    if (s != BFQ_OK) return s;
    if (q) {
        s = check_codes(q, q_dtype, scales, layout, scale_ld, q_eps, scale_fmt, R, K, &a.out);
        if (s != BFQ_OK) return s;
    }
    if (!aligned(dout, 16) || !aligned(rows, 16) || !aligned(d_rows, 16) || !aligned(q, 16) || !aligned(scales, 4) ||
        !aligned(rows_scales, 4) || !aligned(weights, 4) || !aligned(d_weights, 4))
        return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned, weights and scales 4-byte");
    if (!some && !only_padding(a.out, T, R)) {           // without a row the weights have no gradient
        if (T == 0 || !d_weights) return BFQ_OK;
        a.row_kind = R_BF16;
        a.out = CodesOut{};
        d_rows = nullptr;
    }
    a.dout = dout;
    a.dout_f32 = dout_dtype == BFQ_FP32;
    a.weights = weights;
    a.rows = rows;
    a.rows_scales = rows_scales;
    a.d_rows = d_rows;
    a.d_weights = d_weights;
    a.T = T;
    a.K = K;
    return launched(launch_combine_bwd(a, (hipStream_t)stream));
}

}  // extern "C"

// ------------------------------------------------------------------ checkpoints ----

namespace {

// What both directions share: sizes, the checkpoint, the codes that are written.
bfq_status check_checkpoint(const void* ckpt, bfq_dtype ckpt_dtype, const float* ckpt_scales, bfq_activation act,
                            void* q, bfq_dtype q_dtype, float* scales, bfq_scale_layout layout, int64_t scale_ld,
                            float q_eps, bfq_scale_format scale_fmt, const int32_t* live_rows, int64_t M, int64_t F,
                            int64_t q_columns, CheckpointArgs* a) {
    if (M != 0 && (q != nullptr) != (scales != nullptr))
        return fail(BFQ_ERR_NULL, "q and scales must both be given or both be NULL");
    if (M != 0 && (ckpt != nullptr) != (ckpt_scales != nullptr))
        return fail(BFQ_ERR_NULL, "ckpt and ckpt_scales must both be given or both be NULL");
    if (act != BFQ_ACT_SILU && act != BFQ_ACT_GELU_TANH) return fail(BFQ_ERR_ARG, "unknown activation");
    if (ckpt && !code_type(ckpt_dtype)) return fail(BFQ_ERR_DTYPE, "ckpt_dtype must be BFQ_E4M3FN or BFQ_INT8");
    if (M < 0 || F <= 0 || F % 128 != 0) return fail(BFQ_ERR_SHAPE, "need M >= 0 and F a positive multiple of 128");
    if (M >= kMaxRows || F >= (int64_t(1) << 26)) return fail(BFQ_ERR_SHAPE, "need M < 2^24 - 4 and F < 2^26");
    if (!eps_ok(q_eps)) return fail(BFQ_ERR_ARG, "q_eps must be positive and finite");
    if (q) {
        const bfq_status s = check_codes(q, q_dtype, scales, layout, scale_ld, q_eps, scale_fmt, M, q_columns, &a->out);
        if (s != BFQ_OK) return s;
    }
    if (!aligned(ckpt, 16) || !aligned(ckpt_scales, 4) || !aligned(q, 16) || !aligned(scales, 4) || !aligned(live_rows, 4))
        return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned, scales and live_rows 4-byte");
    a->ckpt = const_cast<void*>(ckpt);
    a->ckpt_scales = const_cast<float*>(ckpt_scales);
    a->ckpt_type = qtype_of(ckpt_dtype);
    a->ckpt_eps = q_eps;
    a->live = live_rows;
    a->M = M;
    a->F = F;
    gated_activation((int)act, &a->c1, &a->c3);
    return BFQ_OK;
}

}  // namespace

extern "C" {

bfq_status bfq_gated_checkpoint(const void* preact, bfq_activation act, void* h, void* q, bfq_dtype q_dtype,
                                float* scales, bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                                bfq_scale_format scale_fmt, void* ckpt, bfq_dtype ckpt_dtype, float* ckpt_scales,
                                const int32_t* live_rows, int64_t M, int64_t F, void* stream) {
    if (M != 0 && !preact) return fail(BFQ_ERR_NULL, "preact must be non-NULL");
    if (M != 0 && !h && !q && !ckpt) return fail(BFQ_ERR_NULL, "one of h, q and ckpt must be non-NULL");
    CheckpointArgs a{};
    const bfq_status s = check_checkpoint(ckpt, ckpt_dtype, ckpt_scales, act, q, q_dtype, scales, layout, scale_ld,
                                          q_eps, scale_fmt, live_rows, M, F, F, &a);
    if (s != BFQ_OK) return s;
    if (!aligned(preact, 16) || !aligned(h, 16)) return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned");
    if (M == 0) return BFQ_OK;
    a.pre = preact;
    a.h = h;
    return launched(launch_checkpoint(a, (hipStream_t)stream));
}

bfq_status bfq_gated_checkpoint_backward(const void* ckpt, bfq_dtype ckpt_dtype, const float* ckpt_scales,
                                         const void* dh, bfq_activation act, void* dpre, void* q,
                                         bfq_dtype q_dtype, float* scales, bfq_scale_layout layout,
                                         int64_t scale_ld, float q_eps, bfq_scale_format scale_fmt, void* h,
                                         const int32_t* live_rows, int64_t M, int64_t F, void* stream) {
    if (M != 0 && (!ckpt || !ckpt_scales || !dh)) return fail(BFQ_ERR_NULL, "ckpt, ckpt_scales and dh must be non-NULL");
    if (M != 0 && !dpre && !q && !h) return fail(BFQ_ERR_NULL, "one of dpre, q and h must be non-NULL");
    CheckpointArgs a{};
    const bfq_status s = check_checkpoint(ckpt, ckpt_dtype, ckpt_scales, act, q, q_dtype, scales, layout, scale_ld,
                                          q_eps, scale_fmt, live_rows, M, F, 2 * F, &a);
    if (s != BFQ_OK) return s;
    if (!aligned(dh, 16) || !aligned(dpre, 16) || !aligned(h, 16))
        return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned");
    if (M == 0) return BFQ_OK;
    a.dh = dh;
    a.dpre = dpre;
    a.h = h;
    return launched(launch_checkpoint_bwd(a, (hipStream_t)stream));
}

}  // extern "C"
