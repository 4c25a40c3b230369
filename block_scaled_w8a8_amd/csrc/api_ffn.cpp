// C-ABI entry points of the feed-forward operators (include/bfq.h): the gated product, its
// gradient, the weight transpose, and the norms around a block with their gradients. Arguments
// are validated before any launch, as in api.cpp.
#include <cmath>

#include "api_common.h"

using namespace bfq;

namespace {

// Rows of the kernels with a workgroup of 256 threads a row: a grid dimension holds fewer than 2^32
// threads. (The norm step takes more threads a row, and a launch for each slice of rows that fits.)
constexpr int64_t kMaxRows = (int64_t(1) << 24) - 4;
constexpr int64_t kMaxScaleLd = int64_t(1) << 40;

// Strides of quantizer output scales over M tokens and G groups (layout, leading dimension).
bfq_status out_scale_strides(bfq_scale_layout layout, int64_t ld, int64_t M, int64_t G,
                             bfq_scale_format fmt, bool per_token, int64_t* sm, int64_t* sg,
                             int* packed) {
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

bool eps_ok(float e) { return e > 0.0f && e <= 3.0e38f; }

// ------------------------------------------------------------------ gated tiles ----

// A kernel serves scale format sfmt if it takes any fp32 block scales (S_FP32), or if the scales
// are powers of two (an S_UE8M0 kernel applies them inside the MFMA). Packed activation-scale
// words need an S_PACKED strip kernel, or any standard tile (a run-time flag).
bool serves(const GatedKernel& k, int sfmt) {
    if (sfmt == S_PACKED) return k.sfmt == S_PACKED || k.tile.variant == 0;
    if (k.sfmt == S_PACKED) return false;
    return k.sfmt == S_FP32 || sfmt == S_UE8M0;
}

const GatedKernel* find_gated(bfq_tile t, int wlayout, int sfmt) {
    if (t.bk != 0 && t.bk != 128) return nullptr;
    if (t.variant == 2) t.variant = 0;                     // the same kernels, the last tiles split
    int n = 0;
    const GatedKernel* k = gated_kernels(&n);
    for (int i = 0; i < n; ++i) {
        const bfq_tile& b = k[i].tile;
        if (k[i].wlayout == wlayout && serves(k[i], sfmt) && b.variant == t.variant && b.bm == t.bm &&
            b.bn == t.bn && b.waves_m == t.waves_m && b.waves_n == t.waves_n &&
            b.stages == t.stages && b.sched == t.sched)
            return &k[i];
    }
    return nullptr;
}

// The tile of (bm, bn, sched) among the kernels built for a weight layout.
bfq_tile gated_tile(int variant, int bm, int bn, int sched, int wlayout) {
    int n = 0;
    const GatedKernel* k = gated_kernels(&n);
    for (int i = 0; i < n; ++i) {
        const bfq_tile& t = k[i].tile;
        if (k[i].wlayout == wlayout && t.variant == variant && t.bm == bm && t.bn == bn && t.sched == sched)
            return t;
    }
    return bfq_tile{};
}

// Strips that copy the weights through a ring in LDS.
bool ring_strip(const GatedKernel& k) { return k.tile.variant == 1 && k.tile.sched == 2; }

// Microseconds that a gated product is expected to take with kernel k and its K range in `split`
// parts. The grid runs in rounds of 256 CUs times the workgroups a CU holds; a round's K block
// takes the longer of a workgroup's own latency and the CU's throughput over the workgroups it
// holds (joined smoothly), the whole no less than the weight stream (ring strips take half of it
// again for each further bm tokens); partials cost a second launch and their bytes twice (those of
// a split last round, written by all CUs at the end of it, at a lower rate). The
// constants, here and beside the kernels, are a fit to 840 measured (M, F, K, layout, format,
// output) points of 9 to 100 configurations each, M 1 to 2048 on seven (F, K), weights read from
// HBM as between the layers of a model; over them the pick is on average 1.1 % slower than the
// fastest configuration.
// tail: the parts of the last round's tiles (variant 2), 1 otherwise.
float gated_us(const GatedKernel& k, int64_t M, int64_t F, int64_t K, bool codes, int split, int tail) {
    const bfq_tile& t = k.tile;
    const int64_t groups = ceil_div(M, t.bm) * ceil_div(F, t.bn) * split;
    const int64_t slots = kNumCUs * k.occupancy, full = groups / slots, rest = groups % slots;
    const int kw = t.variant == 1 ? t.waves_m : 1;         // waves that share a strip's K range
    const float blocks = (float)ceil_div(ceil_div(K / 128, split), kw);
    // strips whose waves fetch their own tokens: up to 0.6 of the throughput's time more for them
    const float thr = k.thr * (t.variant == 1 && t.sched == 0
                                   ? 1.f + 0.6f * (float)(M < t.bm ? M : t.bm) / (float)t.bm : 1.f);
    auto round = [&](int64_t held, float n) {
        const float a = k.lat * n, b = (float)held * thr * n * kw;
        return std::sqrt(std::sqrt(a * a * a * a + b * b * b * b)) + k.fix;
    };
    float us = (float)full * round(k.occupancy, blocks) +
               (rest ? round(ceil_div(rest, kNumCUs), std::ceil(blocks / (float)tail)) : 0.f);
    const float rate = t.variant == 0 ? 4.63e6f : ring_strip(k) ? 5.62e6f : 5.93e6f;
    float stream = 2.f * (float)F * (float)K / rate;
    if (ring_strip(k)) stream *= 0.5f + 0.5f * (float)ceil_div(M, t.bm);
    const float x = us > stream ? stream / us : us / stream, x2 = x * x, x4 = x2 * x2;
    us = (us > stream ? us : stream) * std::sqrt(std::sqrt(std::sqrt(1.f + x4 * x4)));
    if (tail > 1) us += 2.74f + (float)(rest * tail) * (float)(t.bm * t.bn) * 16.f / 4.2e6f;
    if (split > 1 || (codes && t.bn != 128)) us += 2.74f + (float)split * (float)M * (float)F * 16.f / 5.54e6f;
    return us;
}

// Variant 2: whole tiles in rounds of one workgroup a CU, the K range of the tiles that are left over
// in as many parts as fill one more round, two K blocks or more each. parts = 1: nothing to split.
struct TailPlan {
    int64_t tiles, first;
    int parts;
};
TailPlan tail_plan(const bfq_tile& t, int64_t M, int64_t F, int64_t K) {
    const int64_t tiles = ceil_div(M, t.bm) * ceil_div(F, t.bn), first = tiles / kNumCUs * kNumCUs;
    if (t.variant != 2 || first == 0 || first == tiles) return {tiles, tiles, 1};
    const int64_t fill = kNumCUs / (tiles - first), parts = fill < K / 256 ? fill : K / 256;
    return parts > 1 ? TailPlan{tiles, first, (int)(parts < 16 ? parts : 16)} : TailPlan{tiles, tiles, 1};
}
size_t tail_bytes(const TailPlan& p, const bfq_tile& t) {
    return p.parts > 1 ? (size_t)(p.tiles - p.first) * (size_t)p.parts * (size_t)t.bm * 2 * (size_t)t.bn * sizeof(float) : 0;
}

// The rule: the kernel and K split with the least expected time. Strips read the weights again
// for every bm tokens, so they are left out where that is more often than was measured.
bfq_tile select_gated(int64_t M, int64_t F, int64_t K, bool codes, int wlayout, int sfmt) {
    const int64_t KB = K / 128;
    if (batch_invariant()) {
        // one MFMA per K block and fp32 scale FMAs in ascending order, whatever M
        if (wlayout == W_PACKED16 && M <= 64) return gated_tile(1, M <= 32 ? 32 : 64, 128, 1, wlayout);
        if (M <= 64) return gated_tile(0, 64, 64, 0, wlayout);
        if (M <= 512) return gated_tile(0, 128, 64, 0, wlayout);
        return gated_tile(0, 256, 128, wlayout == W_PACKED16 ? 0 : 1, wlayout);
    }
    int n = 0;
    const GatedKernel* k = gated_kernels(&n);
    bfq_tile best{};
    float best_us = 3.0e38f;
    for (int i = 0; i < n; ++i) {
        const bfq_tile& t = k[i].tile;
        if (k[i].wlayout != wlayout || k[i].sfmt == S_PACKED || (k[i].sfmt == S_UE8M0 && sfmt != S_UE8M0))
            continue;
        if (t.variant == 1 ? M > (ring_strip(k[i]) ? 4 : 2) * t.bm : M < 24 || M < t.bm / 4) continue;
        const int64_t groups = ceil_div(M, t.bm) * ceil_div(F, t.bn);
        for (int split : {1, 2, 3, 4, 6, 8, 12}) {
            // at least two K blocks a part, and no parts beyond those that fill the CUs (ring
            // strips: none gained from a split that partials alone pay for, nor from over three)
            if (split > 1 && (split * 2 > KB || groups * (split - 1) >= kNumCUs * k[i].occupancy ||
                              (ring_strip(k[i]) && (!codes || split > 3))))
                break;
            const float us = gated_us(k[i], M, F, K, codes, split, 1);
            if (us < best_us) {
                best_us = us;
                best = t;
                best.split_k = split;
            }
        }
        bfq_tile u = t;
        u.variant = 2;
        if (t.variant != 0 || k[i].occupancy != 1 || (codes && t.bn != 128)) continue;
        const int parts = tail_plan(u, M, F, K).parts;
        const float us = parts > 1 ? gated_us(k[i], M, F, K, codes, 1, parts) : best_us;
        if (us < best_us) {
            best_us = us;
            best = u;
        }
    }
    return best;
}

// A tile finishes its outputs itself unless its K range is split or codes need whole groups.
bool needs_partials(const bfq_tile& t, bool codes) { return t.split_k > 1 || (codes && t.bn != 128); }

bool gated_too_large(int64_t M, int64_t F, int64_t K) {
    return M >= kMaxRows || F >= (int64_t(1) << 26) || K > (1 << 23) || too_many_outputs(M, 2 * F) ||
           too_many_outputs(F, K);
}

}  // namespace

extern "C" {

bfq_status bfq_gated_select_tile(int64_t M, int64_t F, int64_t K, bfq_dtype out_dtype,
                                 bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                 bfq_tile* tile_out) {
    if (!tile_out) return fail(BFQ_ERR_NULL, "tile_out must be non-NULL");
    if (out_dtype != BFQ_BF16 && out_dtype != BFQ_FP16 && out_dtype != BFQ_FP32 && out_dtype != BFQ_E4M3FN)
        return fail(BFQ_ERR_DTYPE, "out_dtype must be BF16, FP16, FP32 or E4M3FN");
    if (!wlayout_ok(w_layout)) return fail(BFQ_ERR_ARG, "unknown weight layout");
    if (!sfmt_ok(scale_fmt)) return fail(BFQ_ERR_ARG, "unknown scale format");
    if (M < 0 || F <= 0 || K <= 0 || F % 128 != 0 || K % 128 != 0)
        return fail(BFQ_ERR_SHAPE, "need M >= 0 and F, K positive multiples of 128");
    if (gated_too_large(M, F, K)) return fail(BFQ_ERR_SHAPE, "gated product: shape too large");
    *tile_out = select_gated(M, F, K, out_dtype == BFQ_E4M3FN, (int)w_layout, (int)scale_fmt);
    return BFQ_OK;
}

size_t bfq_gated_gemm_workspace_bytes(int64_t M, int64_t F, int64_t K, bfq_dtype out_dtype,
                                      bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                      const bfq_tile* tile) {
    if (M <= 0 || F <= 0 || K <= 0) return 0;
    if (gated_too_large(M, F, K)) return SIZE_MAX;
    if (!tile && (!wlayout_ok(w_layout) || F % 128 != 0 || K % 128 != 0)) return 0;
    const bool codes = out_dtype == BFQ_E4M3FN;
    const bfq_tile t = tile ? *tile : select_gated(M, F, K, codes, (int)w_layout, (int)scale_fmt);
    if (t.variant == 2) return t.bm > 0 && t.bn > 0 ? tail_bytes(tail_plan(t, M, F, K), t) : 0;
    if (!needs_partials(t, codes) || t.split_k < 1) return 0;
    return (size_t)t.split_k * (size_t)M * 2 * (size_t)F * sizeof(float);
}

int32_t bfq_gated_num_tile_candidates(bfq_weight_layout w_layout, bfq_scale_format scale_fmt) {
    if (!wlayout_ok(w_layout) || !sfmt_ok(scale_fmt)) return 0;
    int n = 0, count = 0;
    const GatedKernel* k = gated_kernels(&n);
    for (int i = 0; i < n; ++i) count += k[i].wlayout == (int)w_layout && serves(k[i], (int)scale_fmt);
    return count;
}

bfq_status bfq_gated_get_tile_candidate(bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                        int32_t index, bfq_tile* tile_out) {
    if (!tile_out) return fail(BFQ_ERR_NULL, "tile_out must be non-NULL");
    if (!wlayout_ok(w_layout)) return fail(BFQ_ERR_ARG, "unknown weight layout");
    if (!sfmt_ok(scale_fmt)) return fail(BFQ_ERR_ARG, "unknown scale format");
    int n = 0, count = 0;
    const GatedKernel* k = gated_kernels(&n);
    for (int i = 0; i < n; ++i) {
        if (k[i].wlayout != (int)w_layout || !serves(k[i], (int)scale_fmt)) continue;
        if (count++ == index) { *tile_out = k[i].tile; return BFQ_OK; }
    }
    return fail(BFQ_ERR_ARG, "candidate index out of range");
}

bfq_status bfq_gated_gemm(const void* a_q, const float* a_scales, bfq_scale_layout a_layout,
                          int64_t a_scale_ld, const void* w_q, const float* w_scales,
                          bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                          bfq_activation act, void* out, float* out_scales,
                          bfq_scale_layout out_layout, int64_t out_scale_ld, float out_eps,
                          void* preact, int64_t M, int64_t F, int64_t K,
                          const int32_t block_shape[2], bfq_dtype in_dtype, bfq_dtype out_dtype,
                          const bfq_tile* tile, void* workspace, size_t workspace_bytes,
                          void* stream) {
    const bool codes = out_dtype == BFQ_E4M3FN;
    if (!w_q || !w_scales || !block_shape || (M != 0 && (!a_q || !a_scales || !out || (codes && !out_scales))))
        return fail(BFQ_ERR_NULL, "a_q, a_scales, w_q, w_scales, out, block_shape and (with codes) "
                                  "out_scales must be non-NULL");
    if (block_shape[0] != 128 || block_shape[1] != 128)
        return fail(BFQ_ERR_SHAPE, "gated product: block_shape must be {128, 128}");
    if (in_dtype != BFQ_E4M3FN) return fail(BFQ_ERR_DTYPE, "gated product: in_dtype must be BFQ_E4M3FN");
    if (out_dtype != BFQ_BF16 && out_dtype != BFQ_FP16 && out_dtype != BFQ_FP32 && !codes)
        return fail(BFQ_ERR_DTYPE, "out_dtype must be BF16, FP16, FP32 or E4M3FN");
    if (!wlayout_ok(w_layout)) return fail(BFQ_ERR_ARG, "unknown weight layout");
    if (!sfmt_ok(scale_fmt)) return fail(BFQ_ERR_ARG, "unknown scale format");
    if (act != BFQ_ACT_SILU && act != BFQ_ACT_GELU_TANH) return fail(BFQ_ERR_ARG, "unknown activation");
    if (M < 0 || F <= 0 || K <= 0 || F % 128 != 0 || K % 128 != 0)
        return fail(BFQ_ERR_SHAPE, "need M >= 0 and F, K positive multiples of 128");
    if (gated_too_large(M, F, K))
        return fail(BFQ_ERR_SHAPE, "need M < 2^24 - 4, F < 2^26, K <= 2^23, M * 2F < 2^40 and F * K < 2^40");
    if (a_scale_ld > (1 << 23)) return fail(BFQ_ERR_SHAPE, "a_scale_ld must be at most 2^23");
    if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(out, 16) || !aligned(preact, 16) ||
        !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(workspace, 16) ||
        (codes && !aligned(out_scales, 4)))
        return fail(BFQ_ERR_ALIGN, "codes, out, preact and workspace must be 16-byte aligned, scales 4-byte");
    const int64_t KB = K / 128;
    int64_t ssm, ssk;
    const bool apacked = a_layout == BFQ_SCALES_PACKED_UE8M0;
    if (a_layout == BFQ_SCALES_ROW_MAJOR) {
        if (a_scale_ld < KB) return fail(BFQ_ERR_SHAPE, "row-major a_scale_ld must be >= K/128");
        ssm = a_scale_ld; ssk = 1;
    } else if (a_layout == BFQ_SCALES_COL_MAJOR) {
        if (a_scale_ld < M) return fail(BFQ_ERR_SHAPE, "column-major a_scale_ld must be >= M");
        ssm = 1; ssk = a_scale_ld;
    } else if (apacked) {
        if (scale_fmt != BFQ_SCALE_UE8M0)
            return fail(BFQ_ERR_ARG, "packed scale words need scales in the UE8M0 format");
        if (a_scale_ld < M) return fail(BFQ_ERR_SHAPE, "packed a_scale_ld must be >= M");
        ssm = 1; ssk = a_scale_ld;
    } else {
        return fail(BFQ_ERR_ARG, "unknown scale layout");
    }
    const int64_t k_rows = apacked ? (KB - 1) / 4 : KB - 1;
    if ((255 * ssm + k_rows * ssk + 1) * 4 >= (int64_t(1) << 32))
        return fail(BFQ_ERR_SHAPE, "activation scales of 256 tokens must span less than 4 GiB");
    GatedArgs ga{};
    if (codes) {
        if (!eps_ok(out_eps)) return fail(BFQ_ERR_ARG, "out_eps must be positive and finite");
        const bfq_status s = out_scale_strides(out_layout, out_scale_ld, M, F / 128, scale_fmt, false,
                                               &ga.os_stride_m, &ga.os_stride_g, &ga.os_packed);
        if (s != BFQ_OK) return s;
    }
    const int wl = (int)w_layout;
    bfq_tile t = tile ? *tile : select_gated(M, F, K, codes, wl, (int)scale_fmt);
    const GatedKernel* gk = find_gated(t, wl, apacked ? S_PACKED : (int)scale_fmt);
    if (!gk || (gk->sfmt == S_UE8M0 && scale_fmt != BFQ_SCALE_UE8M0))
        return fail(BFQ_ERR_TILE, "tile does not name a compiled gated kernel for this weight layout "
                                  "and scale format");
    if (t.split_k < 1 || t.split_k > 256 || t.split_k > KB)
        return fail(BFQ_ERR_TILE, "split_k must be in [1, min(256, K/128)]");
    if (t.variant != 1 && (t.group_m < 1 || t.raster < 0 || t.raster > 1))
        return fail(BFQ_ERR_TILE, "group_m must be >= 1 and raster 0 or 1");
    if (t.variant == 2 && (gk->tile.variant != 0 || t.split_k != 1 || (codes && t.bn != 128)))
        return fail(BFQ_ERR_TILE, "variant 2 takes the tiles of variant 0 with split_k 1 and, for codes, bn 128");
    const TailPlan tail = tail_plan(t, M, F, K);
    const bool parts = needs_partials(t, codes);
    const size_t need = parts ? (size_t)t.split_k * (size_t)M * 2 * (size_t)F * sizeof(float) : tail_bytes(tail, t);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(BFQ_ERR_WORKSPACE, "workspace of " + std::to_string(need) + " bytes required");
    // a grid dimension holds fewer than 2^32 threads
    const int64_t threads = 64 * t.waves_m * t.waves_n;
    if (t.variant != 1 ? (tail.tiles + kNumCUs) * threads >= (int64_t(1) << 32)
                       : ceil_div(M, t.bm) > 65535 || ceil_div(F, t.bn) * threads >= (int64_t(1) << 32))
        return fail(BFQ_ERR_SHAPE, "too many output tiles for one launch");
    if (M == 0) return BFQ_OK;

    ga.a = a_q;
    ga.sa = a_scales;
    ga.sa_stride_m = ssm;
    ga.sa_stride_k = ssk;
    ga.sa_packed = apacked ? 1 : 0;
    ga.w = w_q;
    ga.sw = w_scales;
    ga.out = out;
    ga.partials = parts ? static_cast<float*>(workspace) : nullptr;
    ga.M = M;
    ga.N = F;
    ga.K = K;
    ga.split = t.split_k;
    ga.group_m = t.group_m;
    ga.raster = t.raster;
    gated_activation((int)act, &ga.c1, &ga.c3);
    ga.pre = preact;
    ga.otype = codes ? O_CODES : otype_of(out_dtype);
    ga.out_scales = out_scales;
    ga.os_ue8m0 = scale_fmt == BFQ_SCALE_UE8M0;
    ga.os_eps = out_eps;
    ga.tail_first = tail.first;
    ga.tail_parts = tail.parts;
    ga.tail_bm = t.bm;
    ga.tail_bn = t.bn;
    ga.tail = tail.parts > 1 ? static_cast<float*>(workspace) : nullptr;
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = gk->launch(ga, s);
    if (e == hipSuccess && parts) e = launch_gated_reduce(ga, s);
    if (e == hipSuccess && tail.parts > 1) e = launch_gated_tail(ga, tail.tiles, s);
    if (e != hipSuccess) return fail(BFQ_ERR_HIP, hipGetErrorString(e));
    return BFQ_OK;
}

bfq_status bfq_gated_backward(const void* preact, const void* dh, bfq_activation act, void* dpre,
                              void* q, bfq_dtype q_dtype, float* scales, bfq_scale_layout layout,
                              int64_t scale_ld, float q_eps, bfq_scale_format scale_fmt, void* h,
                              int64_t M, int64_t F, void* stream) {
    if (M != 0 && (!preact || !dh)) return fail(BFQ_ERR_NULL, "preact and dh must be non-NULL");
    if (M != 0 && !dpre && !q && !h) return fail(BFQ_ERR_NULL, "one of dpre, q and h must be non-NULL");
    if (M != 0 && (q != nullptr) != (scales != nullptr))
        return fail(BFQ_ERR_NULL, "q and scales must both be given or both be NULL");
    if (act != BFQ_ACT_SILU && act != BFQ_ACT_GELU_TANH) return fail(BFQ_ERR_ARG, "unknown activation");
    if (q && q_dtype != BFQ_E4M3FN && q_dtype != BFQ_INT8)
        return fail(BFQ_ERR_DTYPE, "q_dtype must be BFQ_E4M3FN or BFQ_INT8");
    if (M < 0 || F <= 0 || F % 8 != 0 || (q && F % 128 != 0))
        return fail(BFQ_ERR_SHAPE, "need M >= 0 and F a positive multiple of 8 (of 128 with codes)");
    if (M >= kMaxRows || F >= (int64_t(1) << 26))
        return fail(BFQ_ERR_SHAPE, "need M < 2^24 - 4 and F < 2^26");
    if (!aligned(preact, 16) || !aligned(dh, 16) || !aligned(dpre, 16) || !aligned(q, 16) ||
        !aligned(h, 16) || !aligned(scales, 4))
        return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned, scales 4-byte");
    GatedBwdArgs a{};
    if (q) {
        if (!eps_ok(q_eps)) return fail(BFQ_ERR_ARG, "q_eps must be positive and finite");
        if (!sfmt_ok(scale_fmt)) return fail(BFQ_ERR_ARG, "unknown scale format");
        const bfq_status s = out_scale_strides(layout, scale_ld, M, 2 * F / 128, scale_fmt, false,
                                               &a.s_stride_m, &a.s_stride_g, &a.packed);
        if (s != BFQ_OK) return s;
        a.qtype = qtype_of(q_dtype);
    }
    if (M == 0) return BFQ_OK;
    a.pre = preact;
    a.dh = dh;
    a.dpre = dpre;
    a.q = q;
    a.scales = scales;
    a.h = h;
    a.M = M;
    a.F = F;
    a.ue8m0 = scale_fmt == BFQ_SCALE_UE8M0;
    a.q_eps = q_eps;
    gated_activation((int)act, &a.c1, &a.c3);
    const hipError_t e = launch_gated_bwd(a, (hipStream_t)stream);
    if (e != hipSuccess) return fail(BFQ_ERR_HIP, hipGetErrorString(e));
    return BFQ_OK;
}

bfq_status bfq_transpose_weights(const void* w_q, const float* w_scales, int64_t N, int64_t K,
                                 bfq_dtype q_dtype, void* wt_q, float* wt_scales, void* stream) {
    if (!w_q || !w_scales || !wt_q || !wt_scales)
        return fail(BFQ_ERR_NULL, "w_q, w_scales, wt_q and wt_scales must be non-NULL");
    if (q_dtype != BFQ_E4M3FN && q_dtype != BFQ_INT8)
        return fail(BFQ_ERR_DTYPE, "q_dtype must be BFQ_E4M3FN or BFQ_INT8");
    if (N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0)
        return fail(BFQ_ERR_SHAPE, "N and K must be non-negative multiples of 128");
    if (N / 64 > 65535 || K > (1 << 23)) return fail(BFQ_ERR_SHAPE, "need N < 2^22 and K <= 2^23");
    if (!aligned(w_q, 16) || !aligned(wt_q, 16) || !aligned(w_scales, 4) || !aligned(wt_scales, 4))
        return fail(BFQ_ERR_ALIGN, "w_q and wt_q must be 16-byte aligned, scales 4-byte");
    const uintptr_t a = (uintptr_t)w_q, b = (uintptr_t)wt_q, n = (uintptr_t)(N * K);
    if (n > 0 && a < b + n && b < a + n) return fail(BFQ_ERR_ARG, "w_q and wt_q must not overlap");
    if (N == 0 || K == 0) return BFQ_OK;
    const hipError_t e = launch_transpose_weights(w_q, w_scales, wt_q, wt_scales, N, K, (hipStream_t)stream);
    if (e != hipSuccess) return fail(BFQ_ERR_HIP, hipGetErrorString(e));
    return BFQ_OK;
}

}  // extern "C"

// ------------------------------------------------------------------------ norms ----

namespace {

// The arguments that the norm step and its gradients share.
bfq_status check_norm(const void* y, const void* residual, bfq_dtype res_dtype, const void* w_post,
                      const void* gate, bfq_gate_kind kind, const void* w_pre, float norm_eps,
                      int64_t M, int64_t K) {
    if (M != 0 && !residual) return fail(BFQ_ERR_NULL, "the residual must be non-NULL");
    if (res_dtype != BFQ_BF16 && res_dtype != BFQ_FP32)
        return fail(BFQ_ERR_DTYPE, "res_dtype must be BFQ_BF16 or BFQ_FP32");
    if (kind != BFQ_GATE_NONE && kind != BFQ_GATE_CHANNEL && kind != BFQ_GATE_TOKEN && kind != BFQ_GATE_FULL)
        return fail(BFQ_ERR_ARG, "unknown gate kind");
    // an empty batch has no rows to point at, so a tensor over rows may be NULL there
    if (kind == BFQ_GATE_NONE ? gate != nullptr : !gate && (M != 0 || kind == BFQ_GATE_CHANNEL))
        return fail(BFQ_ERR_NULL, "gate must be given with a gate kind, and NULL with BFQ_GATE_NONE");
    if (M != 0 && !y && (w_post || gate))
        return fail(BFQ_ERR_NULL, "w_post and gate act on y: NULL without it");
    if (!(norm_eps > 0.0f) || norm_eps > 3.0e38f)
        return fail(BFQ_ERR_ARG, "norm_eps must be positive and finite");
    if (M < 0 || K <= 0 || K % 8 != 0 || K > kNormMaxK)
        return fail(BFQ_ERR_SHAPE, "need M >= 0 and K a positive multiple of 8, at most 16384");
    if (M >= kMaxRows) return fail(BFQ_ERR_SHAPE, "need M < 2^24 - 4");
    if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(w_post, 16) || !aligned(w_pre, 16) ||
        !aligned(gate, kind == BFQ_GATE_TOKEN ? 2 : 16))
        return fail(BFQ_ERR_ALIGN, "row and channel tensors must be 16-byte aligned, a token gate 2-byte");
    return BFQ_OK;
}

}  // namespace

extern "C" {

bfq_status bfq_norm_residual(const void* y, const void* residual, bfq_dtype res_dtype,
                             const void* w_post, const void* gate, bfq_gate_kind gate_kind,
                             float res_scale, const void* w_pre, float norm_eps, void* res_out,
                             void* normed, void* q, bfq_dtype q_dtype, int32_t group_size,
                             float* scales, bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                             bfq_scale_format scale_fmt, int64_t M, int64_t K, void* stream) {
    bfq_status st = check_norm(y, residual, res_dtype, w_post, gate, gate_kind, w_pre, norm_eps, M, K);
    if (st != BFQ_OK) return st;
    if (M != 0 && (y != nullptr) != (res_out != nullptr))
        return fail(BFQ_ERR_NULL, "res_out must be given with y, and NULL without it");
    if (M != 0 && (q != nullptr) != (scales != nullptr))
        return fail(BFQ_ERR_NULL, "q and scales must both be given or both be NULL");
    if (M != 0 && (w_pre != nullptr) != (normed || q))
        return fail(BFQ_ERR_NULL, "normed or q must be given with w_pre, and both be NULL without it");
    if (M != 0 && !y && !w_pre) return fail(BFQ_ERR_NULL, "one of y and w_pre must be non-NULL");
    if (!aligned(res_out, 16) || !aligned(normed, 16) || !aligned(q, 16) || !aligned(scales, 4))
        return fail(BFQ_ERR_ALIGN, "row tensors must be 16-byte aligned, scales 4-byte");
    NormArgs a{};
    if (q) {
        if (q_dtype != BFQ_E4M3FN && q_dtype != BFQ_INT8)
            return fail(BFQ_ERR_DTYPE, "q_dtype must be BFQ_E4M3FN or BFQ_INT8");
        const bool per_token = group_size == K && K != 128;
        if (K % 128 != 0 || (group_size != 128 && !per_token))
            return fail(BFQ_ERR_SHAPE, "codes need K a multiple of 128 and group_size 128 or K");
        if (!eps_ok(q_eps)) return fail(BFQ_ERR_ARG, "q_eps must be positive and finite");
        if (!sfmt_ok(scale_fmt)) return fail(BFQ_ERR_ARG, "unknown scale format");
        st = out_scale_strides(layout, scale_ld, M, K / group_size, scale_fmt, per_token,
                               &a.s_stride_m, &a.s_stride_g, &a.packed);
        if (st != BFQ_OK) return st;
        a.qtype = qtype_of(q_dtype);
        a.per_token = per_token ? 1 : 0;
        a.ue8m0 = scale_fmt == BFQ_SCALE_UE8M0;
        a.q_eps = q_eps;
    }
    if (M == 0) return BFQ_OK;
    a.y = y;
    a.residual = residual;
    a.w_post = w_post;
    a.gate = gate;
    a.gate_kind = (int)gate_kind;
    a.res_scale = res_scale;
    a.w_pre = w_pre;
    a.norm_eps = norm_eps;
    a.M = M;
    a.K = K;
    a.res_out = res_out;
    a.normed = normed;
    a.q = q;
    a.scales = scales;
    a.invariant = batch_invariant() ? 1 : 0;
    const hipError_t e = launch_norm_residual(a, res_dtype == BFQ_FP32, (hipStream_t)stream);
    if (e != hipSuccess) return fail(BFQ_ERR_HIP, hipGetErrorString(e));
    return BFQ_OK;
}

size_t bfq_norm_residual_backward_workspace_bytes(int64_t M, int64_t K) {
    if (M <= 0 || K <= 0) return 0;
    if (M >= kMaxRows || K > kNormMaxK) return SIZE_MAX;
    return (size_t)norm_bwd_groups(M, K) * 2 * (size_t)K * sizeof(float);
}

bfq_status bfq_norm_residual_backward(const void* y, const void* res_out, bfq_dtype res_dtype,
                                      const void* w_post, const void* gate,
                                      bfq_gate_kind gate_kind, float res_scale, const void* w_pre,
                                      float norm_eps, const void* d_normed, const void* d_res_out,
                                      void* d_res, void* d_y, float* d_w_pre, float* d_w_post,
                                      void* d_gate, int64_t M, int64_t K, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    const bfq_status st = check_norm(y, res_out, res_dtype, w_post, gate, gate_kind, w_pre, norm_eps, M, K);
    if (st != BFQ_OK) return st;
    if (M != 0 && !d_res) return fail(BFQ_ERR_NULL, "d_res must be non-NULL");
    if (M != 0 && (y != nullptr) != (d_y != nullptr))
        return fail(BFQ_ERR_NULL, "d_y must be given with y, and NULL without it");
    if (M != 0 && (w_pre != nullptr) != (d_normed != nullptr))
        return fail(BFQ_ERR_NULL, "d_normed must be given with w_pre, and NULL without it");
    if ((d_w_pre && !w_pre) || (d_w_post && !w_post) || (d_gate && gate_kind == BFQ_GATE_NONE))
        return fail(BFQ_ERR_NULL, "d_w_pre, d_w_post and d_gate need w_pre, w_post and a gate");
    if (!aligned(d_normed, 16) || !aligned(d_res_out, 16) || !aligned(d_res, 16) || !aligned(d_y, 16) ||
        !aligned(d_w_pre, 4) || !aligned(d_w_post, 4) || !aligned(workspace, 16) ||
        !aligned(d_gate, gate_kind == BFQ_GATE_FULL ? 16 : 4))
        return fail(BFQ_ERR_ALIGN, "row tensors and workspace must be 16-byte aligned, sums 4-byte");
    const bool columns = d_w_pre || d_w_post || (d_gate && gate_kind == BFQ_GATE_CHANNEL);
    const size_t need = columns ? bfq_norm_residual_backward_workspace_bytes(M, K) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(BFQ_ERR_WORKSPACE, "workspace of " + std::to_string(need) + " bytes required");
    if (M == 0 && !columns) return BFQ_OK;
    NormArgs a{};
    a.y = y;
    a.residual = res_out;
    a.w_post = w_post;
    a.gate = gate;
    a.gate_kind = (int)gate_kind;
    a.res_scale = res_scale;
    a.w_pre = w_pre;
    a.norm_eps = norm_eps;
    a.M = M;
    a.K = K;
    a.d_normed = d_normed;
    a.d_res_out = d_res_out;
    a.d_res = d_res;
    a.d_y = d_y;
    a.d_w_pre = d_w_pre;
    a.d_w_post = d_w_post;
    a.d_gate = d_gate;
    a.columns = columns ? 1 : 0;
    a.partials = static_cast<float*>(workspace);
    const hipError_t e = launch_norm_residual_bwd(a, res_dtype == BFQ_FP32, (hipStream_t)stream);
    if (e != hipSuccess) return fail(BFQ_ERR_HIP, hipGetErrorString(e));
    return BFQ_OK;
}

}  // extern "C"
