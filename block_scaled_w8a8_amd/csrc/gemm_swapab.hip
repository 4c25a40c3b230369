// Decode-shaped block-scaled GEMM for gfx950 ("variant 1", swap-AB streaming) plus the
// deterministic split-K reduction and the int8 block-partials probe.
//
// Pages cited by title and section:
//   [HELION] "Building a High-Performance and Portable vLLM Linear Backend with Helion",
//            kernel section: swap-AB computes the product transposed so that a small M
//            does not waste the wide tile dimension; split-K splits the K range over
//            workgroups to add parallelism when M and/or N are small; the Hopper heuristic
//            picks swap-AB below 32 tokens.
//   [BENCH]  "vLLM DeepGEMM FP8 Block GEMM 基准测试 ..." §4.3: for small m the kernel is
//            bandwidth bound, so GB/s is the number that matters.
//
// gfx950 design: with M <= 64 tokens the whole cost is streaming the weight codes once from
// HBM. Each wave owns NWR weight rows and loads their 16x128-byte MFMA fragments straight
// from global memory into registers (no LDS round trip), keeping D K-blocks in flight in a
// register ring. The token codes (at most 64 x K bytes, L2-resident) ride in the second
// MFMA operand, so the result tile is W*A^T: each lane holds one token and four
// consecutive weight rows, stored back row-major into C. Lane l loads 16-byte chunks
// (l/16) and (l/16)+4 of its row, so each load instruction covers 64 contiguous bytes of
// 16 rows. With packed weights (W_PACKED16) the same two fragment halves are 1 KB of
// contiguous memory each, which is what lets the weight stream approach the HBM peak.
// A workgroup holds NWAVES strips of NWR rows, and KW waves per strip share its K range:
// wave wk streams the wk-th contiguous slice of the strip's K blocks, and the KW partial
// tiles are summed through LDS in ascending wk (deterministic) before one wave stores the
// strip. That gives a weight matrix of few strips (N / 16 = 1536 at N = 24576) enough waves
// to keep HBM busy without a second kernel. Split-K across workgroups writes fp32 partials
// that a second kernel sums in a fixed order.
// CH = 1 (per-token x per-channel scales, [HELION] scope section): no scale loads in the K
// loop; the MFMA accumulates the wave's K range (int8: exact int32 in the accumulator's
// bits) and each wave scales its partial tile by token and channel scale before the
// in-workgroup sum. CH = 2: block scales with the activation scales as packed UE8M0 words
// (four K blocks per word); a compile-time mode, so the other modes keep their registers.
#include "gemm_swapab_body.h"

namespace bfq {

template <int MT, int NWR, int NWAVES, int KW, int D, int QT, int OT, int WL, int CH, int MOE = 0>
__global__ __launch_bounds__(64 * NWAVES * KW) void gemm_swapab_kernel(GemmArgs p) {
    swapab_body<MT, NWR, NWAVES, KW, D, QT, OT, WL, CH, MOE, 0>(p);
}

template <int MT, int NWR, int NWAVES, int KW, int D, int QT, int OT, int WL, int CH, int MOE = 0>
__global__ __launch_bounds__(64 * NWAVES * KW) void gemm_swapab_lds_kernel(GemmArgs p) {
    swapab_lds_body<MT, NWR, NWAVES, KW, D, QT, OT, WL, CH, MOE, 0>(p);
}

template <int MT, int NWR, int NWAVES, int KW, int D, int QT, int OT, int WL, int CH>
hipError_t launch_swapab(const GemmArgs& a, hipStream_t stream) {
    const int64_t strips = (a.N + NWR * NWAVES - 1) / (NWR * NWAVES);
    dim3 grid((unsigned)strips, (unsigned)((a.M + MT - 1) / MT), (unsigned)a.split);
    hipLaunchKernelGGL((gemm_swapab_kernel<MT, NWR, NWAVES, KW, D, QT, OT, WL, CH>), grid,
                       dim3(64 * NWAVES * KW), 0, stream, a);
    return hipGetLastError();
}

template <int MT, int NWR, int NWAVES, int KW, int D, int QT, int OT, int WL, int CH>
hipError_t launch_swapab_lds(const GemmArgs& a, hipStream_t stream) {
    const int64_t strips = (a.N + NWR * NWAVES - 1) / (NWR * NWAVES);
    dim3 grid((unsigned)strips, (unsigned)((a.M + MT - 1) / MT), (unsigned)a.split);
    hipLaunchKernelGGL((gemm_swapab_lds_kernel<MT, NWR, NWAVES, KW, D, QT, OT, WL, CH>), grid,
                       dim3(64 * NWAVES * KW), 0, stream, a);
    return hipGetLastError();
}

// grouped (MoE) forms: grid height = the per-expert row tiles' upper bound
template <int MT, int NWR, int NWAVES, int KW, int D, int QT, int OT, int WL, int CH>
hipError_t launch_moe_swapab(const GemmArgs& a, hipStream_t stream) {
    const int64_t strips = (a.N + NWR * NWAVES - 1) / (NWR * NWAVES);
    dim3 grid((unsigned)strips, (unsigned)moe_max_tiles(a.M, a.moe_experts, MT), (unsigned)a.split);
    hipLaunchKernelGGL((gemm_swapab_kernel<MT, NWR, NWAVES, KW, D, QT, OT, WL, CH, 1>), grid,
                       dim3(64 * NWAVES * KW), 0, stream, a);
    return hipGetLastError();
}

template <int MT, int NWR, int NWAVES, int KW, int D, int QT, int OT, int WL, int CH>
hipError_t launch_moe_swapab_lds(const GemmArgs& a, hipStream_t stream) {
    const int64_t strips = (a.N + NWR * NWAVES - 1) / (NWR * NWAVES);
    dim3 grid((unsigned)strips, (unsigned)moe_max_tiles(a.M, a.moe_experts, MT), (unsigned)a.split);
    hipLaunchKernelGGL((gemm_swapab_lds_kernel<MT, NWR, NWAVES, KW, D, QT, OT, WL, CH, 1>), grid,
                       dim3(64 * NWAVES * KW), 0, stream, a);
    return hipGetLastError();
}

// bfq_tile for variant 1: bm = MT tokens, bn = NWR * NW rows per workgroup, waves_m = KW
// waves sharing each strip's K range, waves_n = NW strips, stages = D K blocks in flight,
// sched 0 = tokens per wave from L2, sched 1 = tokens shared through LDS.
#define BFQ_SAB_ENTRY(MT, NWR, NW, KW, D, QT, OT, WL, CH)                                  \
    KernelEntry{bfq_tile{1, MT, NWR * NW, 128, 1, KW, NW, D, 1, 0, 0, 0}, QT, OT, WL,         \
                (CH) == 1 ? S_CHANNEL : (CH) == 2 ? S_PACKED : S_FP32,                   \
                &launch_swapab<MT, NWR, NW, KW, D, QT, OT, WL, CH>}
#define BFQ_SAB_ALL_OUT(MT, NWR, NW, KW, D, QT, WL, CH)                                    \
    BFQ_SAB_ENTRY(MT, NWR, NW, KW, D, QT, O_BF16, WL, CH),                                 \
        BFQ_SAB_ENTRY(MT, NWR, NW, KW, D, QT, O_FP16, WL, CH),                             \
        BFQ_SAB_ENTRY(MT, NWR, NW, KW, D, QT, O_FP32, WL, CH)
#define BFQ_SAB_BOTH(MT, NWR, NW, KW, D, QT)                                                \
    BFQ_SAB_ALL_OUT(MT, NWR, NW, KW, D, QT, W_ROW, 0), BFQ_SAB_ALL_OUT(MT, NWR, NW, KW, D, QT, W_PACKED16, 0)
// per-token x per-channel scales
#define BFQ_SAB_CH(MT, NWR, NW, KW, D, QT)                                                  \
    BFQ_SAB_ALL_OUT(MT, NWR, NW, KW, D, QT, W_ROW, 1), BFQ_SAB_ALL_OUT(MT, NWR, NW, KW, D, QT, W_PACKED16, 1)
// block scales, activation scales as packed UE8M0 words
#define BFQ_SAB_PK(MT, NWR, NW, KW, D, QT)                                                  \
    BFQ_SAB_ALL_OUT(MT, NWR, NW, KW, D, QT, W_ROW, 2), BFQ_SAB_ALL_OUT(MT, NWR, NW, KW, D, QT, W_PACKED16, 2)

#define BFQ_SABL_ENTRY(MT, NWR, NW, KW, D, QT, OT, WL, CH)                                 \
    KernelEntry{bfq_tile{1, MT, NWR * NW, 128, 1, KW, NW, D, 1, 1, 0, 0}, QT, OT, WL,         \
                (CH) == 1 ? S_CHANNEL : (CH) == 2 ? S_PACKED : S_FP32,                   \
                &launch_swapab_lds<MT, NWR, NW, KW, D, QT, OT, WL, CH>}
#define BFQ_SABL_ALL_OUT(MT, NWR, NW, KW, D, QT, WL, CH)                                   \
    BFQ_SABL_ENTRY(MT, NWR, NW, KW, D, QT, O_BF16, WL, CH),                                \
        BFQ_SABL_ENTRY(MT, NWR, NW, KW, D, QT, O_FP16, WL, CH),                            \
        BFQ_SABL_ENTRY(MT, NWR, NW, KW, D, QT, O_FP32, WL, CH)
#define BFQ_SABL_BOTH(MT, NWR, NW, KW, D, QT)                                               \
    BFQ_SABL_ALL_OUT(MT, NWR, NW, KW, D, QT, W_ROW, 0), BFQ_SABL_ALL_OUT(MT, NWR, NW, KW, D, QT, W_PACKED16, 0)
#define BFQ_SABL_CH(MT, NWR, NW, KW, D, QT)                                                 \
    BFQ_SABL_ALL_OUT(MT, NWR, NW, KW, D, QT, W_ROW, 1), BFQ_SABL_ALL_OUT(MT, NWR, NW, KW, D, QT, W_PACKED16, 1)
#define BFQ_SABL_PK(MT, NWR, NW, KW, D, QT)                                                 \
    BFQ_SABL_ALL_OUT(MT, NWR, NW, KW, D, QT, W_ROW, 2), BFQ_SABL_ALL_OUT(MT, NWR, NW, KW, D, QT, W_PACKED16, 2)

static const KernelEntry kSwapabKernels[] = {
    BFQ_SABL_BOTH(16, 16, 8, 1, 8, Q_FP8),
    BFQ_SABL_BOTH(16, 16, 4, 2, 8, Q_FP8),
    BFQ_SABL_BOTH(32, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(32, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(32, 16, 4, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(48, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(48, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(64, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(64, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(64, 16, 4, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(64, 32, 4, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(96, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(96, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(128, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(128, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(32, 16, 6, 1, 8, Q_FP8),
    BFQ_SABL_BOTH(32, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(64, 16, 6, 1, 8, Q_FP8),
    BFQ_SABL_BOTH(64, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(96, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(128, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(96, 32, 4, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(128, 32, 4, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(128, 32, 6, 1, 4, Q_FP8),
    BFQ_SABL_BOTH(64, 32, 6, 2, 4, Q_FP8),
    BFQ_SABL_BOTH(16, 16, 8, 1, 8, Q_INT8),
    BFQ_SABL_BOTH(32, 16, 8, 1, 4, Q_INT8),
    BFQ_SABL_BOTH(64, 16, 8, 1, 4, Q_INT8),
    BFQ_SABL_BOTH(128, 16, 8, 1, 4, Q_INT8),
    BFQ_SAB_BOTH(16, 32, 4, 1, 4, Q_FP8),
    BFQ_SAB_BOTH(16, 16, 4, 1, 8, Q_FP8),
    BFQ_SAB_BOTH(16, 16, 8, 1, 8, Q_FP8),
    BFQ_SAB_BOTH(16, 32, 8, 1, 4, Q_FP8),
    BFQ_SAB_BOTH(16, 64, 4, 1, 2, Q_FP8),
    BFQ_SAB_BOTH(16, 32, 4, 1, 8, Q_FP8),
    BFQ_SAB_BOTH(32, 32, 4, 1, 4, Q_FP8),
    BFQ_SAB_BOTH(64, 32, 4, 1, 2, Q_FP8),
    BFQ_SAB_BOTH(16, 16, 1, 4, 4, Q_FP8),
    BFQ_SAB_BOTH(16, 16, 1, 4, 8, Q_FP8),
    BFQ_SAB_BOTH(16, 16, 2, 2, 8, Q_FP8),
    BFQ_SAB_BOTH(16, 16, 1, 8, 4, Q_FP8),
    BFQ_SAB_BOTH(16, 32, 1, 4, 4, Q_FP8),
    BFQ_SAB_BOTH(32, 16, 1, 4, 4, Q_FP8),
    BFQ_SAB_BOTH(64, 16, 1, 4, 2, Q_FP8),
    BFQ_SAB_BOTH(32, 32, 1, 4, 4, Q_FP8),
    BFQ_SAB_BOTH(16, 32, 4, 1, 4, Q_INT8),
    BFQ_SAB_BOTH(32, 32, 4, 1, 4, Q_INT8),
    BFQ_SAB_BOTH(64, 32, 4, 1, 2, Q_INT8),
    BFQ_SAB_BOTH(16, 16, 1, 4, 4, Q_INT8),
    BFQ_SAB_BOTH(32, 16, 1, 4, 4, Q_INT8),
    BFQ_SAB_BOTH(64, 16, 1, 4, 2, Q_INT8),
    BFQ_SABL_CH(16, 16, 8, 1, 8, Q_FP8),
    BFQ_SABL_CH(32, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_CH(32, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_CH(32, 16, 4, 2, 4, Q_FP8),
    BFQ_SABL_CH(64, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_CH(64, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_CH(64, 16, 4, 2, 4, Q_FP8),
    BFQ_SABL_CH(96, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_CH(128, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_CH(128, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_CH(16, 16, 8, 1, 8, Q_INT8),
    BFQ_SABL_CH(32, 16, 8, 1, 4, Q_INT8),
    BFQ_SABL_CH(64, 16, 8, 1, 4, Q_INT8),
    BFQ_SABL_CH(128, 16, 8, 1, 4, Q_INT8),
    BFQ_SAB_CH(16, 32, 4, 1, 4, Q_FP8),
    BFQ_SAB_CH(16, 16, 4, 1, 8, Q_FP8),
    BFQ_SAB_CH(16, 16, 8, 1, 8, Q_FP8),
    BFQ_SAB_CH(32, 32, 4, 1, 4, Q_FP8),
    BFQ_SAB_CH(16, 16, 1, 4, 4, Q_FP8),
    BFQ_SAB_CH(16, 16, 1, 4, 8, Q_FP8),
    BFQ_SAB_CH(16, 32, 1, 4, 4, Q_FP8),
    BFQ_SAB_CH(32, 16, 1, 4, 4, Q_FP8),
    BFQ_SAB_CH(64, 16, 1, 4, 2, Q_FP8),
    BFQ_SAB_CH(16, 32, 4, 1, 4, Q_INT8),
    BFQ_SAB_CH(32, 32, 4, 1, 4, Q_INT8),
    BFQ_SAB_CH(16, 16, 1, 4, 4, Q_INT8),
    BFQ_SAB_CH(32, 16, 1, 4, 4, Q_INT8),
    // fp8 block scales read as packed UE8M0 activation-scale words
    BFQ_SABL_PK(96, 32, 4, 1, 4, Q_FP8),
    BFQ_SABL_PK(128, 32, 4, 1, 4, Q_FP8),
    BFQ_SABL_PK(128, 32, 6, 1, 4, Q_FP8),
    BFQ_SABL_PK(64, 32, 6, 2, 4, Q_FP8),
    BFQ_SABL_PK(16, 16, 8, 1, 8, Q_FP8),
    BFQ_SABL_PK(16, 16, 4, 2, 8, Q_FP8),
    BFQ_SABL_PK(32, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_PK(32, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_PK(32, 16, 4, 2, 4, Q_FP8),
    BFQ_SABL_PK(48, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_PK(48, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_PK(64, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_PK(64, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_PK(64, 16, 4, 2, 4, Q_FP8),
    BFQ_SABL_PK(64, 32, 4, 1, 4, Q_FP8),
    BFQ_SABL_PK(96, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_PK(96, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_PK(128, 16, 8, 1, 4, Q_FP8),
    BFQ_SABL_PK(128, 16, 6, 1, 4, Q_FP8),
    BFQ_SABL_PK(32, 16, 6, 1, 8, Q_FP8),
    BFQ_SABL_PK(32, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_PK(64, 16, 6, 1, 8, Q_FP8),
    BFQ_SABL_PK(64, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_PK(96, 16, 6, 2, 4, Q_FP8),
    BFQ_SABL_PK(128, 16, 6, 2, 4, Q_FP8),
    BFQ_SAB_PK(16, 32, 4, 1, 4, Q_FP8),
    BFQ_SAB_PK(16, 16, 4, 1, 8, Q_FP8),
    BFQ_SAB_PK(16, 16, 8, 1, 8, Q_FP8),
    BFQ_SAB_PK(16, 32, 8, 1, 4, Q_FP8),
    BFQ_SAB_PK(16, 64, 4, 1, 2, Q_FP8),
    BFQ_SAB_PK(16, 32, 4, 1, 8, Q_FP8),
    BFQ_SAB_PK(32, 32, 4, 1, 4, Q_FP8),
    BFQ_SAB_PK(64, 32, 4, 1, 2, Q_FP8),
    BFQ_SAB_PK(16, 16, 1, 4, 4, Q_FP8),
    BFQ_SAB_PK(16, 16, 1, 4, 8, Q_FP8),
    BFQ_SAB_PK(16, 16, 2, 2, 8, Q_FP8),
    BFQ_SAB_PK(16, 16, 1, 8, 4, Q_FP8),
    BFQ_SAB_PK(16, 32, 1, 4, 4, Q_FP8),
    BFQ_SAB_PK(32, 16, 1, 4, 4, Q_FP8),
    BFQ_SAB_PK(64, 16, 1, 4, 2, Q_FP8),
    BFQ_SAB_PK(32, 32, 1, 4, 4, Q_FP8),
};

// grouped (MoE) swap-AB kernels, fp8, fp32 or UE8M0 block scales (S_FP32 serves both) and
// packed UE8M0 words
#define BFQ_MOE_SAB_ENTRY(MT, NWR, NW, KW, D, OT, WL, CH)                                      \
    KernelEntry{bfq_tile{1, MT, NWR * NW, 128, 1, KW, NW, D, 1, 0, 0, 0}, Q_FP8, OT, WL,         \
                (CH) == 2 ? S_PACKED : S_FP32, &launch_moe_swapab<MT, NWR, NW, KW, D, Q_FP8, OT, WL, CH>, 1}
#define BFQ_MOE_SABL_ENTRY(MT, NWR, NW, KW, D, OT, WL, CH)                                     \
    KernelEntry{bfq_tile{1, MT, NWR * NW, 128, 1, KW, NW, D, 1, 1, 0, 0}, Q_FP8, OT, WL,         \
                (CH) == 2 ? S_PACKED : S_FP32,                                                 \
                &launch_moe_swapab_lds<MT, NWR, NW, KW, D, Q_FP8, OT, WL, CH>, 1}
#define BFQ_MOE_X6(ENTRY, MT, NWR, NW, KW, D, CH)                                               \
    ENTRY(MT, NWR, NW, KW, D, O_BF16, W_ROW, CH), ENTRY(MT, NWR, NW, KW, D, O_FP16, W_ROW, CH),   \
        ENTRY(MT, NWR, NW, KW, D, O_FP32, W_ROW, CH),                                          \
        ENTRY(MT, NWR, NW, KW, D, O_BF16, W_PACKED16, CH),                                     \
        ENTRY(MT, NWR, NW, KW, D, O_FP16, W_PACKED16, CH),                                     \
        ENTRY(MT, NWR, NW, KW, D, O_FP32, W_PACKED16, CH)
#define BFQ_MOE_SAB(MT, NWR, NW, KW, D)                                                        \
    BFQ_MOE_X6(BFQ_MOE_SAB_ENTRY, MT, NWR, NW, KW, D, 0), BFQ_MOE_X6(BFQ_MOE_SAB_ENTRY, MT, NWR, NW, KW, D, 2)
#define BFQ_MOE_SABL(MT, NWR, NW, KW, D)                                                       \
    BFQ_MOE_X6(BFQ_MOE_SABL_ENTRY, MT, NWR, NW, KW, D, 0), BFQ_MOE_X6(BFQ_MOE_SABL_ENTRY, MT, NWR, NW, KW, D, 2)

static const KernelEntry kMoeSwapabKernels[] = {
    BFQ_MOE_SAB(16, 32, 4, 1, 4),
    BFQ_MOE_SAB(16, 16, 4, 1, 8),
    BFQ_MOE_SAB(16, 16, 1, 4, 4),
    BFQ_MOE_SAB(32, 32, 4, 1, 4),
    BFQ_MOE_SABL(16, 16, 8, 1, 8),
    BFQ_MOE_SABL(32, 16, 8, 1, 4),
    BFQ_MOE_SABL(32, 16, 6, 1, 4),
    BFQ_MOE_SABL(32, 16, 4, 2, 4),
    BFQ_MOE_SABL(64, 16, 8, 1, 4),
    BFQ_MOE_SABL(64, 16, 6, 1, 4),
    BFQ_MOE_SABL(64, 16, 4, 2, 4),
    BFQ_MOE_SABL(96, 16, 6, 1, 4),
    BFQ_MOE_SABL(128, 16, 8, 1, 4),
    BFQ_MOE_SABL(128, 16, 6, 1, 4),
};

const KernelEntry* moe_swapab_kernels(int* count) {
    *count = (int)(sizeof(kMoeSwapabKernels) / sizeof(kMoeSwapabKernels[0]));
    return kMoeSwapabKernels;
}

const KernelEntry* swapab_kernels(int* count) {
    *count = (int)(sizeof(kSwapabKernels) / sizeof(kSwapabKernels[0]));
    return kSwapabKernels;
}

// ------------------------------------------------------------ split-K reduce ----
// out[i] = sum over z of part[z][i], added in z order (so results are run-to-run identical
// and do not depend on the split kernel's timing). The partial loads of B splits are all
// issued before any is waited on (B >= split: one memory round trip, rather than one per
// split, which is what the reduce of a small output costs); slots past the last split
// re-read the last partial, which stays in cache, and are not added.
template <int OT, int B>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ part,
                                                            void* __restrict__ out,
                                                            int64_t MN, int split) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= MN) return;                       // MN is a multiple of 128
    const float* p = part + i;
    v4f s = *reinterpret_cast<const v4f*>(p);
    for (int z0 = 1; z0 < split; z0 += B) {
        v4f t[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int z = z0 + j < split ? z0 + j : split - 1;
            t[j] = *reinterpret_cast<const v4f*>(p + (int64_t)z * MN);
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const bool live = z0 + j < split;
            const v4f u = {s.x + t[j].x, s.y + t[j].y, s.z + t[j].z, s.w + t[j].w};
            s = live ? u : s;
        }
    }
    store4<OT>(out, i, s);
}

template <int OT>
static void launch_reduce_ot(const float* partials, void* out, int64_t MN, int split,
                             hipStream_t stream) {
    dim3 grid((unsigned)((MN / 4 + 255) / 256));
    if (split <= 3)
        hipLaunchKernelGGL((splitk_reduce_kernel<OT, 2>), grid, dim3(256), 0, stream, partials, out, MN, split);
    else if (split <= 5)
        hipLaunchKernelGGL((splitk_reduce_kernel<OT, 4>), grid, dim3(256), 0, stream, partials, out, MN, split);
    else if (split <= 9)
        hipLaunchKernelGGL((splitk_reduce_kernel<OT, 8>), grid, dim3(256), 0, stream, partials, out, MN, split);
    else
        hipLaunchKernelGGL((splitk_reduce_kernel<OT, 16>), grid, dim3(256), 0, stream, partials, out, MN, split);
}

hipError_t launch_splitk_reduce(const float* partials, void* out, int64_t M, int64_t N,
                                int split, int otype, hipStream_t stream) {
    const int64_t MN = M * N;
    if (otype == O_BF16)
        launch_reduce_ot<O_BF16>(partials, out, MN, split, stream);
    else if (otype == O_FP16)
        launch_reduce_ot<O_FP16>(partials, out, MN, split, stream);
    else
        launch_reduce_ot<O_FP32>(partials, out, MN, split, stream);
    return hipGetLastError();
}

// ------------------------------------------------------------ int8 partials probe ----
// One wave per (16 weight rows, 16 tokens, K block): the same two chained int8 MFMAs the
// GEMM kernels use, written out as exact int32 block partials [K/128][M][N].
__global__ __launch_bounds__(64) void block_partials_i32_kernel(const int8_t* __restrict__ A,
                                                                const int8_t* __restrict__ W,
                                                                int32_t* __restrict__ out,
                                                                int64_t M, int64_t N, int64_t K) {
    const int lane = threadIdx.x, frow = lane & 15, fgrp = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16, kb = blockIdx.z;
    int64_t n = n0 + frow, m = m0 + frow;
    m = m < M ? m : M - 1;
    const int8_t* wr = W + n * K + kb * 128 + fgrp * 16;
    const int8_t* ar = A + m * K + kb * 128 + fgrp * 16;
    v4i pi = mfma_i8_16x16x64(*reinterpret_cast<const v4i*>(wr), *reinterpret_cast<const v4i*>(ar),
                              v4i{0, 0, 0, 0});
    pi = mfma_i8_16x16x64(*reinterpret_cast<const v4i*>(wr + 64), *reinterpret_cast<const v4i*>(ar + 64), pi);
    const int64_t mo = m0 + frow;
    if (mo < M) {
        int32_t* o = out + (kb * M + mo) * N + n0 + 4 * fgrp;
        *reinterpret_cast<v4i*>(o) = pi;
    }
}

hipError_t launch_block_partials_i32(const void* a, const void* w, int32_t* out, int64_t M,
                                     int64_t N, int64_t K, hipStream_t stream) {
    dim3 grid((unsigned)(N / 16), (unsigned)((M + 15) / 16), (unsigned)(K / 128));
    hipLaunchKernelGGL(block_partials_i32_kernel, grid, dim3(64), 0, stream, (const int8_t*)a,
                       (const int8_t*)w, out, M, N, K);
    return hipGetLastError();
}

}  // namespace bfq
