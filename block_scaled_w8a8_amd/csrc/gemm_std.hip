// Standard block-scaled GEMM for gfx950 ("variant 0"): one workgroup per BM x BN output
// tile, A (token codes) and W (weight codes) tiles of one 128-wide K block staged through
// LDS with direct global->LDS loads, double-buffered, consumed by MFMA, and the per-K-block
// scale applied in registers right after each block's product.
//
// Pages cited by title and section:
//   [BENCH]  "vLLM DeepGEMM FP8 Block GEMM 基准测试 ..." §4.2: the kernel walks K in
//            block-size steps and multiplies each step's dot product by the activation and
//            weight scales before accumulating; a grouped tile order improves L2 hits.
//   [CONFIG] "vLLM 量化 Kernel 配置机制 ..." §2: a launch is described by its tile sizes,
//            GROUP_SIZE_M, number of warps and pipeline stages.
//   [HELION] "Building a High-Performance and Portable vLLM Linear Backend with Helion",
//            kernel section: split-K divides the K range over several workgroups.
//
// gfx950 design:
//  * MFMA v_mfma_f32_16x16x128_f8f6f4 (e4m3) or v_mfma_i32_16x16x64_i8 (int8): one fp8
//    MFMA covers one whole 128-wide K block for a 16x16 sub-tile, so its result is the
//    block partial P and the scale step is acc = fma(P, sa[m,kb]*sw[nb,kb], acc).
//    sched 2 instead uses 32x32 sub-tiles: two v_mfma_f32_32x32x64_f8f6f4 per K block
//    (each weight fragment feeds twice the MFMA work per LDS read; a lane owns one token and
//    four groups of four output columns).
//  * sched 3 (power-of-two scales only): the scales are applied inside the block-scaled MFMA
//    as E8M0 exponents — the weight scale (one per 128-row block, uniform over a wave) for
//    the first operand, each lane's token scale for the second — and the MFMA accumulates
//    across K blocks itself: no block partial, no FMA. A power-of-two fp32 scale's E8M0
//    byte is its exponent field.
//  * sched 4 (per-token x per-channel scales, [HELION] scope section): no per-block scale at
//    all; the MFMA accumulates the whole K range (fp8 in fp32; int8 in int32, exact, kept in
//    the accumulator registers' bits) and the tile routine multiplies each element by its
//    token and channel scale once at the end.
//  * The weight fragment sits in the MFMA's first operand and the token fragment in the
//    second, so each lane ends up owning one token row and four consecutive output columns:
//    one scale product per lane and sub-tile row, and 8-byte (bf16) row-contiguous stores.
//  * LDS rows are 128 bytes (one K block); the 16-byte chunk c of row r is stored at slot
//    c ^ swz(r) so the 16 rows a fragment read touches fall in different banks.
//  * Workgroup ids are remapped so that each XCD (ids i, i+8, i+16, ...) owns a contiguous
//    range of tiles, ordered in groups of group_m tile rows, keeping shared A/W panels in
//    that XCD's L2.
//  * Weights row-major (W_ROW) or packed (W_PACKED16, see bfq_weight_layout): packed W
//    arrives as whole 1 KB fragment halves, lands in LDS in lane order and is read back by
//    each lane at 16*lane (conflict-free without a swizzle). A 16x16x128 MFMA's K order is
//    free as long as both operands share it, so with packed W the token fragment takes
//    16-byte chunks (l/16) and (l/16)+4 of its row, the placement the packed weights carry
//    (the int8 path uses that placement for both layouts).
#include "gemm_std_tile.h"

namespace bfq {

// Grouped (MoE) store: tile row r < rows holds pair rows[r]; it goes to base[base_off +
// rows[r]*N + n] (the output in pair order); a pair id outside [0, M) is not stored. 16x16
// sub-tiles only.
template <int OT, int BM, int BN, int WM, int WN, int SCHED>
__device__ __forceinline__ void std_store_rows(
    void* base, int64_t base_off, int64_t M, int64_t N, int64_t n0, const int32_t* __restrict__ rows,
    int64_t nrows,
    const typename StdShape<BM, BN, WM, WN, SCHED>::AccT (
        &acc)[StdShape<BM, BN, WM, WN, SCHED>::SM][StdShape<BM, BN, WM, WN, SCHED>::SN]) {
    using Shape = StdShape<BM, BN, WM, WN, SCHED>;
    constexpr int TM = Shape::TM, TN = Shape::TN, SM = Shape::SM, SN = Shape::SN;
    static_assert(Shape::MF == 16, "grouped tiles use 16x16 sub-tiles");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int frow = lane & 15, fgrp = lane >> 4;
#pragma unroll
    for (int sm = 0; sm < SM; ++sm) {
        const int64_t r = wm * TM + sm * 16 + frow;
        if (r >= nrows) continue;
        const int64_t m = rows[r];
        if (m < 0 || m >= M) continue;
#pragma unroll
        for (int sn = 0; sn < SN; ++sn) {
            const int64_t n = n0 + wn * TN + sn * 16 + 4 * fgrp;
            if (n >= N) continue;
            store4<OT>(base, base_off + m * N + n, acc[sm][sn]);
        }
    }
}

// Grouped (MoE) GEMM, standard tiles: grid = N tiles x moe_max_tiles(pairs, E, BM) x split;
// blockIdx.y is the per-expert row tile (moe_tile), workgroups past the last tile exit at
// once (before any LDS traffic, uniformly).
template <int BM, int BN, int WM, int WN, int QT, int OT, int SCHED, int WL>
__global__ __launch_bounds__(64 * WM * WN) void gemm_moe_std_kernel(GemmArgs p) {
    using Shape = StdShape<BM, BN, WM, WN, SCHED>;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    MoeSpan sp;
    if (!moe_tile(p.moe_offsets, p.moe_experts, p.M, BM, blockIdx.y, sp)) return;
    const int64_t N = p.N, KB = p.K / 128;
    const int64_t n0 = (int64_t)blockIdx.x * BN;
    const int split = p.split, z = blockIdx.z;
    const int64_t kb_begin = (int64_t)z * KB / split, kb_end = (int64_t)(z + 1) * KB / split;
    typename Shape::AccT acc[Shape::SM][Shape::SN];
    std_tile<BM, BN, WM, WN, QT, SCHED, 2, WL, 1>(p, lds, sp.p0, n0, kb_begin, kb_end, acc, sp);
    const int32_t* rows = p.moe_rows + sp.p0;
    if (split == 1)
        std_store_rows<OT, BM, BN, WM, WN, SCHED>(p.out, 0, p.M, N, n0, rows, sp.p1 - sp.p0, acc);
    else
        std_store_rows<O_FP32, BM, BN, WM, WN, SCHED>(p.partials, (int64_t)z * p.M * N, p.M, N, n0,
                                                      rows, sp.p1 - sp.p0, acc);
}

// One workgroup per (tile, K split): grid = tiles x 1 x split.
template <int BM, int BN, int WM, int WN, int QT, int OT, int SCHED, int STAGES, int WL>
__global__ __launch_bounds__(64 * WM * WN) void gemm_std_kernel(GemmArgs p) {
    using Shape = StdShape<BM, BN, WM, WN, SCHED>;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int64_t M = p.M, N = p.N, KB = p.K / 128;
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
    int64_t pid_m, pid_n;
    tile_coords(blockIdx.x, tiles_m, tiles_n, p.group_m, p.raster, pid_m, pid_n);
    const int64_t m0 = pid_m * BM, n0 = pid_n * BN;
    const int split = p.split, z = blockIdx.z;
    const int64_t kb_begin = (int64_t)z * KB / split, kb_end = (int64_t)(z + 1) * KB / split;
    typename Shape::AccT acc[Shape::SM][Shape::SN];
    std_tile<BM, BN, WM, WN, QT, SCHED, STAGES, WL>(p, lds, m0, n0, kb_begin, kb_end, acc);
    if (split == 1) std_store<OT, BM, BN, WM, WN, SCHED>(p.out, 0, M, N, m0, n0, acc);
    else std_store<O_FP32, BM, BN, WM, WN, SCHED>(p.partials, (int64_t)z * M * N, M, N, m0, n0, acc);
}

// Stream-K schedule ("variant 2"): a persistent grid of G workgroups (one per CU) takes
// tiles [0, dp_tiles) whole, in rounds of G, then splits the K blocks of the remaining tiles
// evenly: workgroup w owns iterations [w*I/G, (w+1)*I/G) of the I = (tiles - dp_tiles) * KB
// (tile, K block) iterations, in tile-major order, so it may end with part of a tile and
// start with part of another. This fills the last, partial wave of tiles that a plain grid
// leaves half idle. A tile one workgroup covers whole is stored at once; a partial tile is
// parked, as fp32 in the thread's own register order, in the workgroup's slot (0 for the
// first tile of its range, 1 for the last), and a second kernel on the same stream sums each
// split tile's segments in K order and stores it. The kernel boundary publishes the slots,
// so no workgroup ever waits for or synchronises with another, and the sum order is fixed,
// so results are deterministic.
// The iterations are spread over the first Gs = min(G, I) workgroups, so each of those owns at
// least one; the owner of iteration x is max{w : floor(w*I/Gs) <= x} = ceil((x+1)*Gs/I) - 1,
// and a tile's segments are exactly the owners of its first through last iteration.
template <int BM, int BN, int WM, int WN, int SCHED>
struct SlotIO {
    using Shape = StdShape<BM, BN, WM, WN, SCHED>;
    using AccT = typename Shape::AccT;
    static constexpr int SM = Shape::SM, SN = Shape::SN, NT = 64 * WM * WN;
    static constexpr int64_t SLOT = (int64_t)BM * BN;   // floats per partial-tile slot
    // AccT element (sm, sn) is NQ 16-byte pieces; piece q of thread tid sits at byte
    // ((sm*SN + sn)*NQ + q)*NT*16 + tid*16 of the slot: coalesced, one per-lane offset plus a
    // constant scalar offset per access.
    static constexpr int NQ = sizeof(AccT) / 16;
    static __device__ __forceinline__ v4f piece(const AccT& a, int q) {
        if constexpr (NQ == 1) { (void)q; return a; }
        else return v4f{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
    }
    static __device__ __forceinline__ void set_piece(AccT& a, int q, const v4f& v) {
        if constexpr (NQ == 1) { (void)q; a = v; }
        else { a[4 * q] = v.x; a[4 * q + 1] = v.y; a[4 * q + 2] = v.z; a[4 * q + 3] = v.w; }
    }
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(float* slots, int64_t slot) {
        return make_rsrc(slots + uniform_i64(slot) * SLOT, (uint32_t)(SLOT * 4));
    }
    static __device__ __forceinline__ void park(float* slots, int64_t slot, const AccT (&acc)[SM][SN]) {
        const __amdgpu_buffer_rsrc_t r = rsrc(slots, slot);
        const uint32_t voff = threadIdx.x * 16;
#pragma unroll
        for (int sm = 0; sm < SM; ++sm)
#pragma unroll
            for (int sn = 0; sn < SN; ++sn)
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    buf_store_v4f(r, piece(acc[sm][sn], q), voff, (uint32_t)(((sm * SN + sn) * NQ + q) * NT * 16));
    }
    // row band sm of the tile: acc_row = slot (first) or acc_row + slot
    static __device__ __forceinline__ void add_row(float* slots, int64_t slot, bool first, int sm,
                                                   AccT (&acc_row)[SN]) {
        const __amdgpu_buffer_rsrc_t r = rsrc(slots, slot);
        const uint32_t voff = threadIdx.x * 16;
#pragma unroll
        for (int sn = 0; sn < SN; ++sn)
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const v4f v = buf_load_v4f(r, voff, (uint32_t)(((sm * SN + sn) * NQ + q) * NT * 16));
                set_piece(acc_row[sn], q, first ? v : piece(acc_row[sn], q) + v);
            }
    }
};

// Iteration-range helpers shared by the stream-K kernel and its fixup kernel.
__device__ __forceinline__ int64_t sk_owner(int64_t x, int64_t G, int64_t I) {
    return ((x + 1) * G + I - 1) / I - 1;
}

template <int BM, int BN, int WM, int WN, int QT, int OT, int SCHED, int STAGES, int WL>
__global__ __launch_bounds__(64 * WM * WN) void gemm_streamk_kernel(GemmArgs p) {
    using Shape = StdShape<BM, BN, WM, WN, SCHED>;
    using IO = SlotIO<BM, BN, WM, WN, SCHED>;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int64_t M = p.M, N = p.N, KB = p.K / 128;
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
    const int64_t tiles = tiles_m * tiles_n;
    const int64_t G = gridDim.x, w = blockIdx.x;
    typename Shape::AccT acc[Shape::SM][Shape::SN];

    // Work items in order: this workgroup's whole tiles t = w, w+G, ... < dp_tiles (with G a
    // multiple of 8, tile t runs on the XCD that tile_coords assumes), then its stream-K
    // iteration range. One call site of the tile routine keeps the register budget of the
    // plain kernel.
    const int64_t n_whole = w < p.dp_tiles ? (p.dp_tiles - w + G - 1) / G : 0;
    const int64_t I = (tiles - p.dp_tiles) * KB;
    const int64_t Gs = I < G ? I : G;
    const int64_t it_lo = w < Gs ? w * I / Gs : 0, it_hi = w < Gs ? (w + 1) * I / Gs : 0;
    int64_t it = it_lo;
    for (int64_t item = 0;; ++item) {
        int64_t t, ts = 0, k0 = 0, k1 = KB;
        if (item < n_whole) {
            t = w + item * G;
        } else {
            if (it >= it_hi) break;
            ts = it / KB;
            k0 = it - ts * KB;
            k1 = (KB - k0) <= (it_hi - it) ? KB : k0 + (it_hi - it);
            t = p.dp_tiles + ts;
            it += k1 - k0;
        }
        int64_t pm, pn;
        tile_coords(uniform_i64(t), tiles_m, tiles_n, p.group_m, p.raster, pm, pn);
        const int64_t m0 = uniform_i64(pm * BM), n0 = uniform_i64(pn * BN);
        k0 = uniform_i64(k0);
        k1 = uniform_i64(k1);
        std_tile<BM, BN, WM, WN, QT, SCHED, STAGES, WL>(p, lds, m0, n0, k0, k1, acc);
        if (k0 == 0 && k1 == KB) std_store<OT, BM, BN, WM, WN, SCHED>(p.out, 0, M, N, m0, n0, acc);
        else IO::park(p.sk_slots, w * 2 + (ts == it_lo / KB ? 0 : 1), acc);
    }
}

// One workgroup per (stream-K tile, sub-tile row band sm = blockIdx.y): a tile split over
// several workgroups is summed from their parked slots in K order (ascending owner) and
// stored, one band of SM per workgroup so the sum fills the chip; a tile one workgroup covered
// whole was stored by it already. Same block shape as the GEMM, so each thread reads back
// exactly the accumulator pieces it will store.
template <int BM, int BN, int WM, int WN, int OT, int SCHED>
__global__ __launch_bounds__(64 * WM * WN) void gemm_streamk_fixup_kernel(GemmArgs p, int grid) {
    using Shape = StdShape<BM, BN, WM, WN, SCHED>;
    using IO = SlotIO<BM, BN, WM, WN, SCHED>;
    constexpr int TM = Shape::TM, TN = Shape::TN, MF = Shape::MF, SN = Shape::SN;
    const int64_t M = p.M, N = p.N, KB = p.K / 128;
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
    const int64_t tiles = tiles_m * tiles_n;
    const int64_t ts = blockIdx.x;
    const int sm = blockIdx.y;
    const int64_t I = (tiles - p.dp_tiles) * KB;
    const int64_t Gs = I < grid ? I : grid;
    const int64_t w_first = sk_owner(ts * KB, Gs, I), w_last = sk_owner(ts * KB + KB - 1, Gs, I);
    if (w_first == w_last) return;
    typename Shape::AccT acc[SN];
    for (int64_t ws = w_first; ws <= w_last; ++ws) {
        const int sl = ts == (ws * I / Gs) / KB ? 0 : 1;
        IO::add_row(p.sk_slots, ws * 2 + sl, ws == w_first, sm, acc);
    }
    int64_t pm, pn;
    tile_coords(p.dp_tiles + ts, tiles_m, tiles_n, p.group_m, p.raster, pm, pn);
    // the rows of band sm, as std_store writes them
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int frow = lane & (MF - 1), fgrp = lane >> 4, khalf = lane >> 5;
    const int64_t m = pm * BM + wm * TM + sm * MF + frow;
    if (m >= M) return;
    const int64_t n0 = pn * BN + wn * TN;
#pragma unroll
    for (int sn = 0; sn < SN; ++sn) {
        if constexpr (MF == 32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + sn * 32 + 8 * j + 4 * khalf;
                if (n >= N) continue;
                const auto& a = acc[sn];
                const v4f v = {a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]};
                store4<OT>(p.out, m * N + n, v);
            }
        } else {
            (void)khalf;
            const int64_t n = n0 + sn * 16 + 4 * fgrp;
            if (n >= N) continue;
            store4<OT>(p.out, m * N + n, acc[sn]);
        }
    }
}

// Whole rounds first; only the tiles of the last, partial round are split (each split tile
// costs a parked fp32 partial per segment, written and read back once).
int64_t streamk_dp_tiles(int64_t tiles, int grid) { return (tiles / grid) * grid; }

size_t streamk_workspace_bytes(int bm, int bn, int grid) {
    return (size_t)grid * 2 * (size_t)bm * (size_t)bn * sizeof(float);
}

// Workgroups of the stream-K grid: the device's compute units (one resident workgroup each).
int streamk_grid() {
    static int cached[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cached[dev] == 0) {
        int cus = 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
            cus = 256;
        cached[dev] = cus - cus % 8;                   // keep the XCD round-robin aligned
        if (cached[dev] <= 0) cached[dev] = cus;
    }
    return cached[dev];
}

template <int BM, int BN, int WM, int WN, int QT, int OT, int SCHED, int STAGES, int WL>
hipError_t launch_streamk(const GemmArgs& a, hipStream_t stream) {
    constexpr int LDS_BYTES = StdShape<BM, BN, WM, WN, SCHED>::lds_bytes(STAGES);
    const int G = streamk_grid();
    const int64_t tiles = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
    GemmArgs b = a;
    b.dp_tiles = streamk_dp_tiles(tiles, G);
    const int64_t I = (tiles - b.dp_tiles) * (a.K / 128);
    const int64_t grid = b.dp_tiles > 0 ? G : (I < G ? I : G);
    b.sk_slots = a.partials;
    static bool attr_set = false;   // one-time opt-in to more than 64 KB of LDS
    if (!attr_set) {
        hipError_t e = hipFuncSetAttribute(
            reinterpret_cast<const void*>(&gemm_streamk_kernel<BM, BN, WM, WN, QT, OT, SCHED, STAGES, WL>),
            hipFuncAttributeMaxDynamicSharedMemorySize, LDS_BYTES);
        if (e != hipSuccess) return e;
        attr_set = true;
    }
    hipLaunchKernelGGL((gemm_streamk_kernel<BM, BN, WM, WN, QT, OT, SCHED, STAGES, WL>),
                       dim3((unsigned)grid), dim3(64 * WM * WN), LDS_BYTES, stream, b);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || tiles == b.dp_tiles) return e;
    hipLaunchKernelGGL((gemm_streamk_fixup_kernel<BM, BN, WM, WN, OT, SCHED>),
                       dim3((unsigned)(tiles - b.dp_tiles), (unsigned)StdShape<BM, BN, WM, WN, SCHED>::SM),
                       dim3(64 * WM * WN), 0, stream, b, (int)grid);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int QT, int OT, int SCHED, int STAGES, int WL>
hipError_t launch_std(const GemmArgs& a, hipStream_t stream) {
    constexpr int LDS_BYTES = StdShape<BM, BN, WM, WN, SCHED>::lds_bytes(STAGES);
    const int64_t tiles = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
    dim3 grid((unsigned)tiles, 1, (unsigned)a.split);
    static bool attr_set = false;   // one-time opt-in to more than 64 KB of LDS
    if (!attr_set) {
        hipError_t e = hipFuncSetAttribute(
            reinterpret_cast<const void*>(&gemm_std_kernel<BM, BN, WM, WN, QT, OT, SCHED, STAGES, WL>),
            hipFuncAttributeMaxDynamicSharedMemorySize, LDS_BYTES);
        if (e != hipSuccess) return e;
        attr_set = true;
    }
    hipLaunchKernelGGL((gemm_std_kernel<BM, BN, WM, WN, QT, OT, SCHED, STAGES, WL>), grid,
                       dim3(64 * WM * WN), LDS_BYTES, stream, a);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int QT, int OT, int SCHED, int WL>
hipError_t launch_moe_std(const GemmArgs& a, hipStream_t stream) {
    constexpr int LDS_BYTES = StdShape<BM, BN, WM, WN, SCHED>::lds_bytes(2);
    dim3 grid((unsigned)((a.N + BN - 1) / BN), (unsigned)moe_max_tiles(a.M, a.moe_experts, BM),
              (unsigned)a.split);
    static bool attr_set = false;
    if (!attr_set) {
        hipError_t e = hipFuncSetAttribute(
            reinterpret_cast<const void*>(&gemm_moe_std_kernel<BM, BN, WM, WN, QT, OT, SCHED, WL>),
            hipFuncAttributeMaxDynamicSharedMemorySize, LDS_BYTES);
        if (e != hipSuccess) return e;
        attr_set = true;
    }
    hipLaunchKernelGGL((gemm_moe_std_kernel<BM, BN, WM, WN, QT, OT, SCHED, WL>), grid,
                       dim3(64 * WM * WN), LDS_BYTES, stream, a);
    return hipGetLastError();
}

#define BFQ_STD_ENTRY(BM, BN, WM, WN, ST, SC, QT, OT, WL)                                \
    KernelEntry{bfq_tile{0, BM, BN, 128, 1, WM, WN, ST, 8, SC, 0, 0}, QT, OT, WL,         \
                (SC) == 3 ? S_UE8M0 : (SC) == 4 ? S_CHANNEL : S_FP32,                      \
                &launch_std<BM, BN, WM, WN, QT, OT, SC, ST, WL>}

#define BFQ_STD_ALL_OUT(BM, BN, WM, WN, ST, SC, QT, WL)                                   \
    BFQ_STD_ENTRY(BM, BN, WM, WN, ST, SC, QT, O_BF16, WL),                                \
        BFQ_STD_ENTRY(BM, BN, WM, WN, ST, SC, QT, O_FP16, WL),                            \
        BFQ_STD_ENTRY(BM, BN, WM, WN, ST, SC, QT, O_FP32, WL)

static const KernelEntry kStdKernels[] = {
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 0, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 1, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 192, 4, 2, 2, 0, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 3, 1, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 2, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 2, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 0, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 3, 1, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 128, 4, 1, 3, 1, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 0, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 0, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 0, Q_INT8, W_ROW),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 0, Q_INT8, W_ROW),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 0, Q_INT8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 0, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 1, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(256, 192, 4, 2, 2, 0, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 0, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 1, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(256, 128, 4, 2, 2, 0, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(256, 128, 4, 2, 2, 1, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 0, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 0, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 0, Q_INT8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 0, Q_INT8, W_PACKED16),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 0, Q_INT8, W_PACKED16),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 3, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 3, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 3, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 3, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 3, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 3, Q_FP8, W_PACKED16),
    // per-token x per-channel scales
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 4, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 4, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 4, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 4, Q_FP8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 4, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 4, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 4, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 4, Q_FP8, W_PACKED16),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 4, Q_INT8, W_ROW),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 4, Q_INT8, W_ROW),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 4, Q_INT8, W_ROW),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 4, Q_INT8, W_ROW),
    BFQ_STD_ALL_OUT(256, 256, 4, 2, 2, 4, Q_INT8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 256, 2, 2, 2, 4, Q_INT8, W_PACKED16),
    BFQ_STD_ALL_OUT(128, 128, 2, 2, 2, 4, Q_INT8, W_PACKED16),
    BFQ_STD_ALL_OUT(64, 128, 1, 2, 2, 4, Q_INT8, W_PACKED16),
};

#define BFQ_SK_ENTRY(BM, BN, WM, WN, ST, SC, QT, OT, WL)                                 \
    KernelEntry{bfq_tile{2, BM, BN, 128, 1, WM, WN, ST, 8, SC, 0, 0}, QT, OT, WL,         \
                (SC) == 3 ? S_UE8M0 : (SC) == 4 ? S_CHANNEL : S_FP32,                      \
                &launch_streamk<BM, BN, WM, WN, QT, OT, SC, ST, WL>}

#define BFQ_SK_ALL_OUT(BM, BN, WM, WN, ST, SC, QT, WL)                                    \
    BFQ_SK_ENTRY(BM, BN, WM, WN, ST, SC, QT, O_BF16, WL),                                 \
        BFQ_SK_ENTRY(BM, BN, WM, WN, ST, SC, QT, O_FP16, WL),                             \
        BFQ_SK_ENTRY(BM, BN, WM, WN, ST, SC, QT, O_FP32, WL)

static const KernelEntry kStreamKKernels[] = {
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 0, Q_FP8, W_ROW),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 1, Q_FP8, W_ROW),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 0, Q_INT8, W_ROW),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 0, Q_FP8, W_PACKED16),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 1, Q_FP8, W_PACKED16),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 0, Q_INT8, W_PACKED16),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 3, Q_FP8, W_ROW),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 3, Q_FP8, W_PACKED16),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 4, Q_FP8, W_ROW),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 4, Q_FP8, W_PACKED16),
    BFQ_SK_ALL_OUT(256, 256, 4, 2, 2, 4, Q_INT8, W_PACKED16),
};

#define BFQ_MOE_STD_ENTRY(BM, BN, WM, WN, SC, QT, OT, WL)                                  \
    KernelEntry{bfq_tile{0, BM, BN, 128, 1, WM, WN, 2, 1, SC, 0, 0}, QT, OT, WL,              \
                (SC) == 3 ? S_UE8M0 : S_FP32, &launch_moe_std<BM, BN, WM, WN, QT, OT, SC, WL>, 1}
#define BFQ_MOE_STD(BM, BN, WM, WN, SC, QT)                                                 \
    BFQ_MOE_STD_ENTRY(BM, BN, WM, WN, SC, QT, O_BF16, W_ROW),                              \
        BFQ_MOE_STD_ENTRY(BM, BN, WM, WN, SC, QT, O_FP16, W_ROW),                          \
        BFQ_MOE_STD_ENTRY(BM, BN, WM, WN, SC, QT, O_FP32, W_ROW),                          \
        BFQ_MOE_STD_ENTRY(BM, BN, WM, WN, SC, QT, O_BF16, W_PACKED16),                     \
        BFQ_MOE_STD_ENTRY(BM, BN, WM, WN, SC, QT, O_FP16, W_PACKED16),                     \
        BFQ_MOE_STD_ENTRY(BM, BN, WM, WN, SC, QT, O_FP32, W_PACKED16)

// grouped (MoE) standard tiles, fp8 (the gathered rows cost registers: 256x256 with sched 0
// spills with packed weights, the software-pipelined sched 1 fits in 240 VGPRs; it takes
// large token counts, where one 256-row tile covers each expert's rows and its weights
// stream once per expert)
static const KernelEntry kMoeStdKernels[] = {
    BFQ_MOE_STD(128, 256, 2, 2, 0, Q_FP8),
    BFQ_MOE_STD(128, 128, 2, 2, 0, Q_FP8),
    BFQ_MOE_STD(64, 128, 1, 2, 0, Q_FP8),
    BFQ_MOE_STD(256, 256, 4, 2, 1, Q_FP8),
    BFQ_MOE_STD(256, 256, 4, 2, 3, Q_FP8),
    BFQ_MOE_STD(128, 128, 2, 2, 3, Q_FP8),
};

const KernelEntry* moe_std_kernels(int* count) {
    *count = (int)(sizeof(kMoeStdKernels) / sizeof(kMoeStdKernels[0]));
    return kMoeStdKernels;
}

const KernelEntry* streamk_kernels(int* count) {
    *count = (int)(sizeof(kStreamKKernels) / sizeof(kStreamKKernels[0]));
    return kStreamKKernels;
}

const KernelEntry* std_kernels(int* count) {
    *count = (int)(sizeof(kStdKernels) / sizeof(kStdKernels[0]));
    return kStdKernels;
}

}  // namespace bfq
