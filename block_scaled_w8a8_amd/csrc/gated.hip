// The gated product of a feed-forward block and its gradient.
//
// Forward: out[m][f] = act(g) * u with g = sum_k a[m][k] w[f][k] and u = sum_k a[m][k] w[F+f][k]
// (block-scaled e4m3 operands, as the block GEMM), both products, the activation and the product
// in one kernel: a workgroup takes the gate rows and the up rows of the same output columns, so a
// lane's accumulators hold both factors of each of its outputs and the 2F-wide product is never
// stored. Large batches and packed weights at a few tokens use the block GEMM's tile routines
// (gemm_std_tile.h, gemm_swapab_body.h); the sizes between have tiles of their own below.
// Outputs are bf16 / fp16 / fp32, or e4m3 codes with one scale per 128 columns, which is what the
// down projection's GEMM reads: a workgroup that covers 128 output columns holds whole groups.
// A tile whose K range is split, or that covers less than a group when codes are wanted, writes
// fp32 partials of the 2F-wide product instead and gated_reduce_kernel finishes them.
//
// What bounds the forward kernels is what bounds the block GEMM's: the weight stream at decode
// sizes, the operand bytes through a CU's L1 and the scale step at large M. Measured, F 18432 x
// K 7168, packed weights, SILU, bf16 out, on a card under load: 1 token 42 us (6.3 TB/s of weights), 64
// tokens 55 us, 512 tokens 171 us, 1024 tokens 292 us, 4096 tokens 1012 us with fp32 scales (2.14 PFLOP/s)
// and 923 us with powers of two; 1025 to 1055 us where the pre-activations (302 MB) are kept, by the card
// and its clock, which takes some thirty calls to settle (the third one after an idle card: 1370 us, the
// tenth 1145). Pairs of times further down compare two forms in short runs on one card: what they show is
// the difference.
// The two sums carry the e4m3 MFMA's own error, as the block GEMM's do: 3.5e-5 to 4.6e-5 of the
// result (relative, Frobenius) on outlier-bearing tokens, whichever schedule or tile. Where codes
// are wanted it decides the values that lie that near to a rounding boundary: 333 x 2048 codes
// over K 7168 differ from those of the exact product in 0.4 % of places, by one step, and are no
// farther from the unrounded product (2.640 % both).
#include "activation.h"
#include "gemm_std_tile.h"
#include "gemm_swapab_body.h"
#include "quant_device.h"

namespace bfq {

// Four values as bf16 or fp16 (uniform choice).
__device__ __forceinline__ uint2 half4(int otype, const v4f& v) {
    if (otype == O_FP16)
        return make_uint2(f32_to_f16_bits(v.x) | (f32_to_f16_bits(v.y) << 16),
                          f32_to_f16_bits(v.z) | (f32_to_f16_bits(v.w) << 16));
    return make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
}

// Four consecutive outputs, their type chosen at run time (uniform).
__device__ __forceinline__ void store4_any(int otype, void* out, int64_t idx, const v4f& v) {
    if (otype == O_FP32) *reinterpret_cast<v4f*>(static_cast<float*>(out) + idx) = v;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + idx) = half4(otype, v);
}

// One scale of group g of token m; packed: its byte of the word, and by the last group the zero
// bytes after it.
__device__ __forceinline__ void store_scale(float* scales, int64_t sm, int64_t sg, int packed,
                                            int64_t m, int64_t g, int64_t groups, float s) {
    if (!packed) {
        scales[m * sm + g * sg] = s;
        return;
    }
    uint8_t* word = reinterpret_cast<uint8_t*>(scales) + ((g >> 2) * sg + m) * 4;
    word[g & 3] = (uint8_t)e8m0_of(s);
    if (g == groups - 1)
        for (int j = (int)(g & 3) + 1; j < 4; ++j) word[j] = 0;
}

// Stores of a tile whose lane holds, for sub-tile row sm, token row(sm) (or none, < 0) and output
// columns n + 16*sn + 4*(lane/16) .. +3: gate in acc[sm][sn], up in acc[sm][sn + SG].
template <int SM, int SG, typename RowFn>
__device__ __forceinline__ void gated_partials(const GatedArgs& p, const v4f (&acc)[SM][2 * SG],
                                               int64_t n, RowFn row) {
    const int64_t F = p.N, base = (int64_t)blockIdx.z * p.M;
#pragma unroll
    for (int sm = 0; sm < SM; ++sm) {
        const int64_t m = row(sm);
        if (m < 0) continue;
#pragma unroll
        for (int sn = 0; sn < SG; ++sn) {
            float* o = p.partials + (base + m) * 2 * F + n + sn * 16;
            *reinterpret_cast<v4f*>(o) = acc[sm][sn];
            *reinterpret_cast<v4f*>(o + F) = acc[sm][sn + SG];
        }
    }
}

// act(g) * u into acc[sm][0..SG).
template <int SM, int SG>
__device__ __forceinline__ void gated_product(const GatedArgs& p, v4f (&acc)[SM][2 * SG]) {
#pragma unroll
    for (int sm = 0; sm < SM; ++sm)
#pragma unroll
        for (int sn = 0; sn < SG; ++sn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[sm][sn][i] = act_f32(acc[sm][sn][i], p.c1, p.c3) * acc[sm][sn + SG][i];
}

// Pre-activations to p.pre, then the product.
template <int SM, int SG, typename RowFn>
__device__ __forceinline__ void gated_combine(const GatedArgs& p, v4f (&acc)[SM][2 * SG], int64_t n,
                                              RowFn row) {
    const int64_t F = p.N;
    if (p.pre) {
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            const int64_t m = row(sm);
            if (m < 0) continue;
#pragma unroll
            for (int sn = 0; sn < SG; ++sn) {
                store4_any(O_BF16, p.pre, m * 2 * F + n + sn * 16, acc[sm][sn]);
                store4_any(O_BF16, p.pre, m * 2 * F + F + n + sn * 16, acc[sm][sn + SG]);
            }
        }
    }
    gated_product<SM, SG>(p, acc);
}

// Largest magnitudes (bits) of each token's outputs in this wave's columns, in every lane of the
// token (lanes l, l + 16, l + 32, l + 48).
template <int SM, int SG>
__device__ __forceinline__ void gated_amax(const v4f (&acc)[SM][2 * SG], uint32_t (&mx)[SM]) {
#pragma unroll
    for (int sm = 0; sm < SM; ++sm) {
        float a = 0.f;
#pragma unroll
        for (int sn = 0; sn < SG; ++sn)
#pragma unroll
            for (int i = 0; i < 4; ++i) a = max_abs(a, acc[sm][sn][i]);
        uint32_t m = __float_as_uint(a) & 0x7FFFFFFFu;
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        mx[sm] = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    }
}

// Codes of a group's four outputs, given the group's largest magnitude and scale.
__device__ __forceinline__ uint32_t codes4(const v4f& v, uint32_t mx, float s) {
    const float x[8] = {v.x, v.y, v.z, v.w, 0.f, 0.f, 0.f, 0.f};
    return encode8_group<Q_FP8>(x, mx, s).x;
}

// ---------------------------------------------------------------- standard tiles ----

// Output tiles leave through LDS: a lane's accumulators hold four neighbouring columns of 16 rows a
// sub-tile, 32-byte pieces of a row in a store, so the tile is laid out as rows of 16-byte chunks
// and stored as whole rows: with the hardware's bf16 conversion in place of the integer one, 39 us
// less for 4096 x 18432 outputs and their pre-activations (K = 7168). Chunk c of row r sits in slot
// c ^ (r & (chunks - 1)) of its row, which spreads a column of rows over the banks.
// Outputs of more bytes than the L2s hold are stored past them (past_caches): F 18432 x K 7168,
// packed, bf16 out: 1024 tokens 326 -> 298 us, 4096 tokens 991 -> 965 us (with pre-activations
// 1040 -> 990).
template <int ROWB>
__device__ __forceinline__ uint32_t tile_slot(int r, int byte) {
    constexpr int C = ROWB / 16;
    return (uint32_t)(r * ROWB + (((byte >> 4) ^ (r & (C - 1))) << 4) + (byte & 15));
}
// Rows of ROWB bytes from LDS to dst + r * ld, r < rows. `past`: past the caches (see
// past_caches), which the operands that other workgroups still read then keep.
template <int BM, int ROWB, int THREADS>
__device__ __forceinline__ void store_tile(const uint8_t* lds, void* dst, int64_t ld, int64_t rows,
                                           bool past) {
    constexpr int C = ROWB / 16, STEP = THREADS / C;
    const int r0 = threadIdx.x / C, c = threadIdx.x % C;
#pragma unroll
    for (int i = 0; i < BM / STEP; ++i) {
        const int r = r0 + i * STEP;
        if (r < rows) {
            const v4u v = *reinterpret_cast<const v4u*>(lds + tile_slot<ROWB>(r, c * 16));
            v4u* o = reinterpret_cast<v4u*>(static_cast<uint8_t*>(dst) + r * ld + c * 16);
            if (past) {
                asm volatile("");      // or the compiler makes the two stores one, without the hint
                __builtin_nontemporal_store(v, o);
                asm volatile("");
            } else {
                *o = v;
            }
        }
    }
}

// Finishes a tile of BM tokens x BNO output columns from (m0, n0): wave (wm, wn) holds rows wm * TM
// and columns wn * TNO. The LDS is free (the callers end on a barrier).
// slot >= 0: a part of a split tile, whose sums go to that slot of p.tail.
template <int BM, int BNO, int WM, int WN, int SM, int SG>
__device__ __forceinline__ void gated_finish_tile(const GatedArgs& p, uint8_t* lds, v4f (&acc)[SM][2 * SG],
                                                  int64_t m0, int64_t n0, int64_t slot) {
    constexpr int TM = BM / WM, TNO = BNO / WN;
    const int64_t M = p.M, F = p.N;
    const int lane = threadIdx.x & 63, frow = lane & 15, fgrp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t mw = m0 + wm * TM + frow, n = n0 + wn * TNO + 4 * fgrp;
    auto row = [&](int sm) { return mw + sm * 16 < M ? mw + sm * 16 : (int64_t)-1; };
    if (slot >= 0) {
        float* o = p.tail + (slot * BM + wm * TM + frow) * (2 * BNO) + wn * TNO + 4 * fgrp;
#pragma unroll
        for (int sm = 0; sm < SM; ++sm)
#pragma unroll
            for (int n2 = 0; n2 < 2 * SG; ++n2)
                *reinterpret_cast<v4f*>(o + sm * 16 * 2 * BNO + n2 / SG * BNO + n2 % SG * 16) = acc[sm][n2];
        return;
    }
    if (p.partials) {
        gated_partials<SM, SG>(p, acc, n, row);
        return;
    }
    // lr, lc: the lane's first row and column of the tile
    constexpr int THREADS = 64 * WM * WN;
    const int lr = wm * TM + frow, lc = wn * TNO + 4 * fgrp;
    const int64_t live = M - m0 < BM ? M - m0 : BM;
    auto put = [&](int off, int otype, int half) {      // 16-bit values of one half of acc
#pragma unroll
        for (int sm = 0; sm < SM; ++sm)
#pragma unroll
            for (int sn = 0; sn < SG; ++sn)
                *reinterpret_cast<uint2*>(lds + off + tile_slot<2 * BNO>(lr + sm * 16, 2 * (lc + sn * 16))) =
                    half4(otype, acc[sm][sn + half * SG]);
    };
    if (p.pre) {
        put(0, O_BF16, 0);
        put(BM * 2 * BNO, O_BF16, 1);
        lds_barrier();
        uint16_t* pre = static_cast<uint16_t*>(p.pre) + m0 * 2 * F + n0;
        store_tile<BM, 2 * BNO, THREADS>(lds, pre, 4 * F, live, past_caches(4 * M * F));
        store_tile<BM, 2 * BNO, THREADS>(lds + BM * 2 * BNO, pre + F, 4 * F, live, past_caches(4 * M * F));
        lds_barrier();
    }
    gated_product<SM, SG>(p, acc);
    if (p.otype == O_FP32) {
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            const int64_t m = row(sm);
            if (m < 0) continue;
#pragma unroll
            for (int sn = 0; sn < SG; ++sn) store4_any(O_FP32, p.out, m * F + n + sn * 16, acc[sm][sn]);
        }
        return;
    }
    if (p.otype != O_CODES) {
        put(0, p.otype, 0);
        lds_barrier();
        store_tile<BM, 2 * BNO, THREADS>(lds, static_cast<uint16_t*>(p.out) + m0 * F + n0, 2 * F, live,
                                         past_caches(2 * M * F));
        return;
    }
    if constexpr (BNO == 128) {
        // the tile's 128 columns are one group: largest magnitudes over its WN waves through LDS,
        // [wn][tile row], behind the codes
        uint32_t mx[SM];
        gated_amax<SM, SG>(acc, mx);
        uint32_t* red = reinterpret_cast<uint32_t*>(lds + BM * BNO);
        if (fgrp == 0)
#pragma unroll
            for (int sm = 0; sm < SM; ++sm) red[wn * BM + lr + sm * 16] = mx[sm];
        lds_barrier();
        const int64_t g = n0 / 128, G = F / 128;
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < WN; ++w) m = max(m, red[w * BM + lr + sm * 16]);
            const float s = group_scale<Q_FP8>(m, p.os_eps, p.os_ue8m0);
            const int64_t r = mw + sm * 16;
            // packed words have rows up to a multiple of four tokens, zero past the last
            if (wn == 0 && fgrp == 0 && r < (p.os_packed ? (M + 3) / 4 * 4 : M))
                store_scale(p.out_scales, p.os_stride_m, p.os_stride_g, p.os_packed, r, g, G,
                            r < M ? s : 0.f);
#pragma unroll
            for (int sn = 0; sn < SG; ++sn)
                *reinterpret_cast<uint32_t*>(lds + tile_slot<BNO>(lr + sm * 16, lc + sn * 16)) =
                    codes4(acc[sm][sn], m, s);
        }
        lds_barrier();
        store_tile<BM, BNO, THREADS>(lds, static_cast<uint8_t*>(p.out) + m0 * F + n0, F, live, past_caches(M * F));
    }
}

// The tile of this workgroup and its part of the K range: whole tiles (or all of them split alike,
// blockIdx.z), then the parts of the last ones, part by part so that a tile's parts stay on one XCD.
// A grid that fills its last round to an eighth or a quarter leaves the chip idle for most of it:
// F 18432 x K 7168, packed, 256 x 128 tiles: 512 tokens (1.1 rounds) 223 -> 152 us, 1024 (2.25) 321 ->
// 266, 2048 (4.5) 534 -> 517; with 128 tiles left over the parts' bytes cost what they gain.
struct GatedWork {
    int64_t tile, kb0, kb1, slot;
};
__device__ __forceinline__ GatedWork gated_work(const GatedArgs& p, int64_t tiles) {
    const int64_t KB = p.K / 128, t = (int64_t)blockIdx.x - p.tail_first;
    if (p.tail_parts <= 1 || t < 0)
        return {(int64_t)blockIdx.x, (int64_t)blockIdx.z * KB / p.split, (int64_t)(blockIdx.z + 1) * KB / p.split, -1};
    const int64_t tail = tiles - p.tail_first, part = t / tail, j = t % tail;
    return {p.tail_first + j, part * KB / p.tail_parts, (part + 1) * KB / p.tail_parts, j * p.tail_parts + part};
}

// One workgroup per (tile of BM tokens x BN / 2 output columns, K split).
template <int BM, int BN, int WM, int WN, int SCHED, int WL>
__global__ __launch_bounds__(64 * WM * WN) void gemm_gated_std_kernel(GatedArgs p) {
    using Shape = StdShape<BM, BN, WM, WN, SCHED>;
    constexpr int SM = Shape::SM, SG = Shape::SN / 2, BNO = BN / 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int64_t M = p.M, F = p.N;
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (F + BNO - 1) / BNO;
    const GatedWork w = gated_work(p, tiles_m * tiles_n);
    int64_t pid_m, pid_n;
    tile_coords(w.tile, tiles_m, tiles_n, p.group_m, p.raster, pid_m, pid_n);
    const int64_t m0 = pid_m * BM, n0 = pid_n * BNO;
    typename Shape::AccT acc[SM][2 * SG];
    std_tile<BM, BN, WM, WN, Q_FP8, SCHED, 2, WL, 0, 1>(p, lds, m0, n0, w.kb0, w.kb1, acc);
    gated_finish_tile<BM, BNO, WM, WN, SM, SG>(p, lds, acc, m0, n0, w.slot);
}

// Tiles for tens to hundreds of tokens on short products, where a K block's trip to memory costs
// more than its arithmetic: D LDS stages of one K block (BM token rows, BNO gate rows, BNO up rows),
// D - 1 of them in flight. A wave waits for its own loads of the oldest stage, one barrier makes the
// stage whole and frees the one before, which is refilled at once. Token rows and row-major weight
// rows are swizzled as in the standard tiles, packed weights are fragment halves. Scales travel in
// registers, counted with the loads. Against tiles of two stages, which wait out the trip every K
// block: F 4096 x K 4096, 512 tokens, 28.7 us for 38.8; F 2304 x K 7168, 128 tokens, 20.2 for 26.7;
// F 18432 x K 7168, 333 tokens, 138 for 150. At those sizes the fixed costs lead: some 3 us to start
// and drain, 3 us for a split's second launch.
template <int BM, int BNO, int WM, int WN, int D, int SCHED, int WL>
__global__ __launch_bounds__(64 * WM * WN) void gemm_gated_pipe_kernel(GatedArgs p) {
    constexpr int NW = WM * WN, TM = BM / WM, TNO = BNO / WN, SM = TM / 16, SG = TNO / 16;
    constexpr int STAGE = (BM + 2 * BNO) * 128, CA = BM / 8 / NW, CW = BNO / 8 / NW;   // loads a wave
    constexpr int kOps = CA + 2 * CW + SM + 2;
    constexpr bool rows = WL == W_ROW;
    static_assert(NW % 2 == 0 && BM / 8 % NW == 0 && BNO / 8 % NW == 0 && 128 % BNO == 0, "whole loads a wave");
    static_assert((D - 2) * kOps <= 63, "the wait counts loads in six bits");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63, frow = lane & 15, fgrp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t M = p.M, F = p.N, K = p.K, KB = K / 128;
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = F / BNO;
    const GatedWork item = gated_work(p, tiles_m * tiles_n);
    int64_t pid_m, pid_n;
    tile_coords(item.tile, tiles_m, tiles_n, p.group_m, p.raster, pid_m, pid_n);
    const int64_t m0 = pid_m * BM, n0 = pid_n * BNO, kb0 = item.kb0, L = item.kb1 - kb0;
    // past every resource here (inside scales that span over 2 GiB, whose value then goes unused)
    constexpr uint32_t kNoLoad = 0x80000000u;

    const uint8_t* w = static_cast<const uint8_t*>(p.w);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(w + n0 * K, (uint32_t)(BNO * K));
    const __amdgpu_buffer_rsrc_t ru = make_rsrc(w + (F + n0) * K, (uint32_t)(BNO * K));
    const int64_t live = M - m0 < BM ? M - m0 : BM, ssm = p.sa_stride_m, ssk = p.sa_stride_k;
    const int packed = p.sa_packed;
    const uint32_t pmask = packed ? ~0u : 0u;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(static_cast<const uint8_t*>(p.a) + m0 * K, (uint32_t)(live * K));
    const __amdgpu_buffer_rsrc_t rsa = make_rsrc(
        p.sa + m0 * ssm, (uint32_t)(((live - 1) * ssm + (packed ? (KB - 1) / 4 : KB - 1) * ssk + 1) * 4));
    const __amdgpu_buffer_rsrc_t rsg = make_rsrc(p.sw + (n0 / 128) * KB, (uint32_t)(KB * 4));
    const __amdgpu_buffer_rsrc_t rsu = make_rsrc(p.sw + (F / 128 + n0 / 128) * KB, (uint32_t)(KB * 4));
    uint32_t sa_voff[SM];
#pragma unroll
    for (int sm = 0; sm < SM; ++sm) sa_voff[sm] = (uint32_t)((wm * TM + sm * 16 + frow) * ssm * 4);
    // a load of rows: 8 of them, lane l row l / 8, slot l % 8; load i of a wave starts at row
    // 8 * (wave + NW * i), whose swizzle phase is the wave's (NW is even)
    const uint32_t row_voff = (uint32_t)(((lane >> 3) + wave * 8) * K + (((lane & 7) ^ (lane >> 3) ^ (wave & 1)) << 4));
    // packed: 16-row group (wave + NW * i) / 2, half (wave + NW * i) % 2
    const uint32_t w_voff = rows ? row_voff : (uint32_t)((wave >> 1) * KB * 2048 + (wave & 1) * 1024 + lane * 16);

    float sab[D][SM], sgb[D], sub[D];
    int kbs[D];
    auto fetch = [&](int slot, int64_t i) {
        const bool in = i < L;
        const int64_t kb = kb0 + i;
        const uint32_t sk = in ? (uint32_t)kb * 128u : kNoLoad;
        const uint32_t wk = rows ? sk : in ? (uint32_t)kb * 2048u : kNoLoad;
        const uint32_t ss = in ? (uint32_t)((packed ? kb >> 2 : kb) * ssk * 4) : kNoLoad;
        const uint32_t sws = in ? (uint32_t)kb * 4u : kNoLoad;
        const uint32_t at = (uint32_t)(slot * STAGE + wave * 1024);
        // the scales first: they are waited for first
        sgb[slot] = buf_f32(rsg, 0, sws);
        sub[slot] = buf_f32(rsu, 0, sws);
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) sab[slot][sm] = buf_f32(rsa, sa_voff[sm], ss);
        kbs[slot] = (int)(kb & 3);
#pragma unroll
        for (int c = 0; c < CA; ++c)
            dma16(ra, lds, at + c * NW * 1024, row_voff, sk + (uint32_t)(NW * c * 8 * K));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < CW; ++c)
                dma16(h ? ru : rw, lds, at + (uint32_t)(BM * 128 + h * BNO * 128 + c * NW * 1024), w_voff,
                      wk + (rows ? (uint32_t)(NW * c * 8 * K) : (uint32_t)(NW * c / 2 * KB * 2048)));
    };
    v4f acc[SM][2 * SG];
#pragma unroll
    for (int sm = 0; sm < SM; ++sm)
#pragma unroll
        for (int n = 0; n < 2 * SG; ++n) acc[sm][n] = v4f{0.f, 0.f, 0.f, 0.f};
    const uint32_t f0 = (uint32_t)(frow * 128 + ((fgrp ^ swz(frow)) << 4));
    const uint32_t f1 = (uint32_t)(frow * 128 + (((fgrp + 4) ^ swz(frow)) << 4));
    auto frag = [&](const uint8_t* at, uint32_t lo, uint32_t hi) {
        const v4i x = *reinterpret_cast<const v4i*>(at + lo), y = *reinterpret_cast<const v4i*>(at + hi);
        return v8i{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };
    auto compute = [&](int slot) {
        const uint8_t* at = lds + slot * STAGE;
        v8i a[SM];
        float sa[SM];
        int ea[SM];
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            a[sm] = frag(at + (wm * TM + sm * 16) * 128, f0, f1);
            // packed: byte kb % 4 of the word (selects without a branch)
            const uint32_t word = __float_as_uint(sab[slot][sm]), code = e8m0_byte(word, kbs[slot]);
            if constexpr (SCHED == 3)
                ea[sm] = (int)((code & pmask) | (e8m0_of(sab[slot][sm]) & ~pmask));
            else
                sa[sm] = __uint_as_float((__float_as_uint(e8m0_value(code)) & pmask) | (word & ~pmask));
        }
        // the scale step of a sub-tile column runs behind the next one's MFMAs (SCHED 0); powers of
        // two are the MFMA's own scale operands, and it accumulates (SCHED 3)
        v4f q[2][SM];
        auto scale = [&](int n) {
#pragma unroll
            for (int sm = 0; sm < SM; ++sm) {
                const float c = sa[sm] * (n / SG ? sub[slot] : sgb[slot]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[sm][n][j] = __builtin_fmaf(q[n & 1][sm][j], c, acc[sm][n][j]);
            }
        };
#pragma unroll
        for (int n = 0; n < 2 * SG; ++n) {
            const uint8_t* wat = at + BM * 128 + (n / SG * BNO + wn * TNO + (n % SG) * 16) * 128;
            const v8i wf = rows ? frag(wat, f0, f1) : frag(wat, lane * 16, 1024 + lane * 16);
            const int ew = (int)e8m0_of(n / SG ? sub[slot] : sgb[slot]);
#pragma unroll
            for (int sm = 0; sm < SM; ++sm) {
                if constexpr (SCHED == 3) acc[sm][n] = mfma_fp8_16x16x128_e8(wf, a[sm], acc[sm][n], ew, ea[sm]);
                else q[n & 1][sm] = mfma_fp8_16x16x128(wf, a[sm]);
            }
            if constexpr (SCHED == 0) {
                __builtin_amdgcn_sched_barrier(0);
                if (n > 0) scale(n - 1);
            }
        }
        if constexpr (SCHED == 0) scale(2 * SG - 1);
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
        fetch(i, i);
        __builtin_amdgcn_sched_barrier(0);              // stages in order: the waits count
    }
    for (int64_t i0 = 0; i0 < L; i0 += D) {
#pragma unroll
        for (int r = 0; r < D; ++r) {
            if (i0 + r >= L) break;                     // uniform over the workgroup
            __builtin_amdgcn_sched_barrier(0);
            wait_vmem_keep((D - 2) * kOps);
            // a plain barrier: the fences of the others would wait for the copies in flight. This
            // wave's reads of the last stage are done (its MFMAs took them)
            asm volatile("s_barrier" ::: "memory");
            fetch((r + D - 1) % D, i0 + r + D - 1);
            __builtin_amdgcn_sched_barrier(0);
            compute(r);
        }
    }
    wait_vmem_all();       // no copy into LDS may still be in flight
    __syncthreads();
    gated_finish_tile<BM, BNO, WM, WN, SM, SG>(p, lds, acc, m0, n0, item.slot);
}

// ---------------------------------------------------------------- swap-AB strips ----

template <int MT, int NWO, int NWAVES, int SM, int SG, typename Args>
__device__ __forceinline__ void gated_finish(const Args& p, v4f (&acc)[SM][2 * SG], int64_t m0,
                                             int64_t n0, int64_t rows, int wn, int wk, int lane) {
    const int frow = lane & 15, fgrp = lane >> 4;
    const int64_t F = p.N, n = n0 + 4 * fgrp;
    const bool mine = wk == 0 && n0 < F;     // the waves that hold the sums
    auto row = [&](int sm) { return sm * 16 + frow < rows ? m0 + sm * 16 + frow : (int64_t)-1; };
    if (p.partials) {
        if (mine) gated_partials<SM, SG>(p, acc, n, row);
        return;
    }
    if (mine) gated_combine<SM, SG>(p, acc, n, row);
    if (p.otype != O_CODES) {
        if (!mine) return;
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            const int64_t m = row(sm);
            if (m < 0) continue;
#pragma unroll
            for (int sn = 0; sn < SG; ++sn) store4_any(p.otype, p.out, m * F + n + sn * 16, acc[sm][sn]);
        }
        return;
    }
    if constexpr (NWAVES * NWO == 128) {
        __shared__ uint32_t red[NWAVES][MT];
        uint32_t mx[SM];
        gated_amax<SM, SG>(acc, mx);
        if (mine && fgrp == 0)
#pragma unroll
            for (int sm = 0; sm < SM; ++sm) red[wn][sm * 16 + frow] = mx[sm];
        __syncthreads();
        if (!mine) return;
        const int64_t g = n0 / 128, G = F / 128;
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < NWAVES; ++w) m = max(m, red[w][sm * 16 + frow]);
            const float s = group_scale<Q_FP8>(m, p.os_eps, p.os_ue8m0);
            const int64_t r = m0 + sm * 16 + frow;
            if (wn == 0 && fgrp == 0 && r < (p.os_packed ? (p.M + 3) / 4 * 4 : p.M))
                store_scale(p.out_scales, p.os_stride_m, p.os_stride_g, p.os_packed, r, g, G,
                            r < p.M ? s : 0.f);
            if (r >= p.M) continue;
#pragma unroll
            for (int sn = 0; sn < SG; ++sn)
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + r * F + n + sn * 16) =
                    codes4(acc[sm][sn], m, s);
        }
    }
}

template <int MT, int NWR, int NWAVES, int KW, int D, int CH>
__global__ __launch_bounds__(64 * NWAVES * KW) void gemm_gated_swapab_kernel(GatedArgs p) {
    swapab_body<MT, NWR, NWAVES, KW, D, Q_FP8, O_FP32, W_PACKED16, CH, 0, 1>(p);
}

template <int MT, int NWR, int NWAVES, int KW, int D, int CH>
__global__ __launch_bounds__(64 * NWAVES * KW) void gemm_gated_swapab_lds_kernel(GatedArgs p) {
    swapab_lds_body<MT, NWR, NWAVES, KW, D, Q_FP8, O_FP32, W_PACKED16, CH, 0, 1>(p);
}

// 16 bytes per lane from global memory into LDS (dma16), with the non-temporal hint if ONCE.
template <int ONCE>
__device__ __forceinline__ void dma16_weights(__amdgpu_buffer_rsrc_t r, uint8_t* lds_base,
                                              uint32_t lds_off, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)(lds_base + lds_off), 16, voff, soff, 0, ONCE ? 2 : 0);
}

// Strips for a few tokens, the weights through LDS; the weight stream bounds them. A workgroup
// takes 16 output columns (16 gate rows, 16 up rows) and its waves every KW-th K block, so that
// together they walk neighbouring bytes of the weights. Where that leaves CUs without work it takes
// eight (BNO 8: one fragment of eight gate and eight up rows, the factors of an output in lanes l and
// l + 32): F 2048 x K 7168 row-major, 1 token 7.9 us against 10.0, 16 tokens 9.3 against 10.6. Each wave
// copies 1 KB a load (row-major: whole 128-byte lines of 8 rows; packed: a fragment half) into a ring of
// its own, D K blocks of 4 KB (2 KB), and reads its fragments back: no barrier in the K loop, the wave
// waits until the loads of its oldest block have landed, and what is in flight takes no registers, so a
// CU holds up to 10 waves of 16 KB in flight each. Row-major chunk c of row r sits in slot c ^ swz(r), as
// in the standard tiles.
// ONCE (M <= MT): no other workgroup reads these weights, and they are loaded with the non-temporal
// hint: 10 % off the time at F 18432 and 5 to 13 % on short products. With more tokens it would cost
// up to 6 %: the tiles above find the weights in L2.
// Row-major, F 18432 x K 7168: 45.4 us for 1 token (5.8 TB/s of weights), 49.5 for 16; fragment
// loads straight from the rows take half a line of each of 16 rows a request: 61 and 62 us. Packed:
// ahead of the strips above where the products are short (F 4096 x K 4096, 16 tokens: 8.8 us against
// 11.5) and behind on long streams (F 18432 x K 7168, 1 token: 49 against 43).
template <int MT, int BNO, int KW, int D, int WL, int CH, int ONCE>
__global__ __launch_bounds__(64 * KW) void gemm_gated_ring_kernel(GatedArgs p) {
    constexpr int SM = MT / 16, NF = BNO / 8, BLOCK = NF * 2048;   // NF fragments of 16 weight rows
    constexpr bool PK = CH == 2;
    constexpr int kOps = 2 * NF + 2 + 3 * SM;           // vector loads of one K block
    static_assert((D - 1) * kOps <= 63, "the wait counts loads in six bits");
    static_assert((KW - 1) * SM * NF * 1024 <= KW * D * BLOCK, "the slices' sums fit the rings");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int frow = lane & 15, fgrp = lane >> 4;
    const int64_t M = p.M, F = p.N, K = p.K, KB = K / 128;
    const int64_t n0 = (int64_t)blockIdx.x * BNO, m0 = (int64_t)blockIdx.y * MT;
    const int split = p.split, z = blockIdx.z;
    const int64_t ks0 = (int64_t)z * KB / split, ks1 = (int64_t)(z + 1) * KB / split;
    const int64_t L = (ks1 - ks0 - wk + KW - 1) / KW;   // K blocks ks0 + wk, + KW, ..
    // past every resource here (inside scales that span over 2 GiB, whose value then goes unused)
    constexpr uint32_t kNoLoad = 0x80000000u;

    const uint8_t* w = static_cast<const uint8_t*>(p.w);
    // rows n0 / 16 * 16 on: packed weights come as groups of 16 rows
    const int64_t g0 = n0 / 16 * 16, sub = n0 - g0;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(w + g0 * K, (uint32_t)(16 * K));
    const __amdgpu_buffer_rsrc_t ru = make_rsrc(w + (F + g0) * K, (uint32_t)(16 * K));
    const int64_t rows_a = M - m0 < MT ? M - m0 : MT;
    const int64_t ssm = p.sa_stride_m, ssk = p.sa_stride_k, sa_krows = PK ? (KB - 1) / 4 : KB - 1;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(static_cast<const uint8_t*>(p.a) + m0 * K, (uint32_t)(rows_a * K));
    const __amdgpu_buffer_rsrc_t rsa =
        make_rsrc(p.sa + m0 * ssm, (uint32_t)(((rows_a - 1) * ssm + sa_krows * ssk + 1) * 4));
    uint32_t a_voff[SM], sa_voff[SM];
#pragma unroll
    for (int sm = 0; sm < SM; ++sm) {
        a_voff[sm] = (uint32_t)((sm * 16 + frow) * K + fgrp * 16);
        sa_voff[sm] = (uint32_t)((sm * 16 + frow) * ssm * 4);
    }
    const __amdgpu_buffer_rsrc_t rsg = make_rsrc(p.sw + (n0 / 128) * KB, (uint32_t)(KB * 4));
    const __amdgpu_buffer_rsrc_t rsu = make_rsrc(p.sw + (F / 128 + n0 / 128) * KB, (uint32_t)(KB * 4));
    // copy of rows: lane l takes row l / 8 (BNO 16: + 8), slot l % 8; swz of the second eight differs
    // by 1. Eight columns: the fragment's first eight rows are gate rows, the second eight up rows.
    constexpr bool rows = WL == W_ROW;
    const uint32_t row8 = (uint32_t)(((lane >> 3) + (BNO == 8 ? sub : 0)) * K), slot8 = (lane & 7) ^ (lane >> 3);
    const uint32_t c0 = rows ? row8 + (slot8 << 4)
                        : BNO == 8 ? (uint32_t)((lane >> 5) * 1024 + ((lane >> 3) & 3) * 256 + (lane & 7) * 16 + sub * 16)
                                   : (uint32_t)(lane * 16);
    const uint32_t c1 = rows ? row8 + (uint32_t)(BNO == 8 ? 0 : 8 * K) + ((slot8 ^ 1) << 4)
                             : BNO == 8 ? c0 : (uint32_t)(1024 + lane * 16);
    const uint32_t ring = (uint32_t)(wk * D * BLOCK);
    const uint32_t half8 = (uint32_t)((frow >> 3) * 1024 + fgrp * 128 + (frow & 7) * 16);
    const uint32_t f0 = rows ? (uint32_t)(frow * 128 + ((fgrp ^ swz(frow)) << 4))
                             : BNO == 8 ? half8 : (uint32_t)(lane * 16);
    const uint32_t f1 = rows ? (uint32_t)(frow * 128 + (((fgrp + 4) ^ swz(frow)) << 4))
                             : BNO == 8 ? half8 + 512 : (uint32_t)(1024 + lane * 16);

    v4i abuf[D][SM][2];
    float sab[D][SM], swb[D], swu[D];
    int kbs[D];
    auto fetch = [&](int slot, int64_t i) {
        const bool live = i < L;
        const int64_t kb = ks0 + wk + i * KW;
        const uint32_t s = live ? (uint32_t)kb * 128u : kNoLoad;
        const uint32_t ss = live ? (uint32_t)((PK ? kb >> 2 : kb) * ssk * 4) : kNoLoad;
        const uint32_t ws = rows ? s : live ? (uint32_t)kb * 2048u : kNoLoad;
        const uint32_t sws = live ? (uint32_t)kb * 4u : kNoLoad;
        const uint32_t at = ring + (uint32_t)(slot * BLOCK);
        swb[slot] = buf_f32(rsg, 0, sws);
        swu[slot] = buf_f32(rsu, 0, sws);
        kbs[slot] = (int)(kb & 3);
        dma16_weights<ONCE>(rw, lds, at, c0, ws);
        if constexpr (BNO == 16) {
            dma16_weights<ONCE>(rw, lds, at + 1024, c1, ws);
            dma16_weights<ONCE>(ru, lds, at + 2 * 1024, c0, ws);
            dma16_weights<ONCE>(ru, lds, at + 3 * 1024, c1, ws);
        } else {
            dma16_weights<ONCE>(ru, lds, at + 1024, c1, ws);
        }
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            abuf[slot][sm][0] = __builtin_amdgcn_raw_buffer_load_b128(ra, a_voff[sm], s, 0);
            abuf[slot][sm][1] = __builtin_amdgcn_raw_buffer_load_b128(ra, a_voff[sm], s + 64u, 0);
            sab[slot][sm] = buf_f32(rsa, sa_voff[sm], ss);
        }
    };
    v4f acc[SM][NF];
#pragma unroll
    for (int sm = 0; sm < SM; ++sm)
#pragma unroll
        for (int h = 0; h < NF; ++h) acc[sm][h] = v4f{0.f, 0.f, 0.f, 0.f};
    auto consume = [&](int slot) {
        const uint8_t* at = lds + ring + slot * BLOCK;
        v8i wf[NF];
#pragma unroll
        for (int h = 0; h < NF; ++h) {
            const v4i lo = *reinterpret_cast<const v4i*>(at + h * 2048 + f0);
            const v4i hi = *reinterpret_cast<const v4i*>(at + h * 2048 + f1);
            wf[h] = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        }
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            const float sav = PK ? e8m0_value(e8m0_byte(__float_as_uint(sab[slot][sm]), kbs[slot])) : sab[slot][sm];
            const v4i a0 = abuf[slot][sm][0], a1 = abuf[slot][sm][1];
            const v8i af = v8i{a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
            for (int h = 0; h < NF; ++h) {
                const v4f q = mfma_fp8_16x16x128(wf[h], af);
                const bool up = BNO == 16 ? h != 0 : fgrp >= 2;
                const float c = sav * (up ? swu[slot] : swb[slot]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[sm][h][j] = __builtin_fmaf(q[j], c, acc[sm][h][j]);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < D; ++i) {
        fetch(i, i);
        __builtin_amdgcn_sched_barrier(0);                 // slots in order: the waits count
    }
    for (int64_t i0 = 0; i0 < L; i0 += D) {
#pragma unroll
        for (int r = 0; r < D; ++r) {
            // slot r's loads are the oldest in flight; steps past the slice only wait and refill
            __builtin_amdgcn_sched_barrier(0);
            wait_vmem_keep((D - 1) * kOps);
            if (i0 + r < L) consume(r);                    // uniform over the wave
            __builtin_amdgcn_sched_barrier(0);
            fetch(r, i0 + r + D);
        }
    }
    wait_vmem_all();       // no copy into LDS may still be in flight when the wave ends
    // the sums of waves 1 .. KW - 1 through LDS, added in order by wave 0
    __syncthreads();
    v4f* red = reinterpret_cast<v4f*>(lds);
    if (wk > 0) {
#pragma unroll
        for (int sm = 0; sm < SM; ++sm)
#pragma unroll
            for (int h = 0; h < NF; ++h) red[(((wk - 1) * SM + sm) * NF + h) * 64 + lane] = acc[sm][h];
    }
    __syncthreads();
    if (wk == 0) {
#pragma unroll
        for (int w2 = 0; w2 < KW - 1; ++w2)
#pragma unroll
            for (int sm = 0; sm < SM; ++sm)
#pragma unroll
                for (int h = 0; h < NF; ++h) acc[sm][h] += red[((w2 * SM + sm) * NF + h) * 64 + lane];
    }
    if constexpr (BNO == 16) {
        gated_finish<MT, 16, 1, SM, 1>(p, acc, m0, n0, rows_a, 0, wk, lane);
    } else {
        // lanes 0-31 hold columns n0 + 4 * fgrp .. +3 of the gate, lanes 32-63 the same of up
        if (wk > 0) return;
        const int64_t n = n0 + 4 * (fgrp & 1);
#pragma unroll
        for (int sm = 0; sm < SM; ++sm) {
            const int64_t m = m0 + sm * 16 + frow;
            v4f g = acc[sm][0], u;
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = __shfl_xor(g[j], 32, 64);
            if (m >= M) continue;
            const int64_t own = fgrp >= 2 ? F : 0;
            if (p.partials) {
                *reinterpret_cast<v4f*>(p.partials + ((int64_t)z * M + m) * 2 * F + own + n) = g;
                continue;
            }
            if (p.pre) store4_any(O_BF16, p.pre, m * 2 * F + own + n, g);
            if (fgrp >= 2) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = act_f32(g[j], p.c1, p.c3) * u[j];
            store4_any(p.otype, p.out, m * F + n, g);
        }
    }
}

// ---------------------------------------------------------------- reduce ----

// Eight columns of a token (chunk c of its row; `live`: inside the row, `real`: a token, not a padding
// row of packed words): pre-activations, activation, product, output. Groups of 128 columns are 16
// lanes of a wave.
__device__ __forceinline__ void gated_finish8(const GatedArgs& p, int64_t m, int64_t c, bool live,
                                              bool real, const float* g, const float* u) {
    const int lane = threadIdx.x & 63;
    const int64_t F = p.N;
    float h[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live && real) {
        if (p.pre) {
            static_cast<uint4*>(p.pre)[(m * 2 * F) / 8 + c] = pack8(g);
            static_cast<uint4*>(p.pre)[(m * 2 * F + F) / 8 + c] = pack8(u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = act_f32(g[i], p.c1, p.c3) * u[i];
    }
    if (p.otype != O_CODES) {
        if (live && real) {
            store4_any(p.otype, p.out, m * F + c * 8, v4f{h[0], h[1], h[2], h[3]});
            store4_any(p.otype, p.out, m * F + c * 8 + 4, v4f{h[4], h[5], h[6], h[7]});
        }
        return;
    }
    const uint32_t mx = max16(amax8(h));
    const float s = group_scale<Q_FP8>(mx, p.os_eps, p.os_ue8m0);
    if (!live) return;
    if (real) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + m * F + c * 8) = encode8_group<Q_FP8>(h, mx, s);
    if ((lane & 15) == 0)
        store_scale(p.out_scales, p.os_stride_m, p.os_stride_g, p.os_packed, m, c >> 4, F / 128,
                    real ? s : 0.f);
}

// Sums over `parts` partials in order, `step` floats apart: gate columns at s, up columns at s + up.
__device__ __forceinline__ void gated_sum8(const float* s, int parts, int64_t step, int64_t up, float* g, float* u) {
    v4f g0{}, g1{}, u0{}, u1{};
    for (int z = 0; z < parts; ++z, s += step) {
        const v4f a = *reinterpret_cast<const v4f*>(s), b = *reinterpret_cast<const v4f*>(s + 4);
        const v4f d = *reinterpret_cast<const v4f*>(s + up), e = *reinterpret_cast<const v4f*>(s + up + 4);
        if (z == 0) { g0 = a; g1 = b; u0 = d; u1 = e; }
        else { g0 += a; g1 += b; u0 += d; u1 += e; }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) { g[i] = g0[i]; g[i + 4] = g1[i]; u[i] = u0[i]; u[i + 4] = u1[i]; }
}

// Eight columns a thread: g and u summed over the K ranges in order, then as the epilogues above.
// The grid's rows past M (packed words only) write zeros. Bytes bound it, its launch at decode sizes
// (2.7 us): 5.2 us for 333 x 2048 in two parts.
__global__ __launch_bounds__(256) void gated_reduce_kernel(GatedArgs p) {
    const int64_t m = blockIdx.x, F = p.N, c = (int64_t)blockIdx.y * 256 + threadIdx.x;
    const bool live = c * 8 < F, real = m < p.M;
    float g[8], u[8];
    if (live && real) gated_sum8(p.partials + m * 2 * F + c * 8, p.split, p.M * 2 * F, F, g, u);
    gated_finish8(p, m, c, live, real, g, u);
}

// The same for the tiles that were split (GatedArgs::tail): tail_bn / 8 threads a row of the tile.
__global__ __launch_bounds__(256) void gated_tail_kernel(GatedArgs p) {
    const int bm = p.tail_bm, bn = p.tail_bn, per_row = bn / 8;
    const int64_t M = p.M, F = p.N, r = (int64_t)blockIdx.y * (256 / per_row) + threadIdx.x / per_row;
    const int col = threadIdx.x % per_row * 8;
    int64_t pid_m, pid_n;
    tile_coords(p.tail_first + blockIdx.x, (M + bm - 1) / bm, F / bn, p.group_m, p.raster, pid_m, pid_n);
    const int64_t m = pid_m * bm + r;
    const bool live = r < bm && m < (p.otype == O_CODES && p.os_packed ? (M + 3) / 4 * 4 : M), real = live && m < M;
    float g[8], u[8];
    if (real)
        gated_sum8(p.tail + ((int64_t)blockIdx.x * p.tail_parts * bm + r) * (2 * bn) + col, p.tail_parts,
                   (int64_t)bm * 2 * bn, bn, g, u);
    gated_finish8(p, m, (pid_n * bn + col) / 8, live, real, g, u);
}

hipError_t launch_gated_tail(const GatedArgs& a, int64_t tiles, hipStream_t stream) {
    const int rows = 256 / (a.tail_bn / 8);
    hipLaunchKernelGGL(gated_tail_kernel, dim3((unsigned)(tiles - a.tail_first), (unsigned)((a.tail_bm + rows - 1) / rows)),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_gated_reduce(const GatedArgs& a, hipStream_t stream) {
    const int64_t rows = a.otype == O_CODES && a.os_packed ? (a.M + 3) / 4 * 4 : a.M;
    hipLaunchKernelGGL(gated_reduce_kernel, dim3((unsigned)rows, (unsigned)((a.N / 8 + 255) / 256)),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

void gated_activation(int act, float* c1, float* c3) {
    const double t = 1.5957691216057307117597842397375;     // 2 sqrt(2 / pi)
    *c1 = act == BFQ_ACT_SILU ? 1.f : (float)t;
    *c3 = act == BFQ_ACT_SILU ? 0.f : (float)(0.044715 * t);
}

// ---------------------------------------------------------------- registry ----

static int64_t gated_grid(const GatedArgs& a, int64_t tiles) {
    return a.tail_parts > 1 ? a.tail_first + (tiles - a.tail_first) * a.tail_parts : tiles;
}

template <int BM, int BN, int WM, int WN, int SCHED, int WL>
hipError_t launch_gated_std(const GatedArgs& a, hipStream_t stream) {
    constexpr int LDS_BYTES = StdShape<BM, BN, WM, WN, SCHED>::lds_bytes(2);
    const int64_t tiles = ((a.M + BM - 1) / BM) * ((a.N + BN / 2 - 1) / (BN / 2));
    static std::atomic<uint64_t> opted{0};
    const hipError_t e = opt_in_lds(
        opted, reinterpret_cast<const void*>(&gemm_gated_std_kernel<BM, BN, WM, WN, SCHED, WL>), LDS_BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gemm_gated_std_kernel<BM, BN, WM, WN, SCHED, WL>),
                       dim3((unsigned)gated_grid(a, tiles), 1, (unsigned)a.split), dim3(64 * WM * WN), LDS_BYTES,
                       stream, a);
    return hipGetLastError();
}

template <int BM, int BNO, int WM, int WN, int D, int SCHED, int WL>
hipError_t launch_gated_pipe(const GatedArgs& a, hipStream_t stream) {
    constexpr int LDS_BYTES = D * (BM + 2 * BNO) * 128;
    static_assert(LDS_BYTES <= 160 * 1024 && LDS_BYTES >= BM * 4 * BNO, "the stages fit, the epilogue's tiles too");
    const int64_t tiles = ((a.M + BM - 1) / BM) * (a.N / BNO);
    static std::atomic<uint64_t> opted{0};
    const hipError_t e = opt_in_lds(
        opted, reinterpret_cast<const void*>(&gemm_gated_pipe_kernel<BM, BNO, WM, WN, D, SCHED, WL>), LDS_BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gemm_gated_pipe_kernel<BM, BNO, WM, WN, D, SCHED, WL>),
                       dim3((unsigned)gated_grid(a, tiles), 1, (unsigned)a.split), dim3(64 * WM * WN), LDS_BYTES,
                       stream, a);
    return hipGetLastError();
}

template <int MT, int NWR, int NWAVES, int KW, int D, int CH, int LDS>
hipError_t launch_gated_swapab(const GatedArgs& a, hipStream_t stream) {
    const int64_t cols = NWR / 2 * NWAVES, strips = (a.N + cols - 1) / cols;
    const dim3 grid((unsigned)strips, (unsigned)((a.M + MT - 1) / MT), (unsigned)a.split);
    const dim3 block(64 * NWAVES * KW);
    if constexpr (LDS)
        hipLaunchKernelGGL((gemm_gated_swapab_lds_kernel<MT, NWR, NWAVES, KW, D, CH>), grid,
                           block, 0, stream, a);
    else
        hipLaunchKernelGGL((gemm_gated_swapab_kernel<MT, NWR, NWAVES, KW, D, CH>), grid, block,
                           0, stream, a);
    return hipGetLastError();
}

template <int MT, int BNO, int KW, int D, int WL, int CH, int ONCE>
hipError_t launch_gated_ring_once(const GatedArgs& a, hipStream_t stream) {
    constexpr int LDS_BYTES = KW * D * BNO * 256;
    static std::atomic<uint64_t> opted{0};
    const hipError_t e =
        opt_in_lds(opted, reinterpret_cast<const void*>(&gemm_gated_ring_kernel<MT, BNO, KW, D, WL, CH, ONCE>), LDS_BYTES);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.N / BNO), (unsigned)((a.M + MT - 1) / MT), (unsigned)a.split);
    hipLaunchKernelGGL((gemm_gated_ring_kernel<MT, BNO, KW, D, WL, CH, ONCE>), grid, dim3(64 * KW), LDS_BYTES, stream, a);
    return hipGetLastError();
}

template <int MT, int BNO, int KW, int D, int WL, int CH>
hipError_t launch_gated_ring(const GatedArgs& a, hipStream_t stream) {
    return a.M <= MT ? launch_gated_ring_once<MT, BNO, KW, D, WL, CH, 1>(a, stream)
                     : launch_gated_ring_once<MT, BNO, KW, D, WL, CH, 0>(a, stream);
}

// The last four arguments are what the tile rule knows of a kernel: the workgroups a CU holds, and
// its times in microseconds (GatedKernel).
#define BFQ_GATED_STD(BM, BN, WM, WN, SC, WL, OCC, LAT, THR, FIX)                               \
    GatedKernel{bfq_tile{0, BM, (BN) / 2, 128, 1, WM, WN, 2, 8, SC, 0, 0}, WL,                  \
                (SC) == 3 ? S_UE8M0 : S_FP32, &launch_gated_std<BM, BN, WM, WN, SC, WL>, OCC, LAT, THR, FIX}
#define BFQ_GATED_SAB1(MT, NWR, NW, KW, D, CH, L, OCC, LAT, THR, FIX)                           \
    GatedKernel{bfq_tile{1, MT, (NWR) / 2 * (NW), 128, 1, KW, NW, D, 1, L, 0, 0}, W_PACKED16,   \
                (CH) == 2 ? S_PACKED : S_FP32,                                                 \
                &launch_gated_swapab<MT, NWR, NW, KW, D, CH, L>, OCC, LAT, THR, FIX}
#define BFQ_GATED_SAB(MT, NWR, NW, KW, D, L, OCC, LAT, THR, FIX)                                \
    BFQ_GATED_SAB1(MT, NWR, NW, KW, D, 0, L, OCC, LAT, THR, FIX),                           \
        BFQ_GATED_SAB1(MT, NWR, NW, KW, D, 2, L, OCC, LAT, THR, FIX)

#define BFQ_GATED_RING1(MT, BNO, KW, D, WL, CH, OCC, LAT, THR, FIX)                             \
    GatedKernel{bfq_tile{1, MT, BNO, 128, 1, KW, 1, D, 1, 2, 0, 0}, WL, (CH) == 2 ? S_PACKED : S_FP32, \
                &launch_gated_ring<MT, BNO, KW, D, WL, CH>, OCC, LAT, THR, FIX}
#define BFQ_GATED_RING(MT, BNO, KW, D, WL, OCC, LAT, THR, FIX)                                  \
    BFQ_GATED_RING1(MT, BNO, KW, D, WL, 0, OCC, LAT, THR, FIX),                                 \
        BFQ_GATED_RING1(MT, BNO, KW, D, WL, 2, OCC, LAT, THR, FIX)

#define BFQ_GATED_PIPE(BM, BNO, WM, WN, D, SC, WL, OCC, LAT, THR, FIX)                          \
    GatedKernel{bfq_tile{0, BM, BNO, 128, 1, WM, WN, D, 8, SC, 0, 0}, WL,                       \
                (SC) == 3 ? S_UE8M0 : S_FP32, &launch_gated_pipe<BM, BNO, WM, WN, D, SC, WL>, OCC, LAT, THR, FIX}

static const GatedKernel kGatedKernels[] = {
    BFQ_GATED_PIPE(32, 64, 1, 4, 4, 0, W_ROW, 2, 0.351f, 0.332f, 5.060f),
    BFQ_GATED_PIPE(32, 64, 1, 4, 4, 0, W_PACKED16, 2, 0.356f, 0.317f, 4.915f),
    BFQ_GATED_PIPE(32, 64, 1, 4, 4, 3, W_ROW, 2, 0.283f, 0.313f, 5.061f),
    BFQ_GATED_PIPE(32, 64, 1, 4, 4, 3, W_PACKED16, 2, 0.283f, 0.301f, 4.891f),
    BFQ_GATED_PIPE(64, 64, 2, 2, 3, 0, W_ROW, 2, 0.485f, 0.393f, 5.538f),
    BFQ_GATED_PIPE(64, 64, 2, 2, 3, 0, W_PACKED16, 2, 0.477f, 0.365f, 5.461f),
    BFQ_GATED_PIPE(64, 64, 2, 2, 3, 3, W_ROW, 2, 0.379f, 0.379f, 5.470f),
    BFQ_GATED_PIPE(64, 64, 2, 2, 3, 3, W_PACKED16, 2, 0.396f, 0.358f, 5.394f),
    BFQ_GATED_PIPE(64, 128, 2, 4, 3, 0, W_ROW, 1, 0.774f, 0.053f, 6.016f),
    BFQ_GATED_PIPE(64, 128, 2, 4, 3, 0, W_PACKED16, 1, 0.714f, 0.040f, 6.121f),
    BFQ_GATED_PIPE(64, 128, 2, 4, 3, 3, W_ROW, 1, 0.744f, 0.000f, 5.962f),
    BFQ_GATED_PIPE(64, 128, 2, 4, 3, 3, W_PACKED16, 1, 0.691f, 0.040f, 6.057f),
    BFQ_GATED_PIPE(128, 64, 4, 2, 4, 0, W_ROW, 1, 0.690f, 0.323f, 5.539f),
    BFQ_GATED_PIPE(128, 64, 4, 2, 4, 0, W_PACKED16, 1, 0.666f, 0.083f, 5.533f),
    BFQ_GATED_PIPE(128, 64, 4, 2, 4, 3, W_ROW, 1, 0.659f, 0.000f, 5.606f),
    BFQ_GATED_PIPE(128, 64, 4, 2, 4, 3, W_PACKED16, 1, 0.609f, 0.184f, 5.534f),
    BFQ_GATED_PIPE(128, 128, 2, 4, 3, 0, W_ROW, 1, 1.179f, 0.548f, 5.883f),
    BFQ_GATED_PIPE(128, 128, 2, 4, 3, 0, W_PACKED16, 1, 1.136f, 0.611f, 5.883f),
    BFQ_GATED_PIPE(128, 128, 2, 4, 3, 3, W_ROW, 1, 1.032f, 0.155f, 5.811f),
    BFQ_GATED_PIPE(128, 128, 2, 4, 3, 3, W_PACKED16, 1, 1.023f, 0.000f, 5.928f),
    BFQ_GATED_STD(256, 256, 4, 2, 0, W_PACKED16, 1, 1.894f, 0.509f, 4.267f),
    BFQ_GATED_STD(256, 256, 4, 2, 1, W_ROW, 1, 1.951f, 0.000f, 4.198f),
    BFQ_GATED_STD(256, 256, 4, 2, 3, W_ROW, 1, 1.862f, 0.531f, 3.938f),
    BFQ_GATED_STD(256, 256, 4, 2, 3, W_PACKED16, 1, 1.793f, 0.524f, 4.234f),
    BFQ_GATED_RING(16, 16, 1, 4, W_ROW, 10, 0.164f, 0.103f, 3.870f),
    BFQ_GATED_RING(16, 16, 1, 4, W_PACKED16, 10, 0.164f, 0.102f, 3.902f),
    BFQ_GATED_RING(16, 16, 2, 4, W_ROW, 5, 0.000f, 0.129f, 3.611f),
    BFQ_GATED_RING(16, 16, 2, 4, W_PACKED16, 5, 0.000f, 0.126f, 3.507f),
    BFQ_GATED_RING(32, 16, 2, 4, W_ROW, 5, 0.000f, 0.175f, 3.802f),
    BFQ_GATED_RING(32, 16, 2, 4, W_PACKED16, 5, 0.000f, 0.169f, 3.685f),
    BFQ_GATED_RING(16, 8, 4, 4, W_ROW, 5, 0.001f, 0.099f, 3.127f),
    BFQ_GATED_RING(16, 8, 4, 4, W_PACKED16, 5, 0.001f, 0.096f, 3.168f),
    BFQ_GATED_SAB(16, 32, 1, 4, 4, 0, 4, 0.002f, 0.093f, 3.957f),
    BFQ_GATED_SAB(32, 32, 8, 1, 4, 1, 2, 0.000f, 0.750f, 6.568f),
    BFQ_GATED_SAB(64, 32, 8, 1, 4, 1, 1, 0.283f, 0.780f, 7.093f),
};

const GatedKernel* gated_kernels(int* count) {
    *count = (int)(sizeof(kGatedKernels) / sizeof(kGatedKernels[0]));
    return kGatedKernels;
}

// ---------------------------------------------------------------- backward ----

// 16 bytes, with the non-temporal hint if S.
template <int S> __device__ __forceinline__ uint4 stream_load(const uint4* p) {
    if constexpr (S) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p)));
    else return *p;
}
template <int S> __device__ __forceinline__ void stream_store(uint4* p, const uint4& v) {
    if constexpr (S) __builtin_nontemporal_store(__builtin_bit_cast(v4u, v), reinterpret_cast<v4u*>(p));
    else *p = v;
}

// With a = act(g): dg = dh * u * act'(g), du = dh * a, and the product h = a * u again. Eight
// columns a thread, read once and written once; bytes bound it: 4096 x 18432 takes 165 to 169 us, by the
// card, for the pair's gradient and h as bf16 (906 MB, 5.4 TB/s; some 9 us more without the non-temporal
// hints) and 109 us for its codes (604 MB, 5.5 TB/s; a large copy reaches 4.8). Codes: 128-column groups
// of the 2F-wide row, one scale each, 16 lanes a group; rows past M (packed words only) write zeros.
template <int Q, int S>
__global__ __launch_bounds__(256) void gated_bwd_kernel(GatedBwdArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t m = blockIdx.x, F = p.F, c = (int64_t)blockIdx.y * 256 + threadIdx.x;
    const bool live = c * 8 < F, real = m < p.M;
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[i] = du[i] = 0.f;
    if (live && real) {
        const uint4* pre = static_cast<const uint4*>(p.pre) + m * 2 * F / 8;
        const uint4 gc = stream_load<S>(pre + c), uc = stream_load<S>(pre + F / 8 + c);
        const uint4 dc = stream_load<S>(static_cast<const uint4*>(p.dh) + m * F / 8 + c);
        float g[8], u[8], dh[8], h[8];
        unpack8(gc, g);
        unpack8(uc, u);
        unpack8(dc, dh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float slope;
            const float a = act_slope_f32(g[i], p.c1, p.c3, slope);
            h[i] = a * u[i];
            dg[i] = dh[i] * u[i] * slope;
            du[i] = dh[i] * a;
        }
        if (p.h) stream_store<S>(static_cast<uint4*>(p.h) + m * F / 8 + c, pack8(h));
        if (p.dpre) {
            uint4* d = static_cast<uint4*>(p.dpre) + m * 2 * F / 8;
            stream_store<S>(d + c, pack8(dg));
            stream_store<S>(d + F / 8 + c, pack8(du));
        }
    }
    if constexpr (Q >= 0) {
        const uint32_t mg = max16(amax8(dg)), mu = max16(amax8(du));
        if (!live) return;
        const float sg = group_scale<Q>(mg, p.q_eps, p.ue8m0), su = group_scale<Q>(mu, p.q_eps, p.ue8m0);
        if (real) {
            uint2* q = static_cast<uint2*>(p.q) + m * 2 * F / 8;
            q[c] = encode8_group<Q>(dg, mg, sg);
            q[F / 8 + c] = encode8_group<Q>(du, mu, su);
        }
        if ((lane & 15) == 0) {
            const int64_t G = 2 * F / 128, g = c >> 4;
            store_scale(p.scales, p.s_stride_m, p.s_stride_g, p.packed, m, g, G, real ? sg : 0.f);
            store_scale(p.scales, p.s_stride_m, p.s_stride_g, p.packed, m, F / 128 + g, G, real ? su : 0.f);
        }
    }
}

template <int S>
static void launch_bwd(const GatedBwdArgs& a, hipStream_t stream) {
    const int64_t rows = a.q && a.packed ? (a.M + 3) / 4 * 4 : a.M;
    const dim3 grid((unsigned)rows, (unsigned)((a.F / 8 + 255) / 256));
    if (!a.q) hipLaunchKernelGGL((gated_bwd_kernel<-1, S>), grid, dim3(256), 0, stream, a);
    else if (a.qtype == Q_FP8) hipLaunchKernelGGL((gated_bwd_kernel<Q_FP8, S>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((gated_bwd_kernel<Q_INT8, S>), grid, dim3(256), 0, stream, a);
}

hipError_t launch_gated_bwd(const GatedBwdArgs& a, hipStream_t stream) {
    if (past_caches(a.M * a.F * ((a.dpre ? 4 : 0) + (a.q ? 2 : 0) + (a.h ? 2 : 0)))) launch_bwd<1>(a, stream);
    else launch_bwd<0>(a, stream);
    return hipGetLastError();
}

// Codes [N][K] and their 128x128 block scales to [K][N]: one 64 x 64 tile a workgroup through LDS,
// 16-byte rows in and out; the first workgroup of a block moves its scale. An offline step: 129 us
// for 36864 x 7168 (4.1 TB/s).
__global__ __launch_bounds__(256) void transpose_weights_kernel(const uint8_t* __restrict__ w,
                                                                const float* __restrict__ s,
                                                                uint8_t* __restrict__ wt,
                                                                float* __restrict__ st, int64_t N,
                                                                int64_t K) {
    __shared__ uint8_t tile[64][64 + 4];
    const int t = threadIdx.x, r = t >> 2, c = (t & 3) * 16;
    const int64_t k0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
    const uint4 v = *reinterpret_cast<const uint4*>(w + (n0 + r) * K + k0 + c);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(&tile[r][c + 4 * i]) = in[i];
    __syncthreads();
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        out[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) out[i] |= (uint32_t)tile[c + 4 * i + j][r] << (8 * j);
    }
    *reinterpret_cast<uint4*>(wt + (k0 + r) * N + n0 + c) = make_uint4(out[0], out[1], out[2], out[3]);
    if (t == 0 && ((blockIdx.x | blockIdx.y) & 1) == 0)
        st[(k0 / 128) * (N / 128) + n0 / 128] = s[(n0 / 128) * (K / 128) + k0 / 128];
}

hipError_t launch_transpose_weights(const void* w, const float* s, void* wt, float* st, int64_t N,
                                    int64_t K, hipStream_t stream) {
    hipLaunchKernelGGL(transpose_weights_kernel, dim3((unsigned)(K / 64), (unsigned)(N / 64)),
                       dim3(256), 0, stream, static_cast<const uint8_t*>(w), s,
                       static_cast<uint8_t*>(wt), st, N, K);
    return hipGetLastError();
}

}  // namespace bfq
