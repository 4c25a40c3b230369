/*
 * bfq.h — C-ABI of libbfq: block-scaled W8A8 (e4m3fn / int8) linear layer on MI355X (gfx950).
 *
 * Pages cited (by title and section):
 *   [BENCH]  "vLLM DeepGEMM FP8 Block GEMM 基准测试：DeepSeek DeepGEMM 对比 Triton 与 CUTLASS
 *             的块量化 GEMM 内核解析" (blog.gitcode.com)
 *   [CONFIG] "vLLM 量化 Kernel 配置机制：W8A8 Block FP8 Triton 内核的调优、选择与回退原理"
 *             (blog.gitcode.com)
 *   [PR]     vLLM pull request 42153, per_token_group_quant 2-D grid (prhub.com.cn)
 *   [HELION] "Building a High-Performance and Portable vLLM Linear Backend with Helion"
 *             (PyTorch blog, translated)
 *
 * Conventions for every entry point:
 *  - Device pointers unless marked "host". Every buffer is allocated and freed by the
 *    caller; the library never allocates, frees or synchronizes device memory. It owns only
 *    its host-side tile table and the static device buffer of bfq_block_gemm_noalloc.
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream). Work is enqueued
 *    asynchronously; the call returns once the launches are enqueued.
 *  - All arguments are validated before anything is enqueued. On a negative status nothing
 *    was launched and no output was touched; bfq_last_error() holds a detail string
 *    (thread-local). A positive status is success with a warning.
 *  - M = 0 is valid and launches nothing.
 *  - Shapes are int64; K and N must be multiples of 128 (GEMM: M, N < 2^31, M * N < 2^40,
 *    K <= 2^23, scale ld <= 2^23, and the activation scales of 256 tokens over all K blocks
 *    span less than 4 GiB), and x/q/w/out 16-byte aligned.
 *  - Buffers of one call do not overlap unless its description says that they may.
 *  - Two calls on one stream are ordered; calls on different streams that share an output
 *    or workspace race.
 */
#ifndef BFQ_H
#define BFQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BFQ_OK = 0,
    BFQ_WARN_DEFAULT_TILE = 1,  /* success; no tuned entry for (N,K,dtype): default tile used */
    BFQ_ERR_NULL = -1,          /* a required pointer is NULL */
    BFQ_ERR_SHAPE = -2,         /* M<0, K or N not a multiple of 128, group/block not 128 */
    BFQ_ERR_DTYPE = -3,         /* unsupported input/output dtype */
    BFQ_ERR_ALIGN = -4,         /* pointer not 16-byte aligned (scales: 4-byte) */
    BFQ_ERR_WORKSPACE = -5,     /* workspace smaller than bfq_gemm_workspace_bytes() */
    BFQ_ERR_TILE = -6,          /* explicit tile is not one of the compiled kernels */
    BFQ_ERR_TABLE = -7,         /* tile table file missing or malformed */
    BFQ_ERR_HIP = -8,           /* a HIP runtime call or launch failed */
    BFQ_ERR_ARG = -9            /* invalid scalar argument (eps, enum value, index) */
} bfq_status;

/* The *_INT32_MIN_ and *_INT32_RANGE_ enumerators below are not values of their enums: they make each
 * enum a 32-bit type in which every int32 is representable, so that an out-of-range argument from a
 * C or ctypes caller is rejected (BFQ_ERR_ARG / BFQ_ERR_DTYPE) rather than undefined. */
typedef enum {
    BFQ_BF16 = 0,
    BFQ_FP16 = 1,
    BFQ_FP32 = 2,
    BFQ_E4M3FN = 3,   /* OCP float8 e4m3fn, max 448 */
    BFQ_INT8 = 4,     /* symmetric int8 in [-127, 127] */
    BFQ_INT32 = 5,
    BFQ_DTYPE_INT32_MIN_ = -0x7FFFFFFF - 1,
    BFQ_DTYPE_INT32_RANGE_ = 0x7FFFFFFF  /* not a dtype: see below */
} bfq_dtype;

/* Layout of per-(token, group) activation scales, [BENCH] §4.1 (row-major for the Triton
 * kernel, column-major for CUTLASS/DeepGEMM; the TMA-aligned column-major form is
 * column-major with ld = M rounded up to a multiple of 4).
 * BFQ_SCALES_PACKED_UE8M0 ([PR]: the packed output of the per-token-group kernel,
 * output_s_packed): UE8M0 scales as E8M0 codes (2^(code - 127); NaN and Inf -> 255, E8M0
 * has no infinity), four groups per 32-bit word: word (w, m) at ((uint32_t*)s)[w * ld + m],
 * w < ceil(G/4), byte j (bits 8j..8j+7) = group 4w + j, 0 past the last group. The scale
 * pointer then addresses uint32 words. The quantizer needs ld >= M rounded up to a multiple
 * of 4 and writes zero words in rows M .. round_up(M, 4) - 1 (TMA row alignment); the GEMM
 * needs ld >= M. Only with scale_fmt BFQ_SCALE_UE8M0 and 1x128 groups. */
typedef enum {
    BFQ_SCALES_ROW_MAJOR = 0,    /* s[m * ld + g], ld >= K/128 */
    BFQ_SCALES_COL_MAJOR = 1,    /* s[g * ld + m], ld >= M     */
    BFQ_SCALES_PACKED_UE8M0 = 2, /* words[w * ld + m], see above */
    BFQ_SCALES_INT32_MIN_ = -0x7FFFFFFF - 1,
    BFQ_SCALES_INT32_RANGE_ = 0x7FFFFFFF
} bfq_scale_layout;

/* Layout of the weight codes in memory. The values are the same bytes either way; the packed
 * layout puts each MFMA fragment's bytes together so that every wave-wide 16-byte-per-lane
 * load reads 1 KB of contiguous memory (a row-major [N][K] matrix can only give each load
 * 16 rows x 64 bytes, which caps the weight stream well below the HBM peak).
 *   BFQ_W_ROW_MAJOR: w[n][k] at byte n*K + k.
 *   BFQ_W_PACKED16 : for every 16-row group f = n/16 and K block kb, 2048 bytes at
 *                    (f*(K/128) + kb)*2048; inside them byte h*1024 + 16*l + b (h in {0,1},
 *                    lane l in [0,64), b in [0,16)) holds w[16f + l%16][128kb + 64h + 16*(l/16) + b].
 *                    The whole matrix still spans N*K bytes, rows in blocks of 16. */
typedef enum {
    BFQ_W_ROW_MAJOR = 0,
    BFQ_W_PACKED16 = 1,
    BFQ_W_INT32_MIN_ = -0x7FFFFFFF - 1,
    BFQ_W_INT32_RANGE_ = 0x7FFFFFFF
} bfq_weight_layout;

/* Format of the fp32 scales. UE8M0: every scale is a power of two — the block's
 * max(amax, eps)/Qmax rounded up to the next power of two ([BENCH] §4.1: with use_ue8m0 the
 * scale is first rounded up to a power of two, the format DeepGEMM's hardware scaling path
 * requires). The scales are still stored as fp32 (exact); the codes are encode(x / scale).
 * A GEMM told that both scale arrays are UE8M0 may apply them inside gfx950's
 * block-scaled MFMA instead of with one fp32 FMA per output and K block. */
typedef enum {
    BFQ_SCALE_FP32 = 0,
    BFQ_SCALE_UE8M0 = 1,
    BFQ_SCALE_INT32_MIN_ = -0x7FFFFFFF - 1,
    BFQ_SCALE_INT32_RANGE_ = 0x7FFFFFFF
} bfq_scale_format;

/* Activation of a gated product, act(g) * u. SILU: g / (1 + exp(-g)). GELU_TANH: the tanh form,
 * 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))). */
typedef enum {
    BFQ_ACT_SILU = 0,
    BFQ_ACT_GELU_TANH = 1,
    BFQ_ACT_INT32_MIN_ = -0x7FFFFFFF - 1,
    BFQ_ACT_INT32_RANGE_ = 0x7FFFFFFF
} bfq_activation;

/* What one value of a block's gate covers: nothing (no gate), a channel ([K]), a token ([M]) or
 * one element ([M][K]). */
typedef enum {
    BFQ_GATE_NONE = 0,
    BFQ_GATE_CHANNEL = 1,
    BFQ_GATE_TOKEN = 2,
    BFQ_GATE_FULL = 3,
    BFQ_GATE_INT32_MIN_ = -0x7FFFFFFF - 1,
    BFQ_GATE_INT32_RANGE_ = 0x7FFFFFFF
} bfq_gate_kind;

/* A router's score function. SOFTMAX: over the token's experts. SIGMOID: each expert by itself. */
typedef enum {
    BFQ_SCORE_SOFTMAX = 0,
    BFQ_SCORE_SIGMOID = 1,
    BFQ_SCORE_INT32_MIN_ = -0x7FFFFFFF - 1,
    BFQ_SCORE_INT32_RANGE_ = 0x7FFFFFFF
} bfq_score;

/* One launch configuration of the block GEMM ([CONFIG] §2: per-M launch parameters).
 *   variant 0 "standard": bm x bn output tile per workgroup, A and W tiles staged through
 *             LDS (double-buffered), waves_m x waves_n waves, group_m = grouped tile order.
 *   variant 1 "swap_ab": the weight rows stream straight from HBM into the wide MFMA
 *             operand and the bm tokens ride in the narrow one; the output tile is formed
 *             transposed and stored back row-major ([HELION] kernel section). A workgroup
 *             holds waves_n strips of bn/waves_n weight rows; the waves_m waves of a strip
 *             split its K range and are summed in the workgroup, in a fixed order. sched 0:
 *             each wave fetches its token fragments; sched 1: each K block's token fragments
 *             are fetched once per workgroup and shared through LDS.
 *   variant 2 "stream-K": the tiles of variant 0 on a persistent grid of one workgroup per
 *             compute unit; whole tiles in rounds, then the K blocks of the last one to two
 *             rounds of tiles split evenly over the grid; a second kernel sums each split
 *             tile's parked fp32 partials in K order (split_k must be 1). Its workspace holds
 *             two partial tiles per compute unit.
 *   split_k  : K blocks split into split_k contiguous chunks (>= 1), fp32 partials reduced
 *             in a fixed order ([HELION] kernel section).
 *   stages   : LDS stages (variants 0, 2) or weight prefetch depth in K blocks (variant 1).
 *   sched    : variants 0 and 2 instruction schedule (variant 1: see above): 4 = per-token x
 *             per-channel scales (block_shape {1, K}), the MFMA accumulating the whole K; 3 = the scales
 *             applied by the block-scaled MFMA, which accumulates across K blocks (fp8 and
 *             BFQ_SCALE_UE8M0 scales only); 0 = each sub-tile's scale FMAs right after its
 *             MFMAs, 1 = software-pipelined (FMAs one sub-tile behind the MFMAs), 2 = 32x32
 *             sub-tiles (two 32x32x64 MFMAs per K block, FMAs one pair behind; fp8 only).
 *   group_m, raster: variants 0 and 2 tile order (launch arguments, any group_m >= 1): raster 0
 *             gives each of the 8 XCDs a contiguous range of tiles, raster 1 does not.
 *   bk is always 128 (one scale block per K step). */
typedef struct {
    int32_t variant, bm, bn, bk, split_k, waves_m, waves_n, stages, group_m, sched, raster,
        reserved;
} bfq_tile;

/* Per-token-group quantization ([BENCH] §4.1 per_token_group_quant_fp8; [PR] kernel
 * arguments eps/min_8bit/max_8bit). For each row m and 128-wide group g of x:
 *   scale = max(amax, eps) / Qmax   (Qmax = 448 for E4M3FN, 127 for INT8; IEEE division)
 *   q     = encode(x / scale)       (IEEE division; e4m3fn: RNE, saturating; int8: RNE,
 *                                    clamp [-127, 127])
 * scale_fmt BFQ_SCALE_UE8M0 rounds each scale up to a power of two before encoding.
 * A group containing NaN gets a NaN scale and codes 0x7F (e4m3fn) or 0 (int8).
 *   x_bf16 [M][K] row-major bf16; q [M][K] row-major codes (1 byte);
 *   scales: fp32, layout per `layout` with leading dimension scale_ld.
 * group_size 128, or group_size == K for one scale per token (the per-token activation scales
 * of the FP8_Dynamic / W8A8_INT8 formats, [HELION] scope section; K <= 32768): scales then
 * hold one value per row, at scales[m * scale_ld] (row-major, scale_ld >= 1) or scales[m]
 * (column-major, scale_ld >= M). q_dtype must be BFQ_E4M3FN or BFQ_INT8. */
bfq_status bfq_quant_tokens(const void* x_bf16, int64_t M, int64_t K, int32_t group_size,
                            bfq_dtype q_dtype, void* q, float* scales, bfq_scale_layout layout,
                            int64_t scale_ld, float eps, bfq_scale_format scale_fmt,
                            void* stream);

/* Per-block weight quantization, the offline step before the GEMM ([BENCH] §4.1
 * per_block_cast_to_fp8 with fp32 scales): for each block_shape[0] x block_shape[1] block of
 * w [N][K] (fp32, row-major): scale = max(amax, eps)/Qmax, q = encode(w / scale).
 *   q [N][K] codes; scales [N/128][K/128] row-major fp32.
 * block_shape {128, 128}, or {1, K} for one scale per output channel (the per-channel weight
 * scales of FP8_Dynamic / W8A8_INT8, [HELION] scope section; K <= 32768): scales [N]. */
bfq_status bfq_quant_weight_blocks(const float* w, int64_t N, int64_t K,
                                   const int32_t block_shape[2] /* host */, bfq_dtype q_dtype,
                                   void* q, float* scales, float eps,
                                   bfq_scale_format scale_fmt, void* stream);

/* Rearrange weight codes from row-major [N][K] into BFQ_W_PACKED16 (a byte permutation, part
 * of the offline weight preparation like bfq_quant_weight_blocks). w_q and w_packed are
 * separate N*K-byte device buffers (16-byte aligned, not overlapping); q_dtype E4M3FN or
 * INT8 (the permutation does not depend on it). N, K multiples of 128. */
bfq_status bfq_pack_weights(const void* w_q, int64_t N, int64_t K, bfq_dtype q_dtype,
                            void* w_packed, void* stream);

/* Tile selection ([CONFIG] §4.1-§4.2): exact (N, K, dtype, block shape, weight layout, scale format) entry of the loaded
 * tile table, then the bucket nearest to M (ties to the smaller bucket; M past the grid ->
 * last bucket). No entry -> the compiled-in default rule and BFQ_WARN_DEFAULT_TILE ([CONFIG]
 * §4.1 warns and falls back to a default config). tile_out is a host pointer. */
bfq_status bfq_select_tile(int64_t M, int64_t N, int64_t K, const int32_t block_shape[2],
                           bfq_dtype in_dtype, bfq_dtype out_dtype, bfq_weight_layout w_layout,
                           bfq_scale_format scale_fmt, bfq_tile* tile_out);

/* Batch-invariant mode ([CONFIG] §5: with the batch-invariant switch set, tuned configs are
 * not used, so that the output of a token does not depend on how many tokens are in the
 * batch). When enabled, bfq_select_tile ignores the tile table and returns tiles that
 * compute every output element with the same operations in the same order for any M: no
 * split-K, no K split inside a workgroup, no stream-K; with row-major weights only standard
 * tiles (the swap-AB kernels feed the MFMA a different K order there); scales always applied
 * by the fp32 FMA. Rows of the output are then bitwise independent of M. Process-wide;
 * initialized from the environment variable BFQ_BATCH_INVARIANT (1 = on) at first use; must
 * not be changed concurrently with other calls. Explicit tiles passed to bfq_block_gemm are
 * not affected. */
void    bfq_set_batch_invariant(int32_t enable);
int32_t bfq_get_batch_invariant(void);

/* Bytes of device workspace bfq_block_gemm needs for this shape and tile (split-K fp32
 * partials: split_k * M * N * 4 when split_k > 1; stream-K: two partial tiles per compute
 * unit; else 0). tile NULL -> the tile selected for e4m3fn codes in the row-major layout.
 * SIZE_MAX when M * N >= 2^40, a shape bfq_block_gemm rejects. */
size_t bfq_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, const bfq_tile* tile);

/* Block-scaled GEMM ([BENCH] §4.2, w8a8 block-scaled matmul):
 *   out[m][n] = sum_kb ( sum_{k in kb} a_q[m][k] * w_q[n][k] ) * a_scales[m, kb] * w_scales[n/128][kb]
 * with exact per-block products, an fp32 accumulator and one rounding to out_dtype.
 *   a_q [M][K] codes (K-contiguous); w_q N*K codes in w_layout (row-major [N][K] is the
 *   "NT" form of the page; BFQ_W_PACKED16 from bfq_pack_weights);
 *   a_scales per a_layout/a_scale_ld; w_scales [N/128][K/128] row-major;
 *   scale_fmt BFQ_SCALE_UE8M0 states that every a_scales and w_scales value is a power of
 *   two (as the quantizers write in that format); results are then undefined otherwise.
 *   out [M][N] row-major, out_dtype BF16 | FP16 | FP32.
 *   tile NULL -> bfq_select_tile for (w_layout, scale_fmt); an explicit tile must name a
 *   kernel compiled for w_layout whose scale handling allows scale_fmt (else BFQ_ERR_TILE);
 *   workspace may be NULL when the tile needs none.
 * block_shape {1, K} selects the per-token x per-channel format ([HELION] scope section,
 * FP8_Dynamic / W8A8_INT8; K <= 32768):
 *   out[m][n] = ( sum_k a_q[m][k] * w_q[n][k] ) * a_scales[m] * w_scales[n]
 *   with one scale per token (a_layout row-major: a_scales[m * a_scale_ld], a_scale_ld >= 1;
 *   column-major: a_scales[m], a_scale_ld >= M) and w_scales [N]; the codes' product is
 *   accumulated over the whole K (fp8: fp32 MFMA accumulation; int8: exact int32), then
 *   scaled once. scale_fmt does not change how such scales are applied. Those kernels are
 *   tiles with sched 4 (variants 0 and 2) or the variant 1 tiles built for this format.
 * Returns BFQ_WARN_DEFAULT_TILE when tile was NULL and the default rule was used. */
bfq_status bfq_block_gemm(const void* a_q, const float* a_scales, bfq_scale_layout a_layout,
                          int64_t a_scale_ld, const void* w_q, const float* w_scales,
                          bfq_weight_layout w_layout, bfq_scale_format scale_fmt, void* out,
                          int64_t M, int64_t N, int64_t K,
                          const int32_t block_shape[2] /* host */, bfq_dtype in_dtype,
                          bfq_dtype out_dtype, const bfq_tile* tile /* host */,
                          void* workspace, size_t workspace_bytes, void* stream);

/* The block GEMM for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same arguments and
 * result as bfq_block_gemm without a workspace; split-K partials and stream-K slots go to a
 * static device buffer of the library (bfq_noalloc_scratch_bytes() = 32 MiB, one per GPU,
 * held from the library's load until the process ends). It calls no allocator.
 *   tile NULL -> the tile bfq_select_tile gives, made to fit the buffer: a stream-K tile runs
 *   as the plain grid of the same tile, and the K split drops until the partials fit (the
 *   result stays within the parity bar; it may differ in the last bits from bfq_block_gemm,
 *   which runs the selected tile as is).
 *   An explicit tile whose workspace exceeds the buffer -> BFQ_ERR_WORKSPACE (nothing
 *   launched).
 * Every call on one GPU shares that GPU's buffer: calls that overlap on one GPU (different
 * streams, or host threads) race and must be serialised by the caller. The buffer keeps the
 * last call's contents; no call reads what an earlier one left. */
bfq_status bfq_block_gemm_noalloc(const void* a_q, const float* a_scales,
                                  bfq_scale_layout a_layout, int64_t a_scale_ld, const void* w_q,
                                  const float* w_scales, bfq_weight_layout w_layout,
                                  bfq_scale_format scale_fmt, void* out, int64_t M, int64_t N,
                                  int64_t K, const int32_t block_shape[2] /* host */,
                                  bfq_dtype in_dtype, bfq_dtype out_dtype,
                                  const bfq_tile* tile /* host */, void* stream);
size_t bfq_noalloc_scratch_bytes(void);

/* Load a tile table (JSON, host path) and replace the current one ([CONFIG] §2 schema:
 * per (N, K, dtype, block_shape) a map "M bucket -> launch parameters"). Must not run
 * concurrently with other calls. NULL reloads the default location. */
bfq_status bfq_load_tile_table(const char* json_path);

/* Number of compiled kernel configurations usable for (block_shape, in_dtype, w_layout,
 * scale_fmt), and the i-th one (split_k = 1; any split_k >= 1 may be combined with it). Used
 * by the on-device sweep. block_shape (host) {128, 128}, or {1, k} (any k > 0) for the
 * per-token x per-channel kernels. */
int32_t bfq_num_tile_candidates(const int32_t block_shape[2], bfq_dtype in_dtype,
                                bfq_weight_layout w_layout, bfq_scale_format scale_fmt);
bfq_status bfq_get_tile_candidate(const int32_t block_shape[2], bfq_dtype in_dtype,
                                  bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                  int32_t index, bfq_tile* tile_out);

/* ------------------------------------------------------- MoE grouped block GEMM ----
 * [CONFIG] §5: the MoE kernels take the same per-shape, per-batch-size tuned configs with an
 * expert count E in the key. Token t routed to experts topk_ids[t][0..topk-1] forms pairs
 * q = t*topk + j; out[q][n] (pair order, [T*topk][N]) = the block-scaled GEMM (as
 * bfq_block_gemm) of token row t of a_q with row n of expert topk_ids[t][j]'s weights.
 * e4m3fn codes, block_shape {128, 128}; bfq_moe_combine adds up a token's experts.
 */

/* Group the pairs by expert (stable: ascending pair id within an expert), the routing step
 * the grouped GEMM reads. topk_ids [T][topk] int32 (device); expert_offsets [E+1] int32:
 * pairs of expert e are sorted_pairs[expert_offsets[e] .. expert_offsets[e+1]);
 * sorted_pairs int32, at least T*topk entries (the first T*topk are written). An id
 * outside [0, E) goes after every expert (beyond
 * expert_offsets[E]) and its pair is never computed. 1 <= E <= 1023; workspace of
 * bfq_moe_align_workspace_bytes bytes (may be NULL when that is 0). Asynchronous. */
size_t     bfq_moe_align_workspace_bytes(int64_t T, int32_t topk, int32_t E);
bfq_status bfq_moe_align(const int32_t* topk_ids, int64_t T, int32_t topk, int32_t E,
                         int32_t* expert_offsets, int32_t* sorted_pairs, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Tile of the grouped GEMM: the (E, N, K, dtype, weight layout, scale format) table entry,
 * bucket nearest to the token count T; else a default rule from the average rows per active
 * expert and BFQ_WARN_DEFAULT_TILE. Batch-invariant mode applies as in bfq_select_tile. */
bfq_status bfq_moe_select_tile(int64_t T, int32_t topk, int32_t E, int64_t N, int64_t K,
                               const int32_t block_shape[2], bfq_dtype in_dtype,
                               bfq_dtype out_dtype, bfq_weight_layout w_layout,
                               bfq_scale_format scale_fmt, bfq_tile* tile_out);
/* split_k * T * topk * N * 4 bytes when the tile's split_k > 1, else 0; SIZE_MAX when
 * T * topk * N >= 2^40, a shape bfq_moe_block_gemm rejects. */
size_t     bfq_moe_gemm_workspace_bytes(int64_t T, int32_t topk, int64_t N, const bfq_tile* tile);

/* Grouped GEMM over the expert groups of bfq_moe_align.
 *   a_q [T][K] codes and a_scales (a_layout/a_scale_ld over the T tokens; packed UE8M0 words
 *   allowed) as bfq_quant_tokens writes them: each pair's token row is gathered in the kernel;
 *   sorted_pairs, expert_offsets: bfq_moe_align's output (device);
 *   w_q [E][N][K] codes in w_layout (each expert's [N][K] matrix row-major, or packed by
 *   bfq_pack_weights, one after the other); w_scales [E][N/128][K/128];
 *   out [T*topk][N] in pair order; rows of pairs with an expert outside [0, E) are not written
 *   with split_k = 1 and are unspecified with split_k > 1.
 *   tile NULL -> bfq_moe_select_tile. Variants 0 and 1 (grouped forms); T * K < 2^31,
 *   T * topk * N < 2^40. */
bfq_status bfq_moe_block_gemm(const void* a_q, const float* a_scales, bfq_scale_layout a_layout,
                              int64_t a_scale_ld, const int32_t* sorted_pairs,
                              const int32_t* expert_offsets, int32_t topk, const void* w_q,
                              const float* w_scales, bfq_weight_layout w_layout,
                              bfq_scale_format scale_fmt, void* out, int64_t T, int64_t N,
                              int64_t K, int32_t E, const int32_t block_shape[2] /* host */,
                              bfq_dtype in_dtype, bfq_dtype out_dtype,
                              const bfq_tile* tile /* host */, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Compiled grouped kernels usable for (w_layout, scale_fmt) (e4m3fn; split_k = 1). */
int32_t    bfq_moe_num_tile_candidates(bfq_weight_layout w_layout, bfq_scale_format scale_fmt);
bfq_status bfq_moe_get_tile_candidate(bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                      int32_t index, bfq_tile* tile_out);

/* --------------------------------------------- feed-forward blocks: gated product ----
 * The operators between the GEMMs of a feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T:
 * bfq_norm_residual gives the codes of x, bfq_gated_gemm both projections with the activation and
 * the product (as the codes that the down projection's bfq_block_gemm reads), bfq_norm_residual
 * adds the block's output to the residual stream. Backward: the gradient of the down projection's
 * input is bfq_block_gemm of the quantized gradient with the transposed weights
 * (bfq_transpose_weights), bfq_gated_backward carries it to the pre-activations, and another
 * bfq_block_gemm to x. The weights are codes: no gradient of theirs is defined. */

/* Gated product: for each token m and column f < F
 *   g = sum_k a[m][k] w[f][k],  u = sum_k a[m][k] w[F + f][k],  out[m][f] = act(g) * u
 * with both sums as bfq_block_gemm forms them (e4m3fn codes, block_shape {128, 128}) and kept in
 * fp32 until out is rounded once. w_q holds 2F rows, the gate projection's and then the up
 * projection's (row-major, or the 2F x K matrix packed by bfq_pack_weights); w_scales
 * [2F/128][K/128].
 *   out_dtype BF16 | FP16 | FP32: out [M][F]. out_dtype BFQ_E4M3FN: out [M][F] codes and
 *   out_scales, one per 128 columns of a token, in out_layout / out_scale_ld and scale_fmt with
 *   floor out_eps: the token quantizer's formats, formed from the fp32 products (out_scales,
 *   out_layout, out_scale_ld and out_eps are not read otherwise).
 *   preact: bf16 [M][2F] = (g, u), what bfq_gated_backward reads, or NULL.
 * M in [0, 2^24 - 4), F and K positive multiples of 128, F < 2^26, K <= 2^23, M * 2F < 2^40,
 * F * K < 2^40; activation scales as bfq_block_gemm. tile NULL -> bfq_gated_select_tile. The workspace
 * holds bfq_gated_gemm_workspace_bytes bytes (NULL when that is 0). */
bfq_status bfq_gated_gemm(const void* a_q, const float* a_scales, bfq_scale_layout a_layout,
                          int64_t a_scale_ld, const void* w_q, const float* w_scales,
                          bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                          bfq_activation act, void* out, float* out_scales,
                          bfq_scale_layout out_layout, int64_t out_scale_ld, float out_eps,
                          void* preact, int64_t M, int64_t F, int64_t K,
                          const int32_t block_shape[2] /* host */, bfq_dtype in_dtype,
                          bfq_dtype out_dtype, const bfq_tile* tile /* host */, void* workspace,
                          size_t workspace_bytes, void* stream);

/* The tile that bfq_gated_gemm takes: a rule on M, F, K, the layout, the scale format and whether
 * codes are wanted (bn counts output columns: 2 * bn weight rows). Variant 1 with sched 2 (gated
 * tiles only): the waves take every waves_m-th K block and copy the weights through LDS, stages K
 * blocks ahead. Variant 2: the tiles of variant 0 in rounds of one workgroup per compute unit, the K
 * range of those left over in as many parts as fill a last round (split_k 1; for codes bn 128).
 * Batch-invariant mode applies as in bfq_select_tile. */
bfq_status bfq_gated_select_tile(int64_t M, int64_t F, int64_t K, bfq_dtype out_dtype,
                                 bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                 bfq_tile* tile_out);
/* split_k * M * 2F * 4 bytes when the tile's split_k > 1, or when codes are wanted and the tile's
 * bn is not 128; variant 2: at most 256 partial tiles of bm * 2 bn * 4 bytes; else 0. tile NULL -> the
 * selected one. SIZE_MAX for shapes bfq_gated_gemm rejects as too large. */
size_t     bfq_gated_gemm_workspace_bytes(int64_t M, int64_t F, int64_t K, bfq_dtype out_dtype,
                                          bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                          const bfq_tile* tile);
/* Compiled gated kernels usable for (w_layout, scale_fmt) (split_k = 1). */
int32_t    bfq_gated_num_tile_candidates(bfq_weight_layout w_layout, bfq_scale_format scale_fmt);
bfq_status bfq_gated_get_tile_candidate(bfq_weight_layout w_layout, bfq_scale_format scale_fmt,
                                        int32_t index, bfq_tile* tile_out);

/* Gradient of h = act(g) * u at (g, u), from the pre-activations that bfq_gated_gemm kept and the
 * gradient dh of h: dg = dh * u * act'(g), du = dh * act(g), in fp32.
 *   preact bf16 [M][2F]; dh bf16 [M][F]. At least one output, the others NULL:
 *   dpre bf16 [M][2F] = (dg, du); q [M][2F] codes with scales, one per 128 columns (the gradient
 *   as the next bfq_block_gemm reads it; layout, scale_ld, q_eps, scale_fmt as in
 *   bfq_quant_tokens with K = 2F, quantized from the fp32 values); h bf16 [M][F], the product
 *   again. dpre may be preact itself, h may be dh. M < 2^24 - 4; F < 2^26 a positive multiple of
 *   8, of 128 with q. q_dtype is read only with q. */
bfq_status bfq_gated_backward(const void* preact, const void* dh, bfq_activation act, void* dpre,
                              void* q, bfq_dtype q_dtype, float* scales, bfq_scale_layout layout,
                              int64_t scale_ld, float q_eps, bfq_scale_format scale_fmt, void* h,
                              int64_t M, int64_t F, void* stream);

/* Row-major weight codes [N][K] and their block scales [N/128][K/128] transposed: wt_q [K][N],
 * wt_scales [K/128][N/128]. An offline step like bfq_pack_weights (which may follow it); separate
 * buffers. N, K multiples of 128, N < 2^22, K <= 2^23. */
bfq_status bfq_transpose_weights(const void* w_q, const float* w_scales, int64_t N, int64_t K,
                                 bfq_dtype q_dtype, void* wt_q, float* wt_scales, void* stream);

/* ----------------------------------------------- feed-forward blocks: norms, residual ----
 * One step of the residual stream, per token row of K channels, in fp32:
 *   z  = w_post ? y * rms(y) * w_post : y        rms(x) = 1 / sqrt(mean(x^2) + norm_eps)
 *   r' = residual + res_scale * gate * z
 *   n  = r' * rms(r') * w_pre
 *   residual [M][K] of res_dtype BF16 | FP32. y bf16 [M][K], or NULL: r' = residual (w_post, gate
 *   and res_out must then be NULL). gate bf16: [K] (CHANNEL), [M] (TOKEN), [M][K] (FULL) or NULL
 *   (NONE); w_post, w_pre bf16 [K] or NULL.
 *   res_out [M][K] of res_dtype receives r' (may be `residual` itself).
 *   With w_pre, n is stored as normed bf16 [M][K], as codes q [M][K] with scales (the formats of
 *   bfq_quant_tokens: group_size 128 or K, q_dtype E4M3FN | INT8), or both; both are formed from
 *   the fp32 n, and n from the fp32 r'. Without w_pre, normed and q must be NULL.
 * K a positive multiple of 8 (of 128 with q), at most 16384; M < 2^24 - 4; norm_eps positive and
 * finite. Row sums of squares are fp32: values past about 1e17 overflow them. A token's rows do not
 * depend on M for K <= 8192, and in batch-invariant mode for any K. */
bfq_status bfq_norm_residual(const void* y, const void* residual, bfq_dtype res_dtype,
                             const void* w_post, const void* gate, bfq_gate_kind gate_kind,
                             float res_scale, const void* w_pre, float norm_eps, void* res_out,
                             void* normed, void* q, bfq_dtype q_dtype, int32_t group_size,
                             float* scales, bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                             bfq_scale_format scale_fmt, int64_t M, int64_t K, void* stream);

/* Gradients of bfq_norm_residual. res_out is the stored r' (without y: the residual itself);
 * d_normed bf16 [M][K] the gradient at n (with w_pre, else NULL), d_res_out [M][K] of res_dtype
 * the one that reaches r' along the stream, or NULL for zero. Outputs:
 *   d_res [M][K] of res_dtype, the gradient of `residual` (may be d_res_out itself);
 *   d_y bf16 [M][K] with y, else NULL;
 *   d_w_pre, d_w_post fp32 [K], and d_gate (CHANNEL fp32 [K], TOKEN fp32 [M], FULL bf16 [M][K]):
 *   any may be NULL when it is not wanted, and must be when its operand is absent. They are
 *   overwritten, not added to; with M = 0 the column sums become zero.
 * Sums are fp32 in a fixed order: equal calls give equal bits. workspace of
 * bfq_norm_residual_backward_workspace_bytes bytes when a [K] gradient is wanted, else NULL. */
size_t     bfq_norm_residual_backward_workspace_bytes(int64_t M, int64_t K);
bfq_status bfq_norm_residual_backward(const void* y, const void* res_out, bfq_dtype res_dtype,
                                      const void* w_post, const void* gate,
                                      bfq_gate_kind gate_kind, float res_scale, const void* w_pre,
                                      float norm_eps, const void* d_normed, const void* d_res_out,
                                      void* d_res, void* d_y, float* d_w_pre, float* d_w_post,
                                      void* d_gate, int64_t M, int64_t K, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* ------------------------------------------------ MoE layer around the grouped GEMM ----
 * Forward: bfq_moe_route picks each token's experts and weights, bfq_moe_sort groups the pairs,
 * bfq_moe_block_gemm gathers the tokens itself, or bfq_moe_dispatch lays their rows out in expert
 * order (what an exchange between GPUs sends; bfq_moe_block_gemm then takes them with topk 1 and
 * sorted_pairs 0, 1, 2, ..), bfq_gated_checkpoint forms the product between the experts' two GEMMs,
 * and bfq_moe_combine brings their rows back to the tokens. Backward: bfq_moe_combine_backward,
 * bfq_moe_block_gemm with the transposed weights (bfq_transpose_weights on [E * N][K] transposes the
 * whole stack, not each expert: transpose them one by one), bfq_gated_checkpoint_backward, and
 * bfq_moe_combine without weights, which is the dispatch's gradient; bfq_moe_route_backward takes the
 * weights' gradient to the logits.
 *
 * Pairs are q = t*topk + j as above, 0 <= T < 2^22 and 1 <= topk <= 64 (the sort: any with T * topk <
 * 2^31). Rows tensors hold R rows, in expert order (pair_rows given) or in pair order (R = T*topk).
 * A pair without a row (pair_rows[q] outside [0, R), or in pair order an id outside [0, E)) is left
 * out: it adds nothing, whatever its weight, and its row is neither read nor written. In what is
 * written, each row is some pair's at most once, as bfq_moe_sort's places are; where two pairs share
 * one, its contents are those of either, mixed. With R = 0 every tensor over rows may be NULL; with T = 0 every
 * tensor over tokens or pairs, beside rows of any number (both orders are the same then). What belongs to
 * a token does not depend on T, and equal calls give equal bits. K a positive multiple of 8, of 128 where codes are
 * read or written, at most 2^23. */

/* Router: s = score(logits) over a token's E experts, the topk largest keys in descending order
 * (ties: the lowest index first), and their weights
 *   w_j = weight_scale * s_j / (renorm ? sum_k s_k + 1e-20 : 1).
 * The key of an expert is its logit; with a bias ([E], which moves the choice and not the weights) or
 * n_groups > 1 it is s (+ bias), formed in 64 bits. With groups (n_groups of E / n_groups neighbouring
 * experts) only the topk_groups groups with the largest sum of their two largest keys take part (ties:
 * the lowest group). A logit of -inf masks an expert, as does a key of -inf: it is never taken, and
 * where fewer than topk are left (in the groups that take part) the last ids are -1 with weight 0. A
 * logit of +inf counts as the largest finite value; a NaN counts as larger than any key.
 * Scores that are no keys are formed in fp32, and so are their sums; a sigmoid below 2^-126 counts as 0 there.
 *   logits [T][E] BF16 | FP16 | FP32; topk_ids [T][topk] int32; topk_weights [T][topk] fp32.
 * 1 <= E <= 1023, topk <= min(E, 64, the experts of topk_groups groups), n_groups <= 64. */
bfq_status bfq_moe_route(const void* logits, bfq_dtype logits_dtype, const float* bias, int64_t T,
                         int32_t E, int32_t topk, bfq_score score, int32_t n_groups,
                         int32_t topk_groups, int32_t renorm, float weight_scale, int32_t* topk_ids,
                         float* topk_weights, void* stream);

/* Gradient of the weights at the logits, for the ids that were chosen: d_logits [T][E] of
 * logits_dtype, overwritten. Ids outside [0, E) have no weight and no gradient; an id that occurs
 * twice collects both. Sums are fp32 in a fixed order. */
bfq_status bfq_moe_route_backward(const void* logits, bfq_dtype logits_dtype, const int32_t* topk_ids,
                                  const float* d_weights, int64_t T, int32_t E, int32_t topk,
                                  bfq_score score, int32_t renorm, float weight_scale, void* d_logits,
                                  void* stream);

/* The outputs of bfq_moe_align, and the places of the pairs: pair_rows [T][topk] int32 is the
 * position of pair q in sorted_pairs, its row in expert order, or -1 for an id outside [0, E).
 * sorted_pairs holds T*topk entries. workspace of bfq_moe_sort_workspace_bytes bytes, NULL when that
 * is 0 (up to 8192 pairs, which take one launch). */
size_t     bfq_moe_sort_workspace_bytes(int64_t T, int32_t topk, int32_t E);
bfq_status bfq_moe_sort(const int32_t* topk_ids, int64_t T, int32_t topk, int32_t E,
                        int32_t* expert_offsets, int32_t* sorted_pairs, int32_t* pair_rows,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Tokens' rows laid out in expert order: row pair_rows[t*topk + j] of the outputs is row t of x.
 *   x_dtype BF16: x [T][K]; rows [R][K] bf16 receives the rows, and / or q [R][K] their codes with
 *   scales, exactly as bfq_quant_tokens would write them for these rows (group_size 128; layout,
 *   scale_ld, q_eps and scale_fmt over the R rows); x_scales NULL.
 *   x_dtype E4M3FN | INT8: x [T][K] codes with x_scales (x_layout, x_scale_ld over the T tokens), copied
 *   to q (q_dtype the same) and scales in `layout`; packed words stay packed words (both layouts
 *   packed, scale_fmt BFQ_SCALE_UE8M0); rows NULL.
 * Rows without a pair are left as they were (packed words also in rows R .. round_up(R, 4) - 1: 0). */
bfq_status bfq_moe_dispatch(const void* x, bfq_dtype x_dtype, const float* x_scales,
                            bfq_scale_layout x_layout, int64_t x_scale_ld, const int32_t* pair_rows,
                            void* rows, void* q, bfq_dtype q_dtype, float* scales,
                            bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                            bfq_scale_format scale_fmt, int64_t T, int32_t topk, int64_t K, int64_t R,
                            void* stream);

/* Experts' rows back to their tokens:
 *   out[t] = base[t] + sum_j weights[t][j] * rows[row of pair (t, j)]
 * in fp32, added in pair order, rounded once. rows [R][K] BF16 | FP16 | FP32; weights [T][topk] fp32,
 * NULL for ones; out [T][K] BF16 | FP16 | FP32, base of the same type, NULL for zeros (may be out
 * itself). pair_rows [T][topk] (rows in expert order), or NULL (pair order); there topk_ids [T][topk]
 * with E names the pairs that have a row, NULL: all of them.
 * ckpt: codes [R][K] (ckpt_dtype E4M3FN | INT8) with ckpt_scales fp32 [R][K/128], the rows' 8-bit
 * checkpoint for bfq_moe_combine_backward, as bfq_quant_tokens would write it (with floor q_eps; of
 * FP16 and FP32 rows in the same way); both NULL without. Rows without a pair stay as they were. */
bfq_status bfq_moe_combine(const void* rows, bfq_dtype rows_dtype, const float* weights,
                           const int32_t* pair_rows, const int32_t* topk_ids, int32_t E,
                           const void* base, void* out, bfq_dtype out_dtype, void* ckpt,
                           bfq_dtype ckpt_dtype, float* ckpt_scales, float q_eps, int64_t T,
                           int32_t topk, int64_t K, int64_t R, void* stream);

/* Gradients of bfq_moe_combine for dout [T][K] BF16 | FP32 (the base's gradient is dout itself):
 *   d_rows[row of pair (t, j)] = weights[t][j] * dout[t], as d_rows bf16 [R][K] and / or codes q [R][K]
 *   with scales (formats of bfq_quant_tokens over R rows, from the fp32 products); rows without a pair
 *   are left as they were (packed words also in rows R .. round_up(R, 4) - 1: 0).
 *   d_weights fp32 [T][topk]: sum over K of dout[t] * rows[..], 0 without a row; needs rows [R][K] as
 *   BF16 | FP16 | FP32, or as codes E4M3FN | INT8 with rows_scales fp32 [R][K/128].
 * Any output may be NULL, not all; rows NULL without d_weights. Sums are fp32 in a fixed order. */
bfq_status bfq_moe_combine_backward(const void* dout, bfq_dtype dout_dtype, const float* weights,
                                    const void* rows, bfq_dtype rows_dtype, const float* rows_scales,
                                    const int32_t* pair_rows, const int32_t* topk_ids, int32_t E,
                                    void* d_rows, void* q, bfq_dtype q_dtype, float* scales,
                                    bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                                    bfq_scale_format scale_fmt, float* d_weights, int64_t T,
                                    int32_t topk, int64_t K, int64_t R, void* stream);

/* ---------------------------------------- 8-bit checkpoints of a gated product ----
 * From pre-activations preact bf16 [M][2F] = (g, u) (a 2F-wide bfq_block_gemm or bfq_moe_block_gemm,
 * or bfq_gated_gemm's preact): h = act(g) * u in fp32, as h bf16 [M][F] and / or codes q [M][F] with
 * scales (formats of bfq_quant_tokens), and the checkpoint that a backward pass keeps in place of
 * preact: ckpt codes [M][2F] (ckpt_dtype E4M3FN | INT8) with ckpt_scales fp32 [M][2F/128], the codes
 * of bfq_quant_tokens with fp32 scales. Half the bytes of preact; a value is off by at most half a
 * step of its code (e4m3: 2^-4 of itself, int8: 1/254 of its group's largest). Any output may be
 * NULL, not all. live_rows (device, one int32, or NULL for M): rows from *live_rows on are neither
 * read nor written, for instance expert_offsets + E with rows in expert order. F a positive multiple
 * of 128 below 2^26, M < 2^24 - 4; q_eps floors the scales of both. */
bfq_status bfq_gated_checkpoint(const void* preact, bfq_activation act, void* h, void* q,
                                bfq_dtype q_dtype, float* scales, bfq_scale_layout layout,
                                int64_t scale_ld, float q_eps, bfq_scale_format scale_fmt, void* ckpt,
                                bfq_dtype ckpt_dtype, float* ckpt_scales, const int32_t* live_rows,
                                int64_t M, int64_t F, void* stream);

/* bfq_gated_backward from the checkpoint: with (g, u) = codes times scales, dg = dh * u * act'(g) and
 * du = dh * act(g) in fp32, as dpre bf16 [M][2F] and / or codes q [M][2F] with scales; h bf16 [M][F],
 * the product of the checkpoint's values. dh bf16 [M][F] (h may be dh itself). Any output may be NULL,
 * not all. */
bfq_status bfq_gated_checkpoint_backward(const void* ckpt, bfq_dtype ckpt_dtype,
                                         const float* ckpt_scales, const void* dh, bfq_activation act,
                                         void* dpre, void* q, bfq_dtype q_dtype, float* scales,
                                         bfq_scale_layout layout, int64_t scale_ld, float q_eps,
                                         bfq_scale_format scale_fmt, void* h, const int32_t* live_rows,
                                         int64_t M, int64_t F, void* stream);

const char* bfq_status_string(bfq_status s);
const char* bfq_last_error(void);

/* Test support: int8 per-K-block int32 partials, layout [K/128][M][N] (exact). */
bfq_status bfq_debug_block_partials_i32(const void* a_q, const void* w_q, int32_t* partials,
                                        int64_t M, int64_t N, int64_t K, void* stream);

/* Measurement support: `blocks` workgroups of 8 waves, each wave running 8 independent
 * chains of `iters` fp8 16x16x128 MFMAs on register operands and nothing else, so that
 * flops / elapsed is the matrix-core throughput the GPU sustains (at the clock it holds under
 * that load), stated beside the published peak. out: blocks * 512 floats (device), written
 * once per lane to keep the chains live; its values mean nothing. Flops of one launch:
 * bfq_probe_mfma_flops(blocks, iters). blocks in [1, 2^31), iters in [1, 2^40). */
bfq_status bfq_probe_mfma_peak(int64_t blocks, int64_t iters, float* out, void* stream);
double     bfq_probe_mfma_flops(int64_t blocks, int64_t iters);

/* Test support: the element encoder the quantizers use, applied to n fp32 values that are
 * finite with |x| < 464 (e4m3fn) or finite (int8). codes [n] bytes. */
bfq_status bfq_debug_encode(const float* x, int64_t n, bfq_dtype q_dtype, void* codes,
                            void* stream);

#ifdef __cplusplus
}
#endif
#endif /* BFQ_H */
