// The gated product of pre-activations (g, u) with an 8-bit checkpoint of them, and its gradient from
// the checkpoint:
//   h = act(g) u, as bf16 or as codes;  the checkpoint: codes of g and u, one scale per 128 columns
//   dg = dh u act'(g),  du = dh act(g) from the checkpoint's values, as bf16 or codes; h again
// Eight columns of both halves a thread, read once and written once, 16 lanes a group. Rows from *live
// on (what no expert was given) are neither read nor written. Bytes bound both, and the arithmetic is close
// behind: 32768 x 2048 with codes of h, 476 MB in 78 us (6.1 TB/s), its gradient 411 MB in 79 us (5.2),
// a large copy 5.2; over a hundred calls back to back, at the clock they then leave, 90 to 99 us, and 90
// with the encoder's correction left out (some 360 instructions a thread forward). Sixteen columns a thread,
// sharing maxima and scales between more: 4 % less there, 7 % more in single calls, and 14 to 17 % more with
// bf16 outputs. SILU as a kernel of its own, without the cubic term: no difference.
#include "activation.h"
#include "row_access.h"

namespace bfq {

__device__ __forceinline__ int64_t live_rows(const CheckpointArgs& p) {
    if (!p.live) return p.M;
    const int64_t n = *p.live;
    return n < p.M ? n : p.M;
}

// Q: code type of h, or -1; CK: of the checkpoint, or -1 without one. Rows past M exist only to write
// zero words of packed scales.
template <int Q, int CK, int S>
__global__ __launch_bounds__(256) void checkpoint_kernel(CheckpointArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t m = blockIdx.x, F = p.F;
    const uint32_t c = blockIdx.y * blockDim.x + threadIdx.x, half = (uint32_t)(F / 8);
    const bool live = c < half;
    if (m >= p.M) {                                      // uniform
        if constexpr (Q >= 0) {
            if (live && (lane & 15) == 0) put_scale(p.out, m, c >> 4, F / 128, 0.f);
        }
        return;
    }
    if (m >= live_rows(p)) return;                       // uniform
    const __amdgpu_buffer_rsrc_t rg = pair_row(p.pre, 2 * m, (uint32_t)(2 * F)), ru = pair_row(p.pre, 2 * m + 1, (uint32_t)(2 * F));
    RowChunk<R_BF16, S> gc, uc;
    gc.load(rg, c);
    uc.load(ru, c);
    float g[8], u[8], h[8];
    gc.get(g);
    uc.get(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = act_f32(g[i], p.c1, p.c3) * u[i];
    if (p.h) row_store<S>(pair_row(p.h, m, (uint32_t)(2 * F)), c, O_BF16, h);
    if constexpr (CK >= 0) {
        const uint32_t mg = max16(amax8(g)), mu = max16(amax8(u));
        const float sg = group_scale<CK>(mg, p.ckpt_eps, 0), su = group_scale<CK>(mu, p.ckpt_eps, 0);
        row_store8<S>(pair_row(p.ckpt, 2 * m, (uint32_t)F), c * 8, encode8_group<CK>(g, mg, sg));
        row_store8<S>(pair_row(p.ckpt, 2 * m + 1, (uint32_t)F), c * 8, encode8_group<CK>(u, mu, su));
        if (live && (lane & 15) == 0) {
            float* s = p.ckpt_scales + m * (2 * F / 128);
            s[c >> 4] = sg;
            s[F / 128 + (c >> 4)] = su;
        }
    }
    if constexpr (Q >= 0) {
        const uint32_t mh = max16(amax8(h));
        const float s = group_scale<Q>(mh, p.out.eps, p.out.ue8m0);
        row_store8<S>(pair_row(p.out.q, m, (uint32_t)F), c * 8, encode8_group<Q>(h, mh, s));
        if (live && (lane & 15) == 0) put_scale(p.out, m, c >> 4, F / 128, s);
    }
}

template <int CK, int Q, int S>
__global__ __launch_bounds__(256) void checkpoint_bwd_kernel(CheckpointArgs p) {
    constexpr int RK = CK == Q_FP8 ? R_FP8 : R_INT8;
    const int lane = threadIdx.x & 63;
    const int64_t m = blockIdx.x, F = p.F, G = F / 128;
    const uint32_t c = blockIdx.y * blockDim.x + threadIdx.x, half = (uint32_t)(F / 8);
    const bool live = c < half;
    if (m >= p.M) {                                      // uniform
        if constexpr (Q >= 0) {
            if (live && (lane & 15) == 0) {
                put_scale(p.out, m, c >> 4, 2 * G, 0.f);
                put_scale(p.out, m, G + (c >> 4), 2 * G, 0.f);
            }
        }
        return;
    }
    if (m >= live_rows(p)) return;                       // uniform
    RowChunk<RK, S> gc, uc;
    RowChunk<R_BF16, S> dc;
    gc.load(pair_row(p.ckpt, 2 * m, (uint32_t)F), c);
    uc.load(pair_row(p.ckpt, 2 * m + 1, (uint32_t)F), c);
    dc.load(pair_row(p.dh, m, (uint32_t)(2 * F)), c);
    const __amdgpu_buffer_rsrc_t rs = pair_row(p.ckpt_scales, m, (uint32_t)(8 * G));
    const float sg = buf_f32(rs, (c >> 4) * 4, 0), su = buf_f32(rs, (c >> 4) * 4, (uint32_t)(4 * G));
    float g[8], u[8], dh[8], h[8];
    gc.get(g);
    uc.get(u);
    dc.get(dh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float slope;
        const float a = act_slope_f32(g[i] * sg, p.c1, p.c3, slope), uv = u[i] * su;
        h[i] = a * uv;
        g[i] = dh[i] * uv * slope;
        u[i] = dh[i] * a;
    }
    if (p.h) row_store<S>(pair_row(p.h, m, (uint32_t)(2 * F)), c, O_BF16, h);
    if (p.dpre) {
        row_store<S>(pair_row(p.dpre, 2 * m, (uint32_t)(2 * F)), c, O_BF16, g);
        row_store<S>(pair_row(p.dpre, 2 * m + 1, (uint32_t)(2 * F)), c, O_BF16, u);
    }
    if constexpr (Q >= 0) {
        const uint32_t mg = max16(amax8(g)), mu = max16(amax8(u));
        const float tg = group_scale<Q>(mg, p.out.eps, p.out.ue8m0), tu = group_scale<Q>(mu, p.out.eps, p.out.ue8m0);
        row_store8<S>(pair_row(p.out.q, 2 * m, (uint32_t)F), c * 8, encode8_group<Q>(g, mg, tg));
        row_store8<S>(pair_row(p.out.q, 2 * m + 1, (uint32_t)F), c * 8, encode8_group<Q>(u, mu, tu));
        if (live && (lane & 15) == 0) {
            put_scale(p.out, m, c >> 4, 2 * G, tg);
            put_scale(p.out, m, G + (c >> 4), 2 * G, tu);
        }
    }
}

static void checkpoint_grid(const CheckpointArgs& a, dim3* grid, dim3* block) {
    const int64_t chunks = a.F / 8, ny = (chunks + 255) / 256;
    const int64_t rows = a.out.q && a.out.packed ? (a.M + 3) / 4 * 4 : a.M;
    *block = dim3((unsigned)(((chunks + ny - 1) / ny + 63) / 64 * 64));
    *grid = dim3((unsigned)rows, (unsigned)ny);
}

template <int Q, int CK> static void checkpoint_s(const CheckpointArgs& a, hipStream_t stream) {
    dim3 grid, block;
    checkpoint_grid(a, &grid, &block);
    if (past_caches(a.M * a.F * ((a.h ? 2 : 0) + (Q >= 0 ? 1 : 0) + (CK >= 0 ? 2 : 0))))
        hipLaunchKernelGGL((checkpoint_kernel<Q, CK, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((checkpoint_kernel<Q, CK, 0>), grid, block, 0, stream, a);
}
template <int Q> static void checkpoint_q(const CheckpointArgs& a, hipStream_t stream) {
    if (!a.ckpt) checkpoint_s<Q, -1>(a, stream);
    else if (a.ckpt_type == Q_FP8) checkpoint_s<Q, Q_FP8>(a, stream);
    else checkpoint_s<Q, Q_INT8>(a, stream);
}
hipError_t launch_checkpoint(const CheckpointArgs& a, hipStream_t stream) {
    if (!a.out.q) checkpoint_q<-1>(a, stream);
    else if (a.out.qtype == Q_FP8) checkpoint_q<Q_FP8>(a, stream);
    else checkpoint_q<Q_INT8>(a, stream);
    return hipGetLastError();
}

template <int CK, int Q> static void checkpoint_bwd_s(const CheckpointArgs& a, hipStream_t stream) {
    dim3 grid, block;
    checkpoint_grid(a, &grid, &block);
    if (past_caches(a.M * a.F * ((a.h ? 2 : 0) + (a.dpre ? 4 : 0) + (Q >= 0 ? 2 : 0))))
        hipLaunchKernelGGL((checkpoint_bwd_kernel<CK, Q, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((checkpoint_bwd_kernel<CK, Q, 0>), grid, block, 0, stream, a);
}
template <int CK> static void checkpoint_bwd_ck(const CheckpointArgs& a, hipStream_t stream) {
    if (!a.out.q) checkpoint_bwd_s<CK, -1>(a, stream);
    else if (a.out.qtype == Q_FP8) checkpoint_bwd_s<CK, Q_FP8>(a, stream);
    else checkpoint_bwd_s<CK, Q_INT8>(a, stream);
}
hipError_t launch_checkpoint_bwd(const CheckpointArgs& a, hipStream_t stream) {
    if (a.ckpt_type == Q_FP8) checkpoint_bwd_ck<Q_FP8>(a, stream);
    else checkpoint_bwd_ck<Q_INT8>(a, stream);
    return hipGetLastError();
}

}  // namespace bfq
