// Norms around a block of the residual stream, one pass over a token's row:
//   z  = y * rms(y) * w_post           (the norm after the block; without w_post z = y)
//   r' = r + alpha * gate * z          (the block's gate and residual scale)
//   n  = r' * rms(r') * w_pre          (the norm before the next block)
// with rms(x) = 1 / sqrt(mean(x^2) + eps); n is stored as bf16, as the codes and scales that the
// GEMMs read (the token quantizer's formats), or both. All of it in fp32; n is taken from the
// unrounded r' and quantized unrounded, so storing r' or n as bf16 costs the codes nothing.
//
// What bounds it: bytes. A row is read once (y, r) and written once (r', codes), everything
// between stays in registers: P chunks of 8 elements a thread, chunk c of the row held by thread
// c % T in slot c / T, so 16 neighbouring lanes own one 128-element group as in the token
// quantizer. Each norm costs one reduction over the workgroup (DPP within a wave, LDS across).
#include "bfq_internal.h"
#include "quant_device.h"

namespace bfq {

// Eight values of the residual stream: one 16-byte chunk of bf16 or two of fp32.
template <int F32> struct Chunk;
template <> struct Chunk<0> {
    uint4 v;
    __device__ __forceinline__ void load(const void* p, int64_t i) { v = static_cast<const uint4*>(p)[i]; }
    __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float* x) const { unpack8(v, x); }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float* x) {
        static_cast<uint4*>(p)[i] = pack8(x);
    }
};
template <> struct Chunk<1> {
    v4f a, b;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        a = static_cast<const v4f*>(p)[2 * i];
        b = static_cast<const v4f*>(p)[2 * i + 1];
    }
    __device__ __forceinline__ void clear() { a = b = v4f{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float* x) {
        static_cast<v4f*>(p)[2 * i] = v4f{x[0], x[1], x[2], x[3]};
        static_cast<v4f*>(p)[2 * i + 1] = v4f{x[4], x[5], x[6], x[7]};
    }
};

// The gate of 8 elements of row m (chunk c), times alpha.
__device__ __forceinline__ void gate8(const NormArgs& p, int64_t m, int64_t c, int64_t chunks,
                                      float* g) {
    if (p.gate_kind == BFQ_GATE_CHANNEL || p.gate_kind == BFQ_GATE_FULL) {
        unpack8(static_cast<const uint4*>(p.gate)[(p.gate_kind == BFQ_GATE_FULL ? m * chunks : 0) + c], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= p.res_scale;
    } else {
        float a = p.res_scale;
        if (p.gate_kind == BFQ_GATE_TOKEN)
            a *= __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.gate)[m] << 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = a;
    }
}

// Q: -1 no codes, else Q_FP8 / Q_INT8. Rows M .. (packed scale words: up to a multiple of 4)
// exist only to write zero words.
template <int T, int P, int RF32, int Q>
__global__ __launch_bounds__(T) void norm_residual_kernel(NormArgs p) {
    const int t = threadIdx.x, lane = t & 63;
    const int64_t m = blockIdx.x, K = p.K, chunks = K / 8;
    __shared__ float red[2][T / 64];
    __shared__ uint32_t redmax[T / 64];
    if constexpr (Q >= 0) {
        if (m >= p.M) {                                   // uniform: a padding row of packed words
            for (int64_t w = t; w < (K / 128 + 3) / 4; w += T) p.scales[w * p.s_stride_g + m] = 0.f;
            return;
        }
    }
    float r[P][8];
    Chunk<RF32> rc[P];
    uint4 yc[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const int64_t c = (int64_t)u * T + t;
        rc[u].clear();
        yc[u] = make_uint4(0, 0, 0, 0);
        if (c < chunks) {
            rc[u].load(p.residual, m * chunks + c);
            if (p.y) yc[u] = static_cast<const uint4*>(p.y)[m * chunks + c];
        }
    }
    float iy = 1.f;
    if (p.w_post) {
        float s[1] = {0.f};
#pragma unroll
        for (int u = 0; u < P; ++u) {
            float y[8];
            unpack8(yc[u], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] = __builtin_fmaf(y[i], y[i], s[0]);
        }
        block_sum<T, 1>(s, red[0]);
        iy = 1.0f / __builtin_sqrtf(s[0] / (float)K + p.norm_eps);
    }
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const int64_t c = (int64_t)u * T + t;
        rc[u].get(r[u]);
        if (p.y && c < chunks) {
            float y[8], g[8];
            unpack8(yc[u], y);
            gate8(p, m, c, chunks, g);
            if (p.w_post) {
                float w[8];
                unpack8(static_cast<const uint4*>(p.w_post)[c], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * iy * w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) r[u][i] = __builtin_fmaf(g[i], y[i], r[u][i]);
            Chunk<RF32>::store(p.res_out, m * chunks + c, r[u]);
        }
    }
    if (!p.w_pre) return;                                 // uniform

    float s[1] = {0.f};
#pragma unroll
    for (int u = 0; u < P; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = __builtin_fmaf(r[u][i], r[u][i], s[0]);
    block_sum<T, 1>(s, red[1]);
    const float ir = 1.0f / __builtin_sqrtf(s[0] / (float)K + p.norm_eps);
    uint32_t rowmax = 0;
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const int64_t c = (int64_t)u * T + t;
        if (c < chunks) {
            float w[8];
            unpack8(static_cast<const uint4*>(p.w_pre)[c], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[u][i] = r[u][i] * ir * w[i];
            if (p.normed) static_cast<uint4*>(p.normed)[m * chunks + c] = pack8(r[u]);
            if constexpr (Q >= 0) rowmax = max(rowmax, amax8(r[u]));
        }
    }
    if constexpr (Q >= 0) {
        if (p.per_token) {
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1)
                rowmax = max(rowmax, (uint32_t)__shfl_xor((int)rowmax, off, 64));
            if (lane == 0) redmax[t >> 6] = rowmax;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < T / 64; ++w) rowmax = max(rowmax, redmax[w]);
            const float sc = group_scale<Q>(rowmax, p.q_eps, p.ue8m0);
#pragma unroll
            for (int u = 0; u < P; ++u) {
                const int64_t c = (int64_t)u * T + t;
                if (c < chunks) static_cast<uint2*>(p.q)[m * chunks + c] = encode8_group<Q>(r[u], rowmax, sc);
            }
            if (t == 0) p.scales[m * p.s_stride_m] = sc;
            return;
        }
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int64_t c = (int64_t)u * T + t, g = c >> 4;   // 16 lanes own group g
            const bool live = c < chunks;                        // the same for all 16
            const uint32_t mx = max16(live ? amax8(r[u]) : 0u);
            const float sc = group_scale<Q>(mx, p.q_eps, p.ue8m0);
            if (live) static_cast<uint2*>(p.q)[m * chunks + c] = encode8_group<Q>(r[u], mx, sc);
            if (p.packed) {
                // a wave's slot holds the four groups of one word; E8M0 has no Inf: code 255
                const uint32_t word = e8m0_word(live ? e8m0_of(sc) : 0u, lane);
                if (lane == 0 && live) p.scales[(g >> 2) * p.s_stride_g + m] = __uint_as_float(word);
            } else if (live && (lane & 15) == 0) {
                p.scales[m * p.s_stride_m + g * p.s_stride_g] = sc;
            }
        }
    }
}

// Gradients of the same: d_normed at n, d_res_out at r' (from the stream above), both optional;
// r' is the stored sum (`residual` here). With x^ = x * rms(x) and, over the row's K elements,
//   dr  = d_res_out + rms(r') * (w_pre * dn - r^ * mean(w_pre * dn * r^))     = gradient of r
//   dz  = alpha * gate * dr,  dy = rms(y) * (w_post * dz - y^ * mean(w_post * dz * y^))
//   dw_pre = sum_m dn * r^,  dw_post = sum_m dz * y^,  dgate = alpha * dr * z, summed over the
//   rows (CHANNEL) or the row (TOKEN).
// Two reductions a row: {sum r'^2, sum y^2, sum w_pre*dn*r'} together (the means are these times
// powers of rms), then {sum dz*w_post*y}. A workgroup walks rows blockIdx.x, + gridDim.x, ... and
// keeps its share of the column sums in registers, 16 a chunk: dn * r^, and alpha*dr*y^ (CHANNEL:
// times w_post it is the gate's gradient, times the gate w_post's) or dz*y^ (else). Each
// workgroup writes its shares once; norm_columns_kernel adds them in workgroup order, so equal
// inputs give equal sums.
template <int T, int P, int RF32>
__global__ __launch_bounds__(T) void norm_residual_bwd_kernel(NormArgs p) {
    constexpr int W = T / 64;
    const int t = threadIdx.x;
    const int64_t K = p.K, chunks = K / 8;
    const float fK = (float)K;
    __shared__ float red[2][5 * W];
    const bool channel = p.gate_kind == BFQ_GATE_CHANNEL;
    float apre[P][8], apost[P][8];
    uint4 wpre[P], wpost[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const int64_t c = (int64_t)u * T + t;
        wpre[u] = wpost[u] = make_uint4(0, 0, 0, 0);
        if (c < chunks && p.w_pre) wpre[u] = static_cast<const uint4*>(p.w_pre)[c];
        if (c < chunks && p.w_post) wpost[u] = static_cast<const uint4*>(p.w_post)[c];
#pragma unroll
        for (int i = 0; i < 8; ++i) apre[u][i] = apost[u][i] = 0.f;
    }
    int par = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, par ^= 1) {
        Chunk<RF32> rc[P], dc[P];
        uint4 yc[P], nc[P];
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int64_t c = (int64_t)u * T + t;
            rc[u].clear();
            dc[u].clear();
            yc[u] = nc[u] = make_uint4(0, 0, 0, 0);
            if (c < chunks) {
                const int64_t i = m * chunks + c;
                if (p.w_pre) {
                    rc[u].load(p.residual, i);
                    nc[u] = static_cast<const uint4*>(p.d_normed)[i];
                }
                if (p.d_res_out) dc[u].load(p.d_res_out, i);
                if (p.y) yc[u] = static_cast<const uint4*>(p.y)[i];
            }
        }
#pragma unroll
        for (int u = 0; u < P; ++u) {
            float r[8], y[8], dn[8], w[8];
            rc[u].get(r);
            unpack8(yc[u], y);
            unpack8(nc[u], dn);
            unpack8(wpre[u], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[0] = __builtin_fmaf(r[i], r[i], s[0]);
                s[1] = __builtin_fmaf(y[i], y[i], s[1]);
                s[2] = __builtin_fmaf(w[i] * dn[i], r[i], s[2]);
            }
        }
        block_sum<T, 3>(s, red[par]);
        const float ir = 1.0f / __builtin_sqrtf(s[0] / fK + p.norm_eps);
        const float iy = p.w_post ? 1.0f / __builtin_sqrtf(s[1] / fK + p.norm_eps) : 1.f;
        const float cr = ir * ir * s[2] / fK;      // r^ * mean(w_pre * dn * r^) = r' * cr
        float dz[P][8], q[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int64_t c = (int64_t)u * T + t;
            float r[8], dr[8];
            rc[u].get(r);
            dc[u].get(dr);
            if (p.w_pre) {
                float dn[8], w[8];
                unpack8(nc[u], dn);
                unpack8(wpre[u], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dr[i] += ir * (w[i] * dn[i] - r[i] * cr);
                    apre[u][i] = __builtin_fmaf(dn[i], r[i] * ir, apre[u][i]);
                }
            }
            if (c >= chunks) continue;
            Chunk<RF32>::store(p.d_res, m * chunks + c, dr);
            if (!p.y) continue;
            float y[8], g[8], w[8], dg[8];
            gate8(p, m, c, chunks, g);
            unpack8(yc[u], y);
            unpack8(wpost[u], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float yn = y[i] * iy, z = p.w_post ? yn * w[i] : yn;
                const float ad = p.res_scale * dr[i];
                dz[u][i] = g[i] * dr[i];
                dg[i] = ad * z;
                q[0] = __builtin_fmaf(dz[u][i], z, q[0]);
                q[1] += dg[i];
                apost[u][i] = __builtin_fmaf(channel ? ad : dz[u][i], yn, apost[u][i]);
            }
            if (p.gate_kind == BFQ_GATE_FULL && p.d_gate)
                static_cast<uint4*>(p.d_gate)[m * chunks + c] = pack8(dg);
        }
        if (!p.y) continue;                                 // uniform
        block_sum<T, 2>(q, red[par] + 3 * W);
        if (p.gate_kind == BFQ_GATE_TOKEN && p.d_gate && t == 0) static_cast<float*>(p.d_gate)[m] = q[1];
        const float cy = p.w_post ? iy * q[0] / fK : 0.f;
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int64_t c = (int64_t)u * T + t;
            if (c >= chunks) continue;
            if (p.w_post) {
                float y[8], w[8];
                unpack8(yc[u], y);
                unpack8(wpost[u], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) dz[u][i] = iy * (w[i] * dz[u][i] - y[i] * cy);
            }
            static_cast<uint4*>(p.d_y)[m * chunks + c] = pack8(dz[u]);
        }
    }
    if (!p.columns) return;
    float* mine = p.partials + (int64_t)blockIdx.x * 2 * K;
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const int64_t c = (int64_t)u * T + t;
        if (c < chunks) {
            Chunk<1>::store(mine, c, apre[u]);
            Chunk<1>::store(mine + K, c, apost[u]);
        }
    }
}

// Column sums of the workgroups' shares [rows][2][K]: 64 columns a workgroup, 16 threads a column
// each adding every 16th share, then the 16 in order.
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormArgs p, int rows) {
    const int64_t K = p.K, col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const int part = threadIdx.x >> 6;
    __shared__ float sums[16][64];
    float s = 0.f;
    if (col < 2 * K)
        for (int g = part; g < rows; g += 16) s += p.partials[(int64_t)g * 2 * K + col];
    sums[part][threadIdx.x & 63] = s;
    __syncthreads();
    if (part != 0 || col >= 2 * K) return;
#pragma unroll
    for (int g = 1; g < 16; ++g) s += sums[g][threadIdx.x];
    if (col < K) {
        if (p.d_w_pre) p.d_w_pre[col] = s;
        return;
    }
    const int64_t k = col - K;
    auto bf16 = [](const void* v, int64_t i) {
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(v)[i] << 16);
    };
    const bool channel = p.gate_kind == BFQ_GATE_CHANNEL;
    if (p.d_w_post) p.d_w_post[k] = channel ? s * bf16(p.gate, k) : s;
    if (channel && p.d_gate) static_cast<float*>(p.d_gate)[k] = p.w_post ? s * bf16(p.w_post, k) : s;
}

// ---------------------------------------------------------------- launchers ----

template <int T, int P, int RF32>
static hipError_t launch_norm_q(const NormArgs& a, hipStream_t stream) {
    const int64_t rows = a.packed ? (a.M + 3) / 4 * 4 : a.M;
    const dim3 grid((unsigned)rows);
    if (!a.q)
        hipLaunchKernelGGL((norm_residual_kernel<T, P, RF32, -1>), grid, dim3(T), 0, stream, a);
    else if (a.qtype == Q_FP8)
        hipLaunchKernelGGL((norm_residual_kernel<T, P, RF32, Q_FP8>), grid, dim3(T), 0, stream, a);
    else
        hipLaunchKernelGGL((norm_residual_kernel<T, P, RF32, Q_INT8>), grid, dim3(T), 0, stream, a);
    return hipGetLastError();
}

template <int RF32>
static hipError_t launch_norm_p(const NormArgs& a, hipStream_t stream) {
    const int64_t slots = (a.K / 8 + 255) / 256;
    if (slots <= 1) return launch_norm_q<256, 1, RF32>(a, stream);
    if (slots <= 2) return launch_norm_q<256, 2, RF32>(a, stream);
    if (slots <= 4) return launch_norm_q<256, 4, RF32>(a, stream);
    if (slots <= 8) return launch_norm_q<256, 8, RF32>(a, stream);
    return hipErrorInvalidValue;                            // K beyond kNormMaxK (rejected before)
}

hipError_t launch_norm_residual(const NormArgs& a, int res_f32, hipStream_t stream) {
    return res_f32 ? launch_norm_p<1>(a, stream) : launch_norm_p<0>(a, stream);
}

// Workgroups of the backward kernel: one for each row up to a fixed number, whose column sums a
// second kernel adds.
static int64_t bwd_threads(int64_t K) { return K <= 2048 ? 256 : K <= 4096 ? 512 : 1024; }

int64_t norm_bwd_groups(int64_t M, int64_t K) {
    const int64_t most = 256 * (1024 / bwd_threads(K));
    return M < most ? M : most;
}

template <int RF32>
static void launch_bwd(const NormArgs& a, dim3 grid, hipStream_t stream) {
    switch (bwd_threads(a.K)) {
        case 256:
            hipLaunchKernelGGL((norm_residual_bwd_kernel<256, 1, RF32>), grid, dim3(256), 0, stream, a);
            break;
        case 512:
            hipLaunchKernelGGL((norm_residual_bwd_kernel<512, 1, RF32>), grid, dim3(512), 0, stream, a);
            break;
        default:
            if (a.K <= 8192)
                hipLaunchKernelGGL((norm_residual_bwd_kernel<1024, 1, RF32>), grid, dim3(1024), 0, stream, a);
            else
                hipLaunchKernelGGL((norm_residual_bwd_kernel<1024, 2, RF32>), grid, dim3(1024), 0, stream, a);
    }
}

hipError_t launch_norm_residual_bwd(const NormArgs& a, int res_f32, hipStream_t stream) {
    const int64_t groups = norm_bwd_groups(a.M, a.K);
    if (groups > 0) {
        if (res_f32) launch_bwd<1>(a, dim3((unsigned)groups), stream);
        else launch_bwd<0>(a, dim3((unsigned)groups), stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.columns) {
        const int64_t wg = (2 * a.K + 63) / 64;
        hipLaunchKernelGGL(norm_columns_kernel, dim3((unsigned)wg), dim3(1024), 0, stream, a, (int)groups);
    }
    return hipGetLastError();
}

}  // namespace bfq
