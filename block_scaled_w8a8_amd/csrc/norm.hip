// Norms around a block of the residual stream, one pass over a token's row:
//   z  = y * rms(y) * w_post           (the norm after the block; without w_post z = y)
//   r' = r + alpha * gate * z          (the block's gate and residual scale)
//   n  = r' * rms(r') * w_pre          (the norm before the next block)
// with rms(x) = 1 / sqrt(mean(x^2) + eps); n is stored as bf16, as the codes and scales that the
// GEMMs read (the token quantizer's formats), or both. All of it in fp32; n is taken from the
// unrounded r' and quantized unrounded, so storing r' or n as bf16 costs the codes nothing.
//
// What bounds it: bytes. 4096 rows of 7168 with post norm, codes out: 206 MB in 43 us, 4.8 TB/s, the rate
// of a large copy, and in 47 us on average over a hundred calls back to back (without the non-temporal
// hints some 4 us more). A row is read once (y, r) and written once (r', codes), everything between stays
// in registers: P chunks of 8 elements a thread, chunk c of the row held by thread c % T in slot c / T, so
// 16 neighbouring lanes own one 128-element group as in the token quantizer. Each norm costs one
// reduction over the workgroup (DPP within a wave, LDS across).
#include "bfq_internal.h"
#include "quant_device.h"

namespace bfq {

// Row tensors go through buffer resources over one row: a lane past the row's end, and every lane
// of an operand that is absent, reads zero and stores nothing, so the row code has no branches and
// its loads stay in flight until they are used.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* p, int64_t m, uint32_t bytes) {
    const uint8_t* base = static_cast<const uint8_t*>(p) + (p ? m * bytes : 0);
    return make_rsrc(base, p ? bytes : 0);
}
// S = 1: with the non-temporal hint, for rows of a call that writes more than the L2s hold
// (past_caches): nobody finds them there, and the channel vectors keep their place.
constexpr int kNonTemporal = 2;                          // the cache policy operand's bit
template <int S = 0>
__device__ __forceinline__ v4u load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff = 0) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, S ? kNonTemporal : 0);
}
template <int S>
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t r, uint32_t voff, const v4u& v, uint32_t soff = 0) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, voff, soff, S ? kNonTemporal : 0);
}
__device__ __forceinline__ void unpack(const v4u& v, float* x) {
    unpack8(make_uint4(v.x, v.y, v.z, v.w), x);
}
__device__ __forceinline__ v4u pack(const float* x) {
    return v4u{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
}

// Eight values of the residual stream at byte offset voff of a bf16 row (twice that of fp32).
template <int F32, int S> struct Chunk;
template <int S> struct Chunk<0, S> {
    v4u v;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t voff) { v = load16<S>(r, voff); }
    __device__ __forceinline__ void get(float* x) const { unpack(v, x); }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t voff, const float* x) {
        store16<S>(r, voff, pack(x));
    }
};
template <int S> struct Chunk<1, S> {
    v4f a, b;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
        a = __builtin_bit_cast(v4f, load16<S>(r, 2 * voff));
        b = __builtin_bit_cast(v4f, load16<S>(r, 2 * voff, 16));
    }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t voff, const float* x) {
        store16<S>(r, 2 * voff, __builtin_bit_cast(v4u, v4f{x[0], x[1], x[2], x[3]}));
        store16<S>(r, 2 * voff, __builtin_bit_cast(v4u, v4f{x[4], x[5], x[6], x[7]}), 16);
    }
};

// An absent vector operand (zeros from its empty resource) as bf16 ones.
__device__ __forceinline__ v4u ones_unless(const v4u& v, bool present) {
    const uint32_t o = present ? 0u : 0x3F803F80u;
    return v4u{v.x | o, v.y | o, v.z | o, v.w | o};
}

// alpha, times the row's gate value if there is one a token.
__device__ __forceinline__ float row_scale(const NormArgs& p, int64_t m) {
    if (p.gate_kind != BFQ_GATE_TOKEN) return p.res_scale;
    return p.res_scale * __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.gate)[m] << 16);
}

__device__ __forceinline__ float rms_of(float sum_sq, float K, float eps) {
    return 1.0f / __builtin_sqrtf(sum_sq / K + eps);
}

// Most threads of a workgroup that keeps P chunks a thread (K <= kNormMaxK = 8 * 2048).
template <int P> constexpr int kNormThreads = P == 4 ? 512 : 1024;

// One row a workgroup. Q: -1 no codes, else Q_FP8 / Q_INT8. Rows M .. (packed scale words: up to a
// multiple of 4) exist only to write zero words.
template <int P, int RF32, int Q, int S>
__global__ __launch_bounds__(kNormThreads<P>) void norm_residual_kernel(NormArgs p) {
    const int t = threadIdx.x, lane = t & 63, T = blockDim.x;
    const int64_t m = p.row0 + blockIdx.x, K = p.K;
    const uint32_t row16 = (uint32_t)(2 * K), row_res = RF32 ? 2 * row16 : row16;   // bytes of a row
    const float fK = (float)K;
    __shared__ __attribute__((aligned(16))) float red[2][16];
    __shared__ uint32_t redmax[16];
    if constexpr (Q >= 0) {
        if (m >= p.M) {                                   // uniform: a padding row of packed words
            for (int64_t w = t; w < (K / 128 + 3) / 4; w += T) p.scales[w * p.s_stride_g + m] = 0.f;
            return;
        }
    }
    block_sum_init(red[0], 32);
    const bool channel = p.gate_kind == BFQ_GATE_CHANNEL, elements = p.gate_kind == BFQ_GATE_FULL;
    const __amdgpu_buffer_rsrc_t r_res = row_rsrc(p.residual, m, row_res), r_y = row_rsrc(p.y, m, row16),
                                 r_gate = row_rsrc(channel || elements ? p.gate : nullptr,
                                                   elements ? m : 0, row16),
                                 r_post = row_rsrc(p.w_post, 0, row16), r_pre = row_rsrc(p.w_pre, 0, row16),
                                 r_out = row_rsrc(p.res_out, m, row_res), r_n = row_rsrc(p.normed, m, row16);
    // P = 1 (few rows): every load up front, one trip to memory. Else the channel vectors, which
    // hit L2, come only when they are needed: fewer registers, more rows in flight on a CU.
    uint32_t voff[P];
    Chunk<RF32, S> rc[P];
    v4u yc[P], gc[P], wpost[P], wpre[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
        voff[u] = (uint32_t)(u * T + t) * 16;
        yc[u] = load16<S>(r_y, voff[u]);
        rc[u].load(r_res, voff[u]);
    }
    auto load_post = [&]() {
#pragma unroll
        for (int u = 0; u < P; ++u) {
            wpost[u] = load16(r_post, voff[u]);
            gc[u] = load16(r_gate, voff[u]);
        }
    };
    auto load_pre = [&]() {
#pragma unroll
        for (int u = 0; u < P; ++u) wpre[u] = load16(r_pre, voff[u]);
    };
    if constexpr (P == 1) {
        load_post();
        load_pre();
    }
    float c = row_scale(p, m);
    if (p.w_post) {
        float s[1] = {0.f};
#pragma unroll
        for (int u = 0; u < P; ++u) {
            float y[8];
            unpack(yc[u], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] = __builtin_fmaf(y[i], y[i], s[0]);
        }
        block_sum<1>(s, red[0]);
        c *= rms_of(s[0], fK, p.norm_eps);
    }
    if constexpr (P > 1) {
        __builtin_amdgcn_sched_barrier(0);
        load_post();
    }
    float r[P][8], s[1] = {0.f};
#pragma unroll
    for (int u = 0; u < P; ++u) {
        float y[8], g[8], w[8];
        rc[u].get(r[u]);
        unpack(yc[u], y);
        unpack(ones_unless(gc[u], channel || elements), g);
        unpack(ones_unless(wpost[u], p.w_post != nullptr), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[u][i] = __builtin_fmaf(y[i] * w[i] * g[i], c, r[u][i]);   // three bf16: exact in fp32
            s[0] = __builtin_fmaf(r[u][i], r[u][i], s[0]);
        }
        Chunk<RF32, S>::store(r_out, voff[u], r[u]);
    }
    if (!p.w_pre) return;                                 // uniform
    if constexpr (P > 1) {
        __builtin_amdgcn_sched_barrier(0);
        load_pre();
    }
    block_sum<1>(s, red[1]);
    const float ir = rms_of(s[0], fK, p.norm_eps);
#pragma unroll
    for (int u = 0; u < P; ++u) {
        float w[8];
        unpack(wpre[u], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[u][i] = r[u][i] * ir * w[i];
        store16<S>(r_n, voff[u], pack(r[u]));
    }
    if constexpr (Q >= 0) {
        const __amdgpu_buffer_rsrc_t r_q = row_rsrc(p.q, m, (uint32_t)K);
        auto store_codes = [&](int u, uint32_t mx, float sc) {
            const uint2 q = encode8_group<Q>(r[u], mx, sc);
            typedef unsigned int v2u __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(v2u{q.x, q.y}, r_q, voff[u] / 2, 0, S ? kNonTemporal : 0);
        };
        // lanes past the row hold zeros: they join the reductions and store nothing
        if (p.per_token) {
            uint32_t mx = 0;
#pragma unroll
            for (int u = 0; u < P; ++u) mx = max(mx, amax8(r[u]));
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, off, 64));
            if (lane == 0) redmax[t >> 6] = mx;
            lds_barrier();
            for (int w = 0; w < T / 64; ++w) mx = max(mx, redmax[w]);
            const float sc = group_scale<Q>(mx, p.q_eps, p.ue8m0);
#pragma unroll
            for (int u = 0; u < P; ++u) store_codes(u, mx, sc);
            if (t == 0) p.scales[m * p.s_stride_m] = sc;
            return;
        }
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int64_t g = voff[u] >> 8;              // 16 lanes (256 bytes of bf16) own group g
            const bool live = voff[u] < row16;
            const uint32_t mx = max16(amax8(r[u]));
            const float sc = group_scale<Q>(mx, p.q_eps, p.ue8m0);
            store_codes(u, mx, sc);
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
// powers of rms), then {sum dz*z, sum dgate}. A workgroup walks rows blockIdx.x, + gridDim.x, ...
// with the next row's loads in flight and keeps its share of the column sums, 16 a chunk: dn * r^,
// and alpha*dr*y^ (CHANNEL: times w_post it is the gate's gradient, times the gate w_post's) or
// dz*y^ (else). Each workgroup writes its shares once; norm_columns_kernel adds them in workgroup
// order, so equal inputs give equal sums.
// One chunk a thread (P = 1): the sums stay in registers, the channel vectors wait in LDS. Two
// (K > 8192): registers hold a row only, so the sums live in LDS (each thread its own slots), the
// vectors come from L2, and the next row's loads start once their registers are free, all but y's
// before the second reduction.
// Bytes bound it. Measured: 4096 rows of 7168 bf16 with a channel gate 77 us with the column sums (352 MB,
// 4.6 TB/s; 86 on average over a hundred calls back to back), 4096 of 8192 fp32 121 us (5.0 TB/s; two
// chunks a thread were 10 to 13 us slower on both), 1024 of 16384 fp32 78 us (3.9 TB/s: four rows a CU,
// the first and last uncovered; with the sums of two chunks in registers, which spill, more than 50 us
// slower). The column sums' launch is 3 to 5 us of it, and the shares it reads are 8 K bytes a workgroup:
// on a few hundred short rows nearly as many as the operands' (257 rows of 1544: 7 and 3.6 us).
template <int P, int RF32, int S>
__global__ __launch_bounds__(1024) void norm_residual_bwd_kernel(NormArgs p) {
    const int t = threadIdx.x, T = blockDim.x;
    const int64_t K = p.K;
    const uint32_t row16 = (uint32_t)(2 * K), row_res = RF32 ? 2 * row16 : row16;
    const float fK = (float)K;
    __shared__ __attribute__((aligned(16))) float red[2][5 * 16];
    // P = 1: [3][T] vectors (w_pre, w_post, channel gate); P = 2: [2 sums][2 halves][2T] floats
    extern __shared__ v4u vec[];
    v4f* const sums = reinterpret_cast<v4f*>(vec);
    const bool channel = p.gate_kind == BFQ_GATE_CHANNEL, elements = p.gate_kind == BFQ_GATE_FULL;
    const bool post = p.w_post != nullptr;
    struct Row {
        Chunk<RF32, S> r, d;       // the stored sum, the stream's gradient
        v4u y, n;               // the block's output, the gradient at its normed successor
    };
    // element gates of row m
    auto gate_rsrc = [&](int64_t m) { return row_rsrc(elements && m < p.M ? p.gate : nullptr, m, row16); };
    float apre[1][8], apost[1][8];                       // P = 1
    block_sum_init(red[0], 160);
    const __amdgpu_buffer_rsrc_t v_pre = row_rsrc(p.w_pre, 0, row16), v_post = row_rsrc(p.w_post, 0, row16),
                                 v_gate = row_rsrc(channel ? p.gate : nullptr, 0, row16);
    // row m's operands, y and / or the others (constants); the stream's gradient is needed last
    auto load = [&](Row (&x)[P], int64_t m, bool y, bool others) {
        const bool in = m < p.M;
        const __amdgpu_buffer_rsrc_t rr = row_rsrc(in && p.w_pre ? p.residual : nullptr, m, row_res),
                                     rd = row_rsrc(in ? p.d_res_out : nullptr, m, row_res),
                                     ry = row_rsrc(in ? p.y : nullptr, m, row16),
                                     rn = row_rsrc(in ? p.d_normed : nullptr, m, row16);
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const uint32_t voff = (uint32_t)(u * T + t) * 16;
            if (others) {
                x[u].r.load(rr, voff);
                x[u].n = load16<S>(rn, voff);
            }
            if (y) x[u].y = load16<S>(ry, voff);
            if (others) x[u].d.load(rd, voff);
        }
    };
    Row cur[P];
    load(cur, blockIdx.x, true, true);
    auto w_pre_at = [&](int i) { return P == 1 ? vec[i] : load16(v_pre, (uint32_t)i * 16); };
    auto w_post_at = [&](int i) {
        return P == 1 ? vec[T + i] : ones_unless(load16(v_post, (uint32_t)i * 16), post);
    };
    auto gate_at = [&](int i) { return P == 1 ? vec[2 * T + i] : load16(v_gate, (uint32_t)i * 16); };
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const int i = u * T + t;
        if constexpr (P == 1) {
            vec[i] = load16(v_pre, (uint32_t)i * 16);
            vec[T + i] = ones_unless(load16(v_post, (uint32_t)i * 16), post);
            vec[2 * T + i] = load16(v_gate, (uint32_t)i * 16);
#pragma unroll
            for (int j = 0; j < 8; ++j) apre[0][j] = apost[0][j] = 0.f;
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) sums[h * T * P + i] = v4f{0.f, 0.f, 0.f, 0.f};
        }
    }
    // sum k (0: pre, 1: post) of chunk u += x * y
    auto add = [&](int k, int u, const float* x, const float* y) {
        if constexpr (P == 1) {
            float* a = k ? apost[0] : apre[0];
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = __builtin_fmaf(x[i], y[i], a[i]);
        } else {
            v4f* a = sums + (2 * k * P * T + u * T + t);
            v4f lo = a[0], hi = a[T * P];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = __builtin_fmaf(x[i], y[i], lo[i]);
                hi[i] = __builtin_fmaf(x[i + 4], y[i + 4], hi[i]);
            }
            a[0] = lo;
            a[T * P] = hi;
        }
    };
    int par = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, par ^= 1) {
        Row next[P];
        if constexpr (P == 1) load(next, m + gridDim.x, true, true);
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < P; ++u) {
            float r[8], y[8], dn[8], w[8];
            cur[u].r.get(r);
            unpack(cur[u].y, y);
            unpack(cur[u].n, dn);
            unpack(w_pre_at(u * T + t), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[0] = __builtin_fmaf(r[i], r[i], s[0]);
                s[1] = __builtin_fmaf(y[i], y[i], s[1]);
                s[2] = __builtin_fmaf(w[i] * dn[i], r[i], s[2]);
            }
        }
        block_sum<3>(s, red[par]);
        const float ir = rms_of(s[0], fK, p.norm_eps), iy = post ? rms_of(s[1], fK, p.norm_eps) : 1.f;
        const float cr = ir * ir * s[2] / fK;      // r^ * mean(w_pre * dn * r^) = r' * cr
        const float alpha = p.res_scale, a_row = row_scale(p, m);
        const __amdgpu_buffer_rsrc_t rg = gate_rsrc(m), o_r = row_rsrc(p.d_res, m, row_res), o_y = row_rsrc(p.d_y, m, row16),
                                     o_g = row_rsrc(elements ? p.d_gate : nullptr, m, row16);
        float dz[P][8], q[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const uint32_t voff = (uint32_t)(u * T + t) * 16;
            float r[8], dr[8], dn[8], w[8], y[8], g[8], dg[8];
            cur[u].r.get(r);
            cur[u].d.get(dr);
            unpack(cur[u].n, dn);
            unpack(w_pre_at(u * T + t), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dr[i] = __builtin_fmaf(ir, __builtin_fmaf(-r[i], cr, w[i] * dn[i]), dr[i]);
                r[i] *= ir;
            }
            add(0, u, dn, r);
            Chunk<RF32, S>::store(o_r, voff, dr);
            unpack(cur[u].y, y);
            unpack(ones_unless(channel ? gate_at(u * T + t) : load16(rg, voff), channel || elements), g);
            unpack(w_post_at(u * T + t), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float yn = y[i] * iy, z = yn * w[i], ad = alpha * dr[i];
                dz[u][i] = a_row * dr[i] * g[i];
                dg[i] = ad * z;
                q[0] = __builtin_fmaf(dz[u][i], z, q[0]);
                q[1] += dg[i];
                y[i] = yn;
                dr[i] = channel ? ad : dz[u][i];
            }
            add(1, u, dr, y);
            store16<S>(o_g, voff, pack(dg));
        }
        if constexpr (P > 1) load(cur, m + gridDim.x, false, true);
        block_sum<2>(q, red[par] + 3 * 16);
        if (p.gate_kind == BFQ_GATE_TOKEN && p.d_gate && t == 0) static_cast<float*>(p.d_gate)[m] = q[1];
        const float cy = post ? iy * q[0] / fK : 0.f;
#pragma unroll
        for (int u = 0; u < P; ++u) {
            float y[8], w[8];
            unpack(cur[u].y, y);
            unpack(w_post_at(u * T + t), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) dz[u][i] = iy * __builtin_fmaf(-y[i], cy, w[i] * dz[u][i]);
            store16<S>(o_y, (uint32_t)(u * T + t) * 16, pack(dz[u]));
        }
        if constexpr (P == 1) cur[0] = next[0];
        else load(cur, m + gridDim.x, true, false);
    }
    if (!p.columns) return;
    const uint32_t row32 = (uint32_t)(4 * K);
    const __amdgpu_buffer_rsrc_t s0 = row_rsrc(p.partials, 2 * (int64_t)blockIdx.x, row32),
                                 s1 = row_rsrc(p.partials, 2 * (int64_t)blockIdx.x + 1, row32);
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const uint32_t voff = (uint32_t)(u * T + t) * 16;
        if constexpr (P == 1) {
            Chunk<1, 0>::store(s0, voff, apre[0]);
            Chunk<1, 0>::store(s1, voff, apost[0]);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                buf_store_v4f(s0, sums[h * T * P + u * T + t], 2 * voff, 16 * h);
                buf_store_v4f(s1, sums[(2 + h) * T * P + u * T + t], 2 * voff, 16 * h);
            }
        }
    }
}

// Column sums of the workgroups' shares [rows][2][K]: 64 columns a workgroup, four a thread; its 16
// rows of threads each add every 16th share (several loads in flight), then the 16 in order.
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs p, int rows) {
    const int64_t K = p.K;
    const int t = threadIdx.x, part = t >> 4;
    const int64_t c4 = (int64_t)blockIdx.x * 64 + (t & 15) * 4;       // 2K is a multiple of 4
    __shared__ v4f sums[16][16];
    v4f a = {0.f, 0.f, 0.f, 0.f};
    if (c4 < 2 * K) {
        const float* src = p.partials + c4;
#pragma unroll 8
        for (int g = part; g < rows; g += 16) a += *reinterpret_cast<const v4f*>(src + (int64_t)g * 2 * K);
    }
    sums[part][t & 15] = a;
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * 64 + t;
    if (t >= 64 || col >= 2 * K) return;
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < 16; ++g) s += sums[g][t >> 2][t & 3];
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

static unsigned threads_for(int64_t K, int P) {
    return (unsigned)((K / 8 + 64 * P - 1) / (64 * P) * 64);
}

template <int P, int RF32, int S>
static hipError_t launch_norm_q(const NormArgs& a, hipStream_t stream) {
    const int64_t rows = a.packed ? (a.M + 3) / 4 * 4 : a.M;
    // a grid dimension holds fewer than 2^32 threads: at K = 8192 rows past 2^23 - 4 take a second launch
    const int64_t most = ((int64_t(1) << 32) - 1) / threads_for(a.K, P);
    NormArgs b = a;
    for (b.row0 = 0; b.row0 < rows; b.row0 += most) {
        const dim3 grid((unsigned)(rows - b.row0 < most ? rows - b.row0 : most)), block(threads_for(a.K, P));
        if (!a.q)
            hipLaunchKernelGGL((norm_residual_kernel<P, RF32, -1, S>), grid, block, 0, stream, b);
        else if (a.qtype == Q_FP8)
            hipLaunchKernelGGL((norm_residual_kernel<P, RF32, Q_FP8, S>), grid, block, 0, stream, b);
        else
            hipLaunchKernelGGL((norm_residual_kernel<P, RF32, Q_INT8, S>), grid, block, 0, stream, b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int P, int RF32>
static hipError_t launch_norm_s(const NormArgs& a, hipStream_t stream) {
    const int64_t out = (a.res_out ? (RF32 ? 4 : 2) : 0) + (a.normed ? 2 : 0) + (a.q ? 1 : 0);
    return past_caches(a.M * a.K * out) ? launch_norm_q<P, RF32, 1>(a, stream) : launch_norm_q<P, RF32, 0>(a, stream);
}

// Chunks a thread. Few waves a row start and reduce sooner (one row of 1536: 3.4 us with one chunk
// a thread, 3.8 with two); fewer, fatter threads leave room for more rows on a CU (4096 rows of
// 7168: 62.5 us with one chunk, 47.8 with two, 47.2 with four; 1024 rows of 16384: 29.2 with two,
// 25.8 with four). The chunks decide which elements a thread adds up, so past 8192 channels the last
// bits of a row depend on M; in batch-invariant mode four serve every M (one row of 16384, codes out:
// 6.3 us for 6.1; 256 rows 11.9 either way).
template <int RF32>
static hipError_t launch_norm_p(const NormArgs& a, hipStream_t stream) {
    if (a.K <= 2048) return launch_norm_s<1, RF32>(a, stream);
    if (a.K <= 8192 || (a.M <= 256 && !a.invariant)) return launch_norm_s<2, RF32>(a, stream);
    return launch_norm_s<4, RF32>(a, stream);
}

hipError_t launch_norm_residual(const NormArgs& a, int res_f32, hipStream_t stream) {
    return res_f32 ? launch_norm_p<1>(a, stream) : launch_norm_p<0>(a, stream);
}

// Workgroups of the backward kernel: one for each row up to what the CUs hold at once (16 waves
// each at its register count; past K = 8192 one, by its LDS).
int64_t norm_bwd_groups(int64_t M, int64_t K) {
    const int64_t most = 256 * (1024 / threads_for(K, K <= 8192 ? 1 : 2));
    return M < most ? M : most;
}

template <int P, int RF32, int S>
static hipError_t launch_bwd_s(const NormArgs& a, int64_t groups, hipStream_t stream) {
    const unsigned threads = threads_for(a.K, P), lds = threads * (P == 1 ? 48 : 128);
    if constexpr (P > 1) {
        static std::atomic<uint64_t> opted{0};
        const hipError_t e = opt_in_lds(
            opted, reinterpret_cast<const void*>(&norm_residual_bwd_kernel<P, RF32, S>), 1024 * 128);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((norm_residual_bwd_kernel<P, RF32, S>), dim3((unsigned)groups), dim3(threads), lds, stream, a);
    return hipGetLastError();
}

template <int P, int RF32>
static hipError_t launch_bwd(const NormArgs& a, int64_t groups, hipStream_t stream) {
    const int64_t out = (RF32 ? 4 : 2) + (a.d_y ? 2 : 0) + (a.d_gate && a.gate_kind == BFQ_GATE_FULL ? 2 : 0);
    return past_caches(a.M * a.K * out) ? launch_bwd_s<P, RF32, 1>(a, groups, stream)
                                        : launch_bwd_s<P, RF32, 0>(a, groups, stream);
}

hipError_t launch_norm_residual_bwd(const NormArgs& a, int res_f32, hipStream_t stream) {
    const int64_t groups = norm_bwd_groups(a.M, a.K);
    if (groups > 0) {
        const hipError_t e = a.K <= 8192
                                 ? (res_f32 ? launch_bwd<1, 1>(a, groups, stream) : launch_bwd<1, 0>(a, groups, stream))
                                 : (res_f32 ? launch_bwd<2, 1>(a, groups, stream) : launch_bwd<2, 0>(a, groups, stream));
        if (e != hipSuccess) return e;
    }
    if (a.columns) {
        const int64_t wg = (2 * a.K + 63) / 64;
        hipLaunchKernelGGL(norm_columns_kernel, dim3((unsigned)wg), dim3(256), 0, stream, a, (int)groups);
    }
    return hipGetLastError();
}

}  // namespace bfq
