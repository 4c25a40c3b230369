// Access to rows of the expert-ordered operators: 16-byte chunks through buffer resources over one
// row (a lane past the row's end, and every lane of a row that is absent, reads zero and stores
// nothing, so the code between has no branches), conversions of the row types, and codes and scales
// of 128-column groups.
#pragma once
#include "moe_layer.h"
#include "quant_device.h"

namespace bfq {

// Row `r` of `bytes` bytes; empty without a row (r < 0) or a base.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t pair_row(const void* base, int64_t r, uint32_t bytes) {
    const bool there = base && r >= 0;
    return make_rsrc(static_cast<const uint8_t*>(base) + (there ? r * (int64_t)bytes : 0), there ? bytes : 0);
}

// S: the non-temporal hint, for what nobody reads again soon.
template <int S> __device__ __forceinline__ v4u row_load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff = 0) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, S ? kCachePolicyNT : 0);
}
template <int S> __device__ __forceinline__ void row_store16(__amdgpu_buffer_rsrc_t r, uint32_t voff, const v4u& v,
                                                             uint32_t soff = 0) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, voff, soff, S ? kCachePolicyNT : 0);
}
template <int S> __device__ __forceinline__ void row_store8(__amdgpu_buffer_rsrc_t r, uint32_t voff, const uint2& v) {
    typedef unsigned int v2u __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(v2u{v.x, v.y}, r, voff, 0, S ? kCachePolicyNT : 0);
}

// Eight values of a row at column 8c: 16 bits, 32 bits, or codes.
template <int RK, int S> struct RowChunk {
    static constexpr bool wide = RK == R_FP32, codes = RK == R_FP8 || RK == R_INT8;
    static constexpr int size = wide ? 4 : codes ? 1 : 2;     // bytes of a value
    v4u a, b;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t c) {
        if constexpr (codes) {
            typedef unsigned int v2u __attribute__((ext_vector_type(2)));
            const v2u q = __builtin_amdgcn_raw_buffer_load_b64(r, c * 8, 0, S ? kCachePolicyNT : 0);
            a.x = q.x;
            a.y = q.y;
        } else if constexpr (wide) {
            a = row_load16<S>(r, c * 32);
            b = row_load16<S>(r, c * 32, 16);
        } else {
            a = row_load16<S>(r, c * 16);
        }
    }
    __device__ __forceinline__ void get(float* x) const {
        if constexpr (RK == R_BF16) {
            unpack8(make_uint4(a.x, a.y, a.z, a.w), x);
        } else if constexpr (RK == R_FP16) {
            typedef _Float16 h2 __attribute__((ext_vector_type(2)));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const h2 h = __builtin_bit_cast(h2, w[i]);
                x[2 * i] = (float)h.x;
                x[2 * i + 1] = (float)h.y;
            }
        } else if constexpr (RK == R_FP32) {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else if constexpr (RK == R_FP8) {
            code_values<Q_FP8>(make_uint2(a.x, a.y), x);
        } else if constexpr (RK == R_INT8) {
            code_values<Q_INT8>(make_uint2(a.x, a.y), x);
        }
    }
    // Values of eight codes, without their scale.
    template <int QT> static __device__ __forceinline__ void code_values(const uint2& q, float* x) {
        if constexpr (QT == Q_FP8) {
            typedef float f2 __attribute__((ext_vector_type(2)));
            const f2 p0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), p1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true),
                     p2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), p3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
            x[0] = p0.x; x[1] = p0.y; x[2] = p1.x; x[3] = p1.y;
            x[4] = p2.x; x[5] = p2.y; x[6] = p3.x; x[7] = p3.y;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = (float)(int)(int8_t)(q.x >> (8 * i));
                x[4 + i] = (float)(int)(int8_t)(q.y >> (8 * i));
            }
        }
    }
};

// Eight values as bf16, fp16 or fp32 (uniform) at column 8c of a row. Those of fp32 are two halves of a
// line, which meet in L2: never past the caches. (Loads of such halves keep the hint: fp32 rows arrive at 5.0 to
// 5.1 TB/s, a large copy's rate.)
template <int S>
__device__ __forceinline__ void row_store(__amdgpu_buffer_rsrc_t r, uint32_t c, int otype, const float* x) {
    if (otype == O_FP32) {
        row_store16<0>(r, c * 32, __builtin_bit_cast(v4u, v4f{x[0], x[1], x[2], x[3]}));
        row_store16<0>(r, c * 32, __builtin_bit_cast(v4u, v4f{x[4], x[5], x[6], x[7]}), 16);
        return;
    }
    v4u v;
    if (otype == O_BF16) {
        v = v4u{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
    } else {
        v = v4u{f32_to_f16_bits(x[0]) | (f32_to_f16_bits(x[1]) << 16), f32_to_f16_bits(x[2]) | (f32_to_f16_bits(x[3]) << 16),
                f32_to_f16_bits(x[4]) | (f32_to_f16_bits(x[5]) << 16), f32_to_f16_bits(x[6]) | (f32_to_f16_bits(x[7]) << 16)};
    }
    row_store16<S>(r, c * 16, v);
}

__device__ __forceinline__ int type_size(int otype) { return otype == O_FP32 ? 4 : 2; }

// Largest over the L (8 or 16) neighbouring lanes that hold a group, in each of them.
template <int L> __device__ __forceinline__ uint32_t group_max(uint32_t m) {
    m = max(m, dpp_u32<kDppQuadXor1>(m));
    m = max(m, dpp_u32<kDppQuadXor2>(m));
    m = max(m, dpp_u32<kDppHalfMirror>(m));
    return L == 16 ? max(m, dpp_u32<kDppMirror>(m)) : m;
}

// One scale of group g of row m; packed: its byte of the word, and by the last group the zero bytes
// after it.
__device__ __forceinline__ void put_scale(const CodesOut& o, int64_t m, int64_t g, int64_t groups, float s) {
    if (!o.packed) {
        o.scales[m * o.stride_m + g * o.stride_g] = s;
        return;
    }
    uint8_t* word = reinterpret_cast<uint8_t*>(o.scales) + ((g >> 2) * o.stride_g + m) * 4;
    word[g & 3] = (uint8_t)e8m0_of(s);
    if (g == groups - 1)
        for (int j = (int)(g & 3) + 1; j < 4; ++j) word[j] = 0;
}

// The rows that a wave's pairs have: lane j holds that of pair t * topk + j, or -1.
__device__ __forceinline__ int pair_place(const PairPlaces& p, int64_t t, int j) {
    if (j >= p.topk) return -1;
    const int64_t q = t * p.topk + j;
    if (p.pair_rows) {
        const int r = p.pair_rows[q];
        return r >= 0 && r < p.R ? r : -1;
    }
    if (p.ids && (uint32_t)p.ids[q] >= (uint32_t)p.E) return -1;
    return (int)q;
}
__device__ __forceinline__ float lane_f32(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

}  // namespace bfq
