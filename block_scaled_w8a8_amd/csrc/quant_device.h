// Element encoders shared by the quantizing kernels: eight values of a group at a time, given
// the group's scale, and the power-of-two scale format.
//
// Pages cited by title and section:
//   [BENCH] "vLLM DeepGEMM FP8 Block GEMM 基准测试 ..." §4.1 (use_ue8m0)
#pragma once
#include "device_common.h"

namespace bfq {

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
    us2 x = __builtin_bit_cast(us2, a), y = __builtin_bit_cast(us2, b);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}

// Encode 8 values x[0..7] divided by scale s; finite-amax groups only (|x| <= amax of the
// group or row that s was formed from). The quotient is taken as q = x * r with r = 1 / s,
// one IEEE division per lane instead of one per value, then corrected once by the exact
// remainder e = x - q * s (a fused multiply-add): q + e * r, with the sign of x (the
// correction never changes the sign of a nonzero value; it restores -0, which q + e * r would
// turn into +0). For every finite bf16 amax and every bf16 x with |x| <= amax, with fp32 or
// power-of-two scales and either code type, the code of this value equals the code of the
// IEEE quotient x / s (checked exhaustively on the CPU: tests/native/quotient_codes.c); where
// the two fp32 values differ at all (subnormal x in a group whose amax is below eps) both
// encode to zero. (r names the return value below; rs is the reciprocal.)
template <int QT>
__device__ __forceinline__ uint2 encode8(const float* x, float s) {
    const float rs = 1.0f / s;                         // IEEE division, once per lane
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = x[i] * rs;
        const float e = __builtin_fmaf(-q, s, x[i]);   // exact
        y[i] = __builtin_copysignf(__builtin_fmaf(e, rs, q), x[i]);
    }
    uint2 r;
    if constexpr (QT == Q_FP8) {
        r.x = enc_fp8x4(y[0], y[1], y[2], y[3]);
        r.y = enc_fp8x4(y[4], y[5], y[6], y[7]);
    } else {
        r.x = enc_i8x4(y[0], y[1], y[2], y[3]);
        r.y = enc_i8x4(y[4], y[5], y[6], y[7]);
    }
    return r;
}

// Groups whose amax is Inf or NaN. NaN amax: every code is NaN (0x7F) / 0 (int8).
// Inf amax: the scale is Inf, finite values divide to a signed zero, +-Inf to NaN.
template <int QT>
__device__ __forceinline__ uint2 encode8_special(const float* x, bool nan_group) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t code;
        if (nan_group || __builtin_isinf(x[i])) code = (QT == Q_FP8) ? 0x7Fu : 0u;
        else code = (QT == Q_FP8) ? ((__float_as_uint(x[i]) >> 24) & 0x80u) : 0u;
        b[i] = code;
    }
    uint2 r;
    r.x = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
    r.y = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
    return r;
}

// UE8M0 scale format ([BENCH] §4.1, use_ue8m0): the smallest power of two >= s, for a
// positive normal fp32 s (s >= eps / Qmax keeps it normal; s <= FLT_MAX / 127 keeps the
// next power finite). A power of two stays; otherwise the mantissa is cleared and the
// exponent stepped up by one.
__device__ __forceinline__ float pow2_ceil(float s) {
    const uint32_t u = __float_as_uint(s);
    return (u & 0x007FFFFFu) ? __uint_as_float((u & 0xFF800000u) + 0x00800000u) : s;
}

// Encode 8 fp32 values of a finite group (|x| <= amax of the group that s was formed from) to the code
// of the IEEE quotient x / s: q = x * r, r the correctly rounded 1 / s, corrected once by the remainder
// e = q * s - x. With any mantissa of x and s the code of q - e * r is that of the quotient (checked on
// the CPU around every midpoint of two codes: tests/native/quotient_codes_fp32.c; with r a unit off it
// is not), and a zero keeps its sign. v_rcp_f32 is within a unit of 1 / s and one Newton step then
// rounds it correctly, on gfx950 for each of the 2^23 mantissas. The remainder is exact while nothing in
// it is subnormal; scales outside [2^-60, 2^100] (a tiny eps, or amax near the range's ends) take the
// division. Bare products x * r, two operations a value less, gave another code in 2.6e-4 of the places
// where the values are products of two bf16, which meet ties. (encode8 above, on bf16 values, divides
// once a lane and restores signs.)
template <int QT>
__device__ __forceinline__ uint2 encode8_f32(const float* x, float s) {
    float y[8];
    if (s >= 0x1p-60f && s <= 0x1p100f) {
        const float r0 = __builtin_amdgcn_rcpf(s);
        const float rs = __builtin_fmaf(__builtin_fmaf(-s, r0, 1.f), r0, r0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = x[i] * rs, e = __builtin_fmaf(q, s, -x[i]);
            y[i] = __builtin_fmaf(e, -rs, q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] / s;
    }
    uint2 r;
    if constexpr (QT == Q_FP8) {
        r.x = enc_fp8x4(y[0], y[1], y[2], y[3]);
        r.y = enc_fp8x4(y[4], y[5], y[6], y[7]);
    } else {
        r.x = enc_i8x4(y[0], y[1], y[2], y[3]);
        r.y = enc_i8x4(y[4], y[5], y[6], y[7]);
    }
    return r;
}

// The scale of a group whose largest magnitude has the fp32 bits `mx` (NaN > Inf > finite as
// unsigned integers): max(amax, eps) / Qmax, rounded up to a power of two for UE8M0; NaN or
// Inf for a group that holds one. The quotient is the IEEE one: a product with the correctly
// rounded 1 / Qmax and one remainder step round correctly while nothing in them is subnormal
// (Markstein's theorem); the range's ends divide.
template <int QT>
__device__ __forceinline__ float group_scale(uint32_t mx, float eps, int ue8m0) {
    if (mx >= 0x7F800000u) return __uint_as_float(mx > 0x7F800000u ? 0x7FC00000u : 0x7F800000u);
    const float a = __builtin_fmaxf(__uint_as_float(mx), eps);
    float s;
    if (a >= 0x1p-90f && a <= 0x1p120f) {
        constexpr float r = 1.0f / (QT == Q_FP8 ? kFp8Max : kInt8Max);
        const float q = a * r;
        s = __builtin_fmaf(__builtin_fmaf(-q, qmax<QT>(), a), r, q);
    } else {
        s = a / qmax<QT>();
    }
    return ue8m0 ? pow2_ceil(s) : s;
}

// Codes of 8 fp32 values of a group with that largest magnitude and scale.
template <int QT>
__device__ __forceinline__ uint2 encode8_group(const float* x, uint32_t mx, float s) {
    return mx < 0x7F800000u ? encode8_f32<QT>(x, s) : encode8_special<QT>(x, mx > 0x7F800000u);
}

// The larger of m and |x|, a NaN where either is one.
__device__ __forceinline__ float max_abs(float m, float x) {
    return __builtin_elementwise_maximum(m, __builtin_fabsf(x));
}

// Largest magnitude (bits) of 8 values; a NaN among them wins.
__device__ __forceinline__ uint32_t amax8(const float* x) {
    float m = __builtin_fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_abs(m, x[i]);
    return __float_as_uint(m) & 0x7FFFFFFFu;
}

// The value of another lane of the same 16-lane row, through the DPP operand path (no LDS): the
// four patterns below, in this order, combine all 16 lanes of a row.
constexpr int kDppQuadXor1 = 0xB1, kDppQuadXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;
template <int CTRL> __device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, true);
}
template <int CTRL> __device__ __forceinline__ float dpp_f32(float x) {
    return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(x)));
}

// Largest over the 16 lanes of a row (a 128-element group at 8 elements a lane), in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
    m = max(m, dpp_u32<kDppQuadXor1>(m));
    m = max(m, dpp_u32<kDppQuadXor2>(m));
    m = max(m, dpp_u32<kDppHalfMirror>(m));
    return max(m, dpp_u32<kDppMirror>(m));
}

// Sum over the wave, in every lane; the order of the additions is the same in every call.
__device__ __forceinline__ float wave_sum(float x) {
    x += dpp_f32<kDppQuadXor1>(x);
    x += dpp_f32<kDppQuadXor2>(x);
    x += dpp_f32<kDppHalfMirror>(x);
    x += dpp_f32<kDppMirror>(x);
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// Barrier that orders LDS accesses only. __syncthreads() also waits for every outstanding global
// load and store of the wave, which would drain the next row's loads and stall on the last stores.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Sums of N values over a workgroup of up to 1024 threads (blockDim.x a multiple of 64), in every
// thread, added in a fixed order. `slot` is 16 * N floats of LDS, 16-byte aligned, that no thread
// still reads from an earlier call; block_sum_init clears the slots of waves that do not exist, so
// that the sum always takes 16 in four wide reads (a loop over the waves would wait for LDS once
// a wave).
__device__ __forceinline__ void block_sum_init(float* slots, int n) {
    const int W = blockDim.x >> 6;
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if ((i & 15) >= W) slots[i] = 0.f;
}
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* slot) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (blockDim.x == 64) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) slot[16 * i + (threadIdx.x >> 6)] = v[i];
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const v4f* q = reinterpret_cast<const v4f*>(slot + 16 * i);
        const v4f a = q[0], b = q[1], c = q[2], d = q[3];
        const v4f e = (a + b) + (c + d);
        v[i] = (e.x + e.y) + (e.z + e.w);
    }
}

// The E8M0 word of the wave's four groups (16 lanes each, codes of scales s; lanes past the last
// group pass code 0), the same in every lane. E8M0 has no infinity: an Inf scale stores NaN,
// whose code its exponent field already is.
__device__ __forceinline__ uint32_t e8m0_word(uint32_t code, int lane) {
    uint32_t word = code << (8 * (lane >> 4));
    word |= (uint32_t)__shfl_xor((int)word, 16, 64);
    word |= (uint32_t)__shfl_xor((int)word, 32, 64);
    return word;
}

// Eight bf16 values of a 16-byte chunk as fp32, and back.
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
    x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));   // RNE
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

}  // namespace bfq
