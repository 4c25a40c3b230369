// The router of a mixture-of-experts layer: each token's topk experts and their weights from its
// logits, and the gradient at the logits.
//
//   s = softmax(x) or sigmoid(x) over a token's E logits; the key an expert is chosen by is x itself,
//   or (with a bias or groups of experts) s + bias in 64 bits, because keys of neighbouring experts
//   lie within a rounding of fp32; of the groups the topk_groups with the largest sum of two best keys
//   stay. The topk largest keys are taken in descending order, ties by the lowest index.
//   w_j = c s_j / D with D = sum_k s_k + 1e-20 or 1.
//   Gradient: ds_j = c (sum_k s_k (g_j - g_k) + 1e-20 g_j) / D^2, differences first, so that equal
//   gradients cancel exactly; without the division by the sum ds_j = c g_j. Then dx = ds s (1 - s)
//   (sigmoid) or p (ds - sum ds p) (softmax; the sum is c G 1e-20 / D^2 after the division).
//
// What is no key is fp32: scores and weights without bias or groups (the sum over a token's experts too) are
// off by 5.1e-8 in the norm over 4096 tokens of 256 experts, the fp64 form rounded once by 2.3e-8; the
// gradient by 1.1e-7 against 2.5e-8. That is a rounding or two of the fp32 outputs, and no choice
// depends on it.
//
// A wave takes a token: lane l holds experts l*V .. l*V + V-1, so the lowest index among equal keys is
// the lowest lane's, and a choice costs one wave maximum (DPP within rows of 16 lanes, v_readlane
// across them) and one ballot. No workgroup barrier anywhere. Latency and instructions bound it, not bytes:
// 8 tokens of 256 experts in 8 groups 5.8 us, most of it the chain of eight choices and the fp64 scores
// behind a launch; 4096 tokens of 256 logits 5.8 us (softmax; the bytes alone 0.5), with fp64 keys 10.2, with
// groups 11.6; the gradient 6.0. Past 384 experts the lane lists are not sorted: 4096 tokens, fp64 keys, 384 experts
// in 8 groups 12.7 us, 385 in one 16.4, 512 in 8 groups 19.5, 1000 in one 29, in 8 groups 35; softmax 385 8.1, 512
// 8.5, 1000 13.6; the gradient of 512 10.8, of 1000 29. Choices by 64-bit maxima over unsorted keys, logits carried along, sums
// through LDS and loads behind branches: 7.4, 6.9 and 7.0 us.
#include "activation.h"
#include "moe_layer.h"
#include "quant_device.h"

namespace bfq {

constexpr int kRouteWaves = 4;    // tokens of a workgroup

// Order-preserving bits: NaN above everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_bits(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if (x != x) return 0xFFFFFFFFu;
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_bits(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    if (x != x) return ~0ull;
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
constexpr uint32_t kNone32 = 0x007FFFFFu;               // order_bits(-inf): never chosen
constexpr uint64_t kNone64 = 0x000FFFFFFFFFFFFFull;

// Largest over the wave, as a scalar.
__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
    m = max16(m);
    const uint32_t a = __builtin_amdgcn_readlane(m, 0), b = __builtin_amdgcn_readlane(m, 16),
                   c = __builtin_amdgcn_readlane(m, 32), d = __builtin_amdgcn_readlane(m, 48);
    return max(max(a, b), max(c, d));
}
// The lanes that hold the largest key of the wave, and that key. Two keys of 64 bits seldom agree in
// their upper halves: the lower ones are compared only then.
__device__ __forceinline__ uint64_t wave_best(uint32_t m, uint32_t& best) {
    best = wave_max(m);
    return __ballot(m == best);
}
__device__ __forceinline__ uint64_t wave_best(uint64_t m, uint64_t& best) {
    const uint32_t hi = wave_max((uint32_t)(m >> 32));
    uint64_t lanes = __ballot((uint32_t)(m >> 32) == hi);
    uint32_t lo;
    if (lanes & (lanes - 1)) {                           // uniform
        lo = wave_max((uint32_t)(m >> 32) == hi ? (uint32_t)m : 0u);
        lanes &= __ballot((uint32_t)m == lo);
    } else {
        lo = __builtin_amdgcn_readlane((uint32_t)m, __builtin_ctzll(lanes));
    }
    best = ((uint64_t)hi << 32) | lo;
    return lanes;
}

// Sum over the wave: DPP within rows of 16 lanes, then the rows' sums as scalars.
__device__ __forceinline__ float row_of(float x, int lane) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane)); }
__device__ __forceinline__ double row_of(double x, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
template <int CTRL> __device__ __forceinline__ uint64_t dpp_u64(uint64_t x) {
    return ((uint64_t)dpp_u32<CTRL>((uint32_t)(x >> 32)) << 32) | dpp_u32<CTRL>((uint32_t)x);
}
template <int CTRL> __device__ __forceinline__ float dpp_of(float x) { return dpp_f32<CTRL>(x); }
template <int CTRL> __device__ __forceinline__ double dpp_of(double x) {
    return __longlong_as_double((long long)dpp_u64<CTRL>((uint64_t)__double_as_longlong(x)));
}
template <typename R> __device__ __forceinline__ R wave_total(R x) {
    x += dpp_of<kDppQuadXor1>(x);
    x += dpp_of<kDppQuadXor2>(x);
    x += dpp_of<kDppHalfMirror>(x);
    x += dpp_of<kDppMirror>(x);
    return (row_of(x, 0) + row_of(x, 16)) + (row_of(x, 32) + row_of(x, 48));
}

// Experts lane*V .. of a token's row; those past E count as masked. +inf counts as the largest
// finite value, so that a softmax over it is defined. Every load is issued before the first is looked at
// (past E: the last expert's, unused); with a branch around each, one waited for the other.
template <int V>
__device__ __forceinline__ void load_logits(const RouteArgs& p, int64_t t, int lane, float* x) {
    const int64_t at = t * p.E;
    const int e0 = lane * V, last = p.E - 1;
    if (p.otype == O_FP32) {
        const float* row = static_cast<const float*>(p.logits) + at;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = row[min(e0 + i, last)];
    } else {
        const uint16_t* row = static_cast<const uint16_t*>(p.logits) + at;
        uint16_t h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = row[min(e0 + i, last)];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = p.otype == O_BF16 ? bf16_lo(h[i]) : (float)__builtin_bit_cast(_Float16, h[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = x[i] == __builtin_inff() ? 0x1.fffffep127f : x[i];
        x[i] = e0 + i > last ? -__builtin_inff() : x[i];
    }
}

// The wave's largest logit (a NaN wins); 0 where all are masked, whose exponentials are then 0.
template <int V> __device__ __forceinline__ float wave_top(const float* x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, order_bits(x[i]));
    m = wave_max(m);
    if (m == 0xFFFFFFFFu) return __builtin_nanf("");
    const float top = __uint_as_float(m ^ ((m >> 31) ? 0x80000000u : 0xFFFFFFFFu));
    return m <= kNone32 ? 0.f : top;
}

// 1 / d of a positive d: two Newton steps on the hardware's estimate (about 2^-26), each squaring the
// error; a division where d is near the range's end.
__device__ __forceinline__ double inverse_f64(double d) {
    if (!(d < 0x1p1000)) return 1.0 / d;
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// K64: keys are scores plus bias in 64 bits (bias or groups), else the logits.
template <int V, int SG, int K64>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs p) {
    extern __shared__ double group_keys[];               // [kRouteWaves][E] with groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= p.T) return;
    typedef typename std::conditional<K64 != 0, uint64_t, uint32_t>::type Key;
    typedef typename std::conditional<K64 != 0, double, float>::type Real;
    const Key none = K64 ? (Key)kNone64 : (Key)kNone32;
    float x[V], bias[V];
    load_logits<V>(p, t, lane, x);
    if constexpr (K64) {
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < V; ++i) bias[i] = p.bias[min(lane * V + i, p.E - 1)];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) bias[i] = 0.f;
        }
    }
    Real top = 0, rsum = 1, s[V];                        // scores; K64 only where they are keys
    if constexpr (!SG) {
        top = wave_top<V>(x);
        Real sum = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (K64) s[i] = exp((double)x[i] - top);
            else s[i] = expf(x[i] - top);
            sum += s[i];
        }
        sum = wave_total(sum);
        if constexpr (K64) rsum = inverse_f64(sum);
        else rsum = 1.f / sum;
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= rsum;
    } else if constexpr (K64) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = inverse_f64(1.0 + exp(-(double)x[i]));
    }
    Key key[V];
    if constexpr (!K64) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = order_bits(x[i]);
    } else {
        double k[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            k[i] = x[i] == -__builtin_inff() ? -__builtin_inf() : s[i] + (double)bias[i];
        }
        uint64_t kept = ~0ull;                           // bit g * first: group g stays
        int size = p.E, first = 0;                       // experts of a group
        if (p.groups > 1) {
            size = p.E / p.groups;
            double* keys = group_keys + wave * p.E;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i < p.E) keys[lane * V + i] = k[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
            // L lanes a group (a power of two), each the best two of its share, then joined
            int L = 64;
            while (L * p.groups > 64) L >>= 1;
            const int g = lane / L;
            uint64_t a = kNone64, b = kNone64;           // largest, second
            if (g < p.groups)
                for (int e = lane % L; e < size; e += L) {
                    const uint64_t v = order_bits(keys[g * size + e]);
                    if (v > a) { b = a; a = v; }
                    else if (v > b) b = v;
                }
            auto join = [&](uint64_t a2, uint64_t b2) {
                const uint64_t lo = a < a2 ? a : a2;
                a = a < a2 ? a2 : a;
                b = b < b2 ? b2 : b;
                b = b < lo ? lo : b;
            };
            if (L > 1) join(dpp_u64<kDppQuadXor1>(a), dpp_u64<kDppQuadXor1>(b));
            if (L > 2) join(dpp_u64<kDppQuadXor2>(a), dpp_u64<kDppQuadXor2>(b));
            if (L > 4) join(dpp_u64<kDppHalfMirror>(a), dpp_u64<kDppHalfMirror>(b));
            if (L > 8) join(dpp_u64<kDppMirror>(a), dpp_u64<kDppMirror>(b));
            if (L > 16) join(__shfl_xor(a, 16, 64), __shfl_xor(b, 16, 64));
            // sum of the two; a masked one counts as nothing, a group of masked ones never stays
            auto value = [](uint64_t v) {
                return v == ~0ull ? __builtin_nan("")
                                  : __longlong_as_double((long long)(v ^ ((v >> 63) ? 0x8000000000000000ull : ~0ull)));
            };
            uint64_t total = a;
            if (a > kNone64 && b > kNone64) total = order_bits(value(a) + value(b));
            // a group stays if fewer than topk_groups come before it: a larger sum, or an equal one and a
            // lower index
            int before = 0;
            for (int n = 0; n < p.groups; ++n) {
                const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(total >> 32), n * L),
                               lo = __builtin_amdgcn_readlane((uint32_t)total, n * L);
                const uint64_t other = ((uint64_t)hi << 32) | lo;
                before += other > total || (other == total && n < g) ? 1 : 0;
            }
            first = L;
            kept = __ballot(g < p.groups && total > kNone64 && before < p.topk_groups);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;                  // past E: masked
            key[i] = e < p.E && (kept >> (e / size * first)) & 1 ? order_bits(k[i]) : 0;
        }
    }
    // Up to six experts a lane are sorted once (stable), so that a choice takes the head of a list.
    constexpr bool kSorted = V <= 6;
    int e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = lane * V + i;
    if constexpr (kSorted) {
#pragma unroll
        for (int n = V - 1; n > 0; --n) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool swap = key[i + 1] > key[i];
                const Key k0 = key[i], k1 = key[i + 1];
                const int e0 = e[i], e1 = e[i + 1];
                key[i] = swap ? k1 : k0;
                key[i + 1] = swap ? k0 : k1;
                e[i] = swap ? e1 : e0;
                e[i + 1] = swap ? e0 : e1;
            }
        }
    }
    // lane j keeps the j-th choice
    int id = -1;
    for (int j = 0; j < p.topk; ++j) {
        Key m = key[0], best;
        if constexpr (!kSorted) {
#pragma unroll
            for (int i = 1; i < V; ++i) m = key[i] > m ? key[i] : m;
        }
        const uint64_t lanes = wave_best(m, best);
        if (best <= none) break;                         // uniform: only masked experts are left
        const int at = __builtin_ctzll(lanes);
        int pick = kSorted ? 0 : V - 1;
        if constexpr (!kSorted) {
#pragma unroll
            for (int i = V - 2; i >= 0; --i)
                if (key[i] == best) pick = i;
        }
        const int chosen = __builtin_amdgcn_readlane(kSorted ? e[0] : lane * V + pick, at);
        if (lane == j) id = chosen;
        if (lane == at) {
            if constexpr (kSorted) {
#pragma unroll
                for (int i = 0; i < V - 1; ++i) { key[i] = key[i + 1]; e[i] = e[i + 1]; }
                key[V - 1] = 0;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i == pick) key[i] = 0;
            }
        }
    }
    // its score (a sigmoid of fp32 keys: its logit) from the lane that holds it
    constexpr bool kFromLogit = SG && !K64;
    Real w = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const Real v = __shfl(kFromLogit ? (Real)x[i] : s[i], (id < 0 ? 0 : id) / V, 64);
        if (id % V == i) w = v;
    }
    if constexpr (kFromLogit) w = sigmoid_f32(w);
    if (id < 0) w = 0;
    if (p.renorm) {
        w = w / (wave_total(w) + (Real)kRouteEps);
    }
    if (lane < p.topk) {
        p.ids[t * p.topk + lane] = id;
        p.weights[t * p.topk + lane] = (float)(w * (Real)p.weight_scale);
    }
}

template <int V, int SG>
__global__ __launch_bounds__(64 * kRouteWaves) void route_bwd_kernel(RouteArgs p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= p.T) return;
    const int64_t pair = t * p.topk + (lane < p.topk ? lane : 0);
    int id = p.ids[pair];
    float g = p.d_weights[pair], x[V];
    load_logits<V>(p, t, lane, x);
    if (lane >= p.topk) g = 0.f;
    if (lane >= p.topk || id < 0 || id >= p.E) id = -1;
    // the chosen logits from the lanes that hold them
    float xj = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v = __shfl(x[i], (id < 0 ? 0 : id) / V, 64);
        if (id >= 0 && id % V == i) xj = v;
    }
    float top = 0.f, rsum = 1.f, pe[V];
    if constexpr (!SG) {
        top = wave_top<V>(x);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += pe[i] = expf(x[i] - top);
        rsum = 1.f / wave_total(s);
    }
    const float sj = id < 0 ? 0.f : SG ? sigmoid_f32(xj) : expf(xj - top) * rsum;
    float ds = id < 0 ? 0.f : p.weight_scale * g;
    float inner = 0.f;                                   // sum_k ds_k p_k (softmax)
    if (p.renorm) {
        const float D = wave_total(sj) + kRouteEps;
        float acc = 0.f;
        for (int k = 0; k < p.topk; ++k) {
            const float gk = row_of(g, k), sk = row_of(sj, k);
            if (sk != 0.f) acc += sk * (g - gk);         // uniform; a pair without an expert is none
        }
        if (id >= 0) ds = p.weight_scale * ((acc + kRouteEps * g) / D) / D;
        if constexpr (!SG) inner = p.weight_scale * (wave_total(id < 0 ? 0.f : g * sj) * kRouteEps / D) / D;
    } else if constexpr (!SG) {
        inner = wave_total(ds * sj);
    }
    // sigmoid: s (1 - s) ds where it is formed, 1 - s without cancellation; the other experts have none
    if constexpr (SG) ds = id < 0 || ds == 0.f ? 0.f : ds * sj * sigmoid_f32(-xj);
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    for (int k = 0; k < p.topk; ++k) {                   // in pair order: equal calls, equal sums
        const int e = __builtin_amdgcn_readlane(id, k);
        const float dk = row_of(ds, k);
        if (e < 0) continue;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane * V + i == e) d[i] += dk;
    }
    if constexpr (!SG) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = x[i] == -__builtin_inff() ? 0.f : pe[i] * rsum * (d[i] - inner);
    }
    const int64_t at = t * p.E + lane * V;
    if (p.otype == O_FP32) {
        float* row = static_cast<float*>(p.d_logits) + at;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane * V + i < p.E) row[i] = d[i];
    } else {
        uint16_t* row = static_cast<uint16_t*>(p.d_logits) + at;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane * V + i < p.E) row[i] = (uint16_t)(p.otype == O_BF16 ? f32_to_bf16_bits(d[i]) : f32_to_f16_bits(d[i]));
    }
}

template <int V> static void route_fwd(const RouteArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    const bool k64 = a.bias || a.groups > 1;
    const size_t lds = a.groups > 1 ? sizeof(double) * kRouteWaves * a.E : 0;
    if (a.sigmoid && k64) hipLaunchKernelGGL((route_kernel<V, 1, 1>), grid, block, lds, stream, a);
    else if (a.sigmoid) hipLaunchKernelGGL((route_kernel<V, 1, 0>), grid, block, lds, stream, a);
    else if (k64) hipLaunchKernelGGL((route_kernel<V, 0, 1>), grid, block, lds, stream, a);
    else hipLaunchKernelGGL((route_kernel<V, 0, 0>), grid, block, lds, stream, a);
}
template <int V> static void route_bwd(const RouteArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    if (a.sigmoid) hipLaunchKernelGGL((route_bwd_kernel<V, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_bwd_kernel<V, 0>), grid, block, 0, stream, a);
}

// E <= kMoeMaxExperts: at most 16 experts a lane.
hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
    if (a.E <= 64) route_fwd<1>(a, stream);
    else if (a.E <= 128) route_fwd<2>(a, stream);
    else if (a.E <= 192) route_fwd<3>(a, stream);
    else if (a.E <= 256) route_fwd<4>(a, stream);
    else if (a.E <= 384) route_fwd<6>(a, stream);
    else if (a.E <= 512) route_fwd<8>(a, stream);
    else route_fwd<16>(a, stream);
    return hipGetLastError();
}
hipError_t launch_route_bwd(const RouteArgs& a, hipStream_t stream) {
    if (a.E <= 64) route_bwd<1>(a, stream);
    else if (a.E <= 128) route_bwd<2>(a, stream);
    else if (a.E <= 192) route_bwd<3>(a, stream);
    else if (a.E <= 256) route_bwd<4>(a, stream);
    else if (a.E <= 384) route_bwd<6>(a, stream);
    else if (a.E <= 512) route_bwd<8>(a, stream);
    else route_bwd<16>(a, stream);
    return hipGetLastError();
}

}  // namespace bfq
