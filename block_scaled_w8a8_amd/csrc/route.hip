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
// A wave takes a token: lane l holds experts l*V .. l*V + V-1, so the lowest index among equal keys is
// the lowest lane's, and a choice costs one wave maximum (DPP within rows of 16 lanes, v_readlane
// across them) and one ballot. No workgroup barrier anywhere.
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
__device__ __forceinline__ uint64_t wave_max(uint64_t m) {
    const uint32_t hi = wave_max((uint32_t)(m >> 32));
    const uint32_t lo = wave_max((uint32_t)(m >> 32) == hi ? (uint32_t)m : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}

// Experts lane*V .. of a token's row; those past E count as masked. +inf counts as the largest
// finite value, so that a softmax over it is defined.
template <int V>
__device__ __forceinline__ void load_logits(const RouteArgs& p, int64_t t, int lane, float* x) {
    const int64_t at = t * p.E;
    const int e0 = lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = e0 + i;
        x[i] = -__builtin_inff();
        if (e < p.E) {
            if (p.otype == O_FP32) x[i] = static_cast<const float*>(p.logits)[at + e];
            else if (p.otype == O_BF16) x[i] = bf16_lo(static_cast<const uint16_t*>(p.logits)[at + e]);
            else x[i] = (float)static_cast<const _Float16*>(p.logits)[at + e];
            if (x[i] == __builtin_inff()) x[i] = 0x1.fffffep127f;
        }
    }
}
__device__ __forceinline__ float logit_at(const RouteArgs& p, int64_t i) {
    float x;
    if (p.otype == O_FP32) x = static_cast<const float*>(p.logits)[i];
    else if (p.otype == O_BF16) x = bf16_lo(static_cast<const uint16_t*>(p.logits)[i]);
    else x = (float)static_cast<const _Float16*>(p.logits)[i];
    return x == __builtin_inff() ? 0x1.fffffep127f : x;
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

__device__ __forceinline__ double sigmoid_f64(double x) { return 1.0 / (1.0 + exp(-x)); }

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
    float x[V];
    load_logits<V>(p, t, lane, x);
    Real top = 0, sum = 1;
    if constexpr (!SG) {
        top = wave_top<V>(x);
        Real s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (K64) s += exp((double)x[i] - top);
            else s += expf(x[i] - top);
        }
        if constexpr (K64) sum = wave_sum_f64(s);
        else sum = wave_sum(s);
    }
    auto score = [&](float v) -> Real {
        if constexpr (SG) {
            if constexpr (K64) return sigmoid_f64((double)v);
            else return sigmoid_f32(v);
        } else {
            if constexpr (K64) return exp((double)v - top) / sum;
            else return expf(v - top) / sum;
        }
    };
    Key key[V];
    if constexpr (!K64) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = order_bits(x[i]);
    } else {
        double k[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            k[i] = score(x[i]) + (p.bias && e < p.E ? (double)p.bias[e] : 0.0);
            if (x[i] == -__builtin_inff()) k[i] = -__builtin_inf();
        }
        uint64_t kept = ~0ull;                           // groups that stay
        int size = p.E;                                  // experts of a group
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
            for (int d = 1; d < L; d <<= 1) {
                const uint64_t a2 = __shfl_xor(a, d, 64), b2 = __shfl_xor(b, d, 64);
                const uint64_t lo = a < a2 ? a : a2;
                a = a < a2 ? a2 : a;
                b = b < b2 ? b2 : b;
                b = b < lo ? lo : b;
            }
            // sum of the two; a masked one counts as nothing, a group of masked ones never stays
            auto value = [](uint64_t v) {
                return v == ~0ull ? __builtin_nan("")
                                  : __longlong_as_double((long long)(v ^ ((v >> 63) ? 0x8000000000000000ull : ~0ull)));
            };
            uint64_t total = a;
            if (a > kNone64 && b > kNone64) total = order_bits(value(a) + value(b));
            kept = 0;
            for (int n = 0; n < p.topk_groups; ++n) {    // the best one left, lowest index first
                const uint64_t mine = g < p.groups && lane % L == 0 && !((kept >> g) & 1) ? total : 0;
                const uint64_t best = wave_max(mine);
                if (best <= kNone64) break;
                const int at = __builtin_ctzll(__ballot(mine == best));
                kept |= 1ull << (at / L);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = p.groups > 1 ? (lane * V + i) / size : 0;
            const bool in = g < 64 && ((kept >> (g & 63)) & 1);
            key[i] = in ? order_bits(k[i]) : 0;
        }
    }
    // lane j keeps the j-th choice
    int id = -1;
    float xj = 0.f;
    for (int j = 0; j < p.topk; ++j) {
        Key m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = key[i] > m ? key[i] : m;
        const Key best = wave_max(m);
        if (best <= none) break;                         // uniform: only masked experts are left
        const int at = __builtin_ctzll(__ballot(m == best));
        int pick = V - 1;
        float v = x[V - 1];
#pragma unroll
        for (int i = V - 2; i >= 0; --i)
            if (key[i] == best) { pick = i; v = x[i]; }
        if (lane == at) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == pick) key[i] = 0;
        }
        const int e = __builtin_amdgcn_readlane(lane * V + pick, at);
        const float xe = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), at));
        if (lane == j) { id = e; xj = xe; }
    }
    Real w = id >= 0 ? score(xj) : (Real)0;
    if (p.renorm) {
        if constexpr (K64) w = w / (wave_sum_f64(w) + (double)kRouteEps);
        else w = w / (wave_sum(w) + kRouteEps);
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
    float x[V];
    load_logits<V>(p, t, lane, x);
    int id = -1;
    float g = 0.f;
    if (lane < p.topk) {
        id = p.ids[t * p.topk + lane];
        if (id < 0 || id >= p.E) id = -1;
        g = p.d_weights[t * p.topk + lane];
    }
    float xj = id >= 0 ? logit_at(p, t * p.E + id) : -__builtin_inff();
    float top = 0.f, rsum = 1.f;
    if constexpr (!SG) {
        top = wave_top<V>(x);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += expf(x[i] - top);
        rsum = 1.f / wave_sum(s);
    }
    const float sj = id < 0 ? 0.f : SG ? sigmoid_f32(xj) : expf(xj - top) * rsum;
    float ds = id < 0 ? 0.f : p.weight_scale * g;
    float inner = 0.f;                                   // sum_k ds_k p_k (softmax)
    if (p.renorm) {
        const float D = wave_sum(sj) + kRouteEps;
        float acc = 0.f;
        for (int k = 0; k < p.topk; ++k) {
            const float gk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), k)),
                        sk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sj), k));
            if (sk != 0.f) acc += sk * (g - gk);         // uniform; a pair without an expert is none
        }
        if (id >= 0) ds = p.weight_scale * ((acc + kRouteEps * g) / D) / D;
        if constexpr (!SG) inner = p.weight_scale * (wave_sum(id < 0 ? 0.f : g * sj) * kRouteEps / D) / D;
    } else if constexpr (!SG) {
        inner = wave_sum(ds * sj);
    }
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    for (int k = 0; k < p.topk; ++k) {                   // in pair order: equal calls, equal sums
        const int e = __builtin_amdgcn_readlane(id, k);
        const float dk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ds), k));
        if (e < 0) continue;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane * V + i == e) d[i] += dk;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (e >= p.E) continue;
        float r;
        if constexpr (SG) {
            const float s = sigmoid_f32(x[i]), c = sigmoid_f32(-x[i]);   // 1 - s without cancellation
            r = d[i] == 0.f ? 0.f : d[i] * s * c;
        } else {
            r = expf(x[i] - top) * rsum * (d[i] - inner);
            if (x[i] == -__builtin_inff()) r = 0.f;
        }
        const int64_t at = t * p.E + e;
        if (p.otype == O_FP32) static_cast<float*>(p.d_logits)[at] = r;
        else static_cast<uint16_t*>(p.d_logits)[at] =
            (uint16_t)(p.otype == O_BF16 ? f32_to_bf16_bits(r) : f32_to_f16_bits(r));
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
    else if (a.E <= 256) route_fwd<4>(a, stream);
    else if (a.E <= 512) route_fwd<8>(a, stream);
    else route_fwd<16>(a, stream);
    return hipGetLastError();
}
hipError_t launch_route_bwd(const RouteArgs& a, hipStream_t stream) {
    if (a.E <= 64) route_bwd<1>(a, stream);
    else if (a.E <= 128) route_bwd<2>(a, stream);
    else if (a.E <= 256) route_bwd<4>(a, stream);
    else if (a.E <= 512) route_bwd<8>(a, stream);
    else route_bwd<16>(a, stream);
    return hipGetLastError();
}

}  // namespace bfq
