// Rows of a mixture-of-experts layer: the (token, expert) pairs sorted by expert, the tokens' rows
// laid out in that order (dispatch), and the experts' rows back to their tokens with the router's
// weights (combine), with the gradients. The combine without weights is the dispatch's gradient.
//
//   rows[r(t, j)] = x[t]                                            dispatch, as bf16 or codes
//   out[t] = base[t] + sum_j w[t][j] rows[r(t, j)]                  combine
//   d_rows[r(t, j)] = w[t][j] dout[t],  dw[t][j] = <dout[t], rows[r(t, j)]>
//
// All but the sort are bound by bytes. A workgroup takes a token, not a row: what belongs to the
// token (its row, its codes, its gradient) is read and formed once and written topk times, or read
// topk times and summed in registers in pair order: no atomics, equal calls give equal bits.
#include "row_access.h"

namespace bfq {

// ------------------------------------------------------------------------- sort ----
// A stable counting sort in two launches: a histogram a workgroup, then every workgroup adds up what
// lies before it (at most 256 histograms of E + 1 counts, from L2) and places its pairs. One
// workgroup (1024 pairs or fewer) needs no first launch. Against counting, a scan in a workgroup of
// its own and the placing, as three launches, one less round trip through the queue; a decode
// step's pairs take one launch in place of three.

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kSortGroups = 256;

__device__ __forceinline__ int sort_bucket(int32_t id, int E) { return (uint32_t)id < (uint32_t)E ? id : E; }

// Pairs of a workgroup: whole rounds of kSortThreads.
__host__ __device__ inline int64_t sort_share(int64_t pairs) {
    const int64_t rounds = (pairs + kSortThreads - 1) / kSortThreads;
    return (rounds + kSortGroups - 1) / kSortGroups * kSortThreads;
}
static int64_t sort_groups(int64_t pairs) {
    const int64_t share = sort_share(pairs);
    return share > 0 ? (pairs + share - 1) / share : 0;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ ids, int64_t pairs,
                                                                  int64_t share, int E,
                                                                  int32_t* __restrict__ counts) {
    __shared__ int32_t hist[1024];                       // E + 1 <= 1024
    for (int b = threadIdx.x; b <= E; b += kSortThreads) hist[b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * share, hi = lo + share < pairs ? lo + share : pairs;
    for (int64_t q = lo + threadIdx.x; q < hi; q += kSortThreads) atomicAdd(&hist[sort_bucket(ids[q], E)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= E; b += kSortThreads) counts[(int64_t)blockIdx.x * (E + 1) + b] = hist[b];
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t* __restrict__ ids, int64_t pairs,
                                                                  int64_t share, int E,
                                                                  const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ sorted,
                                                                  int32_t* __restrict__ pair_rows) {
    __shared__ int32_t base[1024], sums[kSortWaves];
    __shared__ uint16_t wave_counts[kSortWaves][1024];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = E + 1, G = gridDim.x, g = blockIdx.x;
    const int64_t lo = g * share, hi = lo + share < pairs ? lo + share : pairs;
    // pairs of bucket `tid` in all, and in earlier workgroups
    int32_t total = 0, before = 0;
    if (G == 1) {
        if (tid < B) base[tid] = 0;
        __syncthreads();
        for (int64_t q = lo + tid; q < hi; q += kSortThreads) atomicAdd(&base[sort_bucket(ids[q], E)], 1);
        __syncthreads();
        if (tid < B) total = base[tid];
    } else if (tid < B) {
        for (int i = 0; i < G; ++i) {
            const int32_t c = counts[(int64_t)i * B + tid];
            before += i < g ? c : 0;
            total += c;
        }
    }
    // exclusive prefix over the buckets
    int32_t inc = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t v = __shfl_up(inc, d, 64);
        if (lane >= d) inc += v;
    }
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    int32_t first = inc - total;
    for (int w = 0; w < wave; ++w) first += sums[w];
    if (tid < B) {
        base[tid] = first + before;
        if (g == 0) offsets[tid] = first;
    }
    const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
    for (int64_t q0 = lo; q0 < hi; q0 += kSortThreads) {
        const int64_t q = q0 + tid;
        const bool in = q < hi;
        const int b = in ? sort_bucket(ids[q], E) : 1023;   // E <= 1023: past every expert
        // lanes of the wave with the same bucket: one ballot a bit of its number
        uint64_t same = __ballot(in);
#pragma unroll
        for (int k = 0; k < 10; ++k) {
            const uint64_t bit = __ballot((b >> k) & 1);
            same &= (b >> k) & 1 ? bit : ~bit;
        }
        for (int i = tid; i < kSortWaves * 1024 / 2; i += kSortThreads)
            reinterpret_cast<uint32_t*>(&wave_counts[0][0])[i] = 0;
        __syncthreads();
        const int rank = __builtin_popcountll(same & below);
        if (in && rank == 0) wave_counts[wave][b] = (uint16_t)__builtin_popcountll(same);
        __syncthreads();
        int32_t run = 0;
        if (tid < B) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const int32_t c = wave_counts[w][tid];
                wave_counts[w][tid] = (uint16_t)run;     // at most 1024 in all
                run += c;
            }
        }
        __syncthreads();
        if (in) {
            const int32_t at = base[b] + wave_counts[wave][b] + rank;
            sorted[at] = (int32_t)q;
            pair_rows[q] = b < E ? at : -1;
        }
        __syncthreads();
        if (tid < B) base[tid] += run;                   // read again after the next round's barriers
    }
}

// No pairs: every expert is empty.
__global__ __launch_bounds__(1024) void sort_empty_kernel(int E, int32_t* __restrict__ offsets) {
    if ((int)threadIdx.x <= E) offsets[threadIdx.x] = 0;
}

size_t moe_sort_workspace_bytes(int64_t pairs, int E) {
    const int64_t G = sort_groups(pairs);
    return G > 1 ? (size_t)G * (size_t)(E + 1) * sizeof(int32_t) : 0;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t pairs, int E, int32_t* offsets, int32_t* sorted,
                           int32_t* pair_rows, int32_t* counts, hipStream_t stream) {
    const int64_t G = sort_groups(pairs), share = sort_share(pairs);
    if (G == 0) {
        hipLaunchKernelGGL(sort_empty_kernel, dim3(1), dim3(1024), 0, stream, E, offsets);
        return hipGetLastError();
    }
    if (G > 1) {
        hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)G), dim3(kSortThreads), 0, stream, ids, pairs, share, E,
                           counts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(sort_place_kernel, dim3((unsigned)G), dim3(kSortThreads), 0, stream, ids, pairs, share, E,
                       counts, offsets, sorted, pair_rows);
    return hipGetLastError();
}

// --------------------------------------------------------------------- dispatch ----

// Rows as they are: eight columns a thread.
template <int S>
__global__ __launch_bounds__(256) void dispatch_rows_kernel(DispatchArgs p) {
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63;
    const uint32_t voff = (blockIdx.y * blockDim.x + threadIdx.x) * 16, bytes = (uint32_t)(2 * p.K);
    const int place = pair_place(p.at, t, lane);
    const v4u v = row_load16<S>(pair_row(p.x, t, bytes), voff);
    for (int j = 0; j < p.at.topk; ++j) {
        const int r = __builtin_amdgcn_readlane(place, j);
        if (r >= 0) row_store16<S>(pair_row(p.rows, r, bytes), voff, v);
    }
}

// Codes of a token's row, formed or copied (Q < 0) once and written to each of its rows: 16 columns
// a thread, so 8 lanes hold a group and every lane knows its scale; lane k of the group stores the
// scale of pair k, k + 8, ..: one store for eight rows. Packed scales: 32 lanes hold a word. Blocks
// past the tokens write the zero words of rows R .. round_up(R, 4) - 1.
template <int Q, int S>
__global__ __launch_bounds__(256) void dispatch_codes_kernel(DispatchArgs p) {
    const int64_t t = blockIdx.x, K = p.K, G = K / 128;
    const int lane = threadIdx.x & 63;
    if (t >= p.T) {
        const int64_t m = p.at.R + (t - p.T);
        for (int64_t w = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; w < (G + 3) / 4; w += (int64_t)gridDim.y * blockDim.x)
            p.out.scales[w * p.out.stride_g + m] = 0.f;
        return;
    }
    const int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x, g = c >> 3;
    const bool live = g < G;
    const int place = pair_place(p.at, t, lane);
    v4u code, raw0, raw1;
    float s = 0.f;                                       // packed: the bits of the group's word
    if constexpr (Q >= 0) {
        const __amdgpu_buffer_rsrc_t rx = pair_row(p.x, t, (uint32_t)(2 * K));
        raw0 = row_load16<S>(rx, (uint32_t)c * 32);
        raw1 = row_load16<S>(rx, (uint32_t)c * 32, 16);
        float x[16];
        unpack8(make_uint4(raw0.x, raw0.y, raw0.z, raw0.w), x);
        unpack8(make_uint4(raw1.x, raw1.y, raw1.z, raw1.w), x + 8);
        uint32_t mx = max(amax8(x), amax8(x + 8));       // NaN > Inf > finite as unsigned integers
        mx = max(mx, dpp_u32<kDppQuadXor1>(mx));
        mx = max(mx, dpp_u32<kDppQuadXor2>(mx));
        mx = max(mx, dpp_u32<kDppHalfMirror>(mx));
        s = group_scale<Q>(mx, p.out.eps, p.out.ue8m0);
        const uint2 lo = encode8_group<Q>(x, mx, s), hi = encode8_group<Q>(x + 8, mx, s);
        code = v4u{lo.x, lo.y, hi.x, hi.y};
        if (p.out.packed) {
            uint32_t word = live ? e8m0_of(s) << (8 * ((lane >> 3) & 3)) : 0u;
            word |= (uint32_t)__shfl_xor((int)word, 8, 64);
            word |= (uint32_t)__shfl_xor((int)word, 16, 64);
            s = __uint_as_float(word);
        }
    } else {
        code = row_load16<S>(pair_row(p.x, t, (uint32_t)K), (uint32_t)c * 16);
        const int64_t k = p.out.packed ? g >> 2 : g;
        if (p.out.packed ? k * 4 < G : live) s = p.x_scales[t * p.xs_stride_m + k * p.xs_stride_g];
    }
    const int64_t gs = p.out.packed ? g >> 2 : g;
    const int lanes = p.out.packed ? 32 : 8;             // that hold the same scale
    const bool keeps = p.out.packed ? gs * 4 < G : live;
    for (int j0 = 0; j0 < p.at.topk; j0 += lanes) {
        const int j = j0 + (lane & (lanes - 1));
        const int r = __shfl(place, j & 63, 64);         // j past topk: -1
        if (j < p.at.topk && r >= 0 && keeps) p.out.scales[(int64_t)r * p.out.stride_m + gs * p.out.stride_g] = s;
    }
    for (int j = 0; j < p.at.topk; ++j) {
        const int r = __builtin_amdgcn_readlane(place, j);
        if (r < 0) continue;
        row_store16<S>(pair_row(p.out.q, r, (uint32_t)K), (uint32_t)c * 16, code);
        if constexpr (Q >= 0) {
            if (p.rows) {
                const __amdgpu_buffer_rsrc_t rr = pair_row(p.rows, r, (uint32_t)(2 * K));
                row_store16<S>(rr, (uint32_t)c * 32, raw0);
                row_store16<S>(rr, (uint32_t)c * 32, raw1, 16);
            }
        }
    }
}

// A row's chunks as near to equal blocks of at most 256 threads, whole waves.
static void row_grid(int64_t rows, int64_t chunks, dim3* grid, dim3* block) {
    const int64_t ny = (chunks + 255) / 256;
    *block = dim3((unsigned)(((chunks + ny - 1) / ny + 63) / 64 * 64));
    *grid = dim3((unsigned)rows, (unsigned)ny);
}

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream) {
    dim3 grid, block;
    row_grid(a.T, a.K / 8, &grid, &block);
    if (past_caches(2 * a.K * a.at.R)) hipLaunchKernelGGL((dispatch_rows_kernel<1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((dispatch_rows_kernel<0>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <int S> static void dispatch_codes(const DispatchArgs& a, int copy, hipStream_t stream) {
    dim3 grid, block;
    row_grid(a.T + (a.out.packed ? (4 - a.at.R % 4) % 4 : 0), a.K / 16, &grid, &block);
    if (copy) hipLaunchKernelGGL((dispatch_codes_kernel<-1, S>), grid, block, 0, stream, a);
    else if (a.out.qtype == Q_FP8) hipLaunchKernelGGL((dispatch_codes_kernel<Q_FP8, S>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((dispatch_codes_kernel<Q_INT8, S>), grid, block, 0, stream, a);
}
hipError_t launch_dispatch_codes(const DispatchArgs& a, hipStream_t stream) {
    const int copy = a.x_scales != nullptr;
    if (past_caches(a.K * a.at.R)) dispatch_codes<1>(a, copy, stream);
    else dispatch_codes<0>(a, copy, stream);
    return hipGetLastError();
}

// ---------------------------------------------------------------------- combine ----

// NB rows in flight a thread. CK: -1, or the code type of the rows' checkpoint: 16 lanes hold a
// group, and lane k of them stores the scale of the batch's k-th row.
template <int RK, int CK, int NB, int S>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs p) {
    const int64_t t = blockIdx.x, K = p.K;
    const int lane = threadIdx.x & 63;
    const uint32_t c = blockIdx.y * blockDim.x + threadIdx.x;
    const uint32_t row_bytes = (uint32_t)(K * RowChunk<RK, S>::size), out_bytes = (uint32_t)(K * type_size(p.out_type));
    const int place = pair_place(p.at, t, lane);
    const float weight = p.weights && lane < p.at.topk ? p.weights[t * p.at.topk + lane] : 1.f;
    float y[8];
    {
        const __amdgpu_buffer_rsrc_t rb = pair_row(p.base, t, out_bytes);
        if (p.out_type == O_FP32) { RowChunk<R_FP32, S> b; b.load(rb, c); b.get(y); }
        else if (p.out_type == O_BF16) { RowChunk<R_BF16, S> b; b.load(rb, c); b.get(y); }
        else { RowChunk<R_FP16, S> b; b.load(rb, c); b.get(y); }
    }
    for (int j0 = 0; j0 < p.at.topk; j0 += NB) {
        RowChunk<RK, S> v[NB];
        int r[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            r[i] = __builtin_amdgcn_readlane(place, (j0 + i) & 63);      // past topk: -1
            v[i].load(pair_row(p.rows, r[i], row_bytes), c);
        }
        float scale = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float x[8];
            v[i].get(x);
            const float w = r[i] >= 0 ? lane_f32(weight, (j0 + i) & 63) : 0.f;
            if constexpr (CK >= 0) {
                const uint32_t mx = max16(amax8(x));
                const float s = group_scale<CK>(mx, p.ckpt_eps, 0);
                row_store8<S>(pair_row(p.ckpt, r[i], (uint32_t)K), c * 8, encode8_group<CK>(x, mx, s));
                if ((lane & 15) == i) scale = s;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __builtin_fmaf(w, x[k], y[k]);
        }
        if constexpr (CK >= 0) {
            const int rs = __shfl(place, (j0 + (lane & 15)) & 63, 64);
            if ((lane & 15) < NB && rs >= 0 && j0 + (lane & 15) < p.at.topk && (int64_t)c * 8 < K)
                p.ckpt_scales[(int64_t)rs * (K / 128) + (c >> 4)] = scale;
        }
    }
    row_store<S>(pair_row(p.out, t, out_bytes), c, p.out_type, y);
}

template <int RK, int CK, int NB> static void combine_s(const CombineArgs& a, hipStream_t stream) {
    dim3 grid, block;
    row_grid(a.T, a.K / 8, &grid, &block);
    if (past_caches(2 * a.T * a.K + (CK >= 0 ? a.at.R * a.K : 0)))
        hipLaunchKernelGGL((combine_kernel<RK, CK, NB, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((combine_kernel<RK, CK, NB, 0>), grid, block, 0, stream, a);
}
template <int RK> static void combine_rk(const CombineArgs& a, hipStream_t stream) {
    if (a.ckpt) {
        if (a.ckpt_type == Q_FP8) combine_s<RK, Q_FP8, 8>(a, stream);
        else combine_s<RK, Q_INT8, 8>(a, stream);
    } else if (a.at.topk <= 2) combine_s<RK, -1, 2>(a, stream);
    else if (a.at.topk <= 4) combine_s<RK, -1, 4>(a, stream);
    else combine_s<RK, -1, 8>(a, stream);
}
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
    if (a.rows_type == O_BF16) combine_rk<R_BF16>(a, stream);
    else if (a.rows_type == O_FP16) combine_rk<R_FP16>(a, stream);
    else combine_rk<R_FP32>(a, stream);
    return hipGetLastError();
}

// A workgroup takes a token's whole row, because the weights' gradients are sums over it; eight pairs
// at a time, their rows in flight together. The codes of w * dout come from one maximum for all
// pairs: rounding is monotone, so the largest |w * dout| is |w| times the largest |dout|, rounded.
template <int RK, int Q, int S>
__global__ __launch_bounds__(512) void combine_bwd_kernel(CombineBwdArgs p) {
    constexpr int NB = 8;
    typedef RowChunk<RK == R_NONE ? (int)R_BF16 : RK, S> Chunk;
    const int64_t t = blockIdx.x, K = p.K, G = K / 128;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __shared__ float part[8][NB];
    if constexpr (Q >= 0) {
        if (t >= p.T) {                                  // uniform: a padding row of packed words
            for (int64_t w = tid; w < (G + 3) / 4; w += blockDim.x) p.out.scales[w * p.out.stride_g + p.at.R + (t - p.T)] = 0.f;
            return;
        }
    }
    const uint32_t row_bytes = (uint32_t)(K * Chunk::size);
    const int place = pair_place(p.at, t, lane);
    const float weight = p.weights && lane < p.at.topk ? p.weights[t * p.at.topk + lane] : 1.f;
    const __amdgpu_buffer_rsrc_t rd = pair_row(p.dout, t, (uint32_t)(K * (p.dout_f32 ? 4 : 2)));
    for (int j0 = 0; j0 < p.at.topk; j0 += NB) {
        float acc[NB];
        int r[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            acc[i] = 0.f;
            r[i] = __builtin_amdgcn_readlane(place, (j0 + i) & 63);
        }
        for (uint32_t c0 = 0; c0 < (uint32_t)(K / 8); c0 += blockDim.x) {
            const uint32_t c = c0 + tid;
            const bool live = (int64_t)c * 8 < K;
            float d[8];
            Chunk v[NB];
            float sv[NB];
            if constexpr (RK != R_NONE) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    v[i].load(pair_row(p.rows, r[i], row_bytes), c);
                    if constexpr (Chunk::codes) sv[i] = buf_f32(pair_row(p.rows_scales, r[i], (uint32_t)(4 * G)), (c >> 4) * 4, 0);
                }
            }
            if (p.dout_f32) { RowChunk<R_FP32, 0> b; b.load(rd, c); b.get(d); }
            else { RowChunk<R_BF16, 0> b; b.load(rd, c); b.get(d); }
            uint32_t md = 0;
            if constexpr (Q >= 0) md = max16(amax8(d));
            float scale = 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                if (r[i] < 0) continue;                  // uniform
                const float w = lane_f32(weight, (j0 + i) & 63);
                if constexpr (RK != R_NONE) {
                    float x[8], s = 0.f;
                    v[i].get(x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) s = __builtin_fmaf(d[k], x[k], s);
                    acc[i] += Chunk::codes ? s * sv[i] : s;
                }
                float z[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) z[k] = w * d[k];
                if (p.d_rows) row_store<S>(pair_row(p.d_rows, r[i], (uint32_t)(2 * K)), c, O_BF16, z);
                if constexpr (Q >= 0) {
                    uint32_t mx = __float_as_uint(w * __uint_as_float(md)) & 0x7FFFFFFFu;
                    if (mx >= 0x7F800000u) mx = max16(amax8(z));          // the 16 lanes of a group agree
                    const float s = group_scale<Q>(mx, p.out.eps, p.out.ue8m0);
                    row_store8<S>(pair_row(p.out.q, r[i], (uint32_t)K), c * 8, encode8_group<Q>(z, mx, s));
                    if ((lane & 15) == i) scale = s;
                }
            }
            if constexpr (Q >= 0) {
                const int rs = __shfl(place, (j0 + (lane & 15)) & 63, 64);
                if ((lane & 15) < NB && rs >= 0 && j0 + (lane & 15) < p.at.topk && live)
                    put_scale(p.out, rs, c >> 4, G, scale);
            }
        }
        if constexpr (RK != R_NONE) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const float s = wave_sum(acc[i]);
                if (lane == i) part[wave][i] = s;
            }
            lds_barrier();
            if (tid < NB && j0 + tid < p.at.topk) {
                float s = 0.f;
                for (int w = 0; w < (int)blockDim.x / 64; ++w) s += part[w][tid];
                p.d_weights[t * p.at.topk + j0 + tid] = s;
            }
            lds_barrier();
        }
    }
}

template <int RK, int Q> static void combine_bwd_s(const CombineBwdArgs& a, hipStream_t stream) {
    const int64_t chunks = a.K / 8, rounds = (chunks + 511) / 512;
    const dim3 block((unsigned)(((chunks + rounds - 1) / rounds + 63) / 64 * 64));
    const dim3 grid((unsigned)(a.T + (Q >= 0 && a.out.packed ? (4 - a.at.R % 4) % 4 : 0)));
    if (past_caches(a.at.R * a.K * ((a.d_rows ? 2 : 0) + (Q >= 0 ? 1 : 0))))
        hipLaunchKernelGGL((combine_bwd_kernel<RK, Q, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((combine_bwd_kernel<RK, Q, 0>), grid, block, 0, stream, a);
}
template <int RK> static void combine_bwd_rk(const CombineBwdArgs& a, hipStream_t stream) {
    if (!a.out.q) combine_bwd_s<RK, -1>(a, stream);
    else if (a.out.qtype == Q_FP8) combine_bwd_s<RK, Q_FP8>(a, stream);
    else combine_bwd_s<RK, Q_INT8>(a, stream);
}
hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t stream) {
    switch (a.d_weights ? a.row_kind : R_NONE) {
        case R_NONE: combine_bwd_rk<R_NONE>(a, stream); break;
        case R_BF16: combine_bwd_rk<R_BF16>(a, stream); break;
        case R_FP16: combine_bwd_rk<R_FP16>(a, stream); break;
        case R_FP32: combine_bwd_rk<R_FP32>(a, stream); break;
        case R_FP8: combine_bwd_rk<R_FP8>(a, stream); break;
        default: combine_bwd_rk<R_INT8>(a, stream); break;
    }
    return hipGetLastError();
}

}  // namespace bfq
