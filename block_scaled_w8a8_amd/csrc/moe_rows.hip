// Rows of a mixture-of-experts layer: the (token, expert) pairs sorted by expert, the tokens' rows
// laid out in that order (dispatch), and the experts' rows back to their tokens with the router's
// weights (combine), with the gradients. The combine without weights is the dispatch's gradient.
//
//   rows[r(t, j)] = x[t]                                            dispatch, as bf16 or codes
//   out[t] = base[t] + sum_j w[t][j] rows[r(t, j)]                  combine
//   d_rows[r(t, j)] = w[t][j] dout[t],  dw[t][j] = <dout[t], rows[r(t, j)]>
//
// All but the sort are bound by bytes. A workgroup takes a token, not a row: what belongs to the
// token (its row, its codes) is read and formed once and written topk times, or topk rows are read
// and summed in registers in pair order: no atomics, equal calls give equal bits. In the combine's
// gradient a workgroup takes two, four or eight of a token's pairs, and each reads the token's gradient.
#include "row_access.h"

namespace bfq {

// ------------------------------------------------------------------------- sort ----
// A stable counting sort. Every workgroup places its share of the pairs; what lies before them in other
// shares it takes from the histograms of an earlier launch (at most 256 of E + 1 counts, from L2), or, up
// to kSortAlone pairs, counts itself: reading all ids again costs less than a launch. Latency bounds it:
// 6216 pairs 5.4 us in one launch, 65536 pairs of 256 experts 8.9 us in two (32768: 9.3 in one, and more
// where a router has collapsed onto one expert, whose counts follow one another).

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kSortGroups = 256;
constexpr int64_t kSortAlone = 8192;

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

// Inclusive prefix over the wave, through DPP (row_shr within 16 lanes, row_bcast across them).
__device__ __forceinline__ int32_t wave_prefix(int32_t x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    return x + __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
}

// Counts a wave's buckets in LDS. Additions to one address follow one another, so the pairs of no expert
// here, most of them where several GPUs share the experts, are one addition (6216 pairs, three quarters of
// them elsewhere: 8.0 -> 5.4 us).
__device__ __forceinline__ void count_buckets(int32_t* hist, bool in, int b, int E) {
    const uint64_t none = __ballot(in && b == E);
    if (in && b < E) atomicAdd(&hist[b], 1);
    else if (in && __builtin_ctzll(none) == (threadIdx.x & 63)) atomicAdd(&hist[E], __builtin_popcountll(none));
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ ids, int64_t pairs,
                                                                  int64_t share, int E,
                                                                  int32_t* __restrict__ counts) {
    __shared__ int32_t hist[1024];                       // E + 1 <= 1024
    for (int b = threadIdx.x; b <= E; b += kSortThreads) hist[b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * share, hi = lo + share < pairs ? lo + share : pairs;
    for (int64_t q0 = lo; q0 < hi; q0 += kSortThreads) {
        const int64_t q = q0 + threadIdx.x;
        count_buckets(hist, q < hi, q < hi ? sort_bucket(ids[q], E) : 0, E);
    }
    __syncthreads();
    for (int b = threadIdx.x; b <= E; b += kSortThreads) counts[(int64_t)blockIdx.x * (E + 1) + b] = hist[b];
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t* __restrict__ ids, int64_t pairs,
                                                                  int64_t share, int E,
                                                                  const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ sorted,
                                                                  int32_t* __restrict__ pair_rows) {
    __shared__ int32_t base[1024], prior[1024], sums[kSortWaves];
    __shared__ uint16_t wave_counts[kSortWaves][1024];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = E + 1, G = gridDim.x, g = blockIdx.x;
    const int64_t lo = g * share, hi = lo + share < pairs ? lo + share : pairs;
    // pairs of bucket `tid` in all, and in earlier shares
    int32_t total = 0, before = 0;
    if (!counts) {
        base[tid] = prior[tid] = 0;
        __syncthreads();
        constexpr int rounds = kSortAlone / kSortThreads;
        const int n = (int)pairs;
        int id[rounds];                                  // loads in flight together
#pragma unroll
        for (int i = 0; i < rounds; ++i) id[i] = ids[min(i * kSortThreads + tid, n - 1)];
#pragma unroll
        for (int i = 0; i < rounds; ++i)                 // a round lies within a share
            count_buckets(i * kSortThreads < lo ? prior : base, i * kSortThreads + tid < n, sort_bucket(id[i], E), E);
        __syncthreads();
        before = prior[tid];
        total = before + base[tid];
    } else if (tid < B) {
#pragma unroll 8
        for (int i = 0; i < G; ++i) {
            const int32_t c = counts[(int64_t)i * B + tid];
            before += i < g ? c : 0;
            total += c;
        }
    }
    // exclusive prefix over the buckets
    const int32_t inc = wave_prefix(total);
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    const int32_t earlier = __builtin_amdgcn_readlane(wave_prefix(lane < wave ? sums[lane] : 0), 63);
    const int32_t first = earlier + inc - total;
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
        for (int i = lane; 2 * i < B; i += 64) reinterpret_cast<uint32_t*>(wave_counts[wave])[i] = 0;   // its own
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
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
    return pairs > kSortAlone ? (size_t)G * (size_t)(E + 1) * sizeof(int32_t) : 0;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t pairs, int E, int32_t* offsets, int32_t* sorted,
                           int32_t* pair_rows, int32_t* counts, hipStream_t stream) {
    const int64_t G = sort_groups(pairs), share = sort_share(pairs);
    if (G == 0) {
        hipLaunchKernelGGL(sort_empty_kernel, dim3(1), dim3(1024), 0, stream, E, offsets);
        return hipGetLastError();
    }
    if (pairs > kSortAlone) {
        hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)G), dim3(kSortThreads), 0, stream, ids, pairs, share, E,
                           counts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(sort_place_kernel, dim3((unsigned)G), dim3(kSortThreads), 0, stream, ids, pairs, share, E,
                       pairs > kSortAlone ? counts : nullptr, offsets, sorted, pair_rows);
    return hipGetLastError();
}

// --------------------------------------------------------------------- dispatch ----

// Rows as they are: eight columns a thread (4096 x 7168 to eight rows each: 529 MB in 109 us, 4.9 TB/s).
template <int S>
__global__ __launch_bounds__(256) void dispatch_rows_kernel(DispatchArgs p) {
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63;
    const uint32_t voff = (blockIdx.y * blockDim.x + threadIdx.x) * 16, bytes = (uint32_t)(2 * p.K);
    const int place = pair_place(p.at, t, lane);
    if (!__ballot(place >= 0)) return;                   // uniform: a token of other GPUs' experts
    const v4u v = row_load16<S>(pair_row(p.x, t, bytes), voff);
    for (int j = 0; j < p.at.topk; ++j) {
        const int r = __builtin_amdgcn_readlane(place, j);
        if (r >= 0) row_store16<S>(pair_row(p.rows, r, bytes), voff, v);
    }
}

// Codes of a token's row, formed or copied (Q < 0) once and written to each of its rows: 16 columns
// a thread, so 8 lanes hold a group and every lane knows its scale; lane k of the group stores the
// scale of pair k, k + 8, ..: one store for eight rows. Packed scales: 32 lanes hold a word. Blocks
// past the tokens write the zero words of rows R .. round_up(R, 4) - 1. Bytes bound it: 4096 x 7168 to
// eight rows each, 301 MB in 61 us (4.9 TB/s; a large copy 4.8 to 5.4) with row-major scales, 69 us with
// column-major ones, whose neighbours belong to other tokens.
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
    if (!__ballot(place >= 0)) return;                   // uniform: a token of other GPUs' experts
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
        mx = group_max<8>(mx);
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
                row_store16<0>(rr, (uint32_t)c * 32, raw0);      // halves of a line: not past the caches
                row_store16<0>(rr, (uint32_t)c * 32, raw1, 16);
            }
        }
    }
}

// A row's chunks as near to equal blocks of at most 256 threads, whole waves. Rows of fewer chunks leave
// lanes idle: 4096 tokens to eight rows each, 256 columns as bf16 5.1 us (3.7 TB/s), as codes 5.5 (2.0); 512:
// 7.6 (5.0) and 6.5 (3.3); 1024: 15.7 (4.8) and 8.8 (4.9).
static void row_grid(int64_t rows, int64_t chunks, dim3* grid, dim3* block) {
    const int64_t ny = (chunks + 255) / 256;
    *block = dim3((unsigned)(((chunks + ny - 1) / ny + 63) / 64 * 64));
    *grid = dim3((unsigned)rows, (unsigned)ny);
}

// Stores past the caches go by R, the rows that there may be, because the rows that are written are known
// on the GPU alone. Where a GPU holds a share of the experts and R is one row a pair, ordinary stores would
// be faster. 7168 columns, 8 pairs a token, codes copied, ordinary | past the caches: all pairs here 777
// tokens 10.0 | 11.2 us, a quarter 4.9 | 5.5, an eighth 3.8 | 4.4, an eighth of 4096 tokens 10.2 | 13.8. With the grouped
// GEMM that reads them (4096 outputs) the two are alike: 777 tokens, a quarter 220 | 217, an eighth 209 | 205.
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
// group, and lane k of them stores the scale of the batch's k-th row. Bytes bound it: 4096 x 7168, eight
// rows each and a base, 588 MB in 113 us (5.2 TB/s, a large copy's rate), with the checkpoint 830 MB in
// 163 us (5.1); one token 2.9 us. fp32 rows to bf16 without a base 999 MB in 196 us (5.1), 2048 tokens with
// the checkpoint 617 MB in 114 us (5.4). 4096 tokens of 256 columns 4.5 us (4.2), of 512 7.5 (5.0).
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
template <int RK, int CK> static void combine_nb(const CombineArgs& a, hipStream_t stream) {
    if (a.at.topk <= 2) combine_s<RK, CK, 2>(a, stream);
    else if (a.at.topk <= 4) combine_s<RK, CK, 4>(a, stream);
    else combine_s<RK, CK, 8>(a, stream);
}
template <int RK> static void combine_rk(const CombineArgs& a, hipStream_t stream) {
    if (!a.ckpt) combine_nb<RK, -1>(a, stream);
    else if (a.ckpt_type == Q_FP8) combine_nb<RK, Q_FP8>(a, stream);
    else combine_nb<RK, Q_INT8>(a, stream);
}
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
    if (a.rows_type == O_BF16) combine_rk<R_BF16>(a, stream);
    else if (a.rows_type == O_FP16) combine_rk<R_FP16>(a, stream);
    else combine_rk<R_FP32>(a, stream);
    return hipGetLastError();
}

// Eight values of a row through its address (for a row that exists), S: the non-temporal hint.
template <int S, typename V> __device__ __forceinline__ V stream_load(const void* p) {
    if constexpr (S) return __builtin_nontemporal_load(static_cast<const V*>(p));
    else return *static_cast<const V*>(p);
}
template <int S, typename V> __device__ __forceinline__ void stream_store(void* p, const V& v) {
    if constexpr (S) __builtin_nontemporal_store(v, static_cast<V*>(p));
    else *static_cast<V*>(p) = v;
}

// What a thread loads of a row at once.
template <int BYTES> struct Load { typedef v4u type; };
template <> struct Load<8> { typedef unsigned int type __attribute__((ext_vector_type(2))); };

// A scalar that the compiler takes for a new one: what is formed from it is formed where it stands, not
// ahead of the loop for all rows at once, which the scalar registers have no room for.
__device__ __forceinline__ int here(int x) {
    asm volatile("" : "+s"(x));
    return x;
}

// A workgroup takes a token's whole row, because the weights' gradients are sums over it; NB pairs
// at a time, their rows in flight together. The codes of w * dout come from one maximum for all
// pairs: rounding is monotone, so the largest |w * dout| is |w| times the largest |dout|, rounded.
// Columns of a thread: 16 where rows of codes are read and written (16-byte loads and stores), else 8. A pair
// without a row reads that of another (which is in the caches) and writes nothing: the loads of a
// batch have no branch between them. Bytes bound it: 4096 x 7168, eight pairs, codes in and out, 543 MB
// in 107 to 113 us (4.8 to 5.1 TB/s; a large copy 5.2). Rows through buffer resources, eight times four
// scalar registers that spilled, 8 columns a thread: 142 us; scalar bases and 16 columns, 448 threads
// a token: 121; at most 256 threads, two rounds a row and more tokens on a CU: 107 (192: 114, 128: 114,
// 64: 108). fp32 rows to bf16 1468 MB in 288 us (5.1), to codes 2048 tokens 617 MB in 128 us (4.8). Narrow rows
// leave lanes idle: 4096 tokens of 256 columns, codes 15.2 us (1.3 TB/s), bf16 8.9 (4.0); 512: 17.0 (2.3) and 12.9 (5.5). The block depends on the width and the types alone: a token's sums do not depend on T.
template <int RK, int Q, int NB, int S>
__global__ __launch_bounds__(256) void combine_bwd_kernel(CombineBwdArgs p) {
    constexpr int U = (RK == R_FP8 || RK == R_INT8) && Q >= 0 ? 2 : 1, W = 8 * U, LG = 16 / U;   // lanes of a group
    typedef RowChunk<RK == R_NONE ? (int)R_BF16 : RK, S> Chunk;
    typedef unsigned int v2u __attribute__((ext_vector_type(2)));
    const int64_t t = blockIdx.x, K = p.K, G = K / 128;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __shared__ float part[4][NB];
    if constexpr (Q >= 0) {
        if (t >= p.T) {                                  // uniform: a padding row of packed words
            if (blockIdx.y != 0) return;
            for (int64_t w = tid; w < (G + 3) / 4; w += blockDim.x) p.out.scales[w * p.out.stride_g + p.at.R + (t - p.T)] = 0.f;
            return;
        }
    }
    const int place = pair_place(p.at, t, lane);
    const uint64_t there = __ballot(place >= 0);         // bit j: pair j has a row
    const float weight = p.weights && lane < p.at.topk ? p.weights[t * p.at.topk + lane] : 1.f;
    const uint32_t chunks = (uint32_t)(K / W);
    for (int j0 = blockIdx.y * NB; j0 < p.at.topk; j0 += gridDim.y * NB) {
        const uint32_t alive = (uint32_t)(there >> j0) & ((1u << NB) - 1);
        float acc[NB], w[NB];
        int r[NB];
        // lane k of a group stores pair k's scale (taken here, where every lane of the wave takes part, as the
        // pairs' rows and weights are: below, lanes past the row's end are switched off, and what a register
        // holds for such a lane is the compiler's to lose)
        const int k = lane & (LG - 1), rs = __shfl(place, (j0 + k) & 63, 64);
        const int some = alive ? __builtin_amdgcn_readlane(place, j0 + __builtin_ctz(alive)) : 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            acc[i] = 0.f;
            r[i] = (alive >> i) & 1 ? __builtin_amdgcn_readlane(place, (j0 + i) & 63) : some;
            w[i] = lane_f32(weight, (j0 + i) & 63);
        }
        for (uint32_t c0 = 0; alive && c0 < chunks; c0 += blockDim.x) {
            const uint32_t c = c0 + tid;
            if (c >= chunks) continue;                   // whole groups: K is a multiple of 128 with codes
            float d[W];
            typename Load<Chunk::size * W>::type v[NB][RK == R_FP32 ? 2 : 1];
            float sv[NB];
            if constexpr (RK != R_NONE) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int64_t ri = here(r[i]);
                    const uint8_t* row = static_cast<const uint8_t*>(p.rows) + ri * (K * Chunk::size);
                    const uint32_t at = c * (W * Chunk::size);
                    v[i][0] = stream_load<S, typename Load<Chunk::size * W>::type>(row + at);
                    if constexpr (RK == R_FP32) v[i][1] = stream_load<S, v4u>(row + at + 16);
                    if constexpr (Chunk::codes) sv[i] = (p.rows_scales + ri * G)[c / LG];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p.dout_f32) {
                    const uint8_t* row = static_cast<const uint8_t*>(p.dout) + t * (4 * K);
                    const v4f a = stream_load<0, v4f>(row + c * (4 * W) + 32 * u), b = stream_load<0, v4f>(row + c * (4 * W) + 32 * u + 16);
#pragma unroll
                    for (int n = 0; n < 4; ++n) { d[8 * u + n] = a[n]; d[8 * u + 4 + n] = b[n]; }
                } else {
                    const v4u a = stream_load<0, v4u>(static_cast<const uint8_t*>(p.dout) + t * (2 * K) + c * (2 * W) + 16 * u);
                    unpack8(make_uint4(a.x, a.y, a.z, a.w), d + 8 * u);
                }
            }
            uint32_t md = 0;
            if constexpr (Q >= 0) md = group_max<LG>(U == 2 ? max(amax8(d), amax8(d + W - 8)) : amax8(d));
            float scale = 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                if (!((alive >> i) & 1)) continue;       // uniform
                const int64_t ri = here(r[i]);
                if constexpr (RK != R_NONE) {
                    float s = 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float x[8];
                        Chunk chunk;
                        if constexpr (U == 2) chunk.a = u ? v4u{v[i][0].z, v[i][0].w, 0, 0} : v[i][0];
                        else if constexpr (Chunk::codes) chunk.a = v4u{v[i][0].x, v[i][0].y, 0, 0};
                        else chunk.a = v[i][0];
                        if constexpr (RK == R_FP32) chunk.b = v[i][1];
                        chunk.get(x);
#pragma unroll
                        for (int n = 0; n < 8; ++n) s = __builtin_fmaf(d[8 * u + n], x[n], s);
                    }
                    acc[i] += Chunk::codes ? s * sv[i] : s;
                }
                float z[W];
#pragma unroll
                for (int n = 0; n < W; ++n) z[n] = w[i] * d[n];
                if (p.d_rows) {
                    uint8_t* row = static_cast<uint8_t*>(p.d_rows) + ri * (2 * K);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint4 b = pack8(z + 8 * u);
                        // halves of a line leave together: not past the caches
                        stream_store<U == 2 ? 0 : S>(row + c * (2 * W) + 16 * u, v4u{b.x, b.y, b.z, b.w});
                    }
                }
                if constexpr (Q >= 0) {
                    uint32_t mx = __float_as_uint(w[i] * __uint_as_float(md)) & 0x7FFFFFFFu;
                    if (mx >= 0x7F800000u)               // the lanes of a group agree
                        mx = group_max<LG>(U == 2 ? max(amax8(z), amax8(z + W - 8)) : amax8(z));
                    const float s = group_scale<Q>(mx, p.out.eps, p.out.ue8m0);
                    uint8_t* row = static_cast<uint8_t*>(p.out.q) + ri * K;
                    const uint2 lo = encode8_group<Q>(z, mx, s);
                    if constexpr (U == 2) {
                        const uint2 hi = encode8_group<Q>(z + W - 8, mx, s);
                        stream_store<S>(row + c * W, v4u{lo.x, lo.y, hi.x, hi.y});
                    } else {
                        stream_store<S>(row + c * W, v2u{lo.x, lo.y});
                    }
                    if (k == i) scale = s;
                }
            }
            if constexpr (Q >= 0) {
                if (k < NB && (alive >> k) & 1) put_scale(p.out, rs, c / LG, G, scale);
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

template <int RK, int Q, int NB> static void combine_bwd_nb(const CombineBwdArgs& a, unsigned ys, hipStream_t stream) {
    const int64_t chunks = a.K / ((RK == R_FP8 || RK == R_INT8) && Q >= 0 ? 16 : 8), rounds = (chunks + 255) / 256;
    const dim3 block((unsigned)(((chunks + rounds - 1) / rounds + 63) / 64 * 64));
    const dim3 grid((unsigned)(a.T + (Q >= 0 && a.out.packed ? (4 - a.at.R % 4) % 4 : 0)), ys);
    if (past_caches(a.at.R * a.K * ((a.d_rows ? 2 : 0) + (Q >= 0 ? 1 : 0))))
        hipLaunchKernelGGL((combine_bwd_kernel<RK, Q, NB, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((combine_bwd_kernel<RK, Q, NB, 0>), grid, block, 0, stream, a);
}
// Pairs at a time, and with them the workgroups a token gets: each reads the token's gradient again, and more
// of them fill the card where tokens are few. 7168 columns, rows and codes of 8 bits, 2 | 4 | 8 at a time:
// 8 pairs a token, 300 tokens 13.5 | 15.5 us, 500: 20.1 | 18.6, 1100: 40.2 | 36.8 | 40.8, 2000: 67 | 58.9 | 58.5,
// 4096: 130 | 110.6 | 109.4; 4 pairs a token, 600 tokens 13.4 | 15.6, 1100: 21.9 | 19.9, 4096: 68.6 | 59.9 | 70.6.
// Without the weights' gradient 8192 tokens of 8 pairs: 162 | 146 | 141; rows or output in bf16 take 4 or 8 alike
// (4096 tokens, bf16 in, codes out: 153 | 150 | 153). A pair's sum is the same in each.
// The rule counts T * topk pairs, absent ones too, and no columns; what it takes (marked) is at most 10 % behind
// the fastest at other widths, from bf16 to bf16 14 %. 8 pairs a token, codes: 512 columns, 300 tokens 4.5* | 5.5 | 8.4 us, 1100: 7.2 | 7.8* |
// 10.0, 4096: 17.5 | 16.3 | 17.6*; 1536 columns, 300: 5.5* | 6.7 | 9.8, 500: 6.9 | 7.5* | 10.6, 1100: 12.4 | 12.7* | 15.0,
// 4096: 37.3 | 31.9 | 32.0*; 16384 columns, 300: 23.9* | 25.9 | 33.0, 500: 37.8 | 32.7* | 38.2, 1100: 72.9 | 67.1* | 76.2,
// 4096: 253 | 242 | 253*. An eighth of the pairs here, 7168 columns: 500 tokens 8.7 | 9.5* | 10.6, 1100: 15.2 | 14.4* |
// 15.4, 4096: 41.4 | 36.7 | 38.3*. bf16 to bf16, 1536 columns: 500 tokens 7.5 | 7.9* | 9.0, 2000: 22.2 | 22.7* | 20.0.
template <int RK, int Q> static void combine_bwd_s(const CombineBwdArgs& a, hipStream_t stream) {
    const int64_t pairs = a.T * a.at.topk;
    if (a.at.topk <= 2 || pairs < 3600) combine_bwd_nb<RK, Q, 2>(a, (a.at.topk + 1) / 2, stream);
    else {
        if constexpr (Q >= 0 && (RK == R_FP8 || RK == R_INT8 || RK == R_NONE))
            if (a.at.topk > 4 && pairs >= 24000) return combine_bwd_nb<RK, Q, 8>(a, 1, stream);
        combine_bwd_nb<RK, Q, 4>(a, (a.at.topk + 3) / 4, stream);
    }
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
