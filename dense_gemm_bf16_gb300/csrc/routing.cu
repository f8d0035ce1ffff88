// Tokens to their experts' rows and back (gemm_expert_dispatch, gemm_expert_combine,
// gemm_expert_combine_grad), kernels and entry points.
//
//   dispatch      the pairs (t, j) with an expert, in the order of (expert, t, j), get the
//                 rows 0, 1, ...:  slots[t, j] = row, rows[slots[t, j]] = x[t]
//   combine       y[t] = sum_j w[t, j] rows[slots[t, j]]
//   combine_grad  d_rows[slots[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], rows[slots[t, j]]>
//
// All three are bound by the bytes they move, so each row is read once and written once:
// dispatch walks tokens, not rows (a token is read once and stored `top` times), and the
// gradient makes both of its results from one reading of dy.
//
// The sort is a counting sort over (expert, position), so it is stable and repeats.  Every
// block owns a range of tokens.  For a rank it needs how many pairs of each expert come
// before its range, and for the experts' offsets how many there are in all: with few pairs
// each block counts all of them itself (one launch), with many a first launch leaves each
// range's counts in the workspace and the blocks add those up.  Inside its range a block
// gives every warp a segment; the warp counts and later ranks 32 pairs at a time by
// matching lanes with equal experts, so no order depends on an atomic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "epilogue.cuh"
#include "experts_host.h"
#include "gemm_experts.h"
#include "ptx.cuh"

namespace dg {
namespace {

// ---------------------------------------------------------------- dispatch

constexpr int kRouteThreads = 1024;
constexpr int kRouteBlocks = 304;       // ranges at most (two for each of 152 SMs)
constexpr int kRouteGroups = 4096;      // experts: their counts fit 48 KB of shared memory
constexpr int kRouteInts = 12288;       // ... that many
// Pairs that every block counts by itself; more go through the first launch.
constexpr int64_t kRouteOnePass = 4096;
// Units of a token's row that a thread copies at once where they are less than 16 bytes (16384
// tokens x 4 of 2049, bf16: one 171 us, four 133, eight 106; 16 bytes at a time from shared memory
// 101, but 7.5 against 5.5 for 48 tokens).
__host__ __device__ constexpr int route_apart(int unit) { return unit < 16 ? 8 : 1; }

struct DispatchParams {
    const void* ids;
    int64_t ld_ids;
    int32_t T, top, groups;
    const char* x;
    int64_t x_pitch;        // bytes
    const float* scales;    // or null
    char* rows;
    int64_t rows_pitch;
    float* row_scales;
    int32_t* offsets;
    int32_t* slots;
    int32_t* hist;          // [blocks][groups] of the first launch, or null
    int32_t vecs;           // units of the copy in a row
    int32_t tpt_log2;       // threads that share a token's row
    int32_t warps;          // segments of a block's range
    int32_t ahead;          // tokens of a range that are prefetched
    int* status;
};

// Expert of pair i; negative: none (-2: an id past the last expert).
template <typename ID>
__device__ __forceinline__ int route_id(const DispatchParams& p, int64_t i) {
    const int64_t t = p.ld_ids == p.top ? 0 : i / p.top;
    const ID v = static_cast<const ID*>(p.ids)[p.ld_ids == p.top ? i : t * p.ld_ids + (i - t * p.top)];
    return v < 0 ? -1 : (v >= static_cast<ID>(p.groups) ? -2 : static_cast<int>(v));
}

__device__ __forceinline__ int64_t route_first(const DispatchParams& p, int block, int blocks) {
    return static_cast<int64_t>(p.T) * block / blocks;
}

// Counts of each range.
template <typename ID>
__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const DispatchParams p) {
    extern __shared__ int counts[];
    griddep_launch_dependents();
    for (int e = threadIdx.x; e < p.groups; e += blockDim.x) counts[e] = 0;
    __syncthreads();
    const int b = blockIdx.x, n = gridDim.x;
    const int64_t i1 = route_first(p, b + 1, n) * p.top;
    for (int64_t i = route_first(p, b, n) * p.top + threadIdx.x; i < i1; i += blockDim.x) {
        const int e = route_id<ID>(p, i);
        if (e >= 0) atomicAdd(counts + e, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.groups; e += blockDim.x)
        p.hist[static_cast<int64_t>(b) * p.groups + e] = counts[e];
}

// Offsets, slots and rows.  V: the copy's unit, which divides the rows' size, pitches and
// addresses.
template <typename ID, typename V>
__global__ void __launch_bounds__(kRouteThreads, 1) dispatch_kernel(const DispatchParams p) {
    extern __shared__ int smem[];
    int* before = smem;                  // [groups] first the pairs before this range
    int* total = smem + p.groups;        // [groups] all pairs, then the experts' offsets
    int* counts = smem + 2 * p.groups;   // [warps][groups]
    const int E = p.groups, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x, blocks = gridDim.x;
    const int64_t t0 = route_first(p, b, blocks), t1 = route_first(p, b + 1, blocks);
    const int64_t i0 = t0 * p.top, i1 = t1 * p.top;
    for (int i = tid; i < (2 + p.warps) * E; i += kRouteThreads) smem[i] = 0;
    // this range's tokens are on their way to L2 while their rows are found
    if (sizeof(V) == 16)
        for (int64_t t = t0 + tid; t < t1 && t < t0 + p.ahead; t += kRouteThreads)
            l2_prefetch(p.x + t * p.x_pitch, static_cast<uint32_t>(p.vecs) * 16u);
    __syncthreads();
    if (p.hist) {
        griddep_wait();
        // a thread adds up one expert's counts over some of the ranges
        const int span = E < kRouteThreads ? E : kRouteThreads, sets = kRouteThreads / (span > 0 ? span : 1);
        const int set = span > 0 ? tid / span : sets;
        if (set < sets)
            for (int e = tid - set * span; e < E; e += span) {
                int all = 0, mine = 0;
                for (int r = set; r < blocks; r += sets) {
                    const int v = __ldcg(p.hist + static_cast<int64_t>(r) * E + e);
                    all += v;
                    if (r < b) mine += v;
                }
                atomicAdd(total + e, all);
                atomicAdd(before + e, mine);
            }
    } else {
        const int64_t n = static_cast<int64_t>(p.T) * p.top;
        for (int64_t i = tid; i < n; i += kRouteThreads) {
            const int e = route_id<ID>(p, i);
            if (e < 0) continue;
            atomicAdd(total + e, 1);
            if (i < i0) atomicAdd(before + e, 1);
        }
    }
    // this range's segments: a warp's counts, 32 pairs at a time
    const int64_t seg = ((i1 - i0 + p.warps - 1) / p.warps + 31) & ~int64_t(31);
    const int64_t s0 = i0 + warp * seg < i1 ? i0 + warp * seg : i1;
    const int64_t s1 = s0 + seg < i1 ? s0 + seg : i1;
    int* mine = counts + warp * E;
    if (warp < p.warps) {
        for (int64_t i = s0 + lane; i - lane < s1; i += 32) {
            const int e = i < s1 ? route_id<ID>(p, i) : -1;
            if (e == -2 && p.status) atomicOr(p.status, STATUS_BAD_OFFSETS);
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // offsets: an exclusive sum over the experts
    if (warp == 0) {
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, v = e < E ? total[e] : 0;
            int incl = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            if (e < E) {
                total[e] = run + incl - v;
                if (b == 0) p.offsets[e] = run + incl - v;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (b == 0 && lane == 0) p.offsets[E] = run;
    }
    __syncthreads();
    // the first row of every expert's pairs in each segment
    for (int e = tid; e < E; e += kRouteThreads) {
        int row = total[e] + before[e];
        for (int w = 0; w < p.warps; ++w) {
            const int v = counts[w * E + e];
            counts[w * E + e] = row;
            row += v;
        }
    }
    __syncthreads();
    if (warp < p.warps) {
        for (int64_t i = s0 + lane; i - lane < s1; i += 32) {
            const int e = i < s1 ? route_id<ID>(p, i) : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int row = e >= 0 ? mine[e] + __popc(same & ((1u << lane) - 1u)) : -1;
            __syncwarp();
            if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
            __syncwarp();
            if (i < s1) p.slots[i] = row;
        }
    }
    __syncthreads();
    // the rows: a token is read once and stored once for each of its pairs
    constexpr int W = route_apart(sizeof(V));
    const int tpt = 1 << p.tpt_log2, in = tid & (tpt - 1);
    for (int64_t t = t0 + (tid >> p.tpt_log2); t < t1; t += kRouteThreads >> p.tpt_log2) {
        const int32_t* slot = p.slots + t * p.top;
        const V* src = reinterpret_cast<const V*>(p.x + t * p.x_pitch);
        for (int64_t c = in; c < p.vecs; c += tpt * W) {
            V v[W];
#pragma unroll
            for (int w = 0; w < W; ++w)
                if (w == 0 || c + w * tpt < p.vecs) v[w] = __ldg(src + c + w * tpt);
            for (int j = 0; j < p.top; ++j) {
                const int s = slot[j];
                if (s < 0) continue;
                V* dst = reinterpret_cast<V*>(p.rows + s * p.rows_pitch);
#pragma unroll
                for (int w = 0; w < W; ++w)
                    if (w == 0 || c + w * tpt < p.vecs) dst[c + w * tpt] = v[w];
            }
        }
        if (p.scales && in == 0) {
            const float v = __ldg(p.scales + t);
            for (int j = 0; j < p.top; ++j)
                if (slot[j] >= 0) p.row_scales[slot[j]] = v;
        }
    }
}

template <typename ID, typename V>
cudaError_t dispatch_launch(const DispatchParams& p, int blocks, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kRouteThreads);
    cfg.stream = stream;
    if (p.hist) {
        cfg.dynamicSmemBytes = static_cast<size_t>(p.groups) * 4;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, route_count_kernel<ID>, p);
        if (e != cudaSuccess) return e;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = option_overlap_copy() ? 1 : 0;
    }
    cfg.dynamicSmemBytes = static_cast<size_t>(2 + p.warps) * p.groups * 4;
    return cudaLaunchKernelEx(&cfg, dispatch_kernel<ID, V>, p);
}

template <typename ID>
cudaError_t dispatch_unit(int unit, const DispatchParams& p, int blocks, cudaStream_t stream) {
    switch (unit) {
        case 16: return dispatch_launch<ID, uint4>(p, blocks, stream);
        case 8: return dispatch_launch<ID, uint2>(p, blocks, stream);
        case 4: return dispatch_launch<ID, uint32_t>(p, blocks, stream);
        case 2: return dispatch_launch<ID, uint16_t>(p, blocks, stream);
        default: return dispatch_launch<ID, uint8_t>(p, blocks, stream);
    }
}

// ---------------------------------------------------------------- combine and its gradient

constexpr int kSumThreads = 256;
constexpr int kSumBlocksPerSm = 4;      // all resident at once: no second, partial wave
constexpr int kSumApart = 4;            // pieces of a thread's columns where rows are not aligned

struct CombineParams {
    const int32_t* slots;    // [T][top]
    const void* weights;     // [T][top] of w_dtype, or null: ones
    int64_t ld_w;
    int32_t w_dtype;
    int32_t T, top, K, R;    // R: rows that a slot may name
    const void* rows;        // R x K
    int64_t ld_rows;
    void* y;                 // T x K (combine's result; the gradient's dy)
    int64_t ld_y;
    int32_t y_dtype;         // combine: the rows' type or fp32
    void* d_rows;            // combine_grad
    int64_t ld_drows;
    void* d_weights;         // [T][top] of dw_dtype, or null
    int64_t ld_dw;
    int32_t dw_dtype;
    int32_t tpt_log2;        // threads that share a token
    int* status;
};

// N elements (a power of two, N * size bytes aligned) as fp32.
template <int DT, int N>
struct Pack {
    static constexpr int BYTES = N * (DT == DT_F32 ? 4 : 2);
    using V = std::conditional_t<BYTES == 16, uint4, std::conditional_t<BYTES == 4, uint32_t, uint16_t>>;
};

template <int DT, int N>
__device__ __forceinline__ void unpack(const typename Pack<DT, N>::V& v, float (&f)[N]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (N == 1) {
        if constexpr (DT == DT_BF16)
            f[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
        else
            f[0] = __half2float(__ushort_as_half(v));
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (DT == DT_BF16) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 t = __half22float2(*reinterpret_cast<const __half2*>(w + i));
                f[2 * i] = t.x;
                f[2 * i + 1] = t.y;
            }
        }
    }
}

template <int DT, int N>
__device__ __forceinline__ typename Pack<DT, N>::V pack(const float (&f)[N]) {
    typename Pack<DT, N>::V v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (N == 1) {
        if constexpr (DT == DT_BF16)
            v = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
        else
            v = __half_as_ushort(__float2half_rn(f[0]));
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (DT == DT_BF16) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&t);
            } else {
                const __half2 t = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&t);
            }
        }
    }
    return v;
}

// Row of pair (t, j); negative: none.  A slot past the rows is reported and is none.
__device__ __forceinline__ int combine_slot(const CombineParams& p, int64_t t, int j) {
    const int s = __ldg(p.slots + t * p.top + j);
    if (s < p.R) return s;
    if (p.status) atomicOr(p.status, STATUS_BAD_OFFSETS);
    return -1;
}

__device__ __forceinline__ float combine_weight(const CombineParams& p, int64_t t, int j) {
    if (!p.weights) return 1.0f;
    return load_elem(static_cast<const char*>(p.weights) + (t * p.ld_w + j) * dt_size(p.w_dtype),
                     p.w_dtype);
}

// A pair as the block's threads read it: its row (bytes from the first one, negative: none)
// and weight.
struct alignas(16) CombinePair {
    int64_t row;
    float w;
};
constexpr int kSumPairs = 512;  // pairs that a block holds at once, and choices of a token at most

// The pairs of `n` tokens from t on, by all threads of the block.
__device__ __forceinline__ void combine_pairs(const CombineParams& p, int64_t t, int n, int64_t pitch,
                                              CombinePair* pairs) {
    __syncthreads();  // (the ones before have been read)
    for (int i = threadIdx.x; i < n * p.top; i += kSumThreads) {
        const int64_t tok = t + i / p.top;
        const int j = i % p.top, s = combine_slot(p, tok, j);
        pairs[i].row = s < 0 ? -1 : s * pitch;
        pairs[i].w = s < 0 ? 0.0f : combine_weight(p, tok, j);
    }
    __syncthreads();
}

// N results from element `off` of y on.
template <int DT, int N>
__device__ __forceinline__ void combine_store(const CombineParams& p, int64_t off, const float (&sum)[N]) {
    if (DT != DT_F32 && p.y_dtype == DT_F32) {
        float* dst = static_cast<float*>(p.y) + off;
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4*>(dst + i) =
                    make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) dst[i] = sum[i];
        }
    } else {
        using V = typename Pack<DT, N>::V;
        *reinterpret_cast<V*>(static_cast<char*>(p.y) + off * (DT == DT_F32 ? 4 : 2)) = pack<DT, N>(sum);
    }
}

// A block owns a range of tokens and reads their slots and weights once, some hundred pairs at
// a time (every thread for itself, they were most of the instructions: 16384 tokens x 4 of
// 2048, bf16, 70 us).  A thread takes N neighbouring columns of a token and adds its rows in the
// order of j, in fp32; the next four rows, of this token or the next, are loaded meanwhile.
// Where rows allow no 16 bytes at once it takes W times N columns, a token's threads apart
// (3001 tokens x 6 of 1001, fp16: one column at a time 31 us, two at a time 21, four 17.4; 1002
// columns, two neighbours each: 19 and 12).
template <int DT, int N, int W>
__global__ void __launch_bounds__(kSumThreads, kSumBlocksPerSm) combine_kernel(const CombineParams p) {
    using V = typename Pack<DT, N>::V;
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    __shared__ CombinePair pairs[kSumPairs];
    const int tpt = 1 << p.tpt_log2, in = threadIdx.x & (tpt - 1), mine = threadIdx.x >> p.tpt_log2;
    const int per_block = kSumThreads >> p.tpt_log2;
    const char* rows = static_cast<const char*>(p.rows);
    const int64_t t1 = static_cast<int64_t>(p.T) * (blockIdx.x + 1) / gridDim.x;
    const int batch = kSumPairs / (p.top > 0 ? p.top : 1);
    for (int64_t tb = static_cast<int64_t>(p.T) * blockIdx.x / gridDim.x; tb < t1; tb += batch) {
        const int n = static_cast<int>(t1 - tb < batch ? t1 - tb : batch);
        combine_pairs(p, tb, n, p.ld_rows * ES, pairs);
        // (tokens mine, mine + per_block, ...; of each the columns in * N, ...; of those the
        // pairs by fours)
        int tok = mine, c = in * N, j0 = 0;
        V next[4][W];
        auto load = [&]() {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (j0 + k >= p.top) break;
                const int64_t row = pairs[tok * p.top + j0 + k].row;
                if (row < 0) continue;
                const char* src = rows + row + static_cast<int64_t>(c) * ES;
#pragma unroll
                for (int w = 0; w < W; ++w)
                    if (w == 0 || c + w * tpt * N < p.K)
                        next[k][w] = __ldg(reinterpret_cast<const V*>(src + w * tpt * N * ES));
            }
        };
        bool more = tok < n && c < p.K;
        if (more) load();
        float sum[W][N];
#pragma unroll
        for (int i = 0; i < W * N; ++i) sum[i / N][i % N] = 0.0f;
        while (more) {
            const int at = tok * p.top + j0, left = p.top - j0, col = c;
            const int64_t off = (tb + tok) * p.ld_y + c;
            V v[4][W];
#pragma unroll
            for (int k = 0; k < 4 * W; ++k) v[k / W][k % W] = next[k / W][k % W];
            j0 += 4;
            if (j0 >= p.top) {
                j0 = 0;
                c += tpt * N * W;
                if (c >= p.K) {
                    c = in * N;
                    tok += per_block;
                    more = tok < n;
                }
            }
            if (more) load();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= left) break;
                const CombinePair pair = pairs[at + k];
                if (pair.row < 0) continue;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    float f[N];
                    unpack<DT, N>(v[k][w], f);
#pragma unroll
                    for (int i = 0; i < N; ++i) sum[w][i] = fmaf(pair.w, f[i], sum[w][i]);
                }
            }
            if (left <= 4) {
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (w == 0 || col + w * tpt * N < p.K) combine_store<DT, N>(p, off + w * tpt * N, sum[w]);
#pragma unroll
                    for (int i = 0; i < N; ++i) sum[w][i] = 0.0f;
                }
            }
        }
    }
}

// The gradient's dot products of a token's pairs from j0 on, from its threads' parts.
template <int J>
__device__ __forceinline__ void combine_dots(const CombineParams& p, float (&dot)[J], float (*part)[J],
                                             int64_t t, int j0, bool live) {
    const int warps = 1 << p.tpt_log2 >> 5, in = threadIdx.x & ((1 << p.tpt_log2) - 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < J; ++k)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], d);
    if (warps > 1) {
        __syncthreads();  // (the pairs before have been read)
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < J; ++k) part[warp][k] = dot[k];
        }
        __syncthreads();
        if (in < J) {
            float sum = 0.0f;
            for (int i = 0; i < warps; ++i) sum += part[warp + i][in];
            dot[0] = sum;
        }
    } else {
#pragma unroll
        for (int k = 1; k < J; ++k)
            if (lane == k) dot[0] = dot[k];
    }
    if (live && in < J && j0 + in < p.top)
        store_elem(static_cast<char*>(p.d_weights) + (t * p.ld_dw + j0 + in) * dt_size(p.dw_dtype),
                   p.dw_dtype, dot[0]);
}

// The threads of a token (a warp's worth at least, a block's at most) walk its columns once
// for up to J pairs; their partial dot products meet in shuffles, then in shared memory.
template <int DT, int N, int J>
__global__ void __launch_bounds__(kSumThreads) combine_grad_kernel(const CombineParams p) {
    using V = typename Pack<DT, N>::V;
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    __shared__ CombinePair pairs[kSumPairs];
    __shared__ float part[kSumThreads / 32][J];
    const int tpt = 1 << p.tpt_log2, in = threadIdx.x & (tpt - 1), mine = threadIdx.x >> p.tpt_log2;
    const int per_block = kSumThreads >> p.tpt_log2;
    const char* dy = static_cast<const char*>(p.y);
    const char* rows = static_cast<const char*>(p.rows);
    char* d_rows = static_cast<char*>(p.d_rows);
    const int64_t t1 = static_cast<int64_t>(p.T) * (blockIdx.x + 1) / gridDim.x;
    const int batch = kSumPairs / p.top;
    for (int64_t tb = static_cast<int64_t>(p.T) * blockIdx.x / gridDim.x; tb < t1; tb += batch) {
        const int n = static_cast<int>(t1 - tb < batch ? t1 - tb : batch);
        combine_pairs(p, tb, n, 1, pairs);  // (row numbers: two pitches)
        // (whole blocks walk together: the sums' barriers are the block's)
        for (int t0 = 0; t0 < n; t0 += per_block) {
            const int tok = t0 + mine;
            const int64_t t = tb + tok;
            const bool live = tok < n;
            for (int j0 = 0; j0 < p.top; j0 += J) {
                int64_t s[J];
                float w[J], dot[J];
#pragma unroll
                for (int k = 0; k < J; ++k) {
                    const bool in_range = live && j0 + k < p.top;
                    s[k] = in_range ? pairs[tok * p.top + j0 + k].row : -1;
                    w[k] = in_range ? pairs[tok * p.top + j0 + k].w : 0.0f;
                    dot[k] = 0.0f;
                }
                if (live)
                    for (int c = in * N; c < p.K; c += tpt * N) {
                        V r[J];
                        const V v = *reinterpret_cast<const V*>(dy + (t * p.ld_y + c) * ES);
                        if (p.d_weights) {
#pragma unroll
                            for (int k = 0; k < J; ++k)
                                if (s[k] >= 0)
                                    r[k] = *reinterpret_cast<const V*>(rows + (s[k] * p.ld_rows + c) * ES);
                        }
                        float g[N];
                        unpack<DT, N>(v, g);
#pragma unroll
                        for (int k = 0; k < J; ++k) {
                            if (s[k] < 0) continue;
                            float o[N];
                            if (p.d_weights) {
                                unpack<DT, N>(r[k], o);
#pragma unroll
                                for (int i = 0; i < N; ++i) dot[k] = fmaf(g[i], o[i], dot[k]);
                            }
#pragma unroll
                            for (int i = 0; i < N; ++i) o[i] = w[k] * g[i];
                            *reinterpret_cast<V*>(d_rows + (s[k] * p.ld_drows + c) * ES) = pack<DT, N>(o);
                        }
                    }
                if (p.d_weights) combine_dots<J>(p, dot, part, t, j0, live);
            }
        }
    }
}

// The same for rows on any address.  Units of 16 bytes start where rows and d_rows (alike) have
// their 16-byte boundaries, another column in every row; dy comes to them through shared memory,
// in fp32, a word more for each unit so that neighbouring threads meet no bank twice.  What a row
// has before its first and behind its last whole unit goes to one thread each.  (3001 tokens x 6 of
// 1001, fp16: 23.7 us, 34 with one column at a time and as much with four of them apart; 16384 x
// 4 of 2049, bf16: 147 and 235.  Three barriers and a load's latency for every token of a block's.)
template <int DT, int J>
__global__ void __launch_bounds__(kSumThreads, J > 4 ? 3 : kSumBlocksPerSm)
combine_grad_any_kernel(const CombineParams p) {
    constexpr int ES = DT == DT_F32 ? 4 : 2, N = 16 / ES;
    using V = typename Pack<DT, N>::V;
    using E = typename Pack<DT, 1>::V;
    __shared__ CombinePair pairs[kSumPairs];
    __shared__ float part[kSumThreads / 32][J];
    __shared__ float staged[(kSumThreads + kSumThreads / 32) * (N + 1)];
    const int tpt = 1 << p.tpt_log2, in = threadIdx.x & (tpt - 1), mine = threadIdx.x >> p.tpt_log2;
    const int per_block = kSumThreads >> p.tpt_log2;
    float* dy_at = staged + mine * (tpt + 1) * (N + 1);
    const char* dy = static_cast<const char*>(p.y);
    const char* rows = static_cast<const char*>(p.rows);
    char* d_rows = static_cast<char*>(p.d_rows);
    // columns of a row (K is 16 bytes or more) before its first whole unit
    auto head_of = [&](int64_t row) {
        return static_cast<int>((0 - (reinterpret_cast<uintptr_t>(d_rows) / ES + row * p.ld_drows)) % N);
    };
    const int64_t t1 = static_cast<int64_t>(p.T) * (blockIdx.x + 1) / gridDim.x;
    const int batch = kSumPairs / p.top;
    for (int64_t tb = static_cast<int64_t>(p.T) * blockIdx.x / gridDim.x; tb < t1; tb += batch) {
        const int n = static_cast<int>(t1 - tb < batch ? t1 - tb : batch);
        combine_pairs(p, tb, n, 1, pairs);  // (row numbers: two pitches)
        // (whole blocks walk together: the barriers are the block's)
        for (int t0 = 0; t0 < n; t0 += per_block) {
            const int tok = t0 + mine;
            const int64_t t = tb + tok;
            const bool live = tok < n;
            const char* g_row = dy + t * p.ld_y * ES;
            auto edges = [&](int j0, float (&dot)[J]) {
                for (int i = in; i < J * 2 * N; i += tpt) {
                    const int k = i / (2 * N), at = i % (2 * N);
                    if (!live || j0 + k >= p.top) continue;
                    const CombinePair pair = pairs[tok * p.top + j0 + k];
                    const int head = head_of(pair.row), tail = (p.K - head) % N;
                    if (pair.row < 0 || at >= head + tail) continue;
                    const int c = at < head ? at : p.K - tail + at - head;
                    float g[1], o[1];
                    unpack<DT, 1>(reinterpret_cast<const E*>(g_row)[c], g);
                    if (p.d_weights) {
                        unpack<DT, 1>(reinterpret_cast<const E*>(rows)[pair.row * p.ld_rows + c], o);
#pragma unroll
                        for (int l = 0; l < J; ++l)
                            if (l == k) dot[l] = fmaf(g[0], o[0], dot[l]);
                    }
                    o[0] = pair.w * g[0];
                    reinterpret_cast<E*>(d_rows)[pair.row * p.ld_drows + c] = pack<DT, 1>(o);
                }
            };
            for (int j0 = 0; j0 < p.top; j0 += J) {
                const CombinePair* pair = pairs + tok * p.top + j0;
                const int count = live ? p.top - j0 : 0;
                float dot[J];
#pragma unroll
                for (int k = 0; k < J; ++k) dot[k] = 0.0f;
                for (int64_t c0 = 0; c0 + N <= p.K; c0 += tpt * N) {
                    V r[J];
                    if (p.d_weights) {
#pragma unroll
                        for (int k = 0; k < J; ++k) {
                            if (k >= count) break;
                            const int64_t row = pair[k].row, c = c0 + in * N + head_of(row);
                            if (row >= 0 && c + N <= p.K)
                                r[k] = *reinterpret_cast<const V*>(rows + (row * p.ld_rows + c) * ES);
                        }
                    }
                    // (all of them on their way before the first is waited for)
                    E e[N + 1];
#pragma unroll
                    for (int i = 0; i <= N; ++i) {
                        const int64_t c = c0 + i * tpt + in;
                        e[i] = 0;
                        if (live && c < p.K && (i < N || in < N)) e[i] = reinterpret_cast<const E*>(g_row)[c];
                    }
                    if (c0 == 0) edges(j0, dot);
                    __syncthreads();  // (the columns before have been read)
#pragma unroll
                    for (int i = 0; i <= N; ++i) {
                        const int at = i * tpt + in;
                        float g[1];
                        unpack<DT, 1>(e[i], g);
                        if (i < N || in < N) dy_at[at + at / N] = g[0];
                    }
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < J; ++k) {
                        if (k >= count) break;
                        const int64_t row = pair[k].row;
                        const int head = head_of(row);
                        const int64_t c = c0 + in * N + head;
                        if (row < 0 || c + N > p.K) continue;
                        const float w = pair[k].w;
                        const float* lo = dy_at + in * (N + 1) + head;
                        float g[N], o[N];
#pragma unroll
                        for (int i = 0; i < N; ++i) g[i] = lo[head + i >= N ? i + 1 : i];
                        if (p.d_weights) {
                            unpack<DT, N>(r[k], o);
#pragma unroll
                            for (int i = 0; i < N; ++i) dot[k] = fmaf(g[i], o[i], dot[k]);
                        }
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = w * g[i];
                        *reinterpret_cast<V*>(d_rows + (row * p.ld_drows + c) * ES) = pack<DT, N>(o);
                    }
                }
                if (p.d_weights) combine_dots<J>(p, dot, part, t, j0, live);
            }
        }
    }
}

// Neighbouring elements that a thread takes at once: 16 bytes' worth, two 16-bit ones, or one.
template <int DT>
cudaError_t combine_launch(int n, const CombineParams& p, int blocks, cudaStream_t stream) {
    constexpr int FULL = DT == DT_F32 ? 4 : 8;
    const dim3 g(static_cast<unsigned>(blocks));
    if (n == FULL)
        combine_kernel<DT, FULL, 1><<<g, kSumThreads, 0, stream>>>(p);
    else if (DT != DT_F32 && n == 2)
        combine_kernel<DT, DT == DT_F32 ? 1 : 2, kSumApart><<<g, kSumThreads, 0, stream>>>(p);
    else
        combine_kernel<DT, 1, kSumApart><<<g, kSumThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// The gradient: 16 bytes at a time, from aligned rows or from rows on any address, or one element.
template <int DT>
cudaError_t combine_grad_launch(int n, bool any, const CombineParams& p, int blocks, cudaStream_t stream) {
    constexpr int FULL = DT == DT_F32 ? 4 : 8;
    const dim3 g(static_cast<unsigned>(blocks));
    auto run = [&](auto few) {
        constexpr int J = decltype(few)::value ? 4 : 8;
        if (any)
            combine_grad_any_kernel<DT, J><<<g, kSumThreads, 0, stream>>>(p);
        else if (n == FULL)
            combine_grad_kernel<DT, FULL, J><<<g, kSumThreads, 0, stream>>>(p);
        else
            combine_grad_kernel<DT, 1, J><<<g, kSumThreads, 0, stream>>>(p);
    };
    if (p.top <= 4)
        run(std::true_type());
    else
        run(std::false_type());
    return cudaGetLastError();
}

// Runs combine or its gradient from checked arguments.
gemm_status_t combine_run(CombineParams& p, int dt, bool grad, cudaStream_t stream) {
    DeviceInfo d;
    const gemm_status_t st = device_info(&d);
    if (st != GEMM_OK) return st;
    p.status = d.status;
    const int es = dt_bytes(dt), ys = dt_bytes(p.y_dtype), full = 16 / es;
    auto units = [](const void* ptr, int64_t ld, int bytes) {
        return !ptr || (aligned(ptr, 16) && ld * bytes % 16 == 0);
    };
    auto pairs = [](const void* ptr, int64_t ld) { return !ptr || (aligned(ptr, 4) && ld % 2 == 0); };
    int width = full;
    if (p.K % full != 0 || !units(p.rows, p.ld_rows, es) || !units(p.y, p.ld_y, ys) ||
        (grad && !units(p.d_rows, p.ld_drows, es)))
        width = !grad && es == 2 && p.K % 2 == 0 && pairs(p.rows, p.ld_rows) &&
                        pairs(p.y, p.ld_y) ? 2 : 1;
    // (the gradient takes rows on any address if an element has the same place in its 16 bytes in
    // both tensors)
    auto place = [&](const void* ptr, int64_t ld, int64_t row) {
        return (reinterpret_cast<uintptr_t>(ptr) + static_cast<uintptr_t>(row * ld * es)) % 16;
    };
    const bool any = grad && width != full && p.K >= full &&
                     (!p.rows || (place(p.rows, p.ld_rows, 0) == place(p.d_rows, p.ld_drows, 0) &&
                                  place(p.rows, p.ld_rows, 1) == place(p.d_rows, p.ld_drows, 1)));
    const int64_t n = cdiv(p.K, width == full || any ? full : (grad ? 1 : width * kSumApart));
    int log2 = 5;
    while (log2 < 8 && (int64_t(1) << log2) < n) ++log2;
    p.tpt_log2 = log2;
    int64_t blocks = cdiv(p.T, kSumThreads >> log2);
    // (the gradient of eight pairs at once: 114 registers, or 80)
    const int64_t fit = !grad || p.top <= 4 ? kSumBlocksPerSm : (any ? 3 : (width == full ? 2 : 4));
    if (blocks > d.sm_count * fit) blocks = d.sm_count * fit;
    const int g = static_cast<int>(blocks);
    cudaError_t e;
    if (grad)
        e = dt == DT_BF16  ? combine_grad_launch<DT_BF16>(width, any, p, g, stream)
            : dt == DT_F16 ? combine_grad_launch<DT_F16>(width, any, p, g, stream)
                           : combine_grad_launch<DT_F32>(width, any, p, g, stream);
    else
        e = dt == DT_BF16  ? combine_launch<DT_BF16>(width, p, g, stream)
            : dt == DT_F16 ? combine_launch<DT_F16>(width, p, g, stream)
                           : combine_launch<DT_F32>(width, p, g, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

bool matrix_ok(const void* m, int64_t rows, int64_t cols, int64_t ld, int es) {
    return m && aligned(m, es) && ld >= cols && strided_span_ok(rows, cols, ld, 1, 1, 0) &&
           count_ok(1, rows, cols);
}

// Ranges that a dispatch of this many tokens is cut into, at most.
int64_t route_blocks(int64_t T) { return T < 1 ? 1 : (T < kRouteBlocks ? T : kRouteBlocks); }

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

size_t gemm_expert_dispatch_workspace_size(int64_t T, int64_t top, int64_t groups) {
    if (!size_ok(T) || !size_ok(top) || !size_ok(groups) || groups > kRouteGroups) return 0;
    if (T == 0 || top <= kRouteOnePass / T) return 0;
    return static_cast<size_t>(route_blocks(T) * groups * 4);
}

gemm_status_t gemm_expert_dispatch(int elem_bytes, int64_t T, int64_t K, const void* X, int64_t ldx,
                                   const float* scales, int id_bytes, const void* ids,
                                   int64_t ld_ids, int64_t top, int64_t groups, void* rows,
                                   int64_t ld_rows, float* row_scales, int32_t* offsets,
                                   int32_t* slots, void* workspace, size_t workspace_bytes,
                                   gemm_stream_t stream) {
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return GEMM_ERR_INVALID_ARG;
    if (id_bytes != 4 && id_bytes != 8) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = extents(T, K, top, groups);
    if (st != GEMM_OK) return st;
    if (!offsets || !aligned(offsets, 4)) return GEMM_ERR_INVALID_ARG;
    // (rows are numbered in 32 bits)
    if (groups > kRouteGroups || (T > 0 && top > kMaxExtent / T)) return GEMM_ERR_UNSUPPORTED;
    if (T > 0 && top > 0) {
        if (!ids || !aligned(ids, id_bytes) || ld_ids < top || !slots || !aligned(slots, 4) ||
            !strided_span_ok(T, top, ld_ids, 1, 1, 0))
            return GEMM_ERR_INVALID_ARG;
        if (K > 0 && (!matrix_ok(X, T, K, ldx, elem_bytes) ||
                      !matrix_ok(rows, T * top, K, ld_rows, elem_bytes)))
            return GEMM_ERR_INVALID_ARG;
        if (scales && (!aligned(scales, 4) || !row_scales || !aligned(row_scales, 4)))
            return GEMM_ERR_INVALID_ARG;
    }
    const size_t need = gemm_expert_dispatch_workspace_size(T, top, groups);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo d;
    st = device_info(&d);
    if (st != GEMM_OK) return st;
    DispatchParams p{};
    p.ids = ids;
    p.ld_ids = ld_ids;
    p.T = top > 0 ? static_cast<int32_t>(T) : 0;
    p.top = static_cast<int32_t>(top);
    p.groups = static_cast<int32_t>(groups);
    p.x = static_cast<const char*>(X);
    p.x_pitch = ldx * elem_bytes;
    p.scales = scales;
    p.rows = static_cast<char*>(rows);
    p.rows_pitch = ld_rows * elem_bytes;
    p.row_scales = row_scales;
    p.offsets = offsets;
    p.slots = slots;
    p.hist = need > 0 ? static_cast<int32_t*>(workspace) : nullptr;
    p.status = d.status;
    const int64_t bytes = K * elem_bytes;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(rows) |
                           static_cast<uintptr_t>(bytes) | static_cast<uintptr_t>(p.x_pitch) |
                           static_cast<uintptr_t>(p.rows_pitch);
    int unit = 16;
    while (bits % unit) unit >>= 1;
    if (bytes / unit > kLim) return GEMM_ERR_UNSUPPORTED;
    p.vecs = static_cast<int32_t>(bytes / unit);
    int log2 = 5;
    while (log2 < 10 && (int64_t(route_apart(unit)) << log2) < p.vecs) ++log2;
    p.tpt_log2 = log2;
    // segments: a warp each, as many as shared memory has counts for
    const int64_t fit = groups > 0 ? kRouteInts / groups - 2 : 32;
    p.warps = static_cast<int32_t>(fit < 32 ? fit : 32);
    int64_t blocks = route_blocks(p.T);
    if (blocks > d.sm_count) blocks = d.sm_count;
    // (96 MB in all: what L2 holds beside the rows on their way out)
    p.ahead = bytes > 0 && bytes <= 65536 ? static_cast<int32_t>((int64_t(96) << 20) / (bytes * blocks)) : 0;
    const cudaError_t e =
        id_bytes == 8
            ? dispatch_unit<int64_t>(unit, p, static_cast<int>(blocks), static_cast<cudaStream_t>(stream))
            : dispatch_unit<int32_t>(unit, p, static_cast<int>(blocks), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

gemm_status_t gemm_expert_combine(gemm_dtype_t dtype, int64_t T, int64_t K, int64_t top,
                                  const void* rows, int64_t R, int64_t ld_rows,
                                  const int32_t* slots, const void* weights,
                                  gemm_dtype_t w_dtype, int64_t ld_weights, void* Y, int64_t ldy,
                                  gemm_dtype_t y_dtype, gemm_stream_t stream) {
    if (!is_dt(dtype) || !is_dt(y_dtype) || (weights && !is_dt(w_dtype))) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = extents(T, K, top, R);
    if (st != GEMM_OK) return st;
    if ((y_dtype != dtype && y_dtype != GEMM_DT_F32) || top > kSumPairs) return GEMM_ERR_UNSUPPORTED;
    if (T == 0 || K == 0) return GEMM_OK;
    if (!matrix_ok(Y, T, K, ldy, dt_bytes(y_dtype))) return GEMM_ERR_INVALID_ARG;
    if (top > 0 && (!slots || !aligned(slots, 4))) return GEMM_ERR_INVALID_ARG;
    if (top > 0 && R > 0 && !matrix_ok(rows, R, K, ld_rows, dt_bytes(dtype)))
        return GEMM_ERR_INVALID_ARG;
    if (top > 0 && weights &&
        (!aligned(weights, dt_bytes(w_dtype)) || ld_weights < top ||
         !strided_span_ok(T, top, ld_weights, 1, 1, 0)))
        return GEMM_ERR_INVALID_ARG;
    CombineParams p{};
    p.slots = slots;
    p.weights = weights;
    p.ld_w = ld_weights;
    p.w_dtype = w_dtype;
    p.T = static_cast<int32_t>(T);
    p.top = static_cast<int32_t>(top);
    p.K = static_cast<int32_t>(K);
    p.R = static_cast<int32_t>(R);
    p.rows = top > 0 && R > 0 ? rows : nullptr;
    p.ld_rows = ld_rows;
    p.y = Y;
    p.ld_y = ldy;
    p.y_dtype = y_dtype;
    return combine_run(p, dtype, false, static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_expert_combine_grad(gemm_dtype_t dtype, int64_t T, int64_t K, int64_t top,
                                       const void* DY, int64_t lddy, const int32_t* slots,
                                       const void* weights, gemm_dtype_t w_dtype,
                                       int64_t ld_weights, const void* rows, int64_t R,
                                       int64_t ld_rows, void* d_rows, int64_t ld_drows,
                                       void* d_weights, gemm_dtype_t dw_dtype, int64_t ld_dweights,
                                       gemm_stream_t stream) {
    if (!is_dt(dtype) || (weights && !is_dt(w_dtype)) || (d_weights && !is_dt(dw_dtype)))
        return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = extents(T, K, top, R);
    if (st != GEMM_OK) return st;
    if (top > kSumPairs) return GEMM_ERR_UNSUPPORTED;
    if (T == 0 || top == 0) return GEMM_OK;
    if (!slots || !aligned(slots, 4)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && !matrix_ok(DY, T, K, lddy, dt_bytes(dtype))) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && R > 0 && !matrix_ok(d_rows, R, K, ld_drows, dt_bytes(dtype)))
        return GEMM_ERR_INVALID_ARG;
    if (weights && (!aligned(weights, dt_bytes(w_dtype)) || ld_weights < top ||
                    !strided_span_ok(T, top, ld_weights, 1, 1, 0)))
        return GEMM_ERR_INVALID_ARG;
    if (d_weights) {
        if (!aligned(d_weights, dt_bytes(dw_dtype)) || ld_dweights < top ||
            !strided_span_ok(T, top, ld_dweights, 1, 1, 0))
            return GEMM_ERR_INVALID_ARG;
        if (K > 0 && R > 0 && !matrix_ok(rows, R, K, ld_rows, dt_bytes(dtype)))
            return GEMM_ERR_INVALID_ARG;
    }
    CombineParams p{};
    p.slots = slots;
    p.weights = weights;
    p.ld_w = ld_weights;
    p.w_dtype = w_dtype;
    p.T = static_cast<int32_t>(T);
    p.top = static_cast<int32_t>(top);
    p.K = static_cast<int32_t>(K);
    p.R = static_cast<int32_t>(R);
    p.rows = d_weights && R > 0 ? rows : nullptr;
    p.ld_rows = ld_rows;
    p.y = const_cast<void*>(DY);
    p.ld_y = lddy;
    p.y_dtype = dtype;
    p.d_rows = d_rows;
    p.ld_drows = ld_drows;
    p.d_weights = d_weights;
    p.ld_dw = ld_dweights;
    p.dw_dtype = dw_dtype;
    return combine_run(p, dtype, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
