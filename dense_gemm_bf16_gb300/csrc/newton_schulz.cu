// Element-wise passes of the orthogonalised update: the Frobenius norm of every
// matrix of a batch and X = G / (norm + eps) in scaled fp16.  Both are bound by
// the bytes of G (the second mostly reads it from L2).
//
// The norm sums squares in fp32 with a fixed order (threads, then blocks), so
// results repeat.  Squares of large or small entries would leave fp32's range,
// so entries are summed in three ranges (Blue's method): above 2^40 as
// (2^-88 x)^2, below 2^-40 as (2^88 x)^2, and the rest as they are: every square
// lies in 2^-122 .. 2^96, so that 2^31 of them still fit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "epilogue.cuh"
#include "ragged.h"

namespace dg {
namespace {

constexpr int kThreads = 256;
constexpr float kBig = 1.099511627776e12f;             // 2^40
constexpr float kSmall = 9.094947017729282379e-13f;    // 2^-40
constexpr float kDown = 3.231174267785264355e-27f;     // 2^-88
constexpr float kUp = 3.094850098213450687e26f;        // 2^88

struct Sum3 {
    float big, mid, small;
    __device__ void add(float x) {
        const float ax = fabsf(x);
        if (ax > kBig) {
            const float y = ax * kDown;
            big = fmaf(y, y, big);
        } else if (ax < kSmall) {
            const float y = ax * kUp;
            small = fmaf(y, y, small);
        } else {
            mid = fmaf(ax, ax, mid);  // (a NaN lands here)
        }
    }
};

// Columns c .. c + 7 of row r of matrix b (zeros past N).
template <int GDT>
__device__ __forceinline__ void load8(const NsParams& p, int64_t b, int r, int c, float (&v)[8]) {
    constexpr int ES = GDT == DT_F32 ? 4 : 2;
    const char* src = static_cast<const char*>(p.G) + (b * p.stride_g + r * p.ldg + c) * ES;
    if (p.g_vec && c + 8 <= p.N) {
        if constexpr (GDT == DT_F32) {
            const float4 x = reinterpret_cast<const float4*>(src)[0];
            const float4 y = reinterpret_cast<const float4*>(src)[1];
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
            v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(src);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f;
                if constexpr (GDT == DT_BF16)
                    f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
                else
                    f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < p.N ? load_elem(src + i * ES, GDT) : 0.0f;
}

// Block blockIdx.x = b * parts + part sums rows part, part + parts, ... of matrix b.
template <int GDT>
__global__ void __launch_bounds__(kThreads) ns_norm_kernel(const NsParams p) {
    const int64_t b = blockIdx.x / p.parts;
    const int part = static_cast<int>(blockIdx.x - b * p.parts);
    Sum3 s{0.0f, 0.0f, 0.0f};
    for (int r = part; r < p.M; r += p.parts)
        for (int c = threadIdx.x * 8; c < p.N; c += kThreads * 8) {
            float v[8];
            load8<GDT>(p, b, r, c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s.add(v[i]);
        }
    __shared__ float red[3][kThreads / 32];
    float t[3] = {s.big, s.mid, s.small};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t[k] += __shfl_xor_sync(0xffffffffu, t[k], d);
        if ((threadIdx.x & 31) == 0) red[k][threadIdx.x >> 5] = t[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        float x = 0.0f;
        for (int i = 0; i < kThreads / 32; ++i) x += red[threadIdx.x][i];
        p.partials[static_cast<int64_t>(blockIdx.x) * 3 + threadIdx.x] = x;
    }
}

template <int GDT>
__global__ void __launch_bounds__(kThreads) ns_scale_kernel(const NsParams p) {
    const int64_t b = blockIdx.x / p.parts;
    const int part = static_cast<int>(blockIdx.x - b * p.parts);
    __shared__ float factor[2];
    if (threadIdx.x < 32) {
        // every block adds its matrix's partial sums in the same order
        float s[3] = {0.0f, 0.0f, 0.0f};
        for (int i = threadIdx.x; i < p.parts; i += 32)
            for (int k = 0; k < 3; ++k) s[k] += p.partials[(b * p.parts + i) * 3 + k];
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], d);
        if (threadIdx.x == 0) {
            constexpr double up = kUp, down = kDown;
            const double sq = static_cast<double>(s[0]) * (up * up) + s[1] +
                              static_cast<double>(s[2]) * (down * down);
            // the factor itself may leave fp32's range: its first part is a power of
            // two that brings the entries near 1
            const double f = static_cast<double>(p.scale) / (sqrt(sq) + static_cast<double>(p.eps));
            const double pre = f > up ? up : f < down ? down : 1.0;
            factor[0] = static_cast<float>(pre);
            factor[1] = static_cast<float>(f / pre);
        }
    }
    if (part == 0 && threadIdx.x == 32) p.arrived[b] = 0u;
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1];
    __half* X = static_cast<__half*>(p.X) + b * p.M * p.ldx;
    for (int r = part; r < p.M; r += p.parts)
        for (int c = threadIdx.x * 8; c < p.N; c += kThreads * 8) {
            float v[8];
            load8<GDT>(p, b, r, c, v);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 h = __floats2half2_rn(v[2 * i] * f0 * f1, v[2 * i + 1] * f0 * f1);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            // rows of X are padded to 8 elements, so the last store stays in its row
            *reinterpret_cast<uint4*>(X + r * p.ldx + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
}

}  // namespace

cudaError_t ns_norm_launch(const NsParams& p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.batch * p.parts);
    if (p.g_dtype == DT_F32)
        ns_norm_kernel<DT_F32><<<grid, kThreads, 0, stream>>>(p);
    else if (p.g_dtype == DT_BF16)
        ns_norm_kernel<DT_BF16><<<grid, kThreads, 0, stream>>>(p);
    else
        ns_norm_kernel<DT_F16><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t ns_scale_launch(const NsParams& p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.batch * p.parts);
    if (p.g_dtype == DT_F32)
        ns_scale_kernel<DT_F32><<<grid, kThreads, 0, stream>>>(p);
    else if (p.g_dtype == DT_BF16)
        ns_scale_kernel<DT_BF16><<<grid, kThreads, 0, stream>>>(p);
    else
        ns_scale_kernel<DT_F16><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dg
