// Rows to 8-bit integers with a scale each, and 8-bit operands in the forms that the
// product of i8_kernel.cu reads.
//
//   s = max |x| / 127,   q = 127 x / max |x| to the nearest integer (ties to even)
//
// The quotient is decided exactly: fp32 gives y = x (127 / max |x|) to within 2.5 * 2^-23 of
// itself, at most 3.8e-5; where y lies within 2^-14 of a border between two integers, 254 |x|
// and (2 n + 1) max |x| are compared exactly instead (in fp32: 16-bit rows whose maximum is
// 127 times a power of two have half of their larger elements on a border; with 64-bit products
// for those, 4096 x 4096 took 20 us).  So q does not depend on the reciprocal's rounding, and a
// result computed in 64 bits is the same integer.
//
// One pass over the data: the threads of a row (a warp's worth at least, a block's at
// most) keep its elements in registers between the maximum and the quotients, up to 32
// each (16 of fp32, and where rows are not aligned), and load the next row's meanwhile;
// what a row has beyond is read again, from L2.  4096 x 4096 bf16: 14.5 us, 3.5 TB/s by graph
// replay, where the copy rate would take 7.4; 1001 x 7001 fp32, rows that start anywhere: 13.4
// against 5.2.  The instructions bound it (about six an element), then the load of few rows a
// block (4096 rows on 608 blocks: 6.7 each).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "experts_host.h"
#include "gemm_experts.h"
#include "i8.h"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr int kThreads = 256;
// Elements of a row that a thread keeps (16 registers; the next row's take 16 more).
template <int DT>
__host__ __device__ constexpr int quant_keep(int n) {
    return DT == DT_F32 || n == 1 ? 16 : 32;
}

struct QuantParams {
    const void* x;
    int64_t ld_x;
    int32_t T, K;
    void* q;            // int8, or fp16 (the integers' values, padded with zeros to `pad`)
    int64_t ld_q;       // elements
    int32_t pad;
    float* scales;
    int32_t tpr_log2;   // threads of a row
};

constexpr int kQuantBlocksPerSm = 4;  // all resident at once

template <int BYTES>
struct Raw {
    using Small = std::conditional_t<BYTES == 2, uint16_t, uint8_t>;
    using Half = std::conditional_t<BYTES == 8, uint2, std::conditional_t<BYTES == 4, uint32_t, Small>>;
    using V = std::conditional_t<BYTES == 16, uint4, Half>;
};

// N elements of type DT as fp32 (exact).
template <int DT, int N, typename V>
__device__ __forceinline__ void widen(const V& v, float (&f)[N]) {
    if constexpr (DT == DT_F32) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = DT == DT_BF16 ? __uint_as_float(static_cast<uint32_t>(h[i]) << 16)
                                 : __half2float(__ushort_as_half(h[i]));
    }
}

// The larger magnitudes of a unit's elements and `top`: 16-bit elements two at a time and as
// they are (a NaN stays), fp32 as bit patterns, which order as integers, infinities above all
// numbers and NaN above those.
template <int DT, int N, typename V>
__device__ __forceinline__ uint32_t larger(const V& v, uint32_t top) {
    using E = typename Raw<DT == DT_F32 ? 4 : 2>::V;
    const uint32_t one = N == 1 ? static_cast<uint32_t>(*reinterpret_cast<const E*>(&v)) : 0u;
    const uint32_t* w = N == 1 ? &one : reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < (DT == DT_F32 ? N : (N + 1) / 2); ++i) {
        if constexpr (DT == DT_F32) {
            top = max(top, w[i] & 0x7fffffffu);
        } else if constexpr (DT == DT_BF16) {
            const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(w + i)),
                                                 *reinterpret_cast<const __nv_bfloat162*>(&top));
            top = *reinterpret_cast<const uint32_t*>(&m);
        } else {
            const __half2 m = __hmax2_nan(__habs2(*reinterpret_cast<const __half2*>(w + i)),
                                          *reinterpret_cast<const __half2*>(&top));
            top = *reinterpret_cast<const uint32_t*>(&m);
        }
    }
    return top;
}

// ... of a thread, as fp32 bits.
template <int DT>
__device__ __forceinline__ uint32_t magnitude(uint32_t top) {
    if constexpr (DT == DT_F32) return top;
    const uint32_t h = max(top & 0x7fffu, (top >> 16) & 0x7fffu);
    return DT == DT_BF16 ? h << 16
                         : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(h))));
}

// Adding and subtracting this rounds an fp32 number of at most 2^22 to the nearest integer,
// ties to even; the sum's low bits are the integer.
constexpr float kToInt = 12582912.0f;  // 1.5 * 2^23

// 127 x / top decided exactly, where fp32's y may lie on the wrong side of the border
// lo + 1/2: 254 |x| is compared with (2 lo + 1) top, each as its difference from q, the second
// one's rounded value.  Both differences are exact: the second is a product's rounding error,
// and the first is below 2^-13 of q and a multiple of the last place of 254 |x|, 32 bits down.
__device__ __forceinline__ float quotient_exact(float x, float y, float top) {
    const float lo = floorf(fabsf(y)), odd = 2.0f * lo + 1.0f;
    const float q = odd * top, b = fmaf(odd, top, -q), a = fmaf(254.0f, fabsf(x), -q);
    const bool up = a > b || (a == b && (static_cast<int>(lo) & 1) != 0);
    return copysignf(up ? lo + 1.0f : lo, x);
}

// N quotients 127 x / top as rounded integers + kToInt; r = 127 / top within 2 ulp.
template <int N>
__device__ __forceinline__ void quotients(const float (&x)[N], float top, float r, float (&t)[N]) {
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = x[i] * r;
        t[i] = y + kToInt;
        far = fmaxf(far, fabsf(y - (t[i] - kToInt)));
    }
    if (far > 0.5f - 6.103515625e-5f) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = x[i] * r;
            if (fabsf(y - (t[i] - kToInt)) > 0.5f - 6.103515625e-5f)
                t[i] = quotient_exact(x[i], y, top) + kToInt;
        }
    }
}

// N rounded integers + kToInt as int8 or fp16.
template <int N, bool WIDE>
__device__ __forceinline__ void store_integers(char* dst, const float (&t)[N]) {
    if constexpr (N == 1) {
        if constexpr (WIDE)
            *reinterpret_cast<__half*>(dst) = __float2half_rn(t[0] - kToInt);
        else
            *reinterpret_cast<uint8_t*>(dst) = static_cast<uint8_t>(__float_as_uint(t[0]));
    } else if constexpr (WIDE) {
        typename Raw<N * 2>::V o;
        __half2* h = reinterpret_cast<__half2*>(&o);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) h[i] = __floats2half2_rn(t[2 * i] - kToInt, t[2 * i + 1] - kToInt);
        *reinterpret_cast<typename Raw<N * 2>::V*>(dst) = o;
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint16_t*>(dst) =
            static_cast<uint16_t>(__byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040));
    } else {
        typename Raw<N>::V o;
        uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = __byte_perm(__byte_perm(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]), 0x0040),
                               __byte_perm(__float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]), 0x0040),
                               0x5410);
        *reinterpret_cast<typename Raw<N>::V*>(dst) = o;
    }
}

// A unit of a row that lies partly outside it, zeros there.
template <int ES, int N, typename V>
__device__ __noinline__ V quant_edge(const char* src, int64_t c, int K) {
    using E = typename Raw<ES>::V;
    V v{};
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (c + i >= 0 && c + i < K)
            reinterpret_cast<E*>(&v)[i] = __ldg(reinterpret_cast<const E*>(src + (c + i) * ES));
    return v;
}

// WIDE: fp16 integers, padded; else int8.  EDGE: units may lie partly outside their row (the
// checks cost 4096 x 4096 bf16 1.3 us of 15).
template <int DT, int N, bool WIDE, bool EDGE>
__global__ void __launch_bounds__(kThreads, kQuantBlocksPerSm) quantize_kernel(const QuantParams p) {
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    constexpr int R = quant_keep<DT>(N) / N;
    using V = typename Raw<N * ES>::V;
    __shared__ uint32_t tops[kThreads / 32];
    if (WIDE) griddep_launch_dependents();
    const int tpr = 1 << p.tpr_log2, in = threadIdx.x & (tpr - 1);
    const int per_block = kThreads >> p.tpr_log2;
    const int warp = threadIdx.x >> 5, warps = tpr >> 5, lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
    // A row's units start on the boundaries of N elements in memory, so its first and last one
    // may lie partly outside: `off` elements before the row the first one starts.
    auto before = [&](const char* src) {
        return EDGE ? static_cast<int>(reinterpret_cast<uintptr_t>(src) / ES % N) : 0;
    };
    auto load = [&](const char* src, int64_t c) {
        if (!EDGE || (c >= 0 && c + N <= p.K)) return __ldg(reinterpret_cast<const V*>(src + c * ES));
        return quant_edge<ES, N, V>(src, c, p.K);
    };
    V next[R];
    auto fetch = [&](int64_t row) {
        if (row >= p.T) return;
        const char* src = static_cast<const char*>(p.x) + row * p.ld_x * ES;
        const int off = before(src);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (k * tpr + in) * N - off;
            if (c < p.K) next[k] = load(src, c);
        }
    };
    fetch(static_cast<int64_t>(blockIdx.x) * per_block + (threadIdx.x >> p.tpr_log2));
    // (whole blocks walk together: the maximum's barriers are the block's)
    for (int64_t rb = static_cast<int64_t>(blockIdx.x) * per_block; rb < p.T; rb += step) {
        const int64_t row = rb + (threadIdx.x >> p.tpr_log2);
        const bool live = row < p.T;
        const char* src = static_cast<const char*>(p.x) + row * p.ld_x * ES;
        const int off = before(src);
        V keep[R];
#pragma unroll
        for (int k = 0; k < R; ++k) keep[k] = next[k];
        fetch(row + step);
        uint32_t top = 0;
        if (live) {
#pragma unroll
            for (int k = 0; k < R; ++k)
                if ((k * tpr + in) * N - off < p.K) top = larger<DT, N>(keep[k], top);
            for (int64_t c = (static_cast<int64_t>(R) * tpr + in) * N - off; c < p.K; c += tpr * N)
                top = larger<DT, N>(load(src, c), top);
        }
        top = magnitude<DT>(top);
        top = __reduce_max_sync(0xffffffffu, top);
        if (warps > 1) {
            __syncthreads();  // (the row before has been read)
            if (lane == 0) tops[warp] = top;
            __syncthreads();
            const int first = warp & ~(warps - 1);
            for (int i = 0; i < warps; ++i) top = tops[first + i] > top ? tops[first + i] : top;
        }
        if (!live) continue;
        // (a row with an infinity or a NaN has no integers: a NaN scale says so)
        const bool finite = top < 0x7f800000u;
        const float size = __uint_as_float(top);
        if (in == 0) p.scales[row] = finite ? __fdiv_rn(size, 127.0f) : __uint_as_float(0x7fffffffu);
        // (a power of two keeps 127 / size and x 127 inside fp32; where it rounds an
        // element, that element's integer is zero)
        const float even = size < 0x1p-40f ? 0x1p100f : (size > 0x1p100f ? 0x1p-100f : 1.0f);
        const float big = size * even;
        const bool some = finite && top != 0;
        const float r = some ? __fdividef(127.0f, big) : 0.0f;  // (within 2 ulp)
        char* dst = static_cast<char*>(p.q) + row * p.ld_q * (WIDE ? 2 : 1);
        auto put_integers = [&](int64_t c, const float (&t)[N]) {
            if (!EDGE || (c >= 0 && c + N <= p.K)) {
                store_integers<N, WIDE>(dst + c * (WIDE ? 2 : 1), t);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float one[1] = {t[i]};
                    if (c + i >= 0 && c + i < p.K) store_integers<1, WIDE>(dst + (c + i) * (WIDE ? 2 : 1), one);
                }
            }
        };
        auto put = [&](const V& v, int64_t c) {
            float f[N], t[N];
            widen<DT, N>(v, f);
            if (even != 1.0f) {
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] *= even;
            }
            quotients<N>(f, big, r, t);
            put_integers(c, t);
        };
        if (some) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int c = (k * tpr + in) * N - off;
                if (c < p.K) put(keep[k], c);
            }
            for (int64_t c = (static_cast<int64_t>(R) * tpr + in) * N - off; c < p.K; c += tpr * N)
                put(load(src, c), c);
        } else {
            float zero[N];
#pragma unroll
            for (int i = 0; i < N; ++i) zero[i] = kToInt;
            for (int64_t c = in * N - off; c < p.K; c += tpr * N) put_integers(c, zero);
        }
        if (WIDE)
            for (int c = p.K + in; c < p.pad; c += tpr) reinterpret_cast<uint16_t*>(dst)[c] = 0;
    }
}

int row_threads(int64_t units) {
    int log2 = 5;
    while (log2 < 8 && (int64_t(1) << log2) < units) ++log2;
    return log2;
}

template <int DT, int N, bool WIDE, bool EDGE>
cudaError_t quantize_launch(QuantParams p, int sms, cudaStream_t stream) {
    // as few threads a row as keep it, but enough rows' worth of threads to fill the GPU: what
    // a thread does once a row costs as much as eight elements
    constexpr int keep = quant_keep<DT>(N);
    // (rows that start inside a unit have one more)
    p.tpr_log2 = row_threads((static_cast<int64_t>(p.K) + (EDGE ? N - 1 : 0) + keep - 1) / keep);
    while (p.tpr_log2 < 8 && (int64_t(p.T) << p.tpr_log2) < int64_t(sms) * kThreads) ++p.tpr_log2;
    int64_t blocks = cdiv(p.T, kThreads >> p.tpr_log2);
    if (blocks > int64_t(sms) * kQuantBlocksPerSm) blocks = int64_t(sms) * kQuantBlocksPerSm;
    quantize_kernel<DT, N, WIDE, EDGE><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int DT, bool WIDE>
cudaError_t quantize_width(const QuantParams& p, int sms, cudaStream_t stream) {
    constexpr int ES = DT == DT_F32 ? 4 : 2, FULL = 16 / ES;
    // units of n elements, where an element's place in its unit is the same in X and in Q
    auto fits = [&](int n) {
        return reinterpret_cast<uintptr_t>(p.x) / ES % n ==
                   reinterpret_cast<uintptr_t>(p.q) / (WIDE ? 2 : 1) % n &&
               p.ld_x % n == p.ld_q % n;
    };
    if (fits(FULL) && p.K % FULL == 0 && p.ld_x % FULL == 0 && aligned(p.x, 16))
        return quantize_launch<DT, FULL, WIDE, false>(p, sms, stream);
    if (fits(FULL)) return quantize_launch<DT, FULL, WIDE, true>(p, sms, stream);
    if (fits(2)) return quantize_launch<DT, 2, WIDE, true>(p, sms, stream);
    return quantize_launch<DT, 1, WIDE, false>(p, sms, stream);
}

template <bool WIDE>
cudaError_t quantize_type(int dt, const QuantParams& p, int sms, cudaStream_t stream) {
    return dt == DT_BF16  ? quantize_width<DT_BF16, WIDE>(p, sms, stream)
           : dt == DT_F16 ? quantize_width<DT_F16, WIDE>(p, sms, stream)
                          : quantize_width<DT_F32, WIDE>(p, sms, stream);
}

// int8 rows to fp16 ones, padded with zeros to `pad` (a multiple of 64): a thread takes 8
// neighbouring elements.  VEC: the source's rows start on 8-byte boundaries and K is a
// multiple of 8.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) widen_kernel(const int8_t* x, int64_t ld, int T, int K,
                                                         int pad, uint16_t* out) {
    griddep_launch_dependents();
    const int units = pad / 8;
    const int64_t n = static_cast<int64_t>(T) * units;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride) {
        const int64_t row = i / units;
        const int c = static_cast<int>(i - row * units) * 8;
        const int8_t* src = x + row * ld + c;
        int8_t b[8];
        if (VEC) {
            uint2 v = make_uint2(0, 0);
            if (c < K) v = __ldg(reinterpret_cast<const uint2*>(src));
            *reinterpret_cast<uint2*>(b) = v;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) b[k] = c + k < K ? __ldg(src + k) : int8_t(0);
        }
        uint4 o;
        uint16_t* h = reinterpret_cast<uint16_t*>(&o);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = __half_as_ushort(__short2half_rn(b[k]));
        *reinterpret_cast<uint4*>(out + row * pad + c) = o;
    }
}

// Bytes to rows of `ld_dst` (a multiple of 16), for weights that TMA cannot address.
__global__ void __launch_bounds__(kThreads) pack8_kernel(const uint8_t* src, int64_t ld,
                                                         int64_t stride, int64_t rows, int32_t cols,
                                                         int64_t depth, uint8_t* dst, int64_t ld_dst) {
    const int64_t n = rows * depth, step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); r < n; r += step) {
        const int64_t z = r / rows;
        const uint8_t* from = src + z * stride + (r - z * rows) * ld;
        uint8_t* to = dst + r * ld_dst;
        for (int c = threadIdx.x & 31; c < cols; c += 32) to[c] = __ldg(from + c);
    }
}

}  // namespace

cudaError_t i8_widen_quantized(int dt, const void* x, int64_t ld, int64_t T, int64_t K, int64_t pad,
                               void* out, float* scales, int sms, cudaStream_t stream) {
    QuantParams p{};
    p.x = x;
    p.ld_x = ld;
    p.T = static_cast<int32_t>(T);
    p.K = static_cast<int32_t>(K);
    p.q = out;
    p.ld_q = pad;
    p.pad = static_cast<int32_t>(pad);
    p.scales = scales;
    return quantize_type<true>(dt, p, sms, stream);
}

cudaError_t i8_widen(const void* x, int64_t ld, int64_t T, int64_t K, int64_t pad, void* out, int sms,
                     cudaStream_t stream) {
    const int64_t units = T * (pad / 8);
    int64_t blocks = cdiv(units, kThreads);
    if (blocks > int64_t(sms) * 16) blocks = int64_t(sms) * 16;
    const dim3 g(static_cast<unsigned>(blocks));
    const int8_t* src = static_cast<const int8_t*>(x);
    const int t = static_cast<int>(T), k = static_cast<int>(K), n = static_cast<int>(pad);
    if (aligned(x, 8) && ld % 8 == 0 && K % 8 == 0)
        widen_kernel<true><<<g, kThreads, 0, stream>>>(src, ld, t, k, n, static_cast<uint16_t*>(out));
    else
        widen_kernel<false><<<g, kThreads, 0, stream>>>(src, ld, t, k, n, static_cast<uint16_t*>(out));
    return cudaGetLastError();
}

cudaError_t i8_pack(const void* src, int64_t ld, int64_t stride, int64_t rows, int64_t cols,
                    int64_t depth, void* dst, int64_t ld_dst, int sms, cudaStream_t stream) {
    int64_t blocks = cdiv(rows * depth, kThreads / 32);
    if (blocks > int64_t(sms) * 8) blocks = int64_t(sms) * 8;
    pack8_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
        static_cast<const uint8_t*>(src), ld, stride, rows, static_cast<int32_t>(cols), depth,
        static_cast<uint8_t*>(dst), ld_dst);
    return cudaGetLastError();
}

}  // namespace dg

using namespace dg;

extern "C" gemm_status_t gemm_i8_quantize(gemm_dtype_t dtype, int64_t T, int64_t K, const void* X,
                                          int64_t ldx, int8_t* Q, int64_t ldq, float* scales,
                                          gemm_stream_t stream) {
    if (!is_dt(dtype)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = extents(T, K, 0, 0);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    if (!scales || !aligned(scales, 4)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!X || !aligned(X, dt_bytes(dtype)) || !Q || ldx < K || ldq < K ||
                  !strided_span_ok(T, K, ldx, 1, 1, 0) || !strided_span_ok(T, K, ldq, 1, 1, 0) ||
                  !count_ok(1, T, K)))
        return GEMM_ERR_INVALID_ARG;
    DeviceInfo d;
    st = device_info(&d);
    if (st != GEMM_OK) return st;
    QuantParams p{};
    p.x = X;
    p.ld_x = ldx;
    p.T = static_cast<int32_t>(T);
    p.K = static_cast<int32_t>(K);
    p.q = Q;
    p.ld_q = ldq;
    p.scales = scales;
    if (quantize_type<false>(dtype, p, d.sm_count, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}
