// Rows to 8-bit integers with a scale each, and 8-bit operands in the forms that the
// product of i8_kernel.cu reads.
//
//   s = max |x| / 127,   q = 127 x / max |x| to the nearest integer (ties to even)
//
// The quotient is decided exactly, so q does not depend on the reciprocal's rounding and a
// result computed in 64 bits is the same integer.  Of fp32 rows, y = x (127 / max |x|) is
// within 3.2e-5; where it lies within 2^-14 of a border between two integers, 254 |x| and
// (2 n + 1) max |x| are compared exactly instead.  16-bit rows are often on a border (every
// element of half the maximum; half of all elements where the maximum is 127 times a power of
// two), but never very close to one otherwise, so cutting y's last bits off decides them
// (see quotients; with comparisons 4096 x 4096 took 17.4 us, without 10.7).
//
// One pass over the data: the threads of a row (a warp's worth at least, a block's at
// most) keep its elements in registers between the maximum and the quotients, up to 32
// each (16 where rows are not aligned), and load the next row's meanwhile; what a row has
// beyond is read again, from L2.  Units that need more care (a border, a scale outside fp32's
// middle) are read again element by element in one copy of the code: unrolled beside the
// others it did not stay in the instruction cache (4096 x 4095 fp32: 36 us, now 16.7).
//
// 4096 x 4096 bf16: 9.4 us by graph replay over six inputs in turn, 5.3 TB/s, where the copy rate
// would take 7.4 (the issue slots are 67 % busy; one input again and again: 8.4); 1001 x 7001 fp32,
// rows that start anywhere: 9.6 against 5.2 (3.3 rows for each block; one input: 8.3).
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
// Quantising blocks on an SM, all resident at once.
template <int DT>
constexpr int kQuantBlocksPerSm = DT == DT_F32 ? 2 : 3;
// Elements of a row that a thread keeps (16 or 32 registers; the next row's take as many more).
// fp32 rows of up to 8192 stay on the SM: with 16 elements and twice the blocks, 1001 x 7001
// took 12 us against 9.5, and 16-bit ones with four blocks 10.7 against 9.7 (4096 x 4096).
__host__ __device__ constexpr int quant_keep(int n) { return n == 1 ? 16 : 32; }

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

// An fp32 number of at most 2^22 plus this is rounded to the nearest integer n, ties to even,
// whose bits are the sum's low ones.  For fp16 results (WIDE) the low 16 bits are 0x6480 + n
// instead, the fp16 number 1152 + n.
template <bool WIDE>
constexpr float kToInt = WIDE ? 12582912.0f + 0x6480 : 12582912.0f;  // 1.5 * 2^23

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

// N quotients 127 x / top as rounded integers + kToInt.
//
// fp32: r = 127 / top within 2 ulp (2^-22); what lies close to a border is decided exactly.
//
// 16-bit: 127 x / top is on a border or, m_x below 2^11 being x's significand, at least
// 1 / (254 m_x) > 2^-19 of itself away from one.  r is 127 / top times 1 + 2^-21, within 2 ulp
// again, so that x r exceeds the quotient by 2^-23 to 2^-20.2 of itself, and cutting x r off
// after 20 bits leaves a quotient on a border (8 bits) there and all others on their side of it.
// True: one of them may be wrong (fp32).
template <int DT, bool WIDE, int N>
__device__ __forceinline__ bool quotients(const float (&x)[N], float r, float (&t)[N]) {
    constexpr float C = kToInt<WIDE>;
    if constexpr (DT != DT_F32) {
        if constexpr (N == 1) {
            t[0] = __uint_as_float(__float_as_uint(x[0] * r) & 0xfffffff0u) + C;
        } else {
            // (two at a time: packed fp32 operations)
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float2 y = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(r, r));
                y.x = __uint_as_float(__float_as_uint(y.x) & 0xfffffff0u);
                y.y = __uint_as_float(__float_as_uint(y.y) & 0xfffffff0u);
                y = __fadd2_rn(y, make_float2(C, C));
                t[i] = y.x;
                t[i + 1] = y.y;
            }
        }
        return false;
    } else {
        float far = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            t[i] = fmaf(x[i], r, C);
            far = fmaxf(far, fabsf(fmaf(x[i], r, C - t[i])));
        }
        return far > 0.5f - 6.103515625e-5f;
    }
}

// N rounded integers + kToInt as int8 or fp16.
template <int N, bool WIDE>
__device__ __forceinline__ void store_integers(char* dst, const float (&t)[N]) {
    if constexpr (N == 1) {
        if constexpr (WIDE)
            *reinterpret_cast<__half*>(dst) = __float2half_rn(t[0] - kToInt<WIDE>);
        else
            *reinterpret_cast<uint8_t*>(dst) = static_cast<uint8_t>(__float_as_uint(t[0]));
    } else if constexpr (WIDE) {
        typename Raw<N * 2>::V o;
        __half2* h = reinterpret_cast<__half2*>(&o);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint32_t w =
                __byte_perm(__float_as_uint(t[2 * i]), __float_as_uint(t[2 * i + 1]), 0x5410);
            h[i] = __hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1152.0f));
        }
        *reinterpret_cast<typename Raw<N * 2>::V*>(dst) = o;
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint16_t*>(dst) =
            static_cast<uint16_t>(__byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040));
    } else {
        typename Raw<N>::V o;
        uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint32_t lo = __byte_perm(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]), 0x0040);
            const uint32_t hi = __byte_perm(__float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]), 0x0040);
            w[i] = __byte_perm(lo, hi, 0x5410);
        }
        *reinterpret_cast<typename Raw<N>::V*>(dst) = o;
    }
}

// WIDE: fp16 integers, padded; else int8.  A row's units start on the boundaries of N elements
// in memory; EDGE: what it has before its first and behind its last whole unit, up to 2 (N - 1)
// elements, goes to one thread each.
template <int DT, int N, bool WIDE, bool EDGE>
__global__ void __launch_bounds__(kThreads, kQuantBlocksPerSm<DT>)
quantize_kernel(const QuantParams p) {
    constexpr int ES = DT == DT_F32 ? 4 : 2, QS = WIDE ? 2 : 1;
    constexpr int R = quant_keep(N) / N;
    using V = typename Raw<N * ES>::V;
    using E = typename Raw<ES>::V;
    __shared__ uint32_t tops[2][kThreads / 32];
    if (WIDE) griddep_launch_dependents();
    const int tpr = 1 << p.tpr_log2, in = threadIdx.x & (tpr - 1);
    const int per_block = kThreads >> p.tpr_log2;
    const int warp = threadIdx.x >> 5, warps = tpr >> 5, lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
    // elements before a row's first whole unit; the end of its whole units
    auto head_of = [&](const char* src) {
        if (!EDGE) return 0;
        const int h = static_cast<int>((0 - reinterpret_cast<uintptr_t>(src) / ES) % N);
        return h < p.K ? h : p.K;
    };
    auto end_of = [&](int head) { return EDGE ? p.K - (p.K - head) % N : p.K; };
    // the element beside the units that is this thread's, or K
    auto edge_of = [&](int head, int end) {
        return in < head ? in : (in - head < p.K - end ? end + in - head : p.K);
    };
    auto load = [&](const char* src, int64_t c) { return __ldg(reinterpret_cast<const V*>(src + c * ES)); };
    V next[R];
    E next_edge = 0;
    auto fetch = [&](int64_t row) {
        if (row >= p.T) return;
        const char* src = static_cast<const char*>(p.x) + row * p.ld_x * ES;
        const int head = head_of(src), end = end_of(head);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (k * tpr + in) * N + head;
            if (c < end) next[k] = load(src, c);
        }
        if (EDGE) {
            const int c = edge_of(head, end);
            if (c < p.K) next_edge = __ldg(reinterpret_cast<const E*>(src) + c);
        }
    };
    fetch(static_cast<int64_t>(blockIdx.x) * per_block + (threadIdx.x >> p.tpr_log2));
    int turn = 0;
    // (whole blocks walk together: the maximum's barriers are the block's)
    for (int64_t rb = static_cast<int64_t>(blockIdx.x) * per_block; rb < p.T; rb += step) {
        const int64_t row = rb + (threadIdx.x >> p.tpr_log2);
        const bool live = row < p.T;
        const char* src = static_cast<const char*>(p.x) + row * p.ld_x * ES;
        const int head = head_of(src), end = end_of(head), edge = EDGE ? edge_of(head, end) : p.K;
        const int64_t more = static_cast<int64_t>(R * tpr + in) * N + head;  // units not kept
        V keep[R];
#pragma unroll
        for (int k = 0; k < R; ++k) keep[k] = next[k];
        const E keep_edge = next_edge;
        fetch(row + step);
        uint32_t top = 0;
        if (live) {
#pragma unroll
            for (int k = 0; k < R; ++k)
                if ((k * tpr + in) * N + head < end) top = larger<DT, N>(keep[k], top);
            for (int64_t c = more; c < end; c += tpr * N) top = larger<DT, N>(load(src, c), top);
            if (EDGE && edge < p.K) top = larger<DT, 1>(keep_edge, top);
        }
        top = magnitude<DT>(top);
        top = __reduce_max_sync(0xffffffffu, top);
        if (warps > 1) {
            // (two sets in turn: a warp is at most one row ahead of another's reading)
            if (lane == 0) tops[turn][warp] = top;
            __syncthreads();
            top = tops[turn][(warp & ~(warps - 1)) + (lane & (warps - 1))];
            top = __reduce_max_sync(0xffffffffu, top);
            turn ^= 1;
        }
        if (!live) continue;
        // (a row with an infinity or a NaN has no integers: a NaN scale says so)
        const bool finite = top < 0x7f800000u, some = finite && top != 0;
        const float size = __uint_as_float(top);
        if (in == 0) p.scales[row] = finite ? __fdiv_rn(size, 127.0f) : __uint_as_float(0x7fffffffu);
        // (a power of two keeps 127 / size and x 127 inside fp32; where it rounds an
        // element, that element's integer is zero)
        const float even = size < 0x1p-40f ? 0x1p100f : (size > 0x1p100f ? 0x1p-100f : 1.0f);
        // (within 2 ulp; see quotients)
        constexpr float above = DT == DT_F32 ? 1.0f : 1.0f + 0x1p-21f;
        const float r = some ? __fdividef(127.0f, size * even) * above : 0.0f;
        char* dst = static_cast<char*>(p.q) + row * p.ld_q * QS;
        auto put = [&](const V& v, int64_t c) {
            float f[N], t[N];
            widen<DT, N>(v, f);
            const bool again = quotients<DT, WIDE>(f, r, t);
            store_integers<N, WIDE>(dst + c * QS, t);
            return again;
        };
        auto put_one = [&](E v, int64_t c) {
            float f[1], t[1];
            widen<DT, 1>(v, f);
            f[0] *= even;
            if (quotients<DT, WIDE>(f, r, t))
                t[0] = quotient_exact(f[0], f[0] * r, size * even) + kToInt<WIDE>;
            if (!some) t[0] = kToInt<WIDE>;
            store_integers<1, WIDE>(dst + c * QS, t);
        };
        // units that need more care are read again, element by element, in one copy of the code
        const bool plain = some && even == 1.0f;
        uint32_t again = 0;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int c = (k * tpr + in) * N + head;
            if (c < end && (!plain || put(keep[k], c))) again |= 1u << k;
        }
        int64_t c = more;
        for (;;) {
            int64_t redo;
            if (again) {
                redo = (int64_t(__ffs(again) - 1) * tpr + in) * N + head;
                again &= again - 1;
            } else {
                if (c >= end) break;
                redo = c;
                c += tpr * N;
                if (plain && !put(load(src, redo), redo)) continue;
            }
#pragma unroll 1
            for (int i = 0; i < N; ++i)
                put_one(__ldg(reinterpret_cast<const E*>(src) + redo + i), redo + i);
        }
        if (EDGE && edge < p.K) put_one(keep_edge, edge);
        if (WIDE)
            for (int k = p.K + in; k < p.pad; k += tpr) reinterpret_cast<uint16_t*>(dst)[k] = 0;
    }
}

template <int DT, int N, bool WIDE, bool EDGE>
cudaError_t quantize_launch(QuantParams p, int sms, cudaStream_t stream) {
    // as few threads a row as keep it, but enough rows' worth of threads to fill the GPU: what
    // a thread does once a row costs as much as eight elements
    constexpr int keep = quant_keep(N);
    p.tpr_log2 = 5;
    while ((1 << p.tpr_log2) < kThreads && (p.K > int64_t(keep) << p.tpr_log2 ||
                                      (int64_t(p.T) << p.tpr_log2) < int64_t(sms) * 256))
        ++p.tpr_log2;
    int64_t blocks = cdiv(p.T, kThreads >> p.tpr_log2);
    if (blocks > int64_t(sms) * kQuantBlocksPerSm<DT>) blocks = int64_t(sms) * kQuantBlocksPerSm<DT>;
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
