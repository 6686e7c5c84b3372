// layer_norm.cuh -- shared pieces of the layer norm kernels (layer_norm_fwd.cu,
// layer_norm_bwd.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "gemm_f16.h"
#include "gemm_launch.cuh"
#include "sm103_ptx.cuh"

namespace gemm_sm103 {

struct LayerNormArgs {
    const void *X = nullptr, *gamma = nullptr, *beta = nullptr, *dY = nullptr;
    void *Y = nullptr;                          // forward output, or dX
    float *mean = nullptr, *rstd = nullptr;     // written forward, read backward
    void *dgamma = nullptr, *dbeta = nullptr;
    float *workspace = nullptr;                 // 2 x parts x dim floats (backward)
    int64_t rows = 0;
    int64_t dim = 0;
    float eps = 0.0f;
    int xtype = 0, wtype = 0;
    int sm_count = 0, device = 0;
    cudaStream_t stream = nullptr;
    unsigned long long *status = nullptr;       // device status word
    int withhold = 0;                           // test hook (layer_norm_bwd_selftest_timeout)
    uint64_t timeout_cycles = 0;                // 0: the normal budget
};

int launch_layer_norm_fwd(const LayerNormArgs &a);
int launch_layer_norm_bwd(const LayerNormArgs &a);
// Partial sums of the weights' gradients that a backward call writes per column.
int64_t layer_norm_parts(int64_t rows, int64_t dim, int sm_count);

__device__ __forceinline__ float ln_float(float x) { return x; }
__device__ __forceinline__ float ln_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float ln_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T ln_round(float x);
template <>
__device__ __forceinline__ float ln_round<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half ln_round<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 ln_round<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ float2 ln_pair(uint32_t raw, __half)
{
    __half2 h;
    memcpy(&h, &raw, 4);
    return __half22float2(h);
}
__device__ __forceinline__ float2 ln_pair(uint32_t raw, __nv_bfloat16)
{
    return make_float2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t ln_raw_pair(float2 v, __half)
{
    const __half2 h = __float22half2_rn(v);
    uint32_t raw;
    memcpy(&raw, &h, 4);
    return raw;
}
__device__ __forceinline__ uint32_t ln_raw_pair(float2 v, __nv_bfloat16)
{
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    uint32_t raw;
    memcpy(&raw, &h, 4);
    return raw;
}

// V adjacent elements, loaded and stored in pieces of 16, 8 or 4 bytes where V
// elements make them up (the caller vouches for the alignment), else one by one.
template <class T, int V>
struct LnPack {
    T e[V];

    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (V * sizeof(T) % 16 == 0) {
            uint4 raw[V * sizeof(T) / 16];
#pragma unroll
            for (unsigned i = 0; i < V * sizeof(T) / 16; ++i) raw[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            memcpy(e, raw, sizeof(e));
        } else if constexpr (V * sizeof(T) == 8) {
            const uint2 raw = __ldg(reinterpret_cast<const uint2 *>(p));
            memcpy(e, &raw, sizeof(e));
        } else if constexpr (V * sizeof(T) == 4 && V > 1) {
            const uint32_t raw = __ldg(reinterpret_cast<const uint32_t *>(p));
            memcpy(e, &raw, sizeof(e));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = __ldg(p + i);
        }
    }
    __device__ __forceinline__ void load_shared(const T *p)   // an element, four bytes or whole 16-byte pieces
    {
        if constexpr (V == 1) {
            e[0] = *p;
            return;
        } else if constexpr (V * sizeof(T) == 4) {
            const uint32_t raw = *reinterpret_cast<const uint32_t *>(p);
            memcpy(e, &raw, sizeof(e));
            return;
        }
        constexpr unsigned N = V * sizeof(T) / 16 > 0 ? V * sizeof(T) / 16 : 1;
        uint4 raw[N];
#pragma unroll
        for (unsigned i = 0; i < N; ++i) raw[i] = reinterpret_cast<const uint4 *>(p)[i];
        memcpy(e, raw, sizeof(e));
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (V * sizeof(T) % 16 == 0) {
            uint4 raw[V * sizeof(T) / 16];
            memcpy(raw, e, sizeof(e));
#pragma unroll
            for (unsigned i = 0; i < V * sizeof(T) / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = raw[i];
        } else if constexpr (V * sizeof(T) == 8) {
            uint2 raw;
            memcpy(&raw, e, sizeof(e));
            *reinterpret_cast<uint2 *>(p) = raw;
        } else if constexpr (V * sizeof(T) == 4 && V > 1) {
            uint32_t raw;
            memcpy(&raw, e, sizeof(e));
            *reinterpret_cast<uint32_t *>(p) = raw;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = e[i];
        }
    }
    __device__ __forceinline__ void fill(float v)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = ln_round<T>(v);
    }
    __device__ __forceinline__ float operator[](int i) const { return ln_float(e[i]); }
    // Hides from the compiler that the elements are the ones it has seen.
    __device__ __forceinline__ void opaque()
    {
        if constexpr (V * sizeof(T) % 4 == 0) {
            uint32_t raw[V * sizeof(T) / 4];
            memcpy(raw, e, sizeof(e));
#pragma unroll
            for (unsigned i = 0; i < V * sizeof(T) / 4; ++i) asm volatile("" : "+r"(raw[i]));
            memcpy(e, raw, sizeof(e));
        }
    }
    // Elements 2i and 2i + 1, rounded to T: 16-bit ones by one instruction.
    __device__ __forceinline__ void set_pair(int i, float2 v)
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t raw = ln_raw_pair(v, T{});
            memcpy(e + 2 * i, &raw, 4);
        } else {
            e[2 * i] = v.x;
            e[2 * i + 1] = v.y;
        }
    }
    // Elements 2i and 2i + 1.
    __device__ __forceinline__ float2 pair(int i) const
    {
        if constexpr (sizeof(T) == 2) {
            uint32_t raw;
            memcpy(&raw, e + 2 * i, 4);
            return ln_pair(raw, T{});
        } else {
            return make_float2(e[2 * i], e[2 * i + 1]);
        }
    }
};

// Elements per pack that a call's alignments allow: 16 bytes of X's type, four
// bytes (two 16-bit elements), or one element.  x_bits: the rows' addresses and
// bytes per row, w_bits: the weights' addresses, each or-ed together.  A pack of
// weights has as many elements as one of X, so the same pieces ask for twice the
// alignment where fp32 weights stand beside 16-bit rows.
template <class T, class W>
int ln_pack_elements(uintptr_t x_bits, uintptr_t w_bits)
{
    if (((x_bits | w_bits) & 15u) == 0) return 16 / static_cast<int>(sizeof(T));
    if (sizeof(T) == 2 && (x_bits & 3u) == 0 && (w_bits & (2 * sizeof(W) - 1)) == 0) return 2;
    return 1;
}

// Elements 2m and 2m + 1 of NV packs in order.
template <class T, int V, int NV>
__device__ __forceinline__ float2 ln_pair_of(const LnPack<T, V> (&p)[NV], int m)
{
    if constexpr (V == 1) return make_float2(p[2 * m][0], p[2 * m + 1][0]);
    else return p[m / (V / 2)].pair(m % (V / 2));
}

__device__ __forceinline__ float ln_half(float2 v, int j) { return (j & 1) == 0 ? v.x : v.y; }

// Sum over N neighbouring lanes.
template <int N = 32>
__device__ __forceinline__ float ln_warp_sum(float v)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Threads of a row, as a template argument: TPR <= 32, lanes of a warp; TPR > 32
// (a power of 2), a block; TPR < 0, a block of whole warps chosen at launch, up
// to -TPR threads, so that rows of any length leave few threads idle.
template <int TPR>
__device__ __forceinline__ int ln_threads()
{
    if constexpr (TPR > 0) return TPR;
    else return static_cast<int>(blockDim.x);
}
__host__ __device__ constexpr int ln_warps(int tpr) { return tpr < 0 ? -tpr / 32 : (tpr <= 32 ? 1 : tpr / 32); }

// Sums over the threads of a row, the same bits in each of them; for a block
// through `sh` (ln_warps entries), not in use by an earlier sum that some thread
// may still be reading.  Every warp adds the warps' sums by shuffles: reading
// them one by one costs a load and an add per warp in every thread, a third of
// the backward pass's instructions for 512 threads.
template <int TPR>
__device__ __forceinline__ float ln_row_sum(float v, float *sh)
{
    v = ln_warp_sum<(TPR > 0 && TPR < 32 ? TPR : 32)>(v);
    if constexpr (TPR > 32 || TPR < 0) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
        if constexpr (TPR > 0) v = ln_warp_sum<TPR / 32>(sh[lane & (TPR / 32 - 1)]);
        else v = ln_warp_sum<32>(lane < static_cast<int>(blockDim.x >> 5) ? sh[lane] : 0.0f);
    }
    return v;
}

// Two sums at once.  The first exchange gives each half of the warp one of them,
// so the steps after it add both with one shuffle each: 10 shuffles for 512
// threads where two separate sums take 18.
template <int TPR>
__device__ __forceinline__ float2 ln_row_sum2(float a, float b, float2 *sh)
{
    if constexpr (TPR > 0 && TPR < 32) {
        return make_float2(ln_warp_sum<TPR>(a), ln_warp_sum<TPR>(b));
    } else {
        const int lane = threadIdx.x & 31;
        const bool upper = (lane & 16) != 0;   // holds b's sum, the lower half a's
        float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
        v = ln_warp_sum<16>(v);
        if constexpr (TPR != 32) {
            float *part = reinterpret_cast<float *>(sh);   // (warps, 2)
            if ((lane & 15) == 0) part[2 * (threadIdx.x >> 5) + (upper ? 1 : 0)] = v;
            __syncthreads();
            const int warps = TPR > 0 ? ln_warps(TPR) : static_cast<int>(blockDim.x >> 5);
            const int w = lane & 15, half = upper ? 1 : 0;
            if constexpr (TPR > 0 && ln_warps(TPR) <= 16) {
                v = ln_warp_sum<ln_warps(TPR)>(part[2 * (w & (ln_warps(TPR) - 1)) + half]);
            } else {
                v = w < warps ? part[2 * w + half] : 0.0f;
                if (w + 16 < warps) v += part[2 * (w + 16) + half];
                v = ln_warp_sum<16>(v);
            }
        }
        const float other = __shfl_xor_sync(0xffffffffu, v, 16);
        return upper ? make_float2(other, v) : make_float2(v, other);
    }
}

// s / n, correctly rounded, given 1 / n: the product's error is its remainder, exact
// by one fused multiply-add, over n (P. Markstein, IBM J. Res. Dev. 34, 1990).
// Rows of odd widths are bound by instructions and feel it: 16384 x 4097 fp16
// takes 104.1 us with the product alone, 105.1 so, 108.2 with the operator /.
__device__ __forceinline__ float ln_quotient(float s, float n, float inv)
{
    const float q = s * inv;
    const float r = fmaf(-q, n, s);
    return r == r ? fmaf(r, inv, q) : q;   // infinite or NaN: no remainder
}

// Launch as a programmatic dependent of the previous kernel on the stream (the
// kernels wait for it before touching memory).
template <class... Args>
int ln_launch(void (*kern)(Args...), dim3 grid, unsigned threads, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = dim3(threads, 1, 1);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaLaunchKernelEx(&lc, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// Calls f(T{}, W{}) for the element types of a call: W is X's type or float.
template <class F>
int ln_dispatch(int xtype, int wtype, F f)
{
    if (xtype == GEMM_TYPE_F32) return f(float{}, float{});
    if (xtype == GEMM_TYPE_F16) return wtype == GEMM_TYPE_F32 ? f(__half{}, float{}) : f(__half{}, __half{});
    return wtype == GEMM_TYPE_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}

}  // namespace gemm_sm103
