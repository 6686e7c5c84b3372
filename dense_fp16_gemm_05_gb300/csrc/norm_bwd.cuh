// norm_bwd.cuh -- shared pieces of the norms' backward kernels
// (layer_norm_bwd.cu, rms_norm_bwd.cu): rows through a ring of bulk copies, and
// the second kernel, which adds the blocks' partial sums.
#pragma once

#include <atomic>
#include <type_traits>

#include "gemm_kernel.cuh"
#include "layer_norm.cuh"

namespace gemm_sm103 {

constexpr int kRingStages = 4;   // rows under way per block, at most

// Packs that do not make up 16-byte pieces: rows of other lengths and
// alignments, copied with the whole 16-byte pieces that they lie in.
template <class T, int V>
constexpr bool kRingAny = V * sizeof(T) < 16;

// Bytes of a row's place in the ring.
template <class T, int V>
__host__ __device__ __forceinline__ uint32_t ring_row_bytes(int dim)
{
    const uint32_t bytes = static_cast<uint32_t>(dim) * static_cast<uint32_t>(sizeof(T));
    return kRingAny<T, V> ? (bytes + 15u) / 16u * 16u + 16u : bytes;
}

// The 16-byte pieces of global memory that hold `bytes` bytes at `src`, and what
// of them lies inside the tensor [lo, hi): the rest is not read.
struct RingWindow {
    uint64_t first, begin, end, src, last;

    __device__ __forceinline__ RingWindow(uint64_t src_, uint32_t bytes, uint64_t lo, uint64_t hi)
    {
        src = src_;
        last = src + bytes;
        first = src & ~15ull;
        begin = first < lo ? first + 16 : first;
        end = (last + 15ull) & ~15ull;
        if (end > hi) end -= 16;
        if (end < begin) end = begin;
    }
};

// Adds x to s and what the addition loses to c (Knuth's exact error of a sum): s + c
// then has the terms' sum but for errors of second order.
__device__ __forceinline__ void ln_add_exact(float &s, float &c, float x)
{
    const float t = s + x;
    const float b = t - s;
    c += (s - (t - b)) + (x - b);
    s = t;
}

// Adds the parts of 32 columns: NW warps take every NW-th part, then their sums
// are added in a tree of fixed order.  There are hundreds of parts of both signs,
// so what their additions lose is kept and added last: the result is the parts'
// sum rounded once.  (Both kernels, with plain sums one after another and so:
// 16384 x 4096 fp16 75.0 us and 74.7, 8192 x 768 19.3 and 19.9, 4096 x 5000 fp32
// 45.0 and 45.5; in fp64 the additions alone would be 4 us at 16384 x 4096.)
template <class W, int NW>
__global__ void __launch_bounds__(NW * 32) norm_bwd_finish(const float *__restrict__ part, W *__restrict__ dgamma,
                                                           W *__restrict__ dbeta, int parts, int dim)
{
    __shared__ float sh[NW][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const float *src = part + static_cast<int64_t>(blockIdx.y) * parts * dim;
    float s = 0.0f, c = 0.0f;
    if (k < dim) {
        auto at = [&](int r) { return src[static_cast<int64_t>(r) * dim + k]; };
        // Ten loads under way at a time, or four for the last few: a few hundred parts
        // come at once.  Zeros in the place of parts that are not there change no sum.
        // (RMS norm, both kernels, with eight and the rest by fours: 1000 x 1024 fp16
        // 7.5 us, 6.2 us so; 64 x 4096 5.5 and 5.4.)
        auto batch = [&](auto count, int r0) {
            constexpr int B = decltype(count)::value;
            float x[B];
#pragma unroll
            for (int i = 0; i < B; ++i) x[i] = r0 + i * NW < parts ? at(r0 + i * NW) : 0.0f;
#pragma unroll
            for (int i = 0; i < B; ++i) ln_add_exact(s, c, x[i]);
        };
        int r = w;
        for (; r + 4 * NW < parts; r += 10 * NW) batch(std::integral_constant<int, 10>{}, r);
        if (r < parts) batch(std::integral_constant<int, 4>{}, r);
    }
    // NW neighbouring lanes take a column's sums.  One array for both: with two
    // these blocks started later (1000 x 1023 fp32: 11.3 us, 8.7 us so), likely for
    // another split of the SM between L1 and shared memory than the main kernel's.
    const int column = threadIdx.x / NW, from = threadIdx.x % NW;
    sh[w][lane] = s;
    __syncthreads();
    s = sh[from][column];
    __syncthreads();
    sh[w][lane] = c;
    __syncthreads();
    c = sh[from][column];
#pragma unroll
    for (int o = NW / 2; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, s, o);
        const float other_lost = __shfl_xor_sync(0xffffffffu, c, o);
        ln_add_exact(s, c, other);
        c += other_lost;
    }
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + column;
    // Of a sum that is infinite or NaN the errors are NaN.
    if (from == 0 && out < dim) (blockIdx.y == 0 ? dgamma : dbeta)[out] = ln_round<W>(c == c ? s + c : s);
}

}  // namespace gemm_sm103
