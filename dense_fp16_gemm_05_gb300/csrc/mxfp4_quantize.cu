// mxfp4_quantize.cu -- quantisation to MXFP4 (OCP microscaling formats, version
// 1.0: E2M1 elements, one E8M0 scale per 32 elements along K):
//
//   e = floor(log2 max |x|) - 2 over the block, kept in -127 .. 127
//       (2 = the exponent of E2M1's largest value, 6 = 1.5 * 2^2);
//   code(x) = x 2^-e rounded to the nearest E2M1 value, ties to even,
//             beyond 6 to 6;   scale byte = e + 127.
//
// A block of zeros gets scale byte 0; a block that holds an infinity or a NaN,
// which E2M1 lacks, gets the NaN scale byte 0xFF and zero codes, so that it
// does not vanish from a product.  floor(log2) is read from the exponent bits
// of the block's largest magnitude and 2^-e is a power of two in fp32, so the
// only rounding is the conversion to E2M1.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "gemm_f16.h"
#include "gemm_mxfp4_launch.cuh"

namespace {

using namespace gemm_sm103;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight values -> eight E2M1 codes, element i in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The values of eight codes.
__device__ __forceinline__ void e2m1x8_values(uint32_t codes, float (&v)[8])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Scale byte of a block whose largest |x| has the bit pattern `amax` (fp32).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    const uint32_t ex = amax >> 23;   // sign bit is clear
    if (ex == 255u) return 255u;
    return ex > 2u ? ex - 2u : 0u;
}

// 2^-(byte - 127), and 2^(byte - 127); byte <= 252, or 255 (NaN).
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    if (byte == 255u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);   // 2^-127 is subnormal
}

__device__ __forceinline__ int64_t scale_offset(int64_t row, int b, int k_tiles)
{
    return ((row >> 7) * k_tiles + (b >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (b & 3);
}

struct QuantParams {
    uint8_t *Q;
    uint8_t *S;
    int64_t rows;
    int32_t K, KB, k_tiles;
    int32_t groups;        // 8-element groups per row, 4 KB
    int64_t step_rows;     // grid stride in groups = step_rows * groups + step_groups
    int32_t step_groups;
};

// Eight adjacent elements of X, zeros past the row's end.
template <class T, bool kVec>
struct QuantGroup {
    static constexpr int W = sizeof(T) * 8 / 16;
    uint4 raw[W];

    __device__ __forceinline__ void load(const T *x, int k0, int K)
    {
        if constexpr (kVec) {   // K is a multiple of 8 and the rows are 16-byte aligned
#pragma unroll
            for (int i = 0; i < W; ++i)
                raw[i] = k0 < K ? __ldg(reinterpret_cast<const uint4 *>(x + k0) + i) : make_uint4(0u, 0u, 0u, 0u);
        } else {
            T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = k0 + i < K ? __ldg(x + k0 + i) : from_float<T>(0.0f);
            memcpy(raw, e, sizeof(raw));
        }
    }
};

// Eight elements per thread, a block per four neighbouring lanes; the next
// group's loads are under way while a group is converted.
template <class T, bool kVec, bool kValues>
__global__ void __launch_bounds__(256) mxfp4_quantize_rows(const T *__restrict__ X, T *__restrict__ V, QuantParams p)
{
    griddep_wait();   // X may come from the kernel just before
    griddep_launch_dependents();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    int64_t row = first / p.groups;
    int g = static_cast<int>(first - row * p.groups);
    QuantGroup<T, kVec> next;
    if (row < p.rows) next.load(X + row * p.K, g * 8, p.K);
    // All four lanes of a block have the same row, so they leave together.
    while (row < p.rows) {
        const int k0 = g * 8;
        float v[8];
        {
            T e[8];
            memcpy(e, next.raw, sizeof(e));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
        }
        int64_t next_row = row + p.step_rows;
        int next_g = g + p.step_groups;
        if (next_g >= p.groups) {
            next_g -= p.groups;
            ++next_row;
        }
        if (next_row < p.rows) next.load(X + next_row * p.K, next_g * 8, p.K);
        // Largest magnitude as an integer: NaN's pattern is above infinity's.
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        const uint32_t lanes = 0xFu << (threadIdx.x & 28u);
        amax = max(amax, __shfl_xor_sync(lanes, amax, 1));
        amax = max(amax, __shfl_xor_sync(lanes, amax, 2));
        const uint32_t byte = scale_byte(amax);
        uint32_t codes = 0;
        if (byte != 255u) {
            const float inv = inverse_scale(byte);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= inv;
            codes = e2m1x8(v);
        }
        *reinterpret_cast<uint32_t *>(p.Q + row * (static_cast<int64_t>(p.KB) * 16) + g * 4) = codes;
        if ((g & 3) == 0) {
            const int b = g >> 2;
            uint8_t *s = p.S + scale_offset(row, b, p.k_tiles);
            *s = static_cast<uint8_t>(byte);
            // The blocks that fill up the last tile multiply zero operands: not NaN.
            if (b == p.KB - 1)
                for (int i = 1; b + i < 4 * p.k_tiles; ++i) s[i] = 0;
        }
        if constexpr (kValues) {
            const float sc = scale_value(byte);
            e2m1x8_values(codes, v);
            T *out = V + row * p.K + k0;
            T t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = from_float<T>(v[i] * sc);
            if constexpr (kVec) {
                constexpr int W = sizeof(T) * 8 / 16;
                if (k0 < p.K) {
                    uint4 raw[W];
                    memcpy(raw, t, sizeof(raw));
#pragma unroll
                    for (int i = 0; i < W; ++i) reinterpret_cast<uint4 *>(out)[i] = raw[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k0 + i < p.K) out[i] = t[i];
            }
        }
        row = next_row;
        g = next_g;
    }
}

// X stored (K, rows).  A block takes 128 elements of K (one scale tile's four
// blocks of 32, one per warp) of 32 kCols rows of the result; a thread loads
// kCols adjacent elements of each of its block's 32 rows of X, so a warp reads
// 128 bytes at a time.  Its codes and values then lie along K, 16 adjacent bytes
// here and there in 32 rows: they go through shared memory, so that a row's 64
// bytes of codes and 128 values are written together (stored by each thread
// element by element, values took 144 us at 4096 x 4096 fp16, COLUS this way).
template <class T, int kCols, bool kValues>
__global__ void __launch_bounds__(128) mxfp4_quantize_cols(const T *__restrict__ X, T *__restrict__ V, QuantParams p,
                                                           bool v_vec)
{
    constexpr int R = 32 * kCols;                                    // rows of the result per block
    constexpr int CHUNKS = 128 * static_cast<int>(sizeof(T)) / 16;   // 16-byte pieces of a row's values
    constexpr int PER = 16 / static_cast<int>(sizeof(T));            // values per piece
    // Piece c of row r lies at piece c ^ ((r / kCols) % 8): a warp's writes, one
    // piece of every row, then fall into different banks.
    __shared__ uint4 sv[kValues ? R * CHUNKS : 1];
    __shared__ uint4 sq[R * 4];
    __shared__ uint8_t ss[R * 4];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * R;
    for (int kt = static_cast<int>(blockIdx.y); kt < p.k_tiles; kt += static_cast<int>(gridDim.y)) {
        const int k0 = kt * 128 + w * 32;
        const int n = min(32, p.K - k0);   // <= 0: a block past K
        const int64_t col = row0 + lane * kCols;
        T x[32][kCols];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const T *src = X + static_cast<int64_t>(k0 + i) * p.rows + col;
            if constexpr (kCols == 2) {   // rows is even and X 4-byte aligned
                uint32_t v = 0;
                if (i < n && col < p.rows) v = __ldg(reinterpret_cast<const uint32_t *>(src));
                memcpy(x[i], &v, 4);
            } else {
                x[i][0] = i < n && col < p.rows ? __ldg(src) : from_float<T>(0.0f);
            }
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const int r = lane * kCols + c;
            const int sw = lane & 7;
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) amax = max(amax, __float_as_uint(to_float(x[i][c])) & 0x7FFFFFFFu);
            const uint32_t byte = scale_byte(amax);
            uint32_t codes[4] = {0, 0, 0, 0};
            if (byte != 255u) {
                const float inv = inverse_scale(byte);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = to_float(x[8 * j + i][c]) * inv;
                    codes[j] = e2m1x8(v);
                }
            }
            sq[r * 4 + (w ^ (sw & 3))] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            // A block past K: scale 0, as the blocks that fill up the tile.
            ss[r * 4 + w] = static_cast<uint8_t>(byte);
            if constexpr (kValues) {
                const float sc = scale_value(byte);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v[8];
                    e2m1x8_values(codes[j], v);
                    T t[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = from_float<T>(v[i] * sc);
                    constexpr int W = 8 / PER;
                    uint4 raw[W];
                    memcpy(raw, t, sizeof(raw));
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        sv[r * CHUNKS + ((w * (CHUNKS / 4) + j * W + i) ^ sw)] = raw[i];
                }
            }
        }
        __syncthreads();
        // Codes: 64 bytes per row, as many of them as the row has blocks.
        for (int i = threadIdx.x; i < R * 4; i += 128) {
            const int r = i >> 2, b = i & 3;
            if (row0 + r < p.rows && kt * 4 + b < p.KB)
                *reinterpret_cast<uint4 *>(p.Q + (row0 + r) * (static_cast<int64_t>(p.KB) * 16) + (kt * 4 + b) * 16) =
                    sq[r * 4 + (b ^ ((r / kCols) & 3))];
        }
        // Scales: a row's four bytes of the tile.
        if (threadIdx.x < R && row0 + threadIdx.x < p.rows)
            *reinterpret_cast<uint32_t *>(p.S + scale_offset(row0 + threadIdx.x, kt * 4, p.k_tiles)) =
                *reinterpret_cast<const uint32_t *>(ss + threadIdx.x * 4);
        if constexpr (kValues) {
            if (v_vec) {
                for (int i = threadIdx.x; i < R * CHUNKS; i += 128) {
                    const int r = i / CHUNKS, c = i % CHUNKS;
                    const int k = kt * 128 + c * PER;
                    if (row0 + r < p.rows && k < p.K)
                        *reinterpret_cast<uint4 *>(V + (row0 + r) * p.K + k) = sv[r * CHUNKS + (c ^ ((r / kCols) & 7))];
                }
            } else {
                const T *e = reinterpret_cast<const T *>(sv);
                for (int i = threadIdx.x; i < R * 128; i += 128) {
                    const int r = i >> 7, kk = i & 127;
                    if (row0 + r < p.rows && kt * 128 + kk < p.K)
                        V[(row0 + r) * p.K + kt * 128 + kk] =
                            e[(r * CHUNKS + ((kk / PER) ^ ((r / kCols) & 7))) * PER + kk % PER];
                }
            }
        }
        __syncthreads();   // before the next tile's writes
    }
}

template <class... Args>
int launch_pdl(void (*kern)(Args...), dim3 grid, unsigned threads, cudaStream_t stream, Args... args)
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

template <class T>
int quantize(const Mx4QuantArgs &a)
{
    QuantParams p{};
    p.Q = a.Q;
    p.S = a.S;
    p.rows = a.rows;
    p.K = static_cast<int32_t>(a.K);
    p.KB = static_cast<int32_t>((a.K + 31) / 32);
    p.k_tiles = static_cast<int32_t>(mx4_k_tiles(a.K));
    p.groups = p.KB * 4;
    const T *X = static_cast<const T *>(a.X);
    T *V = static_cast<T *>(a.V);
    if (a.trans) {
        const bool v_vec = a.K % (16 / static_cast<int64_t>(sizeof(T))) == 0 && (reinterpret_cast<uintptr_t>(V) & 15u) == 0;
        const unsigned gy = static_cast<unsigned>(p.k_tiles < 65535 ? p.k_tiles : 65535);
        if constexpr (sizeof(T) == 2) {
            if (a.rows % 2 == 0 && (reinterpret_cast<uintptr_t>(X) & 3u) == 0) {
                const dim3 grid(static_cast<unsigned>((a.rows + 63) / 64), gy, 1);
                return V ? launch_pdl(mxfp4_quantize_cols<T, 2, true>, grid, 128, a.stream, X, V, p, v_vec)
                         : launch_pdl(mxfp4_quantize_cols<T, 2, false>, grid, 128, a.stream, X, V, p, v_vec);
            }
        }
        const dim3 grid(static_cast<unsigned>((a.rows + 31) / 32), gy, 1);
        return V ? launch_pdl(mxfp4_quantize_cols<T, 1, true>, grid, 128, a.stream, X, V, p, v_vec)
                 : launch_pdl(mxfp4_quantize_cols<T, 1, false>, grid, 128, a.stream, X, V, p, v_vec);
    }
    const int64_t total = a.rows * p.groups;
    const int64_t max_blocks = static_cast<int64_t>(a.sm_count) * 8;
    int64_t blocks = (total + 255) / 256;
    if (blocks > max_blocks) blocks = max_blocks;
    const int64_t step = blocks * 256;
    p.step_rows = step / p.groups;
    p.step_groups = static_cast<int32_t>(step % p.groups);
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.V);
    const bool vec = (a.K % 8) == 0 && (bits & 15u) == 0;
    const dim3 grid(static_cast<unsigned>(blocks), 1, 1);
    if (vec)
        return V ? launch_pdl(mxfp4_quantize_rows<T, true, true>, grid, 256, a.stream, X, V, p)
                 : launch_pdl(mxfp4_quantize_rows<T, true, false>, grid, 256, a.stream, X, V, p);
    return V ? launch_pdl(mxfp4_quantize_rows<T, false, true>, grid, 256, a.stream, X, V, p)
             : launch_pdl(mxfp4_quantize_rows<T, false, false>, grid, 256, a.stream, X, V, p);
}

}  // namespace

namespace gemm_sm103 {

int launch_mxfp4_quantize(const Mx4QuantArgs &a)
{
    switch (a.type) {
    case GEMM_TYPE_F16: return quantize<__half>(a);
    case GEMM_TYPE_BF16: return quantize<__nv_bfloat16>(a);
    default: return quantize<float>(a);
    }
}

}  // namespace gemm_sm103
