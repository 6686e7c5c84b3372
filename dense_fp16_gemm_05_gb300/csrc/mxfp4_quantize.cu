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
// does not vanish from a product (with the fused ReLU it does: R(NaN) is +0 in
// every GEMM of the library).  floor(log2) is read from the exponent bits
// of the block's largest magnitude and 2^-e is a power of two in fp32, so the
// only rounding is the conversion to E2M1.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "gemm_f16.h"
#include "gemm_mxfp4_launch.cuh"
#include "sm103_ptx.cuh"

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

// Two values -> a byte of two codes, the first in its low half.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, z;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tmov.b32 %0, {b0, 0, 0, 0};\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// The values of eight codes as four binary16 pairs.
__device__ __forceinline__ void e2m1x8_halves(uint32_t codes, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// The values of eight codes.
__device__ __forceinline__ void e2m1x8_values(uint32_t codes, float (&v)[8])
{
    uint32_t h[4];
    e2m1x8_halves(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Largest magnitude of some elements as an fp32 bit pattern; NaN's pattern is
// above infinity's.  16-bit elements are compared two at a time.
template <class T, int G>
__device__ __forceinline__ uint32_t max_magnitude(const T (&e)[G])
{
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) m = max(m, __float_as_uint(e[i]) & 0x7FFFFFFFu);
        return m;
    } else {
        uint32_t raw[G / 2];
        memcpy(raw, e, sizeof(raw));
        uint32_t m = raw[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < G / 2; ++i) m = __vmaxu2(m, raw[i] & 0x7FFF7FFFu);
        const uint16_t top = static_cast<uint16_t>(max(m & 0xFFFFu, m >> 16));
        T t;
        memcpy(&t, &top, sizeof(top));
        return __float_as_uint(to_float(t)) & 0x7FFFFFFFu;
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

__device__ __forceinline__ int64_t scale_offset(int row, int b, int k_tiles)
{
    return static_cast<int64_t>(row >> 7) * (static_cast<int64_t>(k_tiles) * 512) +
           static_cast<int64_t>(b >> 2) * 512 + ((row & 31) * 16 + ((row >> 5) & 3) * 4 + (b & 3));
}

struct QuantParams {
    uint8_t *Q;
    uint8_t *S;
    int32_t rows;
    int32_t K, KB, k_tiles;
    int32_t groups;        // groups (one thread's elements) per row
    int32_t step_rows;     // grid stride in groups = step_rows * groups + step_groups
    int32_t step_groups;
    int64_t step_x;        // the same stride in elements of X
};

// G adjacent elements of X, of which the row has `left`, zeros past its end;
// rows are whole pieces of 16 bytes, 16-byte aligned.
template <class T, int G>
struct QuantGroup {
    static constexpr int W = G * static_cast<int>(sizeof(T)) / 16;   // pieces of 16 bytes
    uint4 raw[W];

    __device__ __forceinline__ void load(const T *x, int left)
    {
#pragma unroll
        for (int i = 0; i < W; ++i)
            raw[i] = left > G / W * i ? __ldg(reinterpret_cast<const uint4 *>(x) + i) : make_uint4(0u, 0u, 0u, 0u);
    }
};

// The values of G codes (packed in order) times their block's scale, in T.
template <class T, int G>
__device__ __forceinline__ void group_values(const uint32_t *codes, uint32_t byte, T (&t)[G])
{
    if (std::is_same<T, __half>::value && byte >= 103u && byte != 255u) {
        // 2^(byte - 127) is a binary16 number too (a block of binary16 numbers
        // has no larger scale): one rounding, as in fp32.
        const __half2 sc = __float2half2_rn(scale_value(byte));
#pragma unroll
        for (int h = 0; h < G / 8; ++h) {
            uint32_t v[4];
            e2m1x8_halves(codes[h], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __half2 x;
                memcpy(&x, &v[i], 4);
                x = __hmul2(x, sc);
                memcpy(t + 8 * h + 2 * i, &x, 4);
            }
        }
        return;
    }
    const float sc = scale_value(byte);
#pragma unroll
    for (int h = 0; h < (G + 7) / 8; ++h) {
        float v[8];
        e2m1x8_values(codes[h], v);
#pragma unroll
        for (int i = 0; i < (G < 8 ? G : 8); i += 2) {
            const float2 x = mul_f32x2(make_float2(v[i], v[i + 1]), make_float2(sc, sc));
            t[8 * h + i] = from_float<T>(x.x);
            t[8 * h + i + 1] = from_float<T>(x.y);
        }
    }
}

// Elements per thread.  Codes alone: 16, for by counters the pass is then bound
// by instructions before it is by bytes (issue slots 75 % busy with eight).  With
// the values: one 16-byte piece, so that a warp's stores are adjacent.
// (8192^2 fp16: codes 41 us with 8 per thread, 28 us with 16; with the values
// 50 us and 57 us.)
template <class T, bool kValues>
constexpr int kQuantGroup = kValues ? 16 / static_cast<int>(sizeof(T)) : 16;

// Blocks per SM (one wave): as many as the registers allow without spilling.
template <class T, bool kValues>
constexpr int kQuantBlocks = kValues ? 6 : (sizeof(T) == 2 ? 5 : 4);

// A block of 32 per 32 / G neighbouring lanes; the next group's loads are under
// way while a group is converted.
template <class T, bool kValues>
__global__ void __launch_bounds__(256, kQuantBlocks<T, kValues>)
    mxfp4_quantize_rows(const T *__restrict__ X, T *__restrict__ V, QuantParams p)
{
    constexpr int G = kQuantGroup<T, kValues>;
    constexpr int LANES = 32 / G;
    griddep_wait();   // X may come from the kernel just before
    griddep_launch_dependents();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    int row = static_cast<int>(first / p.groups);
    int g = static_cast<int>(first - static_cast<int64_t>(row) * p.groups);
    // Offsets of the thread's group in X (and V) and in Q, whose rows are whole
    // groups.
    int64_t at = static_cast<int64_t>(row) * p.K + g * G;
    uint8_t *q = p.Q + first * (G / 2);
    const int64_t step_q = static_cast<int64_t>(gridDim.x) * blockDim.x * (G / 2);
    const uint32_t lanes = ((1u << LANES) - 1u) << (threadIdx.x & 31u & ~static_cast<uint32_t>(LANES - 1));
    QuantGroup<T, G> next;
    if (row < p.rows) next.load(X + at, p.K - g * G);
    // All lanes of a block have the same row, so they leave together.
    while (row < p.rows) {
        const int left = p.K - g * G;   // elements of the row from here on
        T e[G];
        memcpy(e, next.raw, sizeof(e));
        // Unsigned: rows of the next group may pass 2^31 after the last one.
        uint32_t next_row = static_cast<uint32_t>(row) + static_cast<uint32_t>(p.step_rows);
        int64_t next_at = at + p.step_x;
        int next_g = g + p.step_groups;
        if (next_g >= p.groups) {
            next_g -= p.groups;
            ++next_row;
            next_at += p.K - static_cast<int64_t>(p.groups) * G;
        }
        if (next_row < static_cast<uint32_t>(p.rows)) next.load(X + next_at, p.K - next_g * G);
        uint32_t amax = max_magnitude(e);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(lanes, amax, o));
        const uint32_t byte = scale_byte(amax);
        const float inv = inverse_scale(byte);
        uint32_t codes[(G + 7) / 8];
#pragma unroll
        for (int h = 0; h < (G + 7) / 8; ++h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < (G < 8 ? G : 8); i += 2) {
                const float2 s = mul_f32x2(make_float2(to_float(e[8 * h + i]), to_float(e[8 * h + i + 1])),
                                           make_float2(inv, inv));
                v[i] = s.x;
                v[i + 1] = s.y;
            }
            if constexpr (G >= 8) codes[h] = e2m1x8(v);
            else codes[h] = e2m1x2(v[0], v[1]) | (e2m1x2(v[2], v[3]) << 8);
            if (byte == 255u) codes[h] = 0u;
        }
        if constexpr (G == 16) *reinterpret_cast<uint2 *>(q) = make_uint2(codes[0], codes[1]);
        else if constexpr (G == 8) *reinterpret_cast<uint32_t *>(q) = codes[0];
        else *reinterpret_cast<uint16_t *>(q) = static_cast<uint16_t>(codes[0]);
        if ((g & (LANES - 1)) == 0) {
            const int b = g / LANES;
            uint8_t *s = p.S + scale_offset(row, b, p.k_tiles);
            *s = static_cast<uint8_t>(byte);
            // The blocks that fill up the last tile multiply zero operands: not NaN.
            if (b == p.KB - 1)
                for (int i = 1; b + i < 4 * p.k_tiles; ++i) s[i] = 0;
        }
        if constexpr (kValues) {
            T t[G];
            group_values<T, G>(codes, byte, t);
            uint4 raw;
            memcpy(&raw, t, sizeof(raw));
            if (left > 0) *reinterpret_cast<uint4 *>(V + at) = raw;
        }
        if (next_row >= static_cast<uint32_t>(p.rows)) break;
        row = static_cast<int>(next_row);
        g = next_g;
        at = next_at;
        q += step_q;
    }
}

// Rows of any length and alignment: a warp takes four blocks (a scale tile's
// word) of a row, a lane one element of each, so that loads and stores of single
// elements are adjacent across the warp.
template <class T, bool kValues>
__global__ void __launch_bounds__(256) mxfp4_quantize_rows_any(const T *__restrict__ X, T *__restrict__ V, QuantParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    // Work item: a scale word; items of a row are adjacent.
    const int64_t items = static_cast<int64_t>(p.rows) * p.k_tiles;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); item < items; item += step) {
        const int row = static_cast<int>(item / p.k_tiles), kt = static_cast<int>(item - static_cast<int64_t>(row) * p.k_tiles);
        const int k0 = kt * 128 + lane;
        const int64_t at = static_cast<int64_t>(row) * p.K + k0;
        T e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = k0 + 32 * i < p.K ? __ldg(X + at + 32 * i) : from_float<T>(0.0f);
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = to_float(e[i]);
            const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7FFFFFFFu));
            word |= byte << (8 * i);
            const float v = x * inverse_scale(byte);
            const float w = __shfl_down_sync(0xffffffffu, v, 1);
            const uint32_t code = byte != 255u ? e2m1x2(v, w) : 0u;   // of an even lane and the next
            if ((lane & 1) == 0 && kt * 4 + i < p.KB)
                p.Q[static_cast<int64_t>(row) * (static_cast<int64_t>(p.KB) * 16) + (kt * 4 + i) * 16 + (lane >> 1)] =
                    static_cast<uint8_t>(code);
            if constexpr (kValues) {
                const uint32_t pair = __shfl_sync(0xffffffffu, code, lane & 30);
                const uint32_t nibble = (lane & 1) ? pair >> 4 : pair & 15u;
                float vals[8];
                e2m1x8_values(nibble, vals);
                if (k0 + 32 * i < p.K) V[at + 32 * i] = from_float<T>(vals[0] * scale_value(byte));
            }
        }
        // Blocks past K are zeros: scale 0.
        if (lane == 0) *reinterpret_cast<uint32_t *>(p.S + scale_offset(row, kt * 4, p.k_tiles)) = word;
    }
}

// X stored (K, rows).  A block takes 128 elements of K (one scale tile's four
// blocks of 32, one per warp) of 32 kCols rows of the result; a thread loads
// kCols adjacent elements of each of its block's 32 rows of X, so a warp reads
// 128 bytes at a time.  Its codes and values then lie along K, 16 adjacent bytes
// here and there in 32 rows: they go through shared memory, so that a row's 64
// bytes of codes and 128 values are written together (stored by each thread
// element by element, values took 144 us at 4096 x 4096 fp16, 14.3 us this way).
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
            *reinterpret_cast<uint32_t *>(p.S + scale_offset(static_cast<int>(row0) + static_cast<int>(threadIdx.x), kt * 4, p.k_tiles)) =
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

template <class T, bool kValues>
int launch_rows(const Mx4QuantArgs &a, const T *X, T *V, QuantParams p)
{
    constexpr int G = kQuantGroup<T, kValues>;
    p.groups = p.KB * (32 / G);
    const int64_t total = a.rows * p.groups;
    const int64_t max_blocks = static_cast<int64_t>(a.sm_count) * kQuantBlocks<T, kValues>;
    int64_t blocks = (total + 255) / 256;
    if (blocks > max_blocks) blocks = max_blocks;
    const int64_t step = blocks * 256;
    p.step_rows = static_cast<int32_t>(step / p.groups);
    p.step_groups = static_cast<int32_t>(step % p.groups);
    p.step_x = static_cast<int64_t>(p.step_rows) * a.K + static_cast<int64_t>(p.step_groups) * G;
    return launch_pdl(mxfp4_quantize_rows<T, kValues>, dim3(static_cast<unsigned>(blocks), 1, 1), 256, a.stream, X, V,
                      p);
}

template <class T>
int quantize(const Mx4QuantArgs &a)
{
    QuantParams p{};
    p.Q = a.Q;
    p.S = a.S;
    p.rows = static_cast<int32_t>(a.rows);
    p.K = static_cast<int32_t>(a.K);
    p.KB = static_cast<int32_t>((a.K + 31) / 32);
    p.k_tiles = static_cast<int32_t>(mx4_k_tiles(a.K));
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
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.V) |
                           (static_cast<uintptr_t>(a.K) * sizeof(T));
    if ((bits & 15u) != 0) {
        const int64_t items = a.rows * p.k_tiles, most = static_cast<int64_t>(a.sm_count) * 8;
        const int64_t blocks = (items + 7) / 8 < most ? (items + 7) / 8 : most;
        const dim3 grid(static_cast<unsigned>(blocks), 1, 1);
        return V ? launch_pdl(mxfp4_quantize_rows_any<T, true>, grid, 256, a.stream, X, V, p)
                 : launch_pdl(mxfp4_quantize_rows_any<T, false>, grid, 256, a.stream, X, V, p);
    }
    return V ? launch_rows<T, true>(a, X, V, p) : launch_rows<T, false>(a, X, V, p);
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
