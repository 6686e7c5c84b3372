// fp8_quantize.cu -- quantisation to E4M3 with one scale per block of 1 x 128
// (activations) or 128 x 128 elements (a weight), in the layouts that the
// block-scaled FP8 products take.  Bound by memory: X is read once and kept in
// registers until its block's largest magnitude is known.
#include "fp8_block.cuh"
#include "feed_forward_launch.cuh"
#include "layer_norm.cuh"

namespace {

using namespace gemm_sm103;

template <class T>
struct QuantParams {
    const T *X;
    uint8_t *Q;
    void *S;
    int64_t rows, K;
    uint32_t blocks;     // of a row
    uint32_t total;      // rows * blocks
    uint32_t magic, shift;   // total / blocks by multiplication
};

// Largest magnitude of a pack as an fp32 bit pattern, NaN's above infinity's; 16-bit
// elements are compared two at a time.
template <class T, int V>
__device__ __forceinline__ uint32_t pack_magnitude(const LnPack<T, V> &x)
{
    uint32_t m = 0;
    if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t raw[V / 2];
        memcpy(raw, x.e, sizeof(raw));
#pragma unroll
        for (int i = 0; i < V / 2; ++i) m = __vmaxu2(m, raw[i] & 0x7FFF7FFFu);
        const uint16_t top = static_cast<uint16_t>(max(m & 0xFFFFu, m >> 16));
        T t;
        memcpy(&t, &top, sizeof(top));
        return __float_as_uint(ln_float(t));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, fp8_magnitude(x[i]));
        return m;
    }
}

// Blocks of a row: kUnroll of them per group of eight lanes (single elements: a warp),
// their loads under way together.  V: elements per load, 16 bytes or one.  With
// 16 lanes and one 16-byte pack each the scale's arithmetic came to a third of the
// instructions (8192 x 8192 bf16 with fp32 scales 50 us, 37 us so, 33 us since the way of
// conversion is decided once per block and a quotient takes two instructions; fp16 with
// powers of two 38 us and 31 us, 30.5 us, 6.6 TB/s, since that kind of scale has a kernel
// of its own).
constexpr int kQuantThreads = 256, kUnroll = 2;
__host__ __device__ constexpr int quant_lanes(int v) { return v > 1 ? 8 : 32; }

template <class T, int V, bool kPow2>
__global__ void __launch_bounds__(kQuantThreads) fp8_quantize_rows(QuantParams<T> p)
{
    constexpr int L = quant_lanes(V);               // of a block
    constexpr int E = kFp8Block / L;                // elements of a lane
    constexpr int S = kQuantThreads / L;            // blocks side by side
    griddep_wait();
    griddep_launch_dependents();
    const int lane = static_cast<int>(threadIdx.x) & (L - 1);
    const uint32_t first = blockIdx.x * static_cast<uint32_t>(S * kUnroll) + threadIdx.x / L;
    LnPack<T, V> x[kUnroll][E / V];
    int64_t at[kUnroll];
    int64_t left[kUnroll];   // elements of the lane's place to the row's end
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t i = first + static_cast<uint32_t>(u * S);
        const bool in = i < p.total;
        const uint32_t row = in ? __umulhi(2u * i, p.magic) >> p.shift : 0u;   // i / blocks
        const int64_t k = static_cast<int64_t>(i - row * p.blocks) * kFp8Block + lane * V;
        at[u] = static_cast<int64_t>(row) * p.K + k;
        left[u] = in ? p.K - k : 0;
#pragma unroll
        for (int j = 0; j < E / V; ++j) {
            if (j * L * V < left[u]) x[u][j].load(p.X + at[u] + j * L * V);
            else x[u][j].fill(0.0f);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < E / V; ++j) m = max(m, pack_magnitude(x[u][j]));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t i = first + static_cast<uint32_t>(u * S);
        if (lane == 0 && i < p.total) Fp8Block::store(p.S, i, m, kPow2);
        const Fp8Block b(m, kPow2);
        b.by_way([&](auto way) {
            constexpr int W8 = decltype(way)::value;
#pragma unroll
            for (int j = 0; j < E / V; ++j) {
                if (j * L * V >= left[u]) continue;
                uint8_t *q = p.Q + at[u] + j * L * V;
                if constexpr (V == 1) {
                    *q = static_cast<uint8_t>(b.template codes<W8>(make_float2(x[u][j][0], 0.0f)));
                } else {
                    uint32_t c[V / 4];
#pragma unroll
                    for (int e = 0; e < V / 4; ++e)
                        c[e] = b.template codes<W8>(x[u][j].pair(2 * e)) | (b.template codes<W8>(x[u][j].pair(2 * e + 1)) << 16);
                    if constexpr (V == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(c[0], c[1]);
                    else *reinterpret_cast<uint32_t *>(q) = c[0];
                }
            }
        });
    }
}

// A block of 128 x 128 elements per block of threads, 64 elements per thread.
template <class T, int V, bool kPow2>
__global__ void __launch_bounds__(256) fp8_quantize_square(QuantParams<T> p)
{
    constexpr int L = kFp8Block / V < 32 ? kFp8Block / V : 32;   // lanes of a row
    constexpr int J = kFp8Block / (L * V);                        // packs of a lane in a row
    constexpr int RS = 256 / L, NR = kFp8Block / RS;              // rows side by side, rows of a thread
    __shared__ uint32_t sh[8];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = static_cast<int>(threadIdx.x) % L;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.blocks) * kFp8Block + threadIdx.x / L;
    const int64_t k0 = static_cast<int64_t>(blockIdx.x % p.blocks) * kFp8Block + lane * V;
    LnPack<T, V> x[NR][J];
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t row = row0 + r * RS, k = k0 + j * L * V;
            if (row < p.rows && k < p.K) x[r][j].load(p.X + row * p.K + k);
            else x[r][j].fill(0.0f);
            m = max(m, pack_magnitude(x[r][j]));
        }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, sh[i]);
    if (threadIdx.x == 0) Fp8Block::store(p.S, blockIdx.x, m, kPow2);
    const Fp8Block b(m, kPow2);
    b.by_way([&](auto way) {
        constexpr int W8 = decltype(way)::value;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int64_t row = row0 + r * RS, k = k0 + j * L * V;
                if (row >= p.rows || k >= p.K) continue;
                uint8_t *q = p.Q + row * p.K + k;
                if constexpr (V == 1) {
                    *q = static_cast<uint8_t>(b.template codes<W8>(make_float2(x[r][j][0], 0.0f)));
                } else {
                    uint32_t c[V / 4];
#pragma unroll
                    for (int e = 0; e < V / 4; ++e)
                        c[e] = b.template codes<W8>(x[r][j].pair(2 * e)) | (b.template codes<W8>(x[r][j].pair(2 * e + 1)) << 16);
                    if constexpr (V == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(c[0], c[1]);
                    else *reinterpret_cast<uint32_t *>(q) = c[0];
                }
            }
    });
}

template <class T, int V, bool kPow2>
int launch_kind(const QuantParams<T> &p, int block_rows, cudaStream_t stream)
{
    if (block_rows != 1)
        return ln_launch(fp8_quantize_square<T, V, kPow2>,
                         dim3(static_cast<unsigned>((p.rows + kFp8Block - 1) / kFp8Block * p.blocks), 1, 1), 256, stream,
                         p);
    constexpr uint32_t per = kQuantThreads / quant_lanes(V) * kUnroll;
    return ln_launch(fp8_quantize_rows<T, V, kPow2>, dim3((p.total + per - 1) / per, 1, 1), kQuantThreads, stream, p);
}

template <class T, int V>
int launch_packs(const QuantParams<T> &p, const Fp8QuantArgs &a)
{
    return a.pow2 ? launch_kind<T, V, true>(p, a.block_rows, a.stream) : launch_kind<T, V, false>(p, a.block_rows, a.stream);
}

template <class T>
int quantize(const Fp8QuantArgs &a)
{
    QuantParams<T> p{};
    p.X = static_cast<const T *>(a.X);
    p.Q = static_cast<uint8_t *>(a.Q);
    p.S = a.S;
    p.rows = a.rows;
    p.K = a.K;
    p.blocks = static_cast<uint32_t>((a.K + kFp8Block - 1) / kFp8Block);
    p.total = static_cast<uint32_t>(a.rows * static_cast<int64_t>(p.blocks));
    // Division of i < 2^31 by d: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d),
    // floor(i m / 2^(31 + s)) is the quotient (T. Granlund and P. L. Montgomery,
    // PLDI 1994); m < 2^32, and i m / 2^31 is the high word of 2 i m.
    int s = 0;
    while ((1ull << s) < p.blocks) ++s;
    p.magic = static_cast<uint32_t>(((1ull << (31 + s)) + p.blocks - 1) / p.blocks);
    p.shift = static_cast<uint32_t>(s);
    constexpr int V = 16 / sizeof(T);
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.X) | (static_cast<uintptr_t>(a.K) * sizeof(T));
    if ((bits & 15u) == 0 && (reinterpret_cast<uintptr_t>(a.Q) & (V - 1)) == 0)
        return launch_packs<T, V>(p, a);
    return launch_packs<T, 1>(p, a);
}

}  // namespace

namespace gemm_sm103 {

int launch_fp8_quantize(const Fp8QuantArgs &a)
{
    if (a.type == GEMM_TYPE_F32) return quantize<float>(a);
    if (a.type == GEMM_TYPE_F16) return quantize<__half>(a);
    return quantize<__nv_bfloat16>(a);
}

}  // namespace gemm_sm103
