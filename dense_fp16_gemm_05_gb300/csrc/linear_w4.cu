// linear_w4.cu -- C = R(X W^T) for a few rows of 16-bit X (tokens being generated)
// and 4-bit W with a scale, and optionally a zero point, per row and group of
// columns:  C[m, n] = R( sum over groups  s[n] sum over the group  x[m, k] (q[n, k] - z[n]) ).
//
// Bound by reading W.  The products go through mma.sync m16n8k16 with 16 rows of W
// as the 16-row operand and up to 8 rows of X as the 8-column one: the codes are
// laid out so that one 16-byte load per lane is the operand of four such products,
// and q - z is exact in 16 bits, so what is rounded is the fp32 sum alone; a
// group's sum is scaled in fp32.  (The tensor memory path wants 128 rows of
// operands in shared memory, four times the codes' bytes written there first, for
// an arithmetic that a matrix-vector product does not need.)  K is divided over a
// block's warps and, where there are few rows of W, over the blocks of a cluster,
// whose sums are added through shared memory in a fixed order.
#include "feed_forward_launch.cuh"
#include "layer_norm.cuh"

namespace {

using namespace gemm_sm103;

template <class T>
struct W4Params {
    const T *X;
    const uint4 *Q;   // a lane's 16 bytes
    const T *S;
    const uint8_t *Z;
    T *C;
    int64_t M, N, K;
    int32_t strips, k_tiles, groups, units;   // units of 128 columns
    int32_t relu;
};

constexpr int kWarps = 8;

// The four operand registers of 16 rows x 16 columns from a word of codes:
// register s holds the elements at nibbles s and s + 4, minus the zero point of
// row g (s even) or g + 8 (s odd).
template <class T>
struct W4Codes;

template <>
struct W4Codes<__half> {
    // 1024 + q, and 64 + q by a multiplication with 1/16: both exact.
    static __device__ __forceinline__ uint32_t bias(int z, int odd)
    {
        const __half2 h = __float2half2_rn(odd ? -64.0f - static_cast<float>(z) : -1024.0f - static_cast<float>(z));
        uint32_t r;
        memcpy(&r, &h, 4);
        return r;
    }
    static __device__ __forceinline__ void operands(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&a)[4])
    {
#pragma unroll
        for (int s = 0; s < 4; s += 2) {
            const uint32_t v = w >> (4 * s);
            const uint32_t even = (v & 0x000F000Fu) | 0x64006400u, odd = (v & 0x00F000F0u) | 0x64006400u;
            asm("add.rn.f16x2 %0, %1, %2;" : "=r"(a[s]) : "r"(even), "r"(lo));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(a[s + 1]) : "r"(odd), "r"(0x2C002C00u), "r"(hi));
        }
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <>
struct W4Codes<__nv_bfloat16> {
    // 128 + q: with seven bits behind the point no second nibble fits.
    static __device__ __forceinline__ uint32_t bias(int z, int)
    {
        const __nv_bfloat162 h = __float2bfloat162_rn(-128.0f - static_cast<float>(z));
        uint32_t r;
        memcpy(&r, &h, 4);
        return r;
    }
    static __device__ __forceinline__ void operands(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&a)[4])
    {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t v = ((w >> (4 * s)) & 0x000F000Fu) | 0x43004300u;
            asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(a[s]) : "r"(v), "r"(s & 1 ? hi : lo));
        }
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// NT: groups of 8 rows of X.  RS: strips of 16 rows of W that a warp takes side by
// side, so that X's operands serve them all.  kVec: X's rows are on the 16-byte grid.
template <class T, int NT, int RS, int G, bool kZ, bool kVec>
__global__ void __launch_bounds__(kWarps * 32) linear_w4_kernel(W4Params<T> p)
{
    using Codes = W4Codes<T>;
    constexpr int U = 128 / G;         // groups of a unit
    constexpr int COLS = NT * 8;
    __shared__ float part[kWarps][RS * 16][COLS + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const int g = lane >> 2, t = lane & 3;
    const int strip0 = static_cast<int>(blockIdx.x) * RS;
    const int slices = static_cast<int>(gridDim.y), slice = static_cast<int>(blockIdx.y);
    const int u_begin = static_cast<int>(static_cast<int64_t>(p.units) * slice / slices);
    const int u_end = static_cast<int>(static_cast<int64_t>(p.units) * (slice + 1) / slices);

    struct Unit {
        uint4 q[RS][2];
        T s[RS][U][2];
        uint8_t z[RS][U][2];
    };
    auto load = [&](Unit &b, int u) {
#pragma unroll
        for (int i = 0; i < RS; ++i) {
            // A strip past the last is loaded as the last and not stored.
            const int strip = min(strip0 + i, p.strips - 1);
            const uint4 *q = p.Q + (static_cast<int64_t>(strip) * p.k_tiles + 2 * u) * 32 + lane;
            b.q[i][0] = __ldg(q);
            b.q[i][1] = 2 * u + 1 < p.k_tiles ? __ldg(q + 32) : make_uint4(0, 0, 0, 0);
            const int64_t at = (static_cast<int64_t>(strip) * p.groups + u * U) * kW4Rows + g;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const bool in = u * U + j < p.groups;
                b.s[i][j][0] = in ? __ldg(p.S + at + j * kW4Rows) : ln_round<T>(0.0f);
                b.s[i][j][1] = in ? __ldg(p.S + at + j * kW4Rows + 8) : ln_round<T>(0.0f);
                if constexpr (kZ) {
                    b.z[i][j][0] = in ? __ldg(p.Z + at + j * kW4Rows) : uint8_t{0};
                    b.z[i][j][1] = in ? __ldg(p.Z + at + j * kW4Rows + 8) : uint8_t{0};
                }
            }
        }
    };
    // Eight elements of row `row` of X from column k on, zero past either end.
    auto x_piece = [&](int64_t row, int64_t k) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row >= p.M || k >= p.K) return v;
        const T *x = p.X + row * p.K + k;
        if constexpr (kVec) {
            v = __ldg(reinterpret_cast<const uint4 *>(x));
        } else {
            T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = k + i < p.K ? __ldg(x + i) : ln_round<T>(0.0f);
            memcpy(&v, e, 16);
        }
        return v;
    };

    float sum[RS][NT][4];
#pragma unroll
    for (int i = 0; i < RS; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[i][n][e] = 0.0f;
    Unit next;
    if (u_begin + warp < u_end) load(next, u_begin + warp);
    for (int u = u_begin + warp; u < u_end; u += kWarps) {
        const Unit b = next;
        if (u + kWarps < u_end) load(next, u + kWarps);
        uint4 x[NT][4];   // 32 columns each
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 4; ++h) x[n][h] = x_piece(n * 8 + g, static_cast<int64_t>(u) * 128 + h * 32 + t * 8);
#pragma unroll
        for (int i = 0; i < RS; ++i)
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t lo = Codes::bias(kZ ? b.z[i][j][0] & 15 : 8, 0), hi = Codes::bias(kZ ? b.z[i][j][1] & 15 : 8, 1);
                float d[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
#pragma unroll
                for (int h = j * (G / 32); h < (j + 1) * (G / 32); ++h) {
                    const uint4 &q = b.q[i][h / 2];
                    const uint32_t w[2] = {h % 2 ? q.z : q.x, h % 2 ? q.w : q.y};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t a[4];
                        Codes::operands(w[c], lo, hi, a);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            Codes::mma(d[n], a, c ? x[n][h].z : x[n][h].x, c ? x[n][h].w : x[n][h].y);
                    }
                }
                const float s0 = ln_float(b.s[i][j][0]), s1 = ln_float(b.s[i][j][1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    sum[i][n][0] = fmaf(s0, d[n][0], sum[i][n][0]);
                    sum[i][n][1] = fmaf(s0, d[n][1], sum[i][n][1]);
                    sum[i][n][2] = fmaf(s1, d[n][2], sum[i][n][2]);
                    sum[i][n][3] = fmaf(s1, d[n][3], sum[i][n][3]);
                }
            }
    }
    // Lane (g, t) has rows g and g + 8 of the strip, columns 2t and 2t + 1 of each 8.
#pragma unroll
    for (int i = 0; i < RS; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[warp][i * 16 + g + 8 * (e >> 1)][n * 8 + 2 * t + (e & 1)] = sum[i][n][e];
    __syncthreads();
    constexpr int OUT = RS * 16 * COLS;
    // The block's sums, in place of the first warp's.
    for (int o = threadIdx.x; o < OUT; o += kWarps * 32) {
        const int r = o % (RS * 16), m = o / (RS * 16);
        float v = part[0][r][m];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) v += part[i][r][m];
        part[0][r][m] = v;
    }
    if (slices > 1) {
        cluster_arrive();
        cluster_wait();
    }
    // Every block of the cluster finishes a share of the outputs: a thread the same
    // ones that it summed, if there is one block.
    for (int o = threadIdx.x + slice * kWarps * 32; o < OUT; o += slices * kWarps * 32) {
        const int r = o % (RS * 16), m = o / (RS * 16);
        float v;
        if (slices > 1) {
            v = 0.0f;
            for (int i = 0; i < slices; ++i) {
                const uint32_t at = mapa_shared(smem_addr(&part[0][r][m]), static_cast<uint32_t>(i));
                float other;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(at));
                v += other;
            }
        } else {
            v = part[0][r][m];
        }
        const int64_t n = static_cast<int64_t>(strip0) * 16 + r;
        if (n >= p.N || m >= p.M) continue;
        if (p.relu) v = v > 0.0f ? v : 0.0f;
        p.C[m * p.N + n] = ln_round<T>(v);
    }
    if (slices > 1) {   // nobody leaves while its sums are read
        cluster_arrive();
        cluster_wait();
    }
}

template <class T, int NT, int RS, int G, bool kZ, bool kVec>
int launch_one(const W4Params<T> &p, int sm_count, cudaStream_t stream)
{
    const int64_t blocks = (p.strips + RS - 1) / RS;
    // Blocks of a cluster divide K while the GPU has room for twice as many blocks
    // and every warp keeps a unit.
    int slices = 1;
    while (slices < 8 && blocks * slices < 2 * static_cast<int64_t>(sm_count) && p.units >= 2 * slices * kWarps) slices *= 2;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(slices), 1);
    lc.blockDim = dim3(kWarps * 32, 1, 1);
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = static_cast<unsigned>(slices);
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = slices > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&lc, linear_w4_kernel<T, NT, RS, G, kZ, kVec>, p) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

template <class T, int G, bool kZ, bool kVec>
int launch_rows(const W4Params<T> &p, int sm_count, cudaStream_t stream)
{
    if (p.M <= 8) return launch_one<T, 1, 1, G, kZ, kVec>(p, sm_count, stream);
    if (p.M <= 16) return launch_one<T, 2, 1, G, kZ, kVec>(p, sm_count, stream);
    if (p.M <= 32) return launch_one<T, 4, 1, G, kZ, kVec>(p, sm_count, stream);
    return launch_one<T, 8, 1, G, kZ, kVec>(p, sm_count, stream);
}

template <class T, int G>
int launch_group(const W4Params<T> &p, int sm_count, cudaStream_t stream)
{
    const bool vec = (reinterpret_cast<uintptr_t>(p.X) & 15u) == 0 && p.K % 8 == 0;
    if (p.Z) return vec ? launch_rows<T, G, true, true>(p, sm_count, stream) : launch_rows<T, G, true, false>(p, sm_count, stream);
    return vec ? launch_rows<T, G, false, true>(p, sm_count, stream) : launch_rows<T, G, false, false>(p, sm_count, stream);
}

template <class T>
int linear(const W4LinearArgs &a)
{
    W4Params<T> p{};
    p.X = static_cast<const T *>(a.X);
    p.Q = static_cast<const uint4 *>(a.Q);
    p.S = static_cast<const T *>(a.S);
    p.Z = a.Z;
    p.C = static_cast<T *>(a.C);
    p.M = a.M;
    p.N = a.N;
    p.K = a.K;
    p.strips = static_cast<int32_t>(w4_strips(a.N));
    p.k_tiles = static_cast<int32_t>((a.K + kW4Cols - 1) / kW4Cols);
    p.groups = static_cast<int32_t>((a.K + a.group - 1) / a.group);
    p.units = (p.k_tiles + 1) / 2;
    p.relu = a.relu;
    if (a.group == 32) return launch_group<T, 32>(p, a.sm_count, a.stream);
    if (a.group == 64) return launch_group<T, 64>(p, a.sm_count, a.stream);
    return launch_group<T, 128>(p, a.sm_count, a.stream);
}

}  // namespace

namespace gemm_sm103 {

int launch_linear_w4(const W4LinearArgs &a)
{
    return a.type == GEMM_TYPE_F16 ? linear<__half>(a) : linear<__nv_bfloat16>(a);
}

}  // namespace gemm_sm103
