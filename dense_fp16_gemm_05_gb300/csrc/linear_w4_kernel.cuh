// linear_w4_kernel.cuh -- C = R(X W^T) for a few rows of 16-bit X (tokens being
// generated) and 4-bit W with a scale, and optionally a zero point, per row and
// group of columns:
//
//   C[m, n] = R( sum over groups  s[n]  sum over the group  x[m, k] (q[n, k] - z[n]) ).
//
// Bound by reading W.  The products go through mma.sync m16n8k16 with 16 rows of W
// as the 16-row operand and up to 8 rows of X as the 8-column one: the codes are
// laid out so that one 16-byte load per lane is the operand of four such products,
// and q - z is exact in 16 bits, so what is rounded is the fp32 sum alone; a
// group's sum is scaled in fp32.  (The tensor memory path wants 128 rows of
// operands in shared memory, four times the codes' bytes written there first, for
// an arithmetic that a matrix-vector product does not need.)
//
// Every warp streams its own units -- 16 rows x 128 columns of codes with their
// scales and zero points -- through its own ring of asynchronous copies in shared
// memory: nothing but its own copies makes a warp wait, and the bytes under way are
// not bounded by registers.  Few rows of X stay in shared memory for the whole call
// and a block's sixteen warps divide the columns of 16 rows of W (KW = 16), one
// block per SM walking such strips; their sums are added through shared memory in a
// fixed order.  More rows of X come in chunks for the block's 256 rows of W (KW = 1),
// so that X is read less often than W.  Where W has few rows, K is also divided over
// the blocks of a cluster, whose sums are added through distributed shared memory.
#pragma once

#include <atomic>
#include <type_traits>

#include "feed_forward_launch.cuh"
#include "gemm_launch.cuh"
#include "layer_norm.cuh"
#include "sm103_ptx.cuh"

namespace gemm_sm103 {

template <class T>
struct W4Params {
    const T *X;
    const uint8_t *Q, *S, *Z;   // bytes; Z NULL: 8
    T *C;
    int64_t N, K;
    int32_t M;
    int32_t strips, k_tiles, groups, units;   // 16 rows; 64 columns; scale groups; 128 columns
    int32_t relu;
    int32_t x_row, x_bytes;     // X in shared memory: bytes between rows, bytes of a buffer
};

constexpr int kW4Warps = 16, kW4Threads = kW4Warps * 32;

// Asynchronous copies of 16 and of 8 bytes to shared memory.
__device__ __forceinline__ void w4_copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}
__device__ __forceinline__ void w4_copy8(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}
__device__ __forceinline__ void w4_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void w4_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// (v & mask) | bits in one instruction: of two constants the compiler makes two.
__device__ __forceinline__ uint32_t w4_and_or(uint32_t v, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
    return r;
}

// The four operand registers of 16 rows x 16 columns from a word of codes:
// register s holds the elements at nibbles s and s + 4, minus the zero point of
// row g (s even) or g + 8 (s odd).
template <class T>
struct W4Codes;

template <>
struct W4Codes<__half> {
    // -(1024 + z) for rows g, -(64 + z) for rows g + 8, twice.
    static __device__ __forceinline__ uint32_t bias(uint32_t z, int odd)
    {
        return odd ? 0xD400D400u + z * 0x00100010u : 0xE400E400u + z * 0x00010001u;
    }
    // 1024 + q and, one nibble further up, 1024 + 16 q, times 1/16: all exact.
    static __device__ __forceinline__ void operands(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&a)[4])
    {
#pragma unroll
        for (int s = 0; s < 4; s += 2) {
            const uint32_t v = w >> (4 * s);
            const uint32_t even = w4_and_or(v, 0x000F000Fu, 0x64006400u), odd = w4_and_or(v, 0x00F000F0u, 0x64006400u);
            asm("add.rn.f16x2 %0, %1, %2;" : "=r"(a[s]) : "r"(even), "r"(lo));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(a[s + 1]) : "r"(odd), "r"(0x2C002C00u), "r"(hi));
        }
    }
    // d = a b + c
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                               float c1, float c2, float c3)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    }
};

template <>
struct W4Codes<__nv_bfloat16> {
    // -(128 + z), twice.
    static __device__ __forceinline__ uint32_t bias(uint32_t z, int) { return 0xC300C300u + z * 0x00010001u; }
    // 128 + q: with seven bits behind the point no second nibble fits.
    static __device__ __forceinline__ void operands(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&a)[4])
    {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t v = w4_and_or(w >> (4 * s), 0x000F000Fu, 0x43004300u);
            asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(a[s]) : "r"(v), "r"(s & 1 ? hi : lo));
        }
    }
    // d = a b + c
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                               float c1, float c2, float c3)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    }
};

// Sizes of one kernel: NT groups of 8 rows of X; KW ways (16 or 1) that a strip's
// columns are divided among the warps.  G: columns of a scale group.
template <int NT, int KW, int G>
struct W4Shape {
    static constexpr int STRIPS = kW4Warps / KW, ROWS = STRIPS * kW4Rows, COLS = NT * 8;
    static constexpr int U = 128 / G;                       // scale groups of a unit
    static constexpr int SLOT = 1024 + U * 48;              // bytes: codes, scales, zero points
    static constexpr int DEPTH = KW > 1 || NT <= 2 ? 6 : 4; // units under way per warp
    static constexpr int RING = kW4Warps * DEPTH * SLOT;
    static constexpr int X_UNITS = NT <= 2 ? 8 : 4;         // of a chunk of X, at least DEPTH (KW = 1)
    static constexpr int SUMS = KW * ROWS * (COLS + 1) * 4; // KW = 1: in place of X and the ring
};

// Rows of X half a 128-byte line apart, so that eight lanes' 16-byte loads from two
// rows meet no bank twice.
constexpr int w4_x_row(int64_t units) { return static_cast<int>(units * 256 + 64); }

// kVec: X's rows are on the 16-byte grid and come through shared memory; else their
// elements are read one by one.
template <class T, int NT, int KW, int G, bool kVec>
__global__ void __launch_bounds__(kW4Threads, 1) linear_w4_kernel(W4Params<T> p)
{
    using Codes = W4Codes<T>;
    using Shape = W4Shape<NT, KW, G>;
    constexpr int U = Shape::U, ROWS = Shape::ROWS, COLS = Shape::COLS, D = Shape::DEPTH;
    extern __shared__ uint4 smem[];   // the rings; X (KW = 1: two chunks); KW = 16: two buffers of sums
    typedef float Sums[KW][ROWS][COLS + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const int g = lane >> 2, t = lane & 3;
    const int kw = KW > 1 ? warp : 0, rw = KW > 1 ? 0 : warp;
    const int slices = static_cast<int>(gridDim.y), slice = static_cast<int>(blockIdx.y);
    const int u_begin = static_cast<int>(static_cast<int64_t>(p.units) * slice / slices);
    const int u_end = static_cast<int>(static_cast<int64_t>(p.units) * (slice + 1) / slices);
    const uint8_t *ring = reinterpret_cast<const uint8_t *>(smem) + warp * (D * Shape::SLOT);
    const uint8_t *x_mem = reinterpret_cast<const uint8_t *>(smem) + Shape::RING;
    const uint32_t ring_at = smem_addr(ring), x_at = smem_addr(x_mem);

    // Copies of X: `units` units from unit u on, all threads together.
    auto copy_x = [&](uint32_t dst, int u, int units) {
        const int per_row = units * 16;   // 16-byte pieces
        const int64_t k0 = static_cast<int64_t>(u) * 128;
        for (int i = threadIdx.x; i < p.M * per_row; i += kW4Threads) {
            const int m = i / per_row, c = i - m * per_row;
            if (k0 + c * 8 < p.K) w4_copy16(dst + static_cast<uint32_t>(m * p.x_row + c * 16), p.X + m * p.K + k0 + c * 8);
        }
    };
    // This lane's piece of a unit's scales (the first 4 U lanes) or zero points (2 U).
    const bool side_s = lane < 4 * U, side = side_s || (p.Z && lane < 6 * U);
    const int side_j = side_s ? lane : lane - 4 * U, side_group = side_s ? lane / 4 : side_j / 2;
    const uint8_t *side_base = (side_s ? p.S : p.Z) + side_j * 8;
    const uint32_t side_bytes = side_s ? 32u : 16u;   // of a group
    const uint32_t side_to = 1024u + static_cast<uint32_t>(side_s ? lane * 8 : U * 32 + side_j * 8);
    const uint8_t *q_src = nullptr, *side_src = nullptr;
    auto seek = [&](int strip, int u) {
        strip = min(strip, p.strips - 1);   // one past the last is read as the last and not stored
        q_src = p.Q + (static_cast<int64_t>(strip) * p.k_tiles + 2 * u) * kW4TileBytes + lane * 16;
        side_src = side_base + (static_cast<int64_t>(strip) * p.groups + static_cast<int64_t>(u) * U) * side_bytes;
    };
    auto fetch = [&](int slot, int u) {
        const uint32_t dst = ring_at + static_cast<uint32_t>(slot * Shape::SLOT);
        const bool tail = u == p.units - 1;
        w4_copy16(dst + lane * 16, q_src);
        if (!tail || 2 * u + 1 < p.k_tiles) w4_copy16(dst + 512 + lane * 16, q_src + 512);
        if (side && (!tail || u * U + side_group < p.groups)) w4_copy8(dst + side_to, side_src);
        q_src += KW * 1024;
        side_src += KW * U * side_bytes;
    };

    // A row past X's last is read as the last one: it reaches nothing but its own
    // column of the result, which is not stored.
    uint32_t x_off[NT];
    const T *x_src[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int m = min(n * 8 + g, p.M - 1);
        x_off[n] = static_cast<uint32_t>(m * p.x_row + t * 16);
        x_src[n] = p.X + m * p.K + t * 8;
    }
    float sum[NT][4];
    // Adds unit u's products.  kTail: the last unit, which may reach past K.
    auto unit = [&](const uint8_t *slot, const uint8_t *x_unit, int u, auto tail_) {
        constexpr bool kTail = decltype(tail_)::value;
        const int left = kTail ? static_cast<int>(p.K - static_cast<int64_t>(u) * 128) - t * 8 : 0;
        const uint4 *q = reinterpret_cast<const uint4 *>(slot) + lane;
        // In a last unit of one tile the second one's codes are those of an earlier
        // unit, times zeros.
        const uint4 tile[2] = {q[0], q[32]};
        const uint8_t *scales = slot + 1024 + g * 2, *zeros = slot + 1024 + U * 32 + g;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            uint32_t lo = Codes::bias(8u, 0), hi = Codes::bias(8u, 1);
            if (p.Z) {
                lo = Codes::bias(zeros[j * 16] & 15u, 0);
                hi = Codes::bias(zeros[j * 16 + 8] & 15u, 1);
            }
            // With one product per operand two sums, so that one does not wait for the
            // other.
            constexpr int P = NT == 1 ? 2 : 1;
            float d[P][NT][4];
#pragma unroll
            for (int h = j * (G / 32); h < (j + 1) * (G / 32); ++h) {
                uint4 x[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (kVec) {
                        x[n] = *reinterpret_cast<const uint4 *>(x_unit + x_off[n] + h * 64);
                        if (kTail && h * 32 >= left) x[n] = make_uint4(0, 0, 0, 0);
                    } else {
                        T e[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            e[k] = !kTail || h * 32 + k < left ? __ldg(x_src[n] + static_cast<int64_t>(u) * 128 + h * 32 + k)
                                                               : ln_round<T>(0.0f);
                        memcpy(&x[n], e, 16);
                    }
                }
                const uint4 &v = tile[h / 2];
                const uint32_t w[2] = {h % 2 ? v.z : v.x, h % 2 ? v.w : v.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t a[4];
                    Codes::operands(w[k], lo, hi, a);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float (&e)[4] = d[k % P][n];
                        const uint32_t b0 = k ? x[n].z : x[n].x, b1 = k ? x[n].w : x[n].y;
                        if (h == j * (G / 32) && k < P) Codes::mma(e, a, b0, b1, 0.0f, 0.0f, 0.0f, 0.0f);
                        else Codes::mma(e, a, b0, b1, e[0], e[1], e[2], e[3]);
                    }
                }
            }
            const T *sc = reinterpret_cast<const T *>(scales + j * 32);
            float s0 = ln_float(sc[0]), s1 = ln_float(sc[8]);
            if (kTail && u * U + j >= p.groups) s0 = s1 = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = P == 2 ? d[0][n][e] + d[P - 1][n][e] : d[0][n][e];
                    sum[n][e] = fmaf(e < 2 ? s0 : s1, v, sum[n][e]);
                }
        }
    };
    auto step = [&](int slot, const uint8_t *x_unit, int u) {
        const uint8_t *at = ring + slot * Shape::SLOT;
        if (u < p.units - 1) unit(at, x_unit, u, std::false_type{});
        else unit(at, x_unit, u, std::true_type{});
    };
    auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[n][e] = 0.0f;
    };
    // Lane (g, t) has rows g and g + 8 of a strip, columns 2t and 2t + 1 of each 8.
    auto keep = [&](Sums &sums) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[kw][rw * 16 + g + 8 * (e >> 1)][n * 8 + 2 * t + (e & 1)] = sum[n][e];
    };
    constexpr int OUT = ROWS * COLS;
    auto ways = [&](const Sums &sums, int r, int m) {
        float v = sums[0][r][m];
#pragma unroll
        for (int i = 1; i < KW; ++i) v += sums[i][r][m];
        return v;
    };
    auto store = [&](int64_t n, int m, float v) {
        if (n >= p.N || m >= p.M) return;
        if (p.relu) v = v > 0.0f ? v : 0.0f;
        p.C[m * p.N + n] = ln_round<T>(v);
    };
    auto finish = [&](Sums &sums, int64_t n0) {
        if (slices == 1) {
            for (int o = threadIdx.x; o < OUT; o += kW4Threads) store(n0 + o % ROWS, o / ROWS, ways(sums, o % ROWS, o / ROWS));
            return;
        }
        // The block's sums in place of the first way's, then every block of the cluster
        // adds and stores a share.
        if constexpr (KW > 1)
            for (int o = threadIdx.x; o < OUT; o += kW4Threads) sums[0][o % ROWS][o / ROWS] = ways(sums, o % ROWS, o / ROWS);
        cluster_arrive();
        cluster_wait();
        for (int o = threadIdx.x + slice * kW4Threads; o < OUT; o += slices * kW4Threads) {
            const int r = o % ROWS, m = o / ROWS;
            float v = 0.0f;
            for (int i = 0; i < slices; ++i) {
                const uint32_t at = mapa_shared(smem_addr(&sums[0][r][m]), static_cast<uint32_t>(i));
                float other;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(at));
                v += other;
            }
            store(n0 + r, m, v);
        }
        cluster_arrive();   // nobody leaves while its sums are read
        cluster_wait();
    };

    if constexpr (KW > 1) {
        // Strips blockIdx.x, blockIdx.x + gridDim.x, ...; this warp has units u_begin + kw,
        // u_begin + kw + KW, ... of each, `mine` of them.
        Sums *part = reinterpret_cast<Sums *>(const_cast<uint8_t *>(x_mem) + p.x_bytes);
        const int first = u_begin + kw, mine = first < u_end ? (u_end - first + KW - 1) / KW : 0;
        if (kVec) copy_x(x_at, u_begin, u_end - u_begin);
        w4_commit();
        // The copies run ahead of the products by D units, over the strips' ends.
        int ahead_strip = blockIdx.x, ahead = 0;
        auto next = [&](int slot) {
            if (mine > 0 && ahead_strip < p.strips) {
                if (ahead == 0) seek(ahead_strip, first);
                fetch(slot, first + ahead * KW);
                if (++ahead == mine) {
                    ahead = 0;
                    ahead_strip += static_cast<int>(gridDim.x);
                }
            }
            w4_commit();
        };
#pragma unroll
        for (int i = 0; i < D; ++i) next(i);
        w4_wait<D>();
        __syncthreads();   // X is there
        int slot = 0, buffer = 0;
        for (int strip = blockIdx.x; strip < p.strips; strip += static_cast<int>(gridDim.x)) {
            clear();
            for (int i = 0; i < mine; ++i) {
                w4_wait<D - 1>();
                __syncwarp();
                const int u = first + i * KW;
                step(slot, x_mem + (u - u_begin) * 256, u);
                __syncwarp();
                next(slot);
                if (++slot == D) slot = 0;
            }
            keep(part[buffer]);
            __syncthreads();
            finish(part[buffer], static_cast<int64_t>(strip) * ROWS);
            // Sums of the strip after the next are written behind the next one's barrier.
            buffer ^= 1;
        }
    } else {
        // One strip per warp, units u_begin .. u_end - 1; X in chunks that the block shares.
        constexpr int XU = Shape::X_UNITS;
        static_assert(XU >= D, "a chunk of X is there when the units copied with it are");
        const int n = u_end - u_begin;
        seek(static_cast<int>(blockIdx.x) * Shape::STRIPS + warp, u_begin);
        clear();
        if (kVec) copy_x(x_at, u_begin, XU);
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if (i < n) fetch(i, u_begin + i);
            w4_commit();
        }
        int slot = 0, x_unit = 0, x_buffer = 0;
        for (int i = 0; i < n; ++i) {
            w4_wait<D - 1>();
            if (kVec && x_unit == 0) {
                __syncthreads();   // this chunk is there, and the one before is done with
                if (i + XU < n) copy_x(x_at + static_cast<uint32_t>((x_buffer ^ 1) * p.x_bytes), u_begin + i + XU, XU);
            } else {
                __syncwarp();
            }
            step(slot, x_mem + x_buffer * p.x_bytes + x_unit * 256, u_begin + i);
            __syncwarp();
            if (i + D < n) fetch(slot, u_begin + i + D);
            w4_commit();
            if (++slot == D) slot = 0;
            if (++x_unit == XU) {
                x_unit = 0;
                x_buffer ^= 1;
            }
        }
        w4_wait<0>();
        __syncthreads();
        Sums &sums = *reinterpret_cast<Sums *>(smem);
        keep(sums);
        __syncthreads();
        finish(sums, static_cast<int64_t>(blockIdx.x) * ROWS);
    }
}

constexpr int kW4Budget = 225 * 1024;   // dynamic shared memory of a block

// Rows of X that stay in shared memory beside the rings and the sums (KW = 16).
template <int G>
constexpr int kW4KeepBytes = kW4Budget - W4Shape<1, 16, G>::RING - 2 * W4Shape<1, 16, G>::SUMS;

// Blocks of a cluster that divide K: while the GPU has room for them and every warp
// keeps two of its units.
inline int w4_slices(int64_t row_groups, int64_t units_per_warp, int sm_count)
{
    int slices = 1;
    while (slices < 8 && 2 * slices * row_groups <= sm_count && 4 * slices <= units_per_warp) slices *= 2;
    return slices;
}

template <class T, int NT, int KW, int G, bool kVec>
int launch_w4_kernel(W4Params<T> p, const W4LinearArgs &a)
{
    using Shape = W4Shape<NT, KW, G>;
    auto kern = linear_w4_kernel<T, NT, KW, G, kVec>;
    const int64_t row_groups = (p.strips + Shape::STRIPS - 1) / Shape::STRIPS;
    const int slices = w4_slices(row_groups, (p.units + KW - 1) / KW, a.sm_count);
    int smem = Shape::RING;
    if (kVec) {
        p.x_row = w4_x_row(KW > 1 ? (p.units + slices - 1) / slices : Shape::X_UNITS);
        p.x_bytes = p.M * p.x_row;
        smem += KW > 1 ? p.x_bytes : 2 * p.x_bytes;
    }
    if (KW > 1) smem += 2 * Shape::SUMS;
    else if (smem < Shape::SUMS) smem = Shape::SUMS;
    static std::atomic<int> prepared[kMaxDevices];
    if (!prepared[a.device].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4Budget) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        prepared[a.device].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(KW > 1 && slices == 1 && row_groups > a.sm_count ? a.sm_count : row_groups),
                      static_cast<unsigned>(slices), 1);
    lc.blockDim = dim3(kW4Threads, 1, 1);
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = static_cast<unsigned>(slices);
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = slices > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&lc, kern, p) != cudaSuccess) {
        cudaGetLastError();
        prepared[a.device].store(0, std::memory_order_release);
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// Calls of one scale group width (linear_w4_g32.cu, ...: a translation unit each).
template <class T, int G, bool kVec>
int launch_w4_shape(const W4Params<T> &p, const W4LinearArgs &a)
{
    // Few rows of X that fit beside the rings, and enough columns for half of the
    // warps: M = 1, 16384 x 8192 fp16 17.8 us, 25 us by KW = 1; M = 8 there, whose X
    // does not fit, 21.2 us.
    const bool fits = !kVec || p.M * static_cast<int64_t>(w4_x_row(p.units)) <= kW4KeepBytes<G>;
    if (p.M <= 8 && fits && p.units >= 8) return launch_w4_kernel<T, 1, 16, G, kVec>(p, a);
    if (p.M <= 8) return launch_w4_kernel<T, 1, 1, G, kVec>(p, a);
    if (p.M <= 16) return launch_w4_kernel<T, 2, 1, G, kVec>(p, a);
    if (p.M <= 32) return launch_w4_kernel<T, 4, 1, G, kVec>(p, a);
    return launch_w4_kernel<T, 8, 1, G, kVec>(p, a);
}

template <class T, int G>
int launch_w4(const W4LinearArgs &a)
{
    W4Params<T> p{};
    p.X = static_cast<const T *>(a.X);
    p.Q = static_cast<const uint8_t *>(a.Q);
    p.S = static_cast<const uint8_t *>(a.S);
    p.Z = a.Z;
    p.C = static_cast<T *>(a.C);
    p.M = static_cast<int32_t>(a.M);
    p.N = a.N;
    p.K = a.K;
    p.strips = static_cast<int32_t>(w4_strips(a.N));
    p.k_tiles = static_cast<int32_t>((a.K + kW4Cols - 1) / kW4Cols);
    p.groups = static_cast<int32_t>((a.K + G - 1) / G);
    p.units = (p.k_tiles + 1) / 2;
    p.relu = a.relu;
    const bool vec = (reinterpret_cast<uintptr_t>(p.X) & 15u) == 0 && p.K % 8 == 0;
    return vec ? launch_w4_shape<T, G, true>(p, a) : launch_w4_shape<T, G, false>(p, a);
}

}  // namespace gemm_sm103
