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
// group's sum is scaled in fp32.  (For more than 32 rows of X, and for
// more than 16 beside a large weight: linear_w4_tmem.cuh.)
//
// 1 x 4096 x 4096 takes 4.5 us, 1 x 16384 x 8192 16.9 us (4.1 TB/s), 8 x 16384 x 8192 bf16
// with zero points 22 us, 16 x 16384 x 8192 27.9 us, 24 x 1024 x 8192 8.7 us; with
// the products left out the copies alone take 13 to 17 us at 16384 x 8192.  With one row of
// X the copies and the conversion of the codes share the time, with more it is the
// instructions: for eight codes of a lane some 11 of conversion, and the mma.sync.
//
// Every warp streams its own units -- 16 rows x 128 columns of codes with their
// scales and zero points -- through its own ring of asynchronous copies in shared
// memory: nothing but its own copies makes a warp wait, and the bytes under way are
// not bounded by registers.  A block's sixteen warps are RW strips of 16 rows times
// KW ways that the strips' columns are divided, whose sums are added
// through shared memory in a fixed order.  X stays in shared memory for the whole
// call where it fits, while blocks walk over the strips; else it comes in chunks for
// 16 strips at a time, so that it is read less often than W.  K may also be divided
// over the blocks of a cluster, whose sums are added through distributed shared
// memory: so that X fits, or to have blocks enough.
#pragma once

#include <atomic>

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
    int32_t rw, kw;             // strips of a block, ways of a strip
    int32_t x_row, x_bytes;     // X in shared memory: bytes between rows, bytes of a buffer
    int32_t keep_x;             // one buffer for the block's columns; else two chunks
    int32_t vec;                // X's rows are on the 16-byte grid
};

constexpr int kW4Warps = 16, kW4Threads = kW4Warps * 32;

// Asynchronous copies to shared memory of 16 bytes, of which the first `bytes` are read
// and the others zero, and of 8 bytes, all or none.
__device__ __forceinline__ void w4_copy16(uint32_t dst, const void *src, uint32_t bytes = 16)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void w4_copy8(uint32_t dst, const void *src, bool read)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)),
                 "r"(read ? 8u : 0u)
                 : "memory");
}
__device__ __forceinline__ void w4_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void w4_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Eight elements at `src`, of which `left` lie in the row, the others zero; [lo, hi) is
// the tensor.  From the two 16-byte pieces that hold them where those lie in it.
template <class T>
__device__ __forceinline__ uint4 w4_eight(const T *src, int64_t left, uint64_t lo, uint64_t hi)
{
    const uint64_t at = reinterpret_cast<uint64_t>(src), first = at & ~15ull;
    T e[8];
    if (left >= 8 && first >= lo && first + 32 <= hi) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(first)), b = __ldg(reinterpret_cast<const uint4 *>(first) + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const uint32_t shift = static_cast<uint32_t>(at & 15u) / 2u;   // elements
        uint32_t t[6], u[5], v[4];
#pragma unroll
        for (int i = 0; i < 6; ++i) t[i] = shift & 4u ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = shift & 2u ? t[i + 1] : t[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(u[i], u[i + 1], (shift & 1u) * 16u);
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < left ? __ldg(src + i) : ln_round<T>(0.0f);
    uint4 r;
    memcpy(&r, e, 16);
    return r;
}

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
    static constexpr bool kBf16 = false;
    // -(1024 + z) for rows g, -(64 + z) for rows g + 8, twice.
    static __device__ __forceinline__ uint32_t bias(uint32_t z, int odd)
    {
        return odd ? 0xD400D400u + z * 0x00100010u : 0xE400E400u + z * 0x00010001u;
    }
    // 1024 + q and, one nibble further up, 1024 + 16 q, times 1/16: all exact (codes put
    // into the significand of 1024: Y. J. Kim, R. Henry, R. Fahim, H. H. Awadalla, SustaiNLP 2022).
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
    static constexpr bool kBf16 = true;
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

// Sizes of one kernel: NT groups of 8 rows of X; G columns of a scale group.
template <int NT, int G>
struct W4Shape {
    static constexpr int COLS = NT * 8;
    static constexpr int U = 128 / G;                     // scale groups of a unit
    static constexpr int SLOT = 1024 + U * 48;            // bytes: codes, scales, zero points
    static constexpr int DEPTH = NT == 1 ? 6 : 4;         // units under way per warp
    static constexpr int RING = kW4Warps * DEPTH * SLOT;
    static constexpr int X_UNITS = NT == 2 ? 16 : 8;       // of a chunk of X, at least DEPTH
    static constexpr int SUMS = kW4Warps * 16 * (COLS + 1) * 4;
};

// Rows of X half a 128-byte line apart, so that eight lanes' 16-byte loads from two
// rows meet no bank twice.
constexpr int64_t w4_x_row(int64_t units) { return units * 256 + 64; }

template <class T, int NT, int G>
__global__ void __launch_bounds__(kW4Threads, 1) linear_w4_kernel(W4Params<T> p)
{
    using Codes = W4Codes<T>;
    using Shape = W4Shape<NT, G>;
    constexpr int U = Shape::U, COLS = Shape::COLS, D = Shape::DEPTH;
    extern __shared__ uint4 smem[];   // the rings; X; sums (behind a kept X, else in the place of all)
    typedef float Sums[kW4Warps][16][COLS + 1];   // of a warp's strip
    griddep_wait();
    griddep_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const int g = lane >> 2, t = lane & 3;
    const int kw = warp / p.rw, rw = warp - kw * p.rw;
    const int slices = static_cast<int>(gridDim.y), slice = static_cast<int>(blockIdx.y);
    const int u_begin = static_cast<int>(static_cast<int64_t>(p.units) * slice / slices);
    const int u_end = static_cast<int>(static_cast<int64_t>(p.units) * (slice + 1) / slices);
    uint8_t *x_mem = reinterpret_cast<uint8_t *>(smem) + Shape::RING;
    const uint8_t *ring = reinterpret_cast<const uint8_t *>(smem) + warp * (D * Shape::SLOT);
    const uint32_t ring_at = smem_addr(ring);

    // X's columns of `units` units from unit u on, all threads together, zeros past K.
    auto copy_x = [&](uint8_t *dst, int u, int units) {
        const int per_row = units * 16;   // 16-byte pieces
        const int64_t k0 = static_cast<int64_t>(u) * 128;
        const uint64_t lo = reinterpret_cast<uint64_t>(p.X), hi = lo + static_cast<uint64_t>(p.M) * p.K * sizeof(T);
        for (int i = threadIdx.x; i < p.M * per_row; i += kW4Threads) {
            const int m = i / per_row, c = i - m * per_row;
            const int64_t left = p.K - (k0 + c * 8);
            const T *src = p.X + m * p.K + k0 + c * 8;
            uint8_t *to = dst + m * p.x_row + c * 16;
            if (p.vec) w4_copy16(smem_addr(to), left > 0 ? src : p.X, left > 0 ? 16u : 0u);
            else *reinterpret_cast<uint4 *>(to) = w4_eight(src, left, lo, hi);
        }
    };
    // This lane's piece of a unit's scales (the first 4 U lanes) or zero points (2 U).
    const bool side_s = lane < 4 * U, side = side_s || (p.Z && lane < 6 * U);
    const int side_j = side_s ? lane : lane - 4 * U, side_group = side_s ? lane / 4 : side_j / 2;
    const uint8_t *side_base = (side_s ? p.S : p.Z) + side_j * 8;
    const uint32_t side_bytes = side_s ? 32u : 16u;   // of a group
    const uint32_t side_to = 1024u + static_cast<uint32_t>(side_s ? lane * 8 : U * 32 + side_j * 8);
    const uint32_t q_step = p.kw * 1024u, side_step = p.kw * U * side_bytes;
    const uint8_t *q_src = nullptr, *side_src = nullptr;
    auto seek = [&](int strip, int u) {
        strip = min(strip, p.strips - 1);   // one past the last is read as the last and not stored
        q_src = p.Q + (static_cast<int64_t>(strip) * p.k_tiles + 2 * u) * kW4TileBytes + lane * 16;
        side_src = side_base + (static_cast<int64_t>(strip) * p.groups + static_cast<int64_t>(u) * U) * side_bytes;
    };
    // Unit u into the slot at `dst` bytes.  The last unit may have one tile, and scales of
    // fewer groups: zeros stand for the others.
    const uint32_t q_to = ring_at + lane * 16, s_to = ring_at + side_to;
    auto fetch = [&](uint32_t dst, int u) {
        if (u + 1 < p.units) {
            w4_copy16(q_to + dst, q_src);
            w4_copy16(q_to + dst + 512, q_src + 512);
            if (side) w4_copy8(s_to + dst, side_src, true);
        } else {
            const bool tile2 = 2 * u + 1 < p.k_tiles, in = u * U + side_group < p.groups;
            w4_copy16(q_to + dst, q_src);
            w4_copy16(q_to + dst + 512, tile2 ? q_src + 512 : q_src, tile2 ? 16u : 0u);
            if (side) w4_copy8(s_to + dst, in ? side_src : p.Q, in);
        }
        q_src += q_step;
        side_src += side_step;
    };

    // A row past X's last is read as the last one: it reaches nothing but its own
    // column of the result, which is not stored.
    uint32_t x_off[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x_off[n] = static_cast<uint32_t>(min(n * 8 + g, p.M - 1) * p.x_row + t * 16);
    float sum[NT][4];
    // Adds a unit's products: codes, scales and zero points in `slot`, X's columns at `x_unit`.
    auto unit = [&](const uint8_t *slot, const uint8_t *x_unit) {
        const uint4 *q = reinterpret_cast<const uint4 *>(slot) + lane;
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
                for (int n = 0; n < NT; ++n) x[n] = *reinterpret_cast<const uint4 *>(x_unit + x_off[n] + h * 64);
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
            const float s0 = ln_float(sc[0]), s1 = ln_float(sc[8]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = P == 2 ? d[0][n][e] + d[P - 1][n][e] : d[0][n][e];
                    sum[n][e] = fmaf(e < 2 ? s0 : s1, v, sum[n][e]);
                }
        }
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
            for (int e = 0; e < 4; ++e) sums[warp][g + 8 * (e >> 1)][n * 8 + 2 * t + (e & 1)] = sum[n][e];
    };
    // The block's outputs, of strips strip0 .. strip0 + rw - 1: o is a row of them and of X.
    const int rows = p.rw * 16, out = rows * p.M;
    // `ordered`: room for them, among the blocks of a cluster.
    auto finish = [&](Sums &sums, float *ordered, int strip0) {
        const int64_t n0 = static_cast<int64_t>(strip0) * 16;
        auto ways = [&](int r, int m) {
            float v = sums[r >> 4][r & 15][m];
            for (int i = 1; i < p.kw; ++i) v += sums[i * p.rw + (r >> 4)][r & 15][m];
            return v;
        };
        auto store = [&](int r, int m, float v) {
            if (n0 + r >= p.N) return;
            if (p.relu) v = v > 0.0f ? v : 0.0f;
            p.C[m * p.N + n0 + r] = ln_round<T>(v);
        };
        if (slices == 1) {
            for (int o = threadIdx.x; o < out; o += kW4Threads) {
                const int m = o / rows, r = o - m * rows;
                store(r, m, ways(r, m));
            }
            return;
        }
        // The block's sums in the outputs' order, then every block of the cluster adds and
        // stores a share: loads from another block are worth it in whole 16-byte pieces
        // (64 x 8192 x 1024 over 8 blocks: 98 us element by element).
        for (int o = threadIdx.x; o < out; o += kW4Threads) {
            const int m = o / rows, r = o - m * rows;
            ordered[o] = ways(r, m);
        }
        cluster_arrive();
        cluster_wait();
        for (int o = 4 * (threadIdx.x + slice * kW4Threads); o < out; o += 4 * slices * kW4Threads) {
            const uint32_t at = smem_addr(ordered + o);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, part[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < slices)
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(part[i][0]), "=f"(part[i][1]), "=f"(part[i][2]), "=f"(part[i][3])
                                 : "r"(mapa_shared(at, static_cast<uint32_t>(i))));
            const int m = o / rows, r = o - m * rows;   // rows are a multiple of 16
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < slices) v[e] += part[i][e];
                store(r + e, m, v[e]);
            }
        }
        cluster_arrive();   // nobody goes on while its sums are read
        cluster_wait();
    };

    if (p.keep_x) {
        // Groups of rw strips blockIdx.x, blockIdx.x + gridDim.x, ...; this warp has units
        // u_begin + kw, u_begin + kw + KW, ... of its strip of each, `mine` of them (none, if
        // it is beyond the rw kw warps that there is work for).
        Sums *part = reinterpret_cast<Sums *>(x_mem + p.x_bytes);
        const int first = u_begin + kw, mine = kw < p.kw && first < u_end ? (u_end - first + p.kw - 1) / p.kw : 0;
        copy_x(x_mem, u_begin, u_end - u_begin);
        w4_commit();
        // The copies run ahead of the products by D units, over the strips' ends.
        const int strip_step = static_cast<int>(gridDim.x) * p.rw, strip_first = static_cast<int>(blockIdx.x) * p.rw;
        // Of the strip under way there, the next unit to fetch; of the last, none.
        int ahead_strip = strip_first, ahead = mine > 0 && strip_first < p.strips ? first : u_end;
        seek(ahead_strip + rw, first);
        auto next = [&](uint32_t dst) {
            if (ahead < u_end) {
                fetch(dst, ahead);
                ahead += p.kw;
                if (ahead >= u_end) {
                    ahead_strip += strip_step;
                    if (ahead_strip < p.strips) {
                        ahead = first;
                        seek(ahead_strip + rw, first);
                    }
                }
            }
            w4_commit();
        };
#pragma unroll
        for (int i = 0; i < D; ++i) next(i * Shape::SLOT);
        w4_wait<D>();
        __syncthreads();   // X is there
        const uint8_t *x_first = x_mem + kw * 256;
        uint32_t slot = 0;   // bytes
        int buffer = 0;
        for (int strip0 = strip_first; strip0 < p.strips; strip0 += strip_step) {
            clear();
            const uint8_t *x_unit = x_first;
            for (int i = 0; i < mine; ++i) {
                w4_wait<D - 1>();
                __syncwarp();
                unit(ring + slot, x_unit);
                x_unit += p.kw * 256;
                __syncwarp();
                next(slot);
                slot = slot == (D - 1) * Shape::SLOT ? 0u : slot + Shape::SLOT;
            }
            keep(part[buffer]);
            __syncthreads();
            finish(part[buffer], reinterpret_cast<float *>(part + 1), strip0);
            // Sums of the group after the next are written behind the next one's barrier
            // (among the blocks of a cluster, all of a group behind the last one's).
            if (slices == 1) buffer ^= 1;
        }
    } else {
        // One strip per warp (rw = 16), units u_begin .. u_end - 1; X in chunks that the
        // block shares.
        constexpr int XU = Shape::X_UNITS;
        static_assert(XU >= D, "a chunk of X is there when the units copied with it are");
        const int n = u_end - u_begin;
        seek(static_cast<int>(blockIdx.x) * p.rw + rw, u_begin);
        clear();
        copy_x(x_mem, u_begin, XU);
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if (i < n) fetch(i * Shape::SLOT, u_begin + i);
            w4_commit();
        }
        uint32_t slot = 0;   // bytes
        int x_unit = 0, x_buffer = 0;
        for (int i = 0; i < n; ++i) {
            w4_wait<D - 1>();
            if (x_unit == 0) {
                __syncthreads();   // this chunk is there, and the one before is done with
                if (i + XU < n) copy_x(x_mem + (x_buffer ^ 1) * p.x_bytes, u_begin + i + XU, XU);
            } else {
                __syncwarp();
            }
            unit(ring + slot, x_mem + x_buffer * p.x_bytes + x_unit * 256);
            __syncwarp();
            if (i + D < n) fetch(slot, u_begin + i + D);
            w4_commit();
            slot = slot == (D - 1) * Shape::SLOT ? 0u : slot + Shape::SLOT;
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
        finish(sums, reinterpret_cast<float *>(&sums + 1), static_cast<int>(blockIdx.x) * p.rw);
    }
}

constexpr int kW4Budget = 225 * 1024;   // dynamic shared memory of a block

// Clusters of 1, 2, 4 and 8 blocks that the GPU holds at a time, 0: none.  Of blocks that
// fill an SM a cluster lies within a part of the GPU, whose SMs larger clusters do not
// divide evenly: clusters that are a few too many take as long as twice as many.
struct W4Clusters {
    std::atomic<int> most[4];
};

inline cudaLaunchConfig_t w4_launch_config(int groups, int slices, int threads, int64_t smem, cudaStream_t stream,
                                           cudaLaunchAttribute (&attr)[2])
{
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(groups), static_cast<unsigned>(slices), 1);
    lc.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = static_cast<unsigned>(slices);
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = slices > 1 ? 2 : 1;
    return lc;
}

// Once per kernel and device: its shared memory, and the clusters that fit.
template <class Kernel>
bool w4_prepare(Kernel kern, int threads, int64_t smem, const W4LinearArgs &a, std::atomic<int> (&prepared)[kMaxDevices],
                W4Clusters (&clusters)[kMaxDevices])
{
    if (prepared[a.device].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    clusters[a.device].most[0].store(a.sm_count, std::memory_order_relaxed);
    for (int l = 1; l < 4; ++l) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t lc = w4_launch_config(a.sm_count, 1 << l, threads, smem, a.stream, attr);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &lc) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        clusters[a.device].most[l].store(n, std::memory_order_relaxed);
    }
    prepared[a.device].store(1, std::memory_order_release);
    return true;
}

template <class T, int NT, int G>
int launch_w4_kernel(W4Params<T> p, const W4LinearArgs &a)
{
    using Shape = W4Shape<NT, G>;
    auto kern = linear_w4_kernel<T, NT, G>;
    static std::atomic<int> prepared[kMaxDevices];
    static W4Clusters clusters[kMaxDevices];
    if (!w4_prepare(kern, kW4Threads, kW4Budget, a, prepared, clusters)) return GEMM_ERR_LAUNCH;
    // The division of the work that costs least by this count of nanoseconds, fitted to
    // whole calls under every division; of 25 other shapes (1 to 32 rows, up to
    // 16384 x 8192) it picks the best of all in 23, and in the others one within a
    // twentieth of it (4 x 1024 x 8192 4.8 us of 4.6).  A
    // unit of each of a block's sixteen warps takes 450 with 8 rows of X, 650 with 16,
    // 1030 with 32, and with fewer warps as much less, down to eleven; a group of strips
    // ends with 500, more among the blocks of a cluster, and a quarter for each output; X
    // comes with 60 bytes each, 20 where its rows cannot lie on the 16-byte grid, and in
    // chunks half hidden.  (Where they could and do not is not counted, so that the order
    // of the sums does not go by X's address.)
    const int64_t room = kW4Budget - Shape::RING - 2 * Shape::SUMS;   // for a kept X
    const float unit_cost = NT == 1 ? 450.0f : (NT == 2 ? 650.0f : 1030.0f);
    static constexpr uint8_t kDivisions[][2] = {{16, 1}, {15, 1}, {14, 1}, {8, 2}, {7, 2}, {6, 2},
                                                {5, 3},  {4, 4},  {3, 5},  {2, 8}, {2, 7}, {1, 16}};
    float least = 1e30f;
    int slices = 1;
    for (int l = 0; l < 4 && (1 << l) <= p.units; ++l) {
        const int sl = 1 << l, units = (p.units + sl - 1) / sl, most = clusters[a.device].most[l].load(std::memory_order_relaxed);
        if (most == 0) continue;
        const int64_t x_bytes = p.M * w4_x_row(units);
        const float x_cost = static_cast<float>(x_bytes) / (p.K % 8 == 0 ? 60.0f : 20.0f);
        const float end = sl == 1 ? 500.0f : (sl == 2 ? 1500.0f : (sl == 4 ? 3000.0f : 4000.0f));
        const bool fits = x_bytes <= room;
        for (const auto &d : kDivisions) {
            const int rw = d[0], kw = d[1];
            if (kw > units) continue;
            const int rounds = ((p.strips + rw - 1) / rw + most - 1) / most, warps = rw * kw > 11 ? rw * kw : 11;
            const float group = static_cast<float>((units + kw - 1) / kw * warps) * (unit_cost / 16.0f) + end +
                                static_cast<float>(rw * 4 * p.M);
            auto consider = [&](float cost, int keep) {
                if (cost >= least) return;
                least = cost;
                slices = sl;
                p.keep_x = keep;
                p.rw = rw;
                p.kw = kw;
            };
            if (rw == kW4Warps) consider(static_cast<float>(rounds) * (group + 0.5f * x_cost), 0);
            if (fits) consider(static_cast<float>(rounds) * group + x_cost, 1);
        }
    }
    const int groups = (p.strips + p.rw - 1) / p.rw;
    const int most = slices == 1 ? a.sm_count : clusters[a.device].most[slices == 2 ? 1 : (slices == 4 ? 2 : 3)].load(std::memory_order_relaxed);
    int64_t smem = Shape::RING;
    if (p.keep_x) {
        p.x_row = static_cast<int32_t>(w4_x_row((p.units + slices - 1) / slices));
        p.x_bytes = p.M * p.x_row;
        smem += p.x_bytes + 2 * Shape::SUMS;
    } else {
        p.x_row = static_cast<int32_t>(w4_x_row(Shape::X_UNITS));
        p.x_bytes = p.M * p.x_row;
        smem += 2 * p.x_bytes;
        if (smem < 2 * Shape::SUMS) smem = 2 * Shape::SUMS;
    }
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t lc = w4_launch_config(p.keep_x && groups > most ? most : groups, slices, kW4Threads, smem, a.stream, attr);
    if (cudaLaunchKernelEx(&lc, kern, p) != cudaSuccess) {
        cudaGetLastError();
        prepared[a.device].store(0, std::memory_order_release);
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // namespace gemm_sm103
