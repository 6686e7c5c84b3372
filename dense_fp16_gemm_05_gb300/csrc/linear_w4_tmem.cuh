// linear_w4_tmem.cuh -- the products of linear_w4_kernel.cuh for 17 to 64 rows of X, by
// the tensor core's own path: by mma.sync 64 rows ran at 250 TFLOP/s, an eighth of what
// it does, and with so many rows that, not W's bytes, was what a call took.
//
// A block takes 128 rows of W (8 strips) times some of its columns, 128 at a time (a
// unit).  W's codes become 16-bit q - z in registers and go to tensor memory, which
// tcgen05.mma takes as its 128-row operand: what a lane has of a strip's 16 rows is what
// one store of the shape 16 x 256 bits takes from it.  X's rows are the operand of 32 or
// 64 columns, in shared memory.  A store places two words of a lane side by side, of the four that
// hold its eight neighbouring columns: the product's columns run in the order
//   32 h + 16 k + 4 t + i  for the column  32 h + 8 t + 4 k + i   (t, i < 4, k < 2),
// and X's 8-byte pieces are put down in it.  As in the other kernel a scale group's
// products are summed in fp32 by themselves, in an accumulator of their own, and scaled
// in fp32 on the way into the sums, which a thread keeps for its row of W: q - z is
// exact and nothing is rounded to 16 bits but the result.
//
//   warps 0 - 3   sums: one row of W and 32 columns per thread (0 - 7 for 64 columns);
//                 scales through rings of their own
//   16 warps      W, a strip and every other unit each, through rings of asynchronous
//                 copies; and some rows of X, by registers (8-byte asynchronous copies of
//                 a warp took some 25 cycles each and were the bound)
//   last warp     allocates tensor memory; issues the MMAs, and one commit per unit (or
//                 two), which tells everybody that it is done: a commit holds the lane
//                 for 100 cycles and more
//
// Every warp's code between two waits runs alone on its scheduler for most of the time:
// with a warp per strip for all units a unit took 1400 cycles, of which W's were 1250.
// With two it is bound by instructions (72 % of the issue slots at 64 x 16384 x 8192):
// the codes' conversion and X's way into shared memory, again for every 128 rows of W.
// 64 x 16384 x 8192 bf16 50 us (87 by mma.sync), 64 x 4096 x 4096 fp16 11.1 us (32),
// 64 x 2048 x 2048 7.7 us (12.6), 64 x 1024 x 8192 bf16 12 us (27),
// 32 x 16384 x 8192 40 us (41), 32 x 4096 x 11008 17 us (29).  With 16 rows of X and a
// 16-column operand it takes longer than mma.sync (33 us, 29).
//
// K may be divided over the blocks of a cluster, whose sums are added through
// distributed shared memory.  Every wait is bounded: on expiry the site is recorded in
// the device status word and the block leaves, and no block of its cluster stores.
#pragma once

#include "gemm_kernel.cuh"
#include "linear_w4_kernel.cuh"

namespace gemm_sm103 {

// 32 registers per lane into 16 TMEM lanes x 64 columns: lane (g, t) has of 8 columns
// j the ones 2t and 2t + 1, of rows g (registers 4j, 4j + 1) and g + 8 (4j + 2, 4j + 3).
__device__ __forceinline__ void tmem_store_16x256b_x8(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Starts a load of 16 fp32 columns of the warp's 32 TMEM lanes, one lane per thread; the
// registers are valid behind tcgen05.wait::ld.
__device__ __forceinline__ void tmem_load_start(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Waits for the loads started; the registers are operands, so that no use of them is
// placed before the wait.
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}

// D[tmem] (+)= A[tmem] B[smem] of one 16-bit type, fp32 accumulator.
__device__ __forceinline__ void w4_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ bool w4_elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

struct W4TmemExtra {
    uint64_t limit;   // SM clocks of a wait
    unsigned long long *status;
    int32_t withhold; // test hook: 1 = the last block of a cluster hands over none of W's operands; 0 in every normal call
};

// NX: columns of the MMA, rows of X.
template <int NX, int G>
struct W4TmemShape {
    static constexpr int U = 128 / G;                   // scale groups of a unit
    static constexpr int STRIPS = 8, WAYS = 2;          // warps of W: a strip, every other unit
    static constexpr int SUMS = NX == 64 ? 8 : 4;       // warps that sum
    static constexpr int THREADS = 32 * (SUMS + STRIPS * WAYS + 1);
    static constexpr int COLS = NX * 4 / SUMS;          // of a warp that sums
    static constexpr int DEPTH = 8;                    // units of W under way
    static constexpr int SLOT = 1024 + U * 16;          // bytes: codes, zero points
    static constexpr int S_DEPTH = 8, S_SLOT = 64 * U;  // scales of two strips
    static constexpr int X_ATOM = NX * 128;             // bytes: 64 columns
    static constexpr int X_STAGE = 2 * X_ATOM;
    // A unit's groups are handed over together as far as two of them fit 256 columns.
    static constexpr int PARTS = NX * U > 128 ? NX * U / 128 : 1, PART = U / PARTS;
    static constexpr int A_STAGES = 4;                  // TMEM: 4 x 64 columns
    static constexpr int D_SLOTS = 256 / (NX * PART) < 4 ? 256 / (NX * PART) : 4;   // parts' accumulators, the other 256
    static constexpr int UNITS_DONE = 8;                // barriers of units, more than are under way
    static constexpr int X_OFF = 0, RING_OFF = A_STAGES * X_STAGE;
    static constexpr int S_OFF = RING_OFF + STRIPS * DEPTH * SLOT;
    static constexpr int CTL_OFF = S_OFF + SUMS * S_DEPTH * S_SLOT;
    static constexpr int BARS = UNITS_DONE * PARTS + A_STAGES + D_SLOTS + 1;
    static constexpr int BYTES = 1024 + CTL_OFF + BARS * 8 + 16;   // 1024: alignment
    static_assert(NX * 128 * 4 <= RING_OFF, "a cluster's sums, in the place of X");
    static_assert(DEPTH % WAYS == 0 && A_STAGES % WAYS == 0, "a warp's own units");
    static_assert(UNITS_DONE > A_STAGES && UNITS_DONE * PARTS > D_SLOTS, "phases are told apart");
    static_assert(BYTES <= 227 * 1024, "shared memory of a block");
};

template <class T, int NX, int G>
__global__ void __launch_bounds__(W4TmemShape<NX, G>::THREADS, 1) linear_w4_tmem_sm103a(W4Params<T> p, W4TmemExtra e)
{
    using Codes = W4Codes<T>;
    using Shape = W4TmemShape<NX, G>;
    constexpr int U = Shape::U, D = Shape::DEPTH, AS = Shape::A_STAGES, DS = Shape::D_SLOTS;
    constexpr int WAYS = Shape::WAYS, DW = D / WAYS;   // of a warp of W
    constexpr int SUMS = Shape::SUMS, kMmaWarp = SUMS + Shape::STRIPS * WAYS;
    constexpr int COLS = Shape::COLS, PARTS = Shape::PARTS, PART = Shape::PART, UD = Shape::UNITS_DONE;
    extern __shared__ uint8_t smem_w4[];
    const uint32_t raw = smem_addr(smem_w4), base = (raw + 1023u) & ~1023u;
    uint8_t *mem = smem_w4 + (base - raw);
    const uint32_t bars = base + Shape::CTL_OFF;
    auto done = [&](int i) { return bars + 8u * i; };   // a part's MMAs, of unit % UNITS_DONE
    auto full = [&](int i) { return bars + 8u * (UD * PARTS + i); };   // A in TMEM and X of a unit
    auto d_free = [&](int i) { return bars + 8u * (UD * PARTS + AS + i); };
    const uint32_t drain = bars + 8u * (Shape::BARS - 1);
    volatile uint32_t *slot_ptr = reinterpret_cast<volatile uint32_t *>(mem + Shape::CTL_OFF + 8 * Shape::BARS);
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const int slices = static_cast<int>(gridDim.y), slice = static_cast<int>(blockIdx.y);
    const int u_begin = static_cast<int>(static_cast<int64_t>(p.units) * slice / slices);
    const int u_end = static_cast<int>(static_cast<int64_t>(p.units) * (slice + 1) / slices);
    const int mine = u_end - u_begin;   // units of each of the block's groups of strips
    const int groups = (p.strips + Shape::STRIPS - 1) / Shape::STRIPS;   // this block's: blockIdx.x, + gridDim.x, ...
    const int total = static_cast<int>(blockIdx.x) < groups
                          ? mine * ((groups - static_cast<int>(blockIdx.x) - 1) / static_cast<int>(gridDim.x) + 1) : 0;

    AbortFlag abort;
    abort.local = reinterpret_cast<volatile int *>(const_cast<uint32_t *>(slot_ptr) + 1);
    abort.status = e.status;
    abort.addr = bars + 8u * Shape::BARS + 4u;
    abort.cluster = 1;
    abort.rank = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < UD * PARTS; ++i) mbar_init(done(i), 1);
        for (int i = 0; i < AS; ++i) mbar_init(full(i), Shape::STRIPS);
        for (int i = 0; i < DS; ++i) mbar_init(d_free(i), SUMS);
        mbar_init(drain, 1);
        *abort.local = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc<1>(bars + 8u * Shape::BARS, 512);
        tmem_relinquish<1>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *slot_ptr;
    const uint32_t tmem_d = tmem + AS * 64;
    griddep_wait();
    griddep_launch_dependents();

    if (warp < SUMS) {
        // ---------------------------------------------------------------- sums
        // The first 8 U lanes copy this warp's scales, of strips 2 quarter and 2 quarter + 1.
        const int quarter = warp & 3, first_col = (warp >> 2) * COLS;
        const int half = lane / (4 * U), piece = lane - half * (4 * U), piece_group = piece / 4;
        const bool copies = lane < 8 * U;
        const uint8_t *ring = mem + Shape::S_OFF + warp * (Shape::S_DEPTH * Shape::S_SLOT);
        const uint32_t ring_at = smem_addr(ring) + lane * 8;
        int group = static_cast<int>(blockIdx.x), u = u_begin;   // the next to copy
        const uint8_t *s_src = nullptr;
        auto seek = [&]() {
            const int strip = min(group * Shape::STRIPS + 2 * quarter + half, p.strips - 1);
            s_src = p.S + (static_cast<int64_t>(strip) * p.groups + static_cast<int64_t>(u) * U) * 32 + piece * 8;
        };
        seek();
        auto next = [&](int i) {
            if (i < total) {
                if (copies) {
                    const bool in = u + 1 < p.units || u * U + piece_group < p.groups;
                    w4_copy8(ring_at + (i % Shape::S_DEPTH) * Shape::S_SLOT, in ? s_src : p.S, in);
                }
                s_src += U * 32;
                if (++u == u_end) {
                    u = u_begin;
                    group += static_cast<int>(gridDim.x);
                    seek();
                }
            }
            w4_commit();
        };
        for (int i = 0; i < Shape::S_DEPTH; ++i) next(i);
        float sum[COLS];
#pragma unroll
        for (int n = 0; n < COLS; ++n) sum[n] = 0.0f;
        const uint32_t d_at = tmem_d + (static_cast<uint32_t>(quarter * 32) << 16) + first_col;
        int at_u = 0, at_group = static_cast<int>(blockIdx.x);
        uint32_t part = 0;   // of all units
        bool ok = true;
        for (int i = 0; i < total && ok; ++i) {
            w4_wait<Shape::S_DEPTH - 1>();
            __syncwarp();
            const T *scales = reinterpret_cast<const T *>(ring + (i % Shape::S_DEPTH) * Shape::S_SLOT + (lane >> 4) * (32 * U)) + (lane & 15);
            float s[U];
#pragma unroll
            for (int j = 0; j < U; ++j) s[j] = ln_float(scales[j * 16]);
            __syncwarp();
            next(i + Shape::S_DEPTH);
#pragma unroll
            for (int h = 0; h < PARTS; ++h, ++part) {
                const bool got = wait_phase(done((i % UD) * PARTS + h), (i / UD) & 1u, abort, e.limit, kSiteEpilogueTmemFull);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t at = d_at + (part % DS) * (PART * NX);
#pragma unroll
                for (int j = 0; j < PART; ++j) {
                    uint32_t d[COLS / 16][16];
#pragma unroll
                    for (int k = 0; k < COLS / 16; ++k) tmem_load_start(at + j * NX + k * 16, d[k]);
#pragma unroll
                    for (int k = 0; k < COLS / 16; ++k) tmem_load_wait(d[k]);
                    if (j == PART - 1) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(d_free(part % DS));
                    }
#pragma unroll
                    for (int n = 0; n < COLS; ++n)
                        sum[n] = fmaf(s[h * PART + j], __uint_as_float(d[n / 16][n % 16]), sum[n]);
                }
            }
            if (ok && ++at_u == mine && slices == 1) {
                const int64_t n = static_cast<int64_t>(at_group) * 128 + quarter * 32 + lane;
                if (n < p.N) {
                    T *c = p.C + first_col * p.N + n;
#pragma unroll
                    for (int m = 0; m < COLS; ++m)
                        if (first_col + m < p.M) c[m * p.N] = ln_round<T>(p.relu ? (sum[m] > 0.0f ? sum[m] : 0.0f) : sum[m]);
                }
#pragma unroll
                for (int m = 0; m < COLS; ++m) sum[m] = 0.0f;
                at_u = 0;
                at_group += static_cast<int>(gridDim.x);
            }
        }
        // Behind the last unit's MMAs nothing reads X any more.
        if (slices > 1 && ok) {
            float *ordered = reinterpret_cast<float *>(mem + Shape::X_OFF) + first_col * 128 + quarter * 32 + lane;
#pragma unroll
            for (int m = 0; m < COLS; ++m)
                if (first_col + m < p.M) ordered[m * 128] = sum[m];
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMAs
        // The whole warp walks the loop and one lane issues: what the MMAs take is then in
        // uniform registers already (by one lane alone an MMA took some 100 cycles).
        constexpr uint32_t kType = Codes::kBf16 ? (1u << 7) | (1u << 10) : 0u;
        constexpr uint32_t idesc = idesc_f16_f32(128, NX, false, false) | kType;
        const uint64_t x_desc = smem_desc_sw128(base + Shape::X_OFF, 16, 1024);
        uint32_t part = 0;
        bool ok = true;
        for (int i = 0; i < total && ok; ++i) {
            const int a = i % AS;
            ok = __all_sync(0xffffffffu, wait_phase(full(a), (i / AS) & 1u, abort, e.limit, kSiteMmaFull));
            if (!ok) break;
            fence_proxy_async_smem();   // X, stored by the warps of W
            const uint64_t x_at = x_desc + static_cast<uint64_t>((a * Shape::X_STAGE) >> 4);
            const uint32_t a_at = tmem + a * 64;
#pragma unroll
            for (int h = 0; h < PARTS; ++h, ++part) {
                ok = __all_sync(0xffffffffu, wait_phase(d_free(part % DS), ((part / DS) & 1u) ^ 1u, abort, e.limit, kSiteMmaTmemEmpty));
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d = tmem_d + (part % DS) * (PART * NX);
                const uint32_t bar = done((i % UD) * PARTS + h);
                if (w4_elect_one()) {
                    // The groups in turn: neighbouring MMAs add to different accumulators.
#pragma unroll
                    for (int k = 0; k < G / 16; ++k)
#pragma unroll
                        for (int j = 0; j < PART; ++j) {
                            const int step = (h * PART + j) * (G / 16) + k;   // of the unit's eight
                            w4_mma_ts(d + j * NX, a_at + step * 8,
                                      x_at + static_cast<uint64_t>(((step >> 2) * Shape::X_ATOM + (step & 3) * 32) >> 4), idesc,
                                      k > 0);
                        }
                    mma_commit(bar);
                }
                __syncwarp();
            }
        }
        // Every MMA is complete before tensor memory is freed.
        if (w4_elect_one()) mma_commit(drain);
        __syncwarp();
        wait_phase_drain(drain, 0, e.limit, kSiteDrainMma, e.status);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- W and X
        // Strip j of the eight, of which a quarter of TMEM has two, and units way, way +
        // WAYS, ... of the block's.
        const int j = (warp & 3) * 2 + (((warp - SUMS) >> 2) & 1), way = (warp - SUMS) >> 3;
        const int g = lane >> 2;
        const bool withheld = e.withhold != 0 && slice == slices - 1;
        const uint8_t *ring = mem + Shape::RING_OFF + (way * Shape::STRIPS + j) * (DW * Shape::SLOT);
        const uint32_t q_to = smem_addr(ring) + lane * 16, z_to = smem_addr(ring) + 1024 + lane * 8;
        const bool side = p.Z && lane < 2 * U;
        // The next to copy.
        int i_w = way, u = u_begin, group = static_cast<int>(blockIdx.x);
        const uint8_t *q_src = nullptr, *z_src = nullptr;
        auto seek = [&](int by) {
            u += by;
            q_src += by * 1024;
            z_src += by * (U * 16);
            if (by != 0 && u < u_end) return;
            for (; u >= u_end; u -= mine) group += static_cast<int>(gridDim.x);
            const int strip = min(group * Shape::STRIPS + j, p.strips - 1);
            q_src = p.Q + (static_cast<int64_t>(strip) * p.k_tiles + 2 * u) * kW4TileBytes + lane * 16;
            z_src = p.Z + (static_cast<int64_t>(strip) * p.groups + static_cast<int64_t>(u) * U) * 16 + lane * 8;
        };
        seek(0);
        if (way > 0) seek(way);
        auto next_w = [&](uint32_t dst) {
            if (i_w >= total) return;
            w4_copy16(q_to + dst, q_src);
            if (u + 1 < p.units) {
                w4_copy16(q_to + dst + 512, q_src + 512);
                if (side) w4_copy8(z_to + dst, z_src, true);
            } else {
                const bool tile2 = 2 * u + 1 < p.k_tiles, in = u * U + lane / 2 < p.groups;
                w4_copy16(q_to + dst + 512, tile2 ? q_src + 512 : q_src, tile2 ? 16u : 0u);
                if (side) w4_copy8(z_to + dst, in ? z_src : p.Q, in);
            }
            i_w += WAYS;
            seek(WAYS);
        };
        // Rows j and j + 8 of every 16 of X: this lane's 16 bytes of a row's 256, whose
        // halves go to different places.
        constexpr int XL = NX / 16;
        const int x_row = j + (lane >> 4) * 8, x_piece = lane & 15;
        const int first = (x_piece >> 2) * 64 + (x_piece & 3) * 8, second = first + 32;
        uint8_t *x_to = mem + Shape::X_OFF + (first >> 7) * Shape::X_ATOM + x_row * 128;
        const int x_first = ((((first & 127) >> 4) ^ j) << 4) + (first & 8), x_second = ((((second & 127) >> 4) ^ j) << 4) + (second & 8);
        const int x_loads = x_row < p.M ? (p.M - x_row + 15) / 16 : 0;   // of this lane
        const int64_t x_step = 16 * p.K;
        int x_u = u_begin + way;   // the next to load
        while (x_u >= u_end) x_u -= mine;
        const T *x_src = p.X + x_row * p.K + static_cast<int64_t>(x_u) * 128 + x_piece * 8;
        uint4 xv[XL];
        auto load_x = [&]() {
            const T *src = x_src;
            if (p.vec) {
                const int loads = x_u + 1 < p.units || x_u * 128 + x_piece * 8 < p.K ? x_loads : 0;
#pragma unroll
                for (int m = 0; m < XL; ++m, src += x_step)
                    xv[m] = m < loads ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0u, 0u, 0u, 0u);
            } else {
                const uint64_t lo = reinterpret_cast<uint64_t>(p.X), hi = lo + static_cast<uint64_t>(p.M) * p.K * sizeof(T);
                const int64_t left = p.K - (static_cast<int64_t>(x_u) * 128 + x_piece * 8);
#pragma unroll
                for (int m = 0; m < XL; ++m, src += x_step) {
                    xv[m] = make_uint4(0u, 0u, 0u, 0u);
                    if (m < x_loads && left > 0) xv[m] = w4_eight(src, left, lo, hi);
                }
            }
            x_src += WAYS * 128;
            for (x_u += WAYS; x_u >= u_end; x_u -= mine) x_src -= mine * 128;
        };
        auto store_x = [&](int stage) {
#pragma unroll
            for (int m = 0; m < XL; ++m) {
                uint8_t *to = x_to + stage * Shape::X_STAGE + m * 2048;
                *reinterpret_cast<uint2 *>(to + x_first) = make_uint2(xv[m].x, xv[m].y);
                *reinterpret_cast<uint2 *>(to + x_second) = make_uint2(xv[m].z, xv[m].w);
            }
        };
        load_x();
#pragma unroll
        for (int n = 0; n < DW; ++n) {
            next_w(n * Shape::SLOT);
            w4_commit();
        }
        uint32_t slot = 0;   // bytes
        const uint32_t a_lane = tmem + (static_cast<uint32_t>(j * 16) << 16);
        for (int i = way; i < total; i += WAYS) {
            w4_wait<DW - 1>();
            __syncwarp();
            const uint4 *q = reinterpret_cast<const uint4 *>(ring + slot) + lane;
            const uint4 tile[2] = {q[0], q[32]};
            const uint8_t *zeros = ring + slot + 1024 + g;
            uint32_t r[32];
#pragma unroll
            for (int v = 0; v < U; ++v) {
                uint32_t zlo = Codes::bias(8u, 0), zhi = Codes::bias(8u, 1);
                if (p.Z) {
                    zlo = Codes::bias(zeros[v * 16] & 15u, 0);
                    zhi = Codes::bias(zeros[v * 16 + 8] & 15u, 1);
                }
#pragma unroll
                for (int h = v * (G / 32); h < (v + 1) * (G / 32); ++h) {
                    const uint4 &w = tile[h / 2];
                    const uint32_t words[2] = {h % 2 ? w.z : w.x, h % 2 ? w.w : w.y};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t a[4];
                        Codes::operands(words[k], zlo, zhi, a);
                        uint32_t *o = r + (h * 2 + k) * 4;
                        o[0] = a[0];
                        o[1] = a[2];
                        o[2] = a[1];
                        o[3] = a[3];
                    }
                }
            }
            __syncwarp();
            next_w(slot);
            w4_commit();   // in front of the wait that may give up: w4_wait<0> below covers it
            slot = slot == (DW - 1) * Shape::SLOT ? 0u : slot + Shape::SLOT;
            if (i >= AS) {
                const int before = i - AS;
                const bool got = wait_phase(done((before % UD) * PARTS + PARTS - 1), (before / UD) & 1u, abort, e.limit, kSiteProducerEmpty);
                if (!__all_sync(0xffffffffu, got)) break;
                tc_fence_after_sync();
            }
            store_x(i % AS);
            load_x();   // of the warp's next unit
            tmem_store_16x256b_x8(a_lane + (i % AS) * 64, r);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0 && !withheld) mbar_arrive(full(i % AS));
        }
    }
    w4_wait<0>();   // nothing of this thread's copies is under way
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, 512);
    }
    if (slices == 1) return;
    // Every block of the cluster adds and stores a share of the outputs, 16 bytes of each
    // block at a time.
    const float *ordered = reinterpret_cast<const float *>(mem + Shape::X_OFF);
    cluster_arrive();
    cluster_wait();
    // A block that gave up has left no sums: then nobody stores.
    uint32_t gave_up = 0;
    if (lane < slices)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(gave_up) : "r"(mapa_shared(abort.addr, static_cast<uint32_t>(lane))) : "memory");
    const bool complete = !__any_sync(0xffffffffu, gave_up != 0);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 128;
    for (int o = 4 * (static_cast<int>(threadIdx.x) + slice * Shape::THREADS); o < p.M * 128; o += 4 * slices * Shape::THREADS) {
        const uint32_t at = smem_addr(ordered + o);
        float part[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < slices)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(part[i][0]), "=f"(part[i][1]), "=f"(part[i][2]), "=f"(part[i][3])
                             : "r"(mapa_shared(at, static_cast<uint32_t>(i))));
        const int64_t m = o >> 7, n = n0 + (o & 127);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < slices) v += part[i][b];
            if (p.relu) v = v > 0.0f ? v : 0.0f;
            if (n + b < p.N && complete) p.C[m * p.N + n + b] = ln_round<T>(v);
        }
    }
    cluster_arrive();   // nobody leaves while its sums are read
    cluster_wait();
}

template <class T, int NX, int G>
int launch_w4_tmem(W4Params<T> p, const W4LinearArgs &a)
{
    using Shape = W4TmemShape<NX, G>;
    auto kern = linear_w4_tmem_sm103a<T, NX, G>;
    static std::atomic<int> prepared[kMaxDevices];
    static W4Clusters clusters[kMaxDevices];
    if (!w4_prepare(kern, Shape::THREADS, Shape::BYTES, a, prepared, clusters)) return GEMM_ERR_LAUNCH;
    const int groups = (p.strips + Shape::STRIPS - 1) / Shape::STRIPS;
    // Blocks of a cluster for each group of strips: a unit takes some 720 ns (32 columns:
    // 600), the exchange of the sums as many as this.
    static constexpr float kExchange[] = {0.0f, 1000.0f, 1500.0f, 2500.0f};
    float least = 1e30f;
    int slices = 1;
    for (int l = 0; l < 4 && (1 << l) <= p.units; ++l) {
        const int most = clusters[a.device].most[l].load(std::memory_order_relaxed);
        if (most == 0 || (l > 0 && groups > most)) continue;
        const int units = (p.units + (1 << l) - 1) >> l;
        const float cost = static_cast<float>((groups + most - 1) / most * units) * (NX == 64 ? 720.0f : 600.0f) + kExchange[l];
        if (cost >= least) continue;
        least = cost;
        slices = 1 << l;
    }
    W4TmemExtra extra;
    extra.limit = a.timeout_cycles ? a.timeout_cycles : 1ull << 31;   // about a second
    extra.status = a.status;
    extra.withhold = a.withhold;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t lc = w4_launch_config(slices == 1 && groups > a.sm_count ? a.sm_count : groups, slices,
                                                   Shape::THREADS, Shape::BYTES, a.stream, attr);
    if (cudaLaunchKernelEx(&lc, kern, p, extra) != cudaSuccess) {
        cudaGetLastError();
        prepared[a.device].store(0, std::memory_order_release);
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // namespace gemm_sm103
