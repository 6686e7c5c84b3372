// gemm_mxfp4_kernel.cuh -- microscaled 4-bit GEMM (MXFP4: E2M1 elements, one
// E8M0 scale per 32 elements along K) with a fused ReLU, for sm_103a:
//
//   C[i,j] = R( sum_b 2^(sa[i,b] - 127) * 2^(sw[j,b] - 127) * sum_{k in block b} A[i,k] W[j,k] )
//
// A (M,K) and W (N,K) hold two codes per byte (element 2i in the low half),
// row pitch 16 ceil(K/32) bytes; the scale bytes come in 512-byte tiles of 128
// rows x 4 blocks, byte (r % 32) * 16 + (r / 32) * 4 + b, tiles of a row block
// adjacent along K.  That is the order of the tensor core's scale memory: four
// TMEM columns hold a tile, row r's word at lane r % 32 (in each 32-lane
// quarter), column r / 32, its four bytes the scales of four K blocks of 32.
// tcgen05.mma.kind::mxf4 (K = 64, two scales per row) takes bytes 0-1 or 2-3 of
// the words, as the instruction descriptor's scale ids 0 or 2 say.
//
// The tiles come by TMA beside the operands; four scale warps, one per quarter,
// read a tile's rows (16 bytes per lane) from shared memory and store them into
// TMEM.  tcgen05.cp would move a tile with one instruction, but between the MMAs
// of one K block and the next it drains the tensor pipe: the copies of a K
// block cost about 300 cycles beside 512 of MMAs whether they are two or six
// (8192^3: 231 us with copies, 165 us with the copies left out), while a
// store from another warp runs beside the MMAs (185 us, all else equal).
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "gemm_kernel.cuh"

namespace gemm_sm103 {

// ---------------------------------------------------------------- PTX

// D[tmem] (+)= (A[smem] x scale_A) * (B[smem] x scale_B), E2M1 operands, two
// E8M0 scales per row of A and of B for the instruction's K = 64, fp32
// accumulator.
template <int kCtaGroup>
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate)
{
    if constexpr (kCtaGroup == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
            : "memory");
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint4 ld_shared_u32x4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

// Stores two scale tiles (this lane's 16 bytes of each) into eight consecutive
// columns of the warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_store_scales(uint32_t taddr, const uint4 &a, const uint4 &b)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// Waits until this thread's TMEM stores are complete.
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 3-D tiled load of one box (coordinates x, y, z), completion counted on a
// barrier of this CTA.
__device__ __forceinline__ void tma_load_3d_cta(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x,
                                                int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Loads 16 consecutive fp32 columns of the warp's 32 TMEM lanes and waits.
__device__ __forceinline__ void tmem_load_32x32b_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Instruction descriptor for tcgen05.mma.kind::mxf4: E2M1 A and B (format 1 in
// bits 7-9 and 10-11), both K-major, N >> 3 (17-22), E8M0 scales (bit 23),
// M >> 7 (27-28), K = 64 (bit 31 = 0); scale ids (4-5 for B, 29-30 for A) are
// added per MMA.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N)
{
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 7) << 27);
}

// ---------------------------------------------------------------- CTA pairs, 256 x 256 tiles

// One CTA per SM, a cluster = one CTA pair, a persistent grid over 256 x 256
// output tiles in grouped raster order; each CTA holds 128 rows of the tile's
// accumulator.  A stage is 256 elements of K: a 128-byte swizzle row of A and
// W per row, four MMAs.
struct Mx4Cfg {
    static constexpr int BM = 128;             // rows of C per CTA (TMEM lanes)
    static constexpr int TILE_M = 256;         // rows per pair tile (the MMA's M)
    static constexpr int BN = 256;             // columns of C per tile (the MMA's N)
    static constexpr int BN_CTA = BN / 2;      // rows of W each CTA loads
    static constexpr int BK = 256;             // elements per K block = one 128-byte swizzle row
    static constexpr int ROW_BYTES = BK / 2;
    static constexpr int UMMA_K = 64;
    static constexpr int STEP_BYTES = UMMA_K / 2;
    static constexpr int SF_TILE = 512;        // bytes of a scale tile: 128 rows x 4 blocks of 32
    static constexpr int SF_TILES = BK / 128;  // scale tiles per row block and K block
    static constexpr int STAGES = 5;
    static constexpr int THREADS = 320;
    static constexpr int A_STAGE_BYTES = BM * ROW_BYTES;                // 16 KiB
    static constexpr int W_STAGE_BYTES = BN_CTA * ROW_BYTES;            // 16 KiB
    static constexpr int SFA_STAGE_BYTES = SF_TILES * SF_TILE;          // this CTA's 128 rows
    static constexpr int SFW_STAGE_BYTES = 2 * SF_TILES * SF_TILE;      // all 256 columns, in each CTA
    static constexpr int STAGE_TX_BYTES = A_STAGE_BYTES + W_STAGE_BYTES;
    static constexpr int HALF_TX_BYTES = A_STAGE_BYTES + W_STAGE_BYTES / 2;   // of a half tile
    static constexpr int SF_TX_BYTES = SFA_STAGE_BYTES + SFW_STAGE_BYTES;
    static constexpr int SF_SLOTS = STAGES;    // scale slots in TMEM, one per ring slot
    static constexpr int SFW_COL = 4 * SF_TILES;                        // W words after A's in a slot
    static constexpr int SF_SLOT_COLS = 4 * SF_TILES + 8 * SF_TILES;    // 24 columns
    static constexpr int TMEM_COLS = 512;
    static constexpr int SF_COL0 = TMEM_COLS - SF_SLOTS * SF_SLOT_COLS; // 392
    static constexpr int ACC1_COL = SF_COL0 - BN;                       // 136
    static constexpr int EPI_COLS = 64;
    static constexpr int EPI_CHUNKS = BN / EPI_COLS;    // 4
    static constexpr int C_BUF_BYTES = 32 * EPI_COLS * 2;   // one warp's 32 rows of one chunk
    static constexpr int SMEM_A_OFF = 0;
    static constexpr int SMEM_W_OFF = STAGES * A_STAGE_BYTES;
    static constexpr int SMEM_C_OFF = SMEM_W_OFF + STAGES * W_STAGE_BYTES;
    static constexpr int SMEM_SFA_OFF = SMEM_C_OFF + 4 * 2 * C_BUF_BYTES;
    static constexpr int SMEM_SFW_OFF = SMEM_SFA_OFF + STAGES * SFA_STAGE_BYTES;
    static constexpr int SMEM_CTL_OFF = SMEM_SFW_OFF + STAGES * SFW_STAGE_BYTES;
    static constexpr int SMEM_CTL_BYTES = 256;
    static constexpr int SMEM_BYTES = 1024 + SMEM_CTL_OFF + SMEM_CTL_BYTES;
    static constexpr uint32_t IDESC = idesc_mxf4(TILE_M, BN);
    static constexpr uint32_t IDESC_HALF = idesc_mxf4(TILE_M, BN / 2);

    // The two accumulators share the columns [ACC1_COL, BN); the epilogue reads
    // the RELEASE chunks that hold those first.
    static constexpr int RELEASE = (BN - ACC1_COL + EPI_COLS - 1) / EPI_COLS;
    static_assert(ACC1_COL > 0 && RELEASE == 2 && EPI_CHUNKS == 4, "the epilogue's order of reads");
    static_assert((4 * STAGES + 5) * 8 <= SMEM_CTL_BYTES, "control block");
    static_assert(SF_TILES == 2, "the scale warps' stores");
    static_assert(SMEM_BYTES <= 232448, "shared memory per block on sm_103");
};

struct Mx4Params {
    int32_t M, N;
    int32_t num_m_blocks;   // ceil(M / 256)
    int32_t num_n_blocks;   // ceil(N / 256)
    int32_t num_k_blocks;   // ceil(K / 256)
    int32_t num_units;      // whole tiles, then half tiles
    int32_t split_start;    // tiles from here on are two units of 128 columns each
    int32_t group_m;        // rasterisation panel height, in tiles
    int32_t withhold;       // test hook (gemm_mxfp4_selftest_timeout): loads not issued,
                            // 1 all of them, 2 the scale tiles'; 0 in every normal call
    uint64_t timeout_cycles;
    unsigned long long *status;
};

// Work unit u: tile (mb, nb) and, of a split tile, which half of its columns
// (-1: the whole tile).
__device__ __forceinline__ void mx4_unit_coords(int u, const Mx4Params &p, int &mb, int &nb, int &half)
{
    int t = u;
    half = -1;
    if (u >= p.split_start) {
        t = p.split_start + ((u - p.split_start) >> 1);
        half = (u - p.split_start) & 1;
    }
    const int per_group = p.group_m * p.num_n_blocks;
    const int g = t / per_group;
    const int first_m = g * p.group_m;
    const int rows = min(p.num_m_blocks - first_m, p.group_m);
    const int r = t - g * per_group;
    mb = first_m + r % rows;
    nb = r / rows;
}

// Roles per CTA:
//   warp 0, one lane   TMA producer: per K block a box of A and of W (128 bytes
//                      x 128 rows each), completing on the pair leader's "full"
//                      barrier, and the scale tiles of A's 128 rows and of the
//                      tile's 256 columns, completing on this CTA's "scales
//                      full" barrier
//   warp 1             (leader CTA only) issues the MMAs, M = 256, N = 256, K = 64
//   warps 2..5         epilogue: accumulator -> R -> fp16 -> shared memory ->
//                      TMA store
//   warps 6..9         scale warps: tiles from shared memory to TMEM, then an
//                      arrival on the leader's "scales ready" barrier
// TMEM (512 columns): each ring slot has its own scale slot of 24 columns, free
// again when the ring slot is: the scale warps need no barrier of their own for
// it.  Two accumulators of 256 columns do not fit beside them, so these overlap
// in 120 columns.  The epilogue reads the two chunks that hold those columns
// first and then lets the next tile's MMAs start, which run while it reads and
// stores the rest.
// The tiles of a last wave that fills less than half of the pairs are divided
// into two units of 128 columns each (M = 256, N = 128 MMAs on half of W's rows);
// both read the tile's scales whole and take their half's columns.
// Ragged edges: TMA zero-fills operands and scales outside A and W (a zero
// scale byte is 2^-127, not NaN); rows and columns outside C are not stored.
// Every wait is bounded; on expiry the site is recorded in the device status
// word and all roles leave.
template <bool kRelu>
__global__ void __launch_bounds__(Mx4Cfg::THREADS, 1)
    gemm_mxfp4_sm103a(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                      const __grid_constant__ CUtensorMap tmap_w_half,
                      const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ CUtensorMap tmap_sw,
                      const __grid_constant__ CUtensorMap tmap_c, const Mx4Params p)
{
    using Cfg = Mx4Cfg;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;   // SW128 atoms need 1024-byte alignment
    uint8_t *base_ptr = smem_raw + (base - raw);

    const uint32_t sA = base + Cfg::SMEM_A_OFF;
    const uint32_t sW = base + Cfg::SMEM_W_OFF;
    const uint32_t sC = base + Cfg::SMEM_C_OFF;
    const uint32_t sSFA = base + Cfg::SMEM_SFA_OFF;
    const uint32_t sSFW = base + Cfg::SMEM_SFW_OFF;
    const uint32_t ctl = base + Cfg::SMEM_CTL_OFF;
    constexpr int S = Cfg::STAGES;
    auto full_bar = [&](int s) { return ctl + 8u * s; };
    auto empty_bar = [&](int s) { return ctl + 8u * (S + s); };
    auto sfull_bar = [&](int s) { return ctl + 8u * (2 * S + s); };
    auto sready_bar = [&](int s) { return ctl + 8u * (3 * S + s); };
    const uint32_t tfull_bar = ctl + 8u * (4 * S);
    const uint32_t tempty_bar = ctl + 8u * (4 * S + 1);
    const uint32_t drain_bar = ctl + 8u * (4 * S + 2);
    const uint32_t tmem_slot = ctl + 8u * (4 * S + 3);
    const uint32_t abort_addr = tmem_slot + 4;
    volatile uint32_t *tmem_slot_ptr =
        reinterpret_cast<volatile uint32_t *>(base_ptr + Cfg::SMEM_CTL_OFF + 8 * (4 * S + 3));

    // By shuffle, so that the compiler knows it uniform in the warp.
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();   // 0: the pair leader, which issues the MMAs
    const bool leader = rank == 0;
    constexpr uint16_t kPairMask = 0x3u;

    AbortFlag abort;
    abort.local = reinterpret_cast<volatile int *>(tmem_slot_ptr + 1);
    abort.status = p.status;
    abort.addr = abort_addr;
    abort.cluster = 2;
    abort.rank = rank;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 2);    // each CTA's arrive.expect_tx (used on the leader)
            mbar_init(empty_bar(s), 1);   // one MMA commit, sent to both CTAs
            mbar_init(sfull_bar(s), 1);   // this CTA's scale tiles
            mbar_init(sready_bar(s), 8);  // one arrive per scale warp of both CTAs (used on the leader)
        }
        mbar_init(tfull_bar, 1);          // one MMA commit, sent to both CTAs
        mbar_init(tempty_bar, 8);         // one arrive per epilogue warp of both CTAs
        mbar_init(drain_bar, 1);
        *abort.local = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmap_a);
        prefetch_tensormap(&tmap_w);
        if (p.split_start < p.num_units) prefetch_tensormap(&tmap_w_half);
        prefetch_tensormap(&tmap_sa);
        prefetch_tensormap(&tmap_sw);
        prefetch_tensormap(&tmap_c);
    }
    if (warp == 1) {
        tmem_alloc<2>(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish<2>();
    }
    tc_fence_before_sync();
    __syncthreads();
    // Both CTAs' barriers are initialised and their TMEM allocated before
    // either signals the other.
    cluster_arrive();
    cluster_wait();
    tc_fence_after_sync();
    griddep_launch_dependents();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot_ptr, 0);
    const uint64_t limit = p.timeout_cycles;
    const int KB = p.num_k_blocks;
    const int first = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);
    // The producer's ring slots in use, and the parity of their last load.
    volatile uint32_t *issued_ptr = tmem_slot_ptr + 2;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            uint32_t issued_mask = 0, issued_parity = 0;
            bool ok = true;
            const uint32_t full_base = leader ? full_bar(0) : mapa_shared(full_bar(0), 0);
            griddep_wait();   // A, W and the scales may come from the kernel just before
            for (int u = first; ok && u < p.num_units && p.withhold != 1; u += stride) {
                int mb, nb, half;
                mx4_unit_coords(u, p, mb, nb, half);
                const uint32_t tx = half < 0 ? Cfg::STAGE_TX_BYTES : Cfg::HALF_TX_BYTES;
                const CUtensorMap *map_w = half < 0 ? &tmap_w : &tmap_w_half;
                const int m0 = mb * Cfg::TILE_M + static_cast<int>(rank) * Cfg::BM;
                const int n0 = nb * Cfg::BN + (half < 0 ? static_cast<int>(rank) * Cfg::BN_CTA
                                                        : half * Cfg::BN_CTA + static_cast<int>(rank) * (Cfg::BN_CTA / 2));
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wait_phase(empty_bar(s), ph ^ 1u, abort, limit, kSiteProducerEmpty)) {
                        ok = false;
                        break;
                    }
                    // Both CTAs' bytes are counted on the leader's barrier; each
                    // announces its own.
                    const uint32_t fb = full_base + 8u * s;
                    if (leader) mbar_arrive_expect_tx(fb, tx);
                    else mbar_arrive_expect_tx_cluster(fb, tx);
                    tma_load_2d_pair(sA + s * Cfg::A_STAGE_BYTES, &tmap_a, fb, kb * Cfg::ROW_BYTES, m0);
                    tma_load_2d_pair(sW + s * Cfg::W_STAGE_BYTES, map_w, fb, kb * Cfg::ROW_BYTES, n0);
                    // Scale tiles: (word in the tile, tile along K, row block).
                    if (p.withhold == 0) {
                        mbar_arrive_expect_tx(sfull_bar(s), Cfg::SF_TX_BYTES);
                        tma_load_3d_cta(sSFA + s * Cfg::SFA_STAGE_BYTES, &tmap_sa, sfull_bar(s), 0,
                                        kb * Cfg::SF_TILES, mb * 2 + static_cast<int>(rank));
                        tma_load_3d_cta(sSFW + s * Cfg::SFW_STAGE_BYTES, &tmap_sw, sfull_bar(s), 0,
                                        kb * Cfg::SF_TILES, nb * 2);
                    }
                    issued_mask |= 1u << s;
                    issued_parity = (issued_parity & ~(1u << s)) | (ph << s);
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            issued_ptr[0] = issued_mask;
            issued_ptr[1] = issued_parity;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (leader CTA)
        // The whole warp walks the loop and one lane issues: what the MMAs take
        // (descriptors, addresses) is then in uniform registers already.  With a
        // single lane in the loop each MMA waited for some ten moves there, and
        // a K block's four MMAs, 512 cycles of work, took some 640 to issue
        // (8192^3 with this and the epilogue's early reads: 185 us -> 156 us).
        if (leader) {
            int s = 0;
            uint32_t ph = 0, acc_it = 0;
            bool ok = true, issued_any = false;
            // K-major SW128 operands: 8-row groups 1024 B apart; a K step of 64
            // elements is +32 B inside the swizzle row.
            const uint64_t a_desc0 = smem_desc_sw128(sA, 16, 1024);
            const uint64_t w_desc0 = smem_desc_sw128(sW, 16, 1024);
            for (int u = first; ok && u < p.num_units; u += stride, ++acc_it) {
                int mb, nb, half;
                mx4_unit_coords(u, p, mb, nb, half);
                const uint32_t idesc = half < 0 ? Cfg::IDESC : Cfg::IDESC_HALF;
                const uint32_t sfw_col = Cfg::SFW_COL + (half > 0 ? 4u : 0u);
                // The epilogue has read the columns that this tile's accumulator
                // shares with the previous one's (and all of the one before).
                if (acc_it > 0)
                    ok = __all_sync(0xffffffffu,
                                    wait_phase(tempty_bar, (acc_it - 1) & 1u, abort, limit, kSiteMmaTmemEmpty));
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t acc = tmem_base + ((acc_it & 1u) ? Cfg::ACC1_COL : 0);
                for (int kb = 0; kb < KB; ++kb) {
                    ok = __all_sync(0xffffffffu, wait_phase(full_bar(s), ph, abort, limit, kSiteMmaFull) &&
                                                     wait_phase(sready_bar(s), ph, abort, limit, kSiteMmaFull));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t sf = tmem_base + Cfg::SF_COL0 + static_cast<uint32_t>(s * Cfg::SF_SLOT_COLS);
                    const uint64_t a_st = a_desc0 + static_cast<uint64_t>((s * Cfg::A_STAGE_BYTES) >> 4);
                    const uint64_t w_st = w_desc0 + static_cast<uint64_t>((s * Cfg::W_STAGE_BYTES) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < Cfg::BK / Cfg::UMMA_K; ++ks) {
                            const uint64_t step = static_cast<uint64_t>((ks * Cfg::STEP_BYTES) >> 4);
                            const uint32_t id = (ks & 1) * 2;   // bytes 0-1 or 2-3 of the words
                            mma_mxf4<2>(acc, a_st + step, w_st + step, idesc | (id << 4) | (id << 29),
                                        sf + 4u * (ks / 2), sf + sfw_col + 8u * (ks / 2),
                                        (kb != 0 || ks != 0) ? 1u : 0u);
                        }
                        // Operand slot s is free in both CTAs once these MMAs have read it.
                        mma_commit_pair_mc(empty_bar(s), kPairMask);
                        // The tile's accumulator is complete in both CTAs.
                        if (kb == KB - 1) mma_commit_pair_mc(tfull_bar, kPairMask);
                    }
                    __syncwarp();
                    issued_any = true;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok && issued_any) {
                // Wait for this warp's MMAs before the TMEM is freed.
                if (elect_one()) mma_commit_pair_mc(drain_bar, static_cast<uint16_t>(1u << rank));
                __syncwarp();
                wait_phase_drain(drain_bar, 0, limit, kSiteDrainMma, p.status);
            }
        }
        __syncwarp();
    } else if (warp >= 6) {
        // ------------------------------------------------------------ scale warps (6..9)
        const int q = warp & 3;        // TMEM lane quarter this warp may access
        const uint32_t sready0 = leader ? sready_bar(0) : mapa_shared(sready_bar(0), 0);
        const uint32_t row = static_cast<uint32_t>(lane) * 16u;
        const int total = first < p.num_units ? (p.num_units - first + stride - 1) / stride * KB : 0;
        int s = 0;
        uint32_t ph = 0;
        for (int blk = 0; blk < total; ++blk) {
            int ok = 1;
            if (lane == 0) ok = wait_phase(sfull_bar(s), ph, abort, limit, kSiteMmaTmemEmpty) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            // The producer refilled this ring slot after the MMAs that read the
            // scale slot had completed.
            tc_fence_after_sync();
            const uint32_t a = sSFA + static_cast<uint32_t>(s * Cfg::SFA_STAGE_BYTES) + row;
            const uint32_t w = sSFW + static_cast<uint32_t>(s * Cfg::SFW_STAGE_BYTES) + row;
            const uint32_t sf = tmem_base + Cfg::SF_COL0 + static_cast<uint32_t>(s * Cfg::SF_SLOT_COLS) +
                                (static_cast<uint32_t>(q * 32) << 16);
            // Shared memory holds W's tiles as (row block, K tile); in TMEM the
            // eight columns of one K tile are adjacent.
            tmem_store_scales(sf, ld_shared_u32x4(a), ld_shared_u32x4(a + Cfg::SF_TILE));
            tmem_store_scales(sf + Cfg::SFW_COL, ld_shared_u32x4(w), ld_shared_u32x4(w + 2 * Cfg::SF_TILE));
            tmem_store_scales(sf + Cfg::SFW_COL + 8, ld_shared_u32x4(w + Cfg::SF_TILE),
                              ld_shared_u32x4(w + 3 * Cfg::SF_TILE));
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(sready_bar(s));
                else mbar_arrive_cluster(sready0 + 8u * static_cast<uint32_t>(s));
            }
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue (warps 2..5)
        const int ew = warp - 2;       // owner of smem staging buffers
        const int q = warp & 3;        // TMEM lane quarter this warp may access
        const uint32_t row_off = static_cast<uint32_t>(lane) * 128u;
        const uint32_t sw = static_cast<uint32_t>(lane & 7);
        const uint32_t tempty_leader = leader ? tempty_bar : mapa_shared(tempty_bar, 0);
        const uint32_t cbuf0 = sC + static_cast<uint32_t>(ew * 2 * Cfg::C_BUF_BYTES);
        uint32_t acc_it = 0;
        for (int u = first; u < p.num_units; u += stride, ++acc_it) {
            int mb, nb, half;
            mx4_unit_coords(u, p, mb, nb, half);
            int ok = 1;
            if (lane == 0) ok = wait_phase(tfull_bar, acc_it & 1u, abort, limit, kSiteEpilogueTmemFull) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (acc_it == 0) griddep_wait();   // before this warp's first store of C
            tc_fence_after_sync();
            const int row0 = mb * Cfg::TILE_M + static_cast<int>(rank) * Cfg::BM + q * 32;
            const uint32_t odd = acc_it & 1u;
            const uint32_t acc_addr =
                tmem_base + (odd ? Cfg::ACC1_COL : 0) + (static_cast<uint32_t>(q * 32) << 16);
            // The shared columns lie in the last chunks of accumulator 0 and the
            // first of accumulator 1; both are read before anything is packed, so
            // that the next tile's MMAs wait only for the reads (with one chunk
            // packed and stored before the next is read, 1700 cycles per tile).
            // A half tile has the first two chunks only.
            const bool reversed = !odd && half < 0;
            auto chunk = [&](int i) { return reversed ? Cfg::EPI_CHUNKS - 1 - i : i; };
            auto store_chunk = [&](const uint32_t (&r)[64], int i) {
                // The store that used this staging buffer two chunks ago has read it.
                if (lane == 0) bulk_wait_group_read<1>();
                __syncwarp();
                const uint32_t cbuf = cbuf0 + static_cast<uint32_t>((i & 1) * Cfg::C_BUF_BYTES);
                // 16-byte piece jj of a row at piece jj ^ (row % 8): the layout a
                // SWIZZLE_128B tensor-map store expects.
#pragma unroll
                for (int jj = 0; jj < 8; ++jj)
                    st_shared_v4(cbuf + row_off + ((static_cast<uint32_t>(jj) ^ sw) << 4),
                                 pack_f16x2<kRelu>(r[8 * jj + 0], r[8 * jj + 1]),
                                 pack_f16x2<kRelu>(r[8 * jj + 2], r[8 * jj + 3]),
                                 pack_f16x2<kRelu>(r[8 * jj + 4], r[8 * jj + 5]),
                                 pack_f16x2<kRelu>(r[8 * jj + 6], r[8 * jj + 7]));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    const int col0 = nb * Cfg::BN + (half > 0 ? Cfg::BN_CTA : 0) + chunk(i) * Cfg::EPI_COLS;
                    if (row0 < p.M && col0 < p.N) tma_store_2d(&tmap_c, cbuf, col0, row0);
                    bulk_commit_group();
                }
            };
            uint32_t ra[64], rb[64];
            tmem_load_32x32b_x64_async(acc_addr + static_cast<uint32_t>(chunk(0) * Cfg::EPI_COLS), ra);
            tmem_load_32x32b_x64_async(acc_addr + static_cast<uint32_t>(chunk(1) * Cfg::EPI_COLS), rb);
            tmem_wait_ld_x64(ra);
            tmem_wait_ld_x64(rb);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(tempty_bar);
                else mbar_arrive_cluster(tempty_leader);
            }
            store_chunk(ra, 0);
            if (half >= 0) {
                store_chunk(rb, 1);
                continue;
            }
            tmem_load_32x32b_x64_async(acc_addr + static_cast<uint32_t>(chunk(2) * Cfg::EPI_COLS), ra);
            store_chunk(rb, 1);
            tmem_wait_ld_x64(ra);
            tmem_load_32x32b_x64_async(acc_addr + static_cast<uint32_t>(chunk(3) * Cfg::EPI_COLS), rb);
            store_chunk(ra, 2);
            tmem_wait_ld_x64(rb);
            store_chunk(rb, 3);
        }
        if (lane == 0) bulk_wait_group<0>();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && abort.raised()) {
        // Let the loads in flight land before the CTA exits.  Here, where the roles
        // have met, and not in the producer: it may have issued its last load before
        // another role gave up.  Without an abort every load has been waited for.
        const uint32_t issued_mask = issued_ptr[0], issued_parity = issued_ptr[1];
        for (int i = 0; i < S; ++i)
            if (issued_mask & (1u << i))
                wait_phase_drain(sfull_bar(i), (issued_parity >> i) & 1u, limit, kSiteDrainLoads, p.status);
        if (leader) {
            for (int i = 0; i < S; ++i)
                if (issued_mask & (1u << i))
                    wait_phase_drain(full_bar(i), (issued_parity >> i) & 1u, limit, kSiteDrainLoads, p.status);
        } else {
            // This CTA's operand loads complete on the leader's barrier, which it
            // cannot probe: give them a bounded time (~1e6 cycles) to land.
            const long long t0 = clock64();
            while (clock64() - t0 < 1000000) {
            }
        }
    }
    // A warp's lanes meet again for the aligned barrier.
    __syncwarp();
    // Neither CTA exits while the other may still signal its barriers or its
    // MMAs may still use this CTA's shared or tensor memory.
    cluster_arrive();
    cluster_wait();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc<2>(tmem_base, Cfg::TMEM_COLS);
    }
}

// ---------------------------------------------------------------- narrow tiles, K divided over a cluster

// For problems that 256 x 256 tiles leave most SMs idle on: few rows of A (one,
// when tokens are generated one at a time), where the time is that of reading
// W.  The operands change places: 128 rows of W are the MMA's M (TMEM lanes),
// kBN rows of A its N, so a single row of A costs an MMA of N = 16 and not a
// 128-row tile, and the ring holds mostly W.  The K loop of a tile is divided
// over the S = 1, 2, 4 or 8 CTAs of a cluster; each leaves its fp32 partial tile
// in its shared memory, and after a cluster barrier every CTA adds a share of
// the tile over the S partials in rank order (a fixed order: equal calls give
// equal bits) and stores fp16.
//
// Few CTAs each with a short K loop make this a matter of latencies.  Timed by
// clocks written at each step (1 x 4096 x 4096), a K block cost the MMA thread
// some 670 cycles whatever it held, for two barrier waits, the issue of its
// MMAs and a commit; so a ring slot holds 512 elements of K, two swizzle rows
// and eight MMAs (256 elements: 7.9 us with one CTA per tile, 512: 6.4 us).  The
// first loads are issued before the CTA's other set-up, and the cluster's
// first barrier is waited for only when the partial tiles are exchanged.
template <int kBN, int kStages>
struct Mx4NarrowCfg {
    static constexpr int BM = 128;             // rows of W per tile (TMEM lanes)
    static constexpr int BN = kBN;             // rows of A per tile
    static constexpr int BK = 512;             // elements of K per ring slot: two swizzle rows
    static constexpr int HALVES = 2;
    static constexpr int ROW_BYTES = 128;      // of one half
    static constexpr int UMMA_K = 64;
    static constexpr int STEP_BYTES = UMMA_K / 2;
    static constexpr int STEPS = 4;            // MMAs per half
    static constexpr int SF_TILE = 512;
    static constexpr int SF_TILES = BK / 128;
    static constexpr int STAGES = kStages;
    static constexpr int THREADS = 192;
    static constexpr int W_HALF_BYTES = BM * ROW_BYTES;
    static constexpr int X_HALF_BYTES = BN * ROW_BYTES;
    static constexpr int W_STAGE_BYTES = HALVES * W_HALF_BYTES;
    static constexpr int X_STAGE_BYTES = HALVES * X_HALF_BYTES;
    static constexpr int SF_STAGE_BYTES = SF_TILES * SF_TILE;   // of W and of A each
    static constexpr int STAGE_TX_BYTES = W_STAGE_BYTES + X_STAGE_BYTES;
    static constexpr int SF_TX_BYTES = 2 * SF_STAGE_BYTES;
    static constexpr int SF_SLOTS = STAGES;                     // one per ring slot
    static constexpr int SF_SLOT_COLS = 8 * SF_TILES;           // W's words, then A's
    static constexpr int SF_COL0 = BN;
    static constexpr int TMEM_USED = BN + SF_SLOTS * SF_SLOT_COLS;
    static constexpr int TMEM_COLS = TMEM_USED <= 64 ? 64 : (TMEM_USED <= 128 ? 128 : 256);
    static constexpr int PART_BYTES = BM * BN * 4;              // in the ring, once the MMAs are done
    static constexpr int SMEM_W_OFF = 0;
    static constexpr int SMEM_X_OFF = STAGES * W_STAGE_BYTES;
    static constexpr int SMEM_SFW_OFF = SMEM_X_OFF + STAGES * X_STAGE_BYTES;
    static constexpr int SMEM_SFX_OFF = SMEM_SFW_OFF + STAGES * SF_STAGE_BYTES;
    static constexpr int SMEM_CTL_OFF = SMEM_SFX_OFF + STAGES * SF_STAGE_BYTES;
    static constexpr int SMEM_CTL_BYTES = 512;
    static constexpr int SMEM_BYTES = 1024 + SMEM_CTL_OFF + SMEM_CTL_BYTES;
    static constexpr uint32_t IDESC = idesc_mxf4(BM, BN);

    static_assert(SF_TILES == 2 * HALVES && X_HALF_BYTES % 1024 == 0, "tiles of a half; swizzle atoms");
    static_assert(BN % 16 == 0 && BN <= 128, "N of the MMA; scale words of one row block");
    static_assert(PART_BYTES <= STAGES * (W_STAGE_BYTES + X_STAGE_BYTES), "the partial tile fits in the ring");
    static_assert((4 * STAGES + 3) * 8 <= SMEM_CTL_BYTES, "control block");
    static_assert(SMEM_BYTES <= 232448, "shared memory per block on sm_103");
};

struct Mx4NarrowParams {
    int32_t M, N;
    int32_t num_m_tiles;    // ceil(M / BN)
    int32_t num_k_blocks;   // ceil(K / 512)
    int32_t k_per_cta;      // K blocks of each CTA of a cluster
    int32_t withhold;       // test hook, as above
    uint64_t timeout_cycles;
    __half *C;
    unsigned long long *status;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Adds CTA crank's share of the tile over the S partial tiles in rank order.
// Item i: row i / 16 of A and rows 8 (i % 16) .. + 7 of W, consecutive items to
// a CTA.  All S pairs of loads are issued before the first is used, so that
// their round trips through the cluster overlap: with N = K = 4096, 1 row
// 5.1 us against 5.3 and 16 rows 5.5 against 6.0 for one pair after another,
// and no difference beyond 1.5 % at 64 and 128 rows.
template <int S, bool kRelu, int kBN>
__device__ __forceinline__ void mx4_reduce(const Mx4NarrowParams &p, uint32_t part, uint32_t crank, int m0, int n0,
                                           int t)
{
    constexpr int PER_ROW = 128 / 8;
    const int items = min(kBN, p.M - m0) * PER_ROW;
    const int per = (items + S - 1) / S;
    const int i1 = min(items, per * (static_cast<int>(crank) + 1));
    uint32_t src[S];
#pragma unroll
    for (int c = 0; c < S; ++c) src[c] = S == 1 ? part : mapa_shared(part, static_cast<uint32_t>(c));
    for (int i = per * static_cast<int>(crank) + t; i < i1; i += 128) {
        const int j = i / PER_ROW, w8 = i % PER_ROW;
        if (n0 + 8 * w8 >= p.N) continue;   // N is a multiple of 8
        const uint32_t off = static_cast<uint32_t>(j * 512 + w8 * 32);
        float4 lo[S], hi[S];
#pragma unroll
        for (int c = 0; c < S; ++c) {
            lo[c] = ld_cluster_f32x4(src[c] + off);
            hi[c] = ld_cluster_f32x4(src[c] + off + 16u);
        }
#pragma unroll
        for (int c = 1; c < S; ++c) {
            lo[0].x += lo[c].x;
            lo[0].y += lo[c].y;
            lo[0].z += lo[c].z;
            lo[0].w += lo[c].w;
            hi[0].x += hi[c].x;
            hi[0].y += hi[c].y;
            hi[0].z += hi[c].z;
            hi[0].w += hi[c].w;
        }
        st_global_v4(p.C + static_cast<int64_t>(m0 + j) * p.N + n0 + 8 * w8,
                     pack_f16x2<kRelu>(__float_as_uint(lo[0].x), __float_as_uint(lo[0].y)),
                     pack_f16x2<kRelu>(__float_as_uint(lo[0].z), __float_as_uint(lo[0].w)),
                     pack_f16x2<kRelu>(__float_as_uint(hi[0].x), __float_as_uint(hi[0].y)),
                     pack_f16x2<kRelu>(__float_as_uint(hi[0].z), __float_as_uint(hi[0].w)));
    }
}

// Warp 0: TMA producer.  Warp 1: MMAs.  Warps 2..5: scale tiles to TMEM; then
// the partial tile to shared memory and the sum over the cluster.
template <bool kRelu, int kBN, int kStages>
__global__ void __launch_bounds__(192, 1)
    gemm_mxfp4_narrow_sm103a(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                             const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ CUtensorMap tmap_sw,
                             const Mx4NarrowParams p)
{
    using Cfg = Mx4NarrowCfg<kBN, kStages>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);

    const uint32_t sW = base + Cfg::SMEM_W_OFF;
    const uint32_t sX = base + Cfg::SMEM_X_OFF;
    const uint32_t sSFW = base + Cfg::SMEM_SFW_OFF;
    const uint32_t sSFX = base + Cfg::SMEM_SFX_OFF;
    const uint32_t ctl = base + Cfg::SMEM_CTL_OFF;
    constexpr int S = Cfg::STAGES;
    auto full_bar = [&](int s) { return ctl + 8u * s; };
    auto empty_bar = [&](int s) { return ctl + 8u * (S + s); };
    auto sfull_bar = [&](int s) { return ctl + 8u * (2 * S + s); };
    auto sready_bar = [&](int s) { return ctl + 8u * (3 * S + s); };
    const uint32_t tfull_bar = ctl + 8u * (4 * S);
    const uint32_t tmem_slot = ctl + 8u * (4 * S + 1);
    volatile uint32_t *tmem_slot_ptr =
        reinterpret_cast<volatile uint32_t *>(base_ptr + Cfg::SMEM_CTL_OFF + 8 * (4 * S + 1));

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // uniform
    const int lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    const uint32_t ncl = cluster_nctarank();

    AbortFlag abort;
    abort.local = reinterpret_cast<volatile int *>(tmem_slot_ptr + 1);
    abort.status = p.status;
    abort.addr = tmem_slot + 4;
    abort.cluster = ncl;
    abort.rank = crank;

    if (warp == 0) {
        // One thread per ring slot: 4 S initialisations one after another would
        // hold back the first load by some 400 cycles.
        if (lane < S) {
            mbar_init(full_bar(lane), 1);
            mbar_init(empty_bar(lane), 1);
            mbar_init(sfull_bar(lane), 1);
            mbar_init(sready_bar(lane), 4);   // one arrive per scale warp
        }
        if (lane == 31) {
            mbar_init(tfull_bar, 1);
            *abort.local = 0;
        }
        fence_mbar_init();
        __syncwarp();
    }
    const uint64_t limit = p.timeout_cycles;
    const int unit = static_cast<int>(blockIdx.x / ncl);
    const int mt = unit % p.num_m_tiles, wb = unit / p.num_m_tiles;   // neighbours share W's rows
    const int m0 = mt * Cfg::BN, n0 = wb * Cfg::BM;
    const int kb0 = static_cast<int>(crank) * p.k_per_cta;
    const int kb1 = min(p.num_k_blocks, kb0 + p.k_per_cta);   // the launch leaves no CTA without K blocks

    auto load = [&](int kb, int s) {
        mbar_arrive_expect_tx(full_bar(s), Cfg::STAGE_TX_BYTES);
#pragma unroll
        for (int h = 0; h < Cfg::HALVES; ++h) {
            const int x = (kb * Cfg::HALVES + h) * Cfg::ROW_BYTES;   // past K: zeros
            tma_load_2d(sW + s * Cfg::W_STAGE_BYTES + h * Cfg::W_HALF_BYTES, &tmap_w, full_bar(s), x, n0);
            tma_load_2d(sX + s * Cfg::X_STAGE_BYTES + h * Cfg::X_HALF_BYTES, &tmap_a, full_bar(s), x, m0);
        }
        if (p.withhold != 0) return;
        mbar_arrive_expect_tx(sfull_bar(s), Cfg::SF_TX_BYTES);
        tma_load_3d_cta(sSFW + s * Cfg::SF_STAGE_BYTES, &tmap_sw, sfull_bar(s), 0, kb * Cfg::SF_TILES, wb);
        tma_load_3d_cta(sSFX + s * Cfg::SF_STAGE_BYTES, &tmap_sa, sfull_bar(s), 0, kb * Cfg::SF_TILES, m0 / 128);
    };
    // The thread that initialised the barriers fills the ring before it joins
    // the others, whose set-up runs while the first loads are on their way.
    const int filled = p.withhold != 1 ? min(S, kb1 - kb0) : 0;
    // The producer's ring slots in use, and the parity of their last load.
    volatile uint32_t *issued_ptr = tmem_slot_ptr + 2;
    if (threadIdx.x == 0) {
        griddep_wait();   // A, W and the scales may come from the kernel just before
        for (int s = 0; s < filled; ++s) load(kb0 + s, s);
    }
    if (warp == 1) {
        tmem_alloc<1>(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish<1>();
    }
    tc_fence_before_sync();
    __syncthreads();
    // Waited for only when the partial tiles are exchanged: until then no CTA
    // touches another, but for abort flags raised a second or more from now.
    if (ncl > 1) cluster_arrive();
    tc_fence_after_sync();
    griddep_launch_dependents();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot_ptr, 0);

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t issued_mask = (1u << filled) - 1u;
            uint32_t issued_parity = 0;
            int s = 0;
            uint32_t ph = 1;
            for (int kb = kb0 + filled; kb < kb1 && p.withhold != 1; ++kb) {
                if (!wait_phase(empty_bar(s), ph ^ 1u, abort, limit, kSiteProducerEmpty)) break;
                load(kb, s);
                issued_parity = (issued_parity & ~(1u << s)) | (ph << s);
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            issued_ptr[0] = issued_mask;
            issued_ptr[1] = issued_parity;
        }
        __syncwarp();
    } else if (warp == 1) {
        // The whole warp walks the loop, one lane issues (see the pair kernel).
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        const uint64_t w_desc0 = smem_desc_sw128(sW, 16, 1024);
        const uint64_t x_desc0 = smem_desc_sw128(sX, 16, 1024);
        // Row m0 of A is at word column (m0 % 128) / 32 of its scale tiles.
        const uint32_t sfx_word = static_cast<uint32_t>((m0 % 128) / 32);
        for (int kb = kb0; kb < kb1; ++kb) {
            ok = __all_sync(0xffffffffu, wait_phase(full_bar(s), ph, abort, limit, kSiteMmaFull) &&
                                             wait_phase(sready_bar(s), ph, abort, limit, kSiteMmaFull));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t sf = tmem_base + Cfg::SF_COL0 + static_cast<uint32_t>(s * Cfg::SF_SLOT_COLS);
            const uint64_t w_st = w_desc0 + static_cast<uint64_t>((s * Cfg::W_STAGE_BYTES) >> 4);
            const uint64_t x_st = x_desc0 + static_cast<uint64_t>((s * Cfg::X_STAGE_BYTES) >> 4);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < Cfg::HALVES * Cfg::STEPS; ++ks) {
                    const int half = ks / Cfg::STEPS, step = (ks % Cfg::STEPS) * Cfg::STEP_BYTES;
                    const uint32_t id = (ks & 1) * 2;
                    mma_mxf4<1>(tmem_base, w_st + static_cast<uint64_t>((half * Cfg::W_HALF_BYTES + step) >> 4),
                                x_st + static_cast<uint64_t>((half * Cfg::X_HALF_BYTES + step) >> 4),
                                Cfg::IDESC | (id << 4) | (id << 29), sf + 4u * (ks / 2),
                                sf + 4u * (Cfg::SF_TILES + ks / 2) + sfx_word, (kb != kb0 || ks != 0) ? 1u : 0u);
                }
                mma_commit(empty_bar(s));
            }
            __syncwarp();
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
        }
        // Also after an abort: the wait below frees the TMEM only once this warp's
        // MMAs are done.
        if (elect_one()) mma_commit(tfull_bar);
        __syncwarp();
        if (!ok) wait_phase_drain(tfull_bar, 0, limit, kSiteDrainMma, p.status);
        __syncwarp();
    } else {
        const int q = warp & 3;
        const int rows = min(Cfg::BN, p.M - m0);   // rows of A in this tile
        int ok = 1;
        // Scale tiles from shared memory to TMEM, as long as there are K blocks.
        {
            const uint32_t row = static_cast<uint32_t>(lane) * 16u;
            int s = 0;
            uint32_t ph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (lane == 0) ok = wait_phase(sfull_bar(s), ph, abort, limit, kSiteMmaTmemEmpty) ? 1 : 0;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t w = sSFW + static_cast<uint32_t>(s * Cfg::SF_STAGE_BYTES) + row;
                const uint32_t x = sSFX + static_cast<uint32_t>(s * Cfg::SF_STAGE_BYTES) + row;
                const uint32_t sf = tmem_base + Cfg::SF_COL0 + static_cast<uint32_t>(s * Cfg::SF_SLOT_COLS) +
                                    (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
                for (int h = 0; h < Cfg::HALVES; ++h) {
                    const uint32_t o = static_cast<uint32_t>(2 * h * Cfg::SF_TILE);
                    tmem_store_scales(sf + 8u * h, ld_shared_u32x4(w + o), ld_shared_u32x4(w + o + Cfg::SF_TILE));
                    tmem_store_scales(sf + 8u * (Cfg::HALVES + h), ld_shared_u32x4(x + o),
                                      ld_shared_u32x4(x + o + Cfg::SF_TILE));
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(sready_bar(s));
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (ok && lane == 0) ok = wait_phase(tfull_bar, 0, abort, limit, kSiteEpilogueTmemFull) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok) {
            tc_fence_after_sync();
            // Partial tile: value (row j of A, row w of W) at float j * 128 + w.
            const uint32_t part = sW + static_cast<uint32_t>(q * 32 + lane) * 4u;
            const uint32_t acc = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int j0 = 0; j0 < rows; j0 += 16) {
                uint32_t r[16];
                tmem_load_32x32b_x16(acc + static_cast<uint32_t>(j0), r);
#pragma unroll
                for (int j = 0; j < 16; ++j) st_shared_u32(part + static_cast<uint32_t>(j0 + j) * 512u, r[j]);
            }
        }
    }

    // Every partial tile of the cluster is written.
    tc_fence_before_sync();
    __syncwarp();
    if (ncl > 1) {
        cluster_wait();   // of the arrival after the set-up
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp >= 2 && !abort.raised()) {
        griddep_wait();   // before this thread's first store of C
        const int t = static_cast<int>(threadIdx.x) - 64;
        switch (ncl) {
        case 1: mx4_reduce<1, kRelu, Cfg::BN>(p, sW, crank, m0, n0, t); break;
        case 2: mx4_reduce<2, kRelu, Cfg::BN>(p, sW, crank, m0, n0, t); break;
        case 4: mx4_reduce<4, kRelu, Cfg::BN>(p, sW, crank, m0, n0, t); break;
        default: mx4_reduce<8, kRelu, Cfg::BN>(p, sW, crank, m0, n0, t); break;
        }
    }
    if (threadIdx.x == 0 && abort.raised()) {
        // Let the loads in flight land before the CTA exits (see the pair kernel).
        const uint32_t issued_mask = issued_ptr[0], issued_parity = issued_ptr[1];
        for (int i = 0; i < S; ++i)
            if (issued_mask & (1u << i)) {
                wait_phase_drain(full_bar(i), (issued_parity >> i) & 1u, limit, kSiteDrainLoads, p.status);
                wait_phase_drain(sfull_bar(i), (issued_parity >> i) & 1u, limit, kSiteDrainLoads, p.status);
            }
    }
    __syncwarp();
    if (ncl > 1) {
        // No CTA exits while another may still read its shared memory.
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace gemm_sm103
