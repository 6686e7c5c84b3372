// gemm_mxfp4.cu -- host-side launch of the 4-bit microscaled GEMM
// (gemm_mxfp4_kernel.cuh).  The C ABI entry, gemm_mxfp4 in gemm_f16.cu,
// validates every argument and calls launch_mxfp4.
#include "gemm_mxfp4_launch.cuh"

#include "gemm_mxfp4_kernel.cuh"

namespace gemm_sm103 {

namespace {

// Per device and ReLU variant: the shared-memory attribute is set once and
// the number of co-resident CTA pairs cached (one CTA per SM).
template <bool kRelu>
struct Mx4Prepared {
    static std::atomic<int> slots[kMaxDevices];

    static int get(int dev, int sm_count)
    {
        int v = slots[dev].load(std::memory_order_acquire);
        if (v > 0) return v;
        auto kern = gemm_mxfp4_sm103a<kRelu>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Mx4Cfg::SMEM_BYTES) !=
            cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        v = sm_count / 2;
        cudaLaunchConfig_t lc{};
        lc.blockDim = dim3(Mx4Cfg::THREADS, 1, 1);
        lc.dynamicSmemBytes = Mx4Cfg::SMEM_BYTES;
        lc.gridDim = dim3(2 * v, 1, 1);
        cudaLaunchAttribute attrs[1];
        attrs[0].id = cudaLaunchAttributeClusterDimension;
        attrs[0].val.clusterDim.x = 2;
        attrs[0].val.clusterDim.y = 1;
        attrs[0].val.clusterDim.z = 1;
        lc.attrs = attrs;
        lc.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kern, &lc) == cudaSuccess && clusters > 0)
            v = clusters < v ? clusters : v;
        else
            cudaGetLastError();
        if (v > 0) slots[dev].store(v, std::memory_order_release);
        return v;
    }

    static void forget(int dev) { slots[dev].store(0, std::memory_order_release); }
};

template <bool kRelu>
std::atomic<int> Mx4Prepared<kRelu>::slots[kMaxDevices];

template <bool kRelu>
int launch_pairs(const Mx4LaunchArgs &a)
{
    using Cfg = Mx4Cfg;
    CUtensorMap ta, tw, tw_half, tsa, tsw, tc;
    int st;
    if ((st = encode_codes_u4(&ta, a.A, a.M, a.K, Cfg::BM)) != GEMM_OK) return st;
    if ((st = encode_codes_u4(&tw, a.W, a.N, a.K, Cfg::BN_CTA)) != GEMM_OK) return st;
    if ((st = encode_codes_u4(&tw_half, a.W, a.N, a.K, Cfg::BN_CTA / 2)) != GEMM_OK) return st;
    if ((st = encode_scale_tiles(&tsa, a.SA, a.M, a.K, Cfg::SF_TILES, 1)) != GEMM_OK) return st;
    if ((st = encode_scale_tiles(&tsw, a.SW, a.N, a.K, Cfg::SF_TILES, 2)) != GEMM_OK) return st;
    if ((st = encode_matrix(&tc, a.C, a.M, a.N, Cfg::EPI_COLS, 32)) != GEMM_OK) return st;

    Mx4Params p{};
    p.M = static_cast<int32_t>(a.M);
    p.N = static_cast<int32_t>(a.N);
    p.num_m_blocks = static_cast<int32_t>((a.M + Cfg::TILE_M - 1) / Cfg::TILE_M);
    p.num_n_blocks = static_cast<int32_t>((a.N + Cfg::BN - 1) / Cfg::BN);
    p.num_k_blocks = static_cast<int32_t>((a.K + Cfg::BK - 1) / Cfg::BK);
    const int64_t tiles = static_cast<int64_t>(p.num_m_blocks) * p.num_n_blocks;
    if (tiles > INT32_MAX - 1024) return GEMM_ERR_INVALID_ARG;
    // 2048-row panels, as the fp16 kernels.  Panels of 16 tiles gain 0.7 % at 8192^3
    // (152.0 against 153.1 us) and lose 2-5 % on smaller outputs (4096 x 8192 x
    // 1024: 19.4 against 18.4 us).
    p.group_m = 8;
    p.withhold = a.withhold;
    p.timeout_cycles = a.timeout_cycles ? a.timeout_cycles : timeout_cycles_for(a.K);
    p.status = a.status;

    using Prep = Mx4Prepared<kRelu>;
    const int64_t slots = Prep::get(a.dev.device, a.dev.sm_count);
    if (slots <= 0) return GEMM_ERR_LAUNCH;
    // Half tiles for a last wave that leaves half of the pairs idle (4096^3, the
    // last 28 of 256 tiles on 76 pairs: 27.0 us whole, 26.0 us halved; 8192^3, the
    // last 36 of 1024: 154.2 us, 151.7 us).
    const int64_t rest = tiles % slots;
    const int64_t split = tiles > slots && 2 * rest <= slots ? rest : 0;
    p.split_start = static_cast<int32_t>(tiles - split);
    p.num_units = static_cast<int32_t>(tiles + split);
    const int64_t clusters = tiles < slots ? tiles : slots;
    auto kern = gemm_mxfp4_sm103a<kRelu>;
    cudaLaunchConfig_t lc{};
    lc.blockDim = dim3(Cfg::THREADS, 1, 1);
    lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
    lc.stream = a.stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = 2;
    attrs[0].val.clusterDim.y = 1;
    attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // programmatic dependent launch
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attrs;
    lc.numAttrs = 2;
    lc.gridDim = dim3(static_cast<unsigned>(2 * clusters), 1, 1);
    if (cudaLaunchKernelEx(&lc, kern, ta, tw, tw_half, tsa, tsw, tc, p) != cudaSuccess) {
        cudaGetLastError();
        Prep::forget(a.dev.device);
        if (Prep::get(a.dev.device, a.dev.sm_count) <= 0 ||
            cudaLaunchKernelEx(&lc, kern, ta, tw, tw_half, tsa, tsw, tc, p) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
    }
    return GEMM_OK;
}

template <bool kRelu, int kBN, int kStages>
int launch_narrow(const Mx4LaunchArgs &a, int splits)
{
    using Cfg = Mx4NarrowCfg<kBN, kStages>;
    CUtensorMap ta, tw, tsa, tsw;
    int st;
    if ((st = encode_codes_u4(&ta, a.A, a.M, a.K, Cfg::BN)) != GEMM_OK) return st;
    if ((st = encode_codes_u4(&tw, a.W, a.N, a.K, Cfg::BM)) != GEMM_OK) return st;
    if ((st = encode_scale_tiles(&tsa, a.SA, a.M, a.K, Cfg::SF_TILES, 1)) != GEMM_OK) return st;
    if ((st = encode_scale_tiles(&tsw, a.SW, a.N, a.K, Cfg::SF_TILES, 1)) != GEMM_OK) return st;

    Mx4NarrowParams p{};
    p.M = static_cast<int32_t>(a.M);
    p.N = static_cast<int32_t>(a.N);
    p.num_m_tiles = static_cast<int32_t>((a.M + Cfg::BN - 1) / Cfg::BN);
    p.num_k_blocks = static_cast<int32_t>((a.K + Cfg::BK - 1) / Cfg::BK);
    p.k_per_cta = (p.num_k_blocks + splits - 1) / splits;
    p.withhold = a.withhold;
    p.timeout_cycles = a.timeout_cycles ? a.timeout_cycles : timeout_cycles_for(a.K);
    p.C = static_cast<__half *>(a.C);
    p.status = a.status;
    const int64_t ctas = static_cast<int64_t>(p.num_m_tiles) * ((a.N + Cfg::BM - 1) / Cfg::BM) * splits;
    if (ctas > INT32_MAX) return GEMM_ERR_INVALID_ARG;

    // Per device: the shared-memory attribute is set once.
    static std::atomic<int> prepared[kMaxDevices];
    auto kern = gemm_mxfp4_narrow_sm103a<kRelu, kBN, kStages>;
    for (int attempt = 0;; ++attempt) {
        if (!prepared[a.dev.device].load(std::memory_order_acquire)) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) !=
                cudaSuccess) {
                cudaGetLastError();
                return GEMM_ERR_LAUNCH;
            }
            prepared[a.dev.device].store(1, std::memory_order_release);
        }
        cudaLaunchConfig_t lc{};
        lc.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
        lc.blockDim = dim3(Cfg::THREADS, 1, 1);
        lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
        lc.stream = a.stream;
        cudaLaunchAttribute attrs[2];
        attrs[0].id = cudaLaunchAttributeClusterDimension;
        attrs[0].val.clusterDim.x = static_cast<unsigned>(splits);
        attrs[0].val.clusterDim.y = 1;
        attrs[0].val.clusterDim.z = 1;
        attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[1].val.programmaticStreamSerializationAllowed = 1;
        lc.attrs = attrs;
        lc.numAttrs = 2;
        if (cudaLaunchKernelEx(&lc, kern, ta, tw, tsa, tsw, p) == cudaSuccess) return GEMM_OK;
        cudaGetLastError();
        prepared[a.dev.device].store(0, std::memory_order_release);
        if (attempt > 0) return GEMM_ERR_LAUNCH;
    }
}

// CTAs of a cluster that divide a tile's K loop, for `tiles` tiles of k_blocks
// ring slots each: doubled while every CTA still has an SM to itself and at
// least min_blocks ring slots of K.  A second wave of clusters costs as much as
// the first (1 x 8192 x 8192: 2 CTAs per tile 9.7 us, 4 CTAs 13.9 us), and
// clusters of 8 do not pack a GPC's SMs, so those are held to half of them
// (1 x 2048 x 8192, 16 tiles: 4 CTAs 6.0 us, 8 CTAs 9.2 us).
int narrow_splits(int64_t tiles, int64_t k_blocks, int64_t min_blocks, int sm_count)
{
    int s = 1;
    while (s < 8 && tiles * 2 * s <= (s == 4 ? sm_count / 2 : sm_count) && k_blocks >= 2 * s * min_blocks) s *= 2;
    // No CTA without K blocks: ceil(k_blocks / s) each.
    while (s > 1 && (k_blocks + s - 1) / s * (s - 1) >= k_blocks) s /= 2;
    return s;
}

// The choice between the two kernels and their tiles.  A narrow tile's time
// hardly depends on its width (4096 x 4096 weight, 64 rows of A: 7.2 us with one
// CTA per tile, 512 rows in 128-row tiles 9.5 us), so the narrowest that holds
// M, or that leaves every tile an SM, is taken; with more tiles than SMs the
// 256 x 256 pair tiles win (768 x 4096 x 4096: 11.4 us, 192 narrow tiles 18 us; 512 x
// 4096 x 4096: 11.2 us, 128 narrow tiles 9.5 us), unless A has so few rows that
// W's bytes are the time (1 x 131072 x 4096: 54 us against 86 us; 64 x 24576 x 4096:
// 16.6 against 19.8 us, 64 x 65536 x 2048: 24.8 against 22.9 us).  Dividing K pays where the
// partial tiles are small (16 rows: 6.4 -> 5.3 us at 4096 x 4096, two ring slots
// per CTA); for 64 rows the exchange costs what it saves until K is long.
template <bool kRelu>
int launch_variant(const Mx4LaunchArgs &a)
{
    const int64_t w_tiles = (a.N + 127) / 128, k_blocks = (a.K + 511) / 512;
    const int64_t sms = a.dev.sm_count;
    auto tiles = [&](int bn) { return w_tiles * ((a.M + bn - 1) / bn); };
    auto splits = [&](int bn) { return narrow_splits(tiles(bn), k_blocks, bn <= 32 ? 2 : 8, a.dev.sm_count); };
    if (a.M <= 16) return launch_narrow<kRelu, 16, 5>(a, splits(16));
    if (a.M <= 32) return launch_narrow<kRelu, 32, 5>(a, splits(32));
    if (tiles(64) <= (a.M <= 64 ? 2 * sms : sms)) return launch_narrow<kRelu, 64, 4>(a, splits(64));
    if (tiles(128) <= sms) return launch_narrow<kRelu, 128, 3>(a, splits(128));
    return launch_pairs<kRelu>(a);
}

}  // namespace

int launch_mxfp4(const Mx4LaunchArgs &a)
{
    return a.relu ? launch_variant<true>(a) : launch_variant<false>(a);
}

}  // namespace gemm_sm103
