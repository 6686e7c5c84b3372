// gemm_f16.cu -- host side of the GB300 fp16 GEMM + ReLU library: argument
// checks, TMA tensor-map encoding, configuration choice, the device status
// word, and the extern "C" entry points declared in include/gemm_f16.h.  The
// kernel instances themselves are launched from gemm_cfg_<id>.cu.
//
// Nothing here computes the product on the host; every element of C is
// written by the sm_103a kernel in gemm_kernel.cuh (or, for K == 0, by one
// cudaMemsetAsync of +0, the value of the empty sum).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "gemm_f16.h"
#include "attention_launch.cuh"
#include "feed_forward_launch.cuh"
#include "gemm_fp8_launch.cuh"
#include "gemm_launch.cuh"
#include "gemm_mxfp4_launch.cuh"
#include "layer_norm.cuh"
#include "rms_norm.cuh"

using namespace gemm_sm103;

// Device status word of each GPU: 0 = fine; otherwise the first timeout record
// written by a kernel (wait site | block << 8).  Kernels get its address.
__device__ unsigned long long g_gemm_f16_status;

namespace {

// Reason for the last rejected call on this thread (static strings only).
thread_local const char *t_last_detail = "";

constexpr int kMaxFromHostPanels = 8;   // row panels of gemm_f16_from_host

int reject(int status, const char *why)
{
    t_last_detail = why;
    return status;
}

// ---------------------------------------------------------------- configurations

struct ConfigInfo {
    const char *name;
    int tile_m;       // rows of C per work unit (all CTAs of the unit together)
    int tile_n;       // columns of C per work unit
    int all_layouts;  // 1: NN, NT, TN and TT operand layouts; 0: NN only
};

// id 1..kNumConfigs; index 0 is "auto".
constexpr ConfigInfo kConfigs[] = {
    {"auto", 0, 0, 1},
    {"1sm_128x256_s4", Cfg1x256::SUPER_M, Cfg1x256::BN, 1},
    {"1sm_128x128_s6", Cfg1x128::SUPER_M, Cfg1x128::BN, 1},
    {"2sm_256x256_s6", Cfg2x256::SUPER_M, Cfg2x256::BN, 1},
    {"2sm_256x256_s7_direct", Cfg2x256d::SUPER_M, Cfg2x256d::BN, 0},
    {"2sm_256x512_s4", Cfg2x512::SUPER_M, Cfg2x512::BN, 1},
    {"1sm_128x128_ck_s6", Cfg1x128ck::SUPER_M, Cfg1x128ck::BN, 0},
};
// The configuration whose K split runs across a cluster (no workspace).
constexpr int kClusterKConfig = 6;
constexpr int kNumConfigs = static_cast<int>(sizeof(kConfigs) / sizeof(kConfigs[0])) - 1;

// ---------------------------------------------------------------- driver entry points

struct DriverFns {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    PFN_cuMemGetAddressRange_v3020 range = nullptr;
    PFN_cuPointerGetAttributes_v7000 attributes = nullptr;   // may be missing
    bool ok = false;
};

const DriverFns &driver()
{
    static DriverFns fns;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q1 = cudaDriverEntryPointSymbolNotFound;
        cudaDriverEntryPointQueryResult q2 = cudaDriverEntryPointSymbolNotFound;
        void *f1 = nullptr, *f2 = nullptr;
        cudaError_t e1 = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f1, 12000, cudaEnableDefault, &q1);
        cudaError_t e2 = cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &f2, 3020, cudaEnableDefault, &q2);
        if (e1 == cudaSuccess && q1 == cudaDriverEntryPointSuccess && f1 && e2 == cudaSuccess &&
            q2 == cudaDriverEntryPointSuccess && f2) {
            fns.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f1);
            fns.range = reinterpret_cast<PFN_cuMemGetAddressRange_v3020>(f2);
            fns.ok = true;
        }
        cudaDriverEntryPointQueryResult q3 = cudaDriverEntryPointSymbolNotFound;
        void *f3 = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &f3, 7000, cudaEnableDefault, &q3) ==
                cudaSuccess &&
            q3 == cudaDriverEntryPointSuccess)
            fns.attributes = reinterpret_cast<PFN_cuPointerGetAttributes_v7000>(f3);
        else
            cudaGetLastError();
    });
    return fns;
}

// ---------------------------------------------------------------- per-device facts

// Filled once per device; read without locking afterwards.
std::atomic<int> g_device_state[kMaxDevices];   // 0 unknown, 1 supported, 2 unsupported
int g_device_sms[kMaxDevices];
std::atomic<unsigned long long *> g_status_addr[kMaxDevices];

int current_device_info(DeviceInfo *out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED_DEVICE;
    // Driver-level calls (cuMemGetAddressRange) need the device's primary
    // context current on this thread; a thread whose first CUDA work is this
    // call (e.g. the autograd engine's backward thread) has none yet.
    // cudaSetDevice initialises the primary context and makes it current.
    thread_local int t_bound_device = -1;
    if (t_bound_device != dev) {
        if (cudaSetDevice(dev) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        t_bound_device = dev;
    }
    int state = g_device_state[dev].load(std::memory_order_acquire);
    if (state == 0) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        g_device_sms[dev] = sms;
        state = (major == 10 && minor == 3) ? 1 : 2;
        g_device_state[dev].store(state, std::memory_order_release);
    }
    out->device = dev;
    out->sm_count = g_device_sms[dev];
    out->supported = state == 1;
    return state == 1 ? GEMM_OK : GEMM_ERR_UNSUPPORTED_DEVICE;
}

// Device address of this GPU's status word (cached per device).
unsigned long long *status_word(int dev)
{
    unsigned long long *p = g_status_addr[dev].load(std::memory_order_acquire);
    if (p) return p;
    void *q = nullptr;
    if (cudaGetSymbolAddress(&q, g_gemm_f16_status) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    p = static_cast<unsigned long long *>(q);
    g_status_addr[dev].store(p, std::memory_order_release);
    return p;
}

// ---------------------------------------------------------------- argument checks

// A device buffer of `bytes` bytes starting at p: device (or managed) memory of
// device `dev`, entirely inside one allocation.
int check_device_buffer(const void *p, uint64_t bytes, int dev, uintptr_t align = 16)
{
    if (p == nullptr) return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    if ((reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0)
        return reject(GEMM_ERR_ALIGNMENT, "a buffer pointer is not aligned (16 bytes for GEMM operands)");
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return reject(GEMM_ERR_INVALID_ARG, "cudaPointerGetAttributes failed on a buffer pointer");
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
        return reject(GEMM_ERR_INVALID_ARG, "a buffer is not device or managed memory");
    if (attr.type == cudaMemoryTypeDevice && attr.device != dev)
        return reject(GEMM_ERR_INVALID_ARG, "a buffer lives on another device than the current one");
    const DriverFns &fns = driver();
    if (!fns.ok) return reject(GEMM_ERR_CUDA, "driver entry points unavailable");
    CUdeviceptr base = 0;
    size_t size = 0;
    if (fns.range(&base, &size, reinterpret_cast<CUdeviceptr>(p)) != CUDA_SUCCESS)
        return reject(GEMM_ERR_INVALID_ARG, "cuMemGetAddressRange does not know a buffer pointer");
    const uint64_t off = static_cast<uint64_t>(reinterpret_cast<CUdeviceptr>(p) - base);
    if (off > size || bytes > size - off)
        return reject(GEMM_ERR_INVALID_ARG, "a buffer is smaller than its matrix (runs past its allocation)");
    return GEMM_OK;
}

// check_device_buffer with one driver call instead of two runtime and driver
// calls: what it cannot vouch for goes to check_device_buffer, which accepts
// or names the reason.
int check_device_buffer_fast(const void *p, uint64_t bytes, int dev, uintptr_t align = 16)
{
    const DriverFns &fns = driver();
    if (fns.attributes != nullptr && p != nullptr && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0) {
        unsigned int type = 0;
        int ordinal = -1;
        CUdeviceptr base = 0;
        size_t size = 0;
        CUpointer_attribute what[4] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL,
                                       CU_POINTER_ATTRIBUTE_RANGE_START_ADDR, CU_POINTER_ATTRIBUTE_RANGE_SIZE};
        void *out[4] = {&type, &ordinal, &base, &size};
        if (fns.attributes(4, what, out, reinterpret_cast<CUdeviceptr>(p)) == CUDA_SUCCESS &&
            type == CU_MEMORYTYPE_DEVICE && ordinal == dev && base != 0) {
            const uint64_t off = static_cast<uint64_t>(reinterpret_cast<CUdeviceptr>(p) - base);
            if (off <= size && bytes <= size - off) return GEMM_OK;
        }
    }
    return check_device_buffer(p, bytes, dev, align);
}

bool ranges_overlap(const void *a, uint64_t abytes, const void *b, uint64_t bbytes)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bbytes && b0 < a0 + abytes;
}

int check_sizes(int64_t M, int64_t N, int64_t K, int relu)
{
    if (M < 0 || N < 0 || K < 0) return reject(GEMM_ERR_INVALID_ARG, "a size is negative");
    if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return reject(GEMM_ERR_INVALID_ARG, "a size exceeds INT32_MAX");
    if (relu != 0 && relu != 1) return reject(GEMM_ERR_INVALID_ARG, "relu is not 0 or 1");
    return GEMM_OK;
}

}  // namespace

namespace gemm_sm103 {

// Row-major fp16 matrix rows x cols (leading dimension cols), boxes of
// box_cols x box_rows with 128-byte swizzle; out-of-range loads read zero.
int encode_matrix(CUtensorMap *map, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_cols,
                  uint32_t box_rows)
{
    const DriverFns &fns = driver();
    if (!fns.ok) return GEMM_ERR_CUDA;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fns.encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(ptr), dims, strides, box,
                            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_CUDA;
}

// Row-major one-byte-element matrix (E4M3 codes) rows x cols, leading
// dimension cols bytes, boxes of box_cols x box_rows with 128-byte swizzle.
int encode_matrix_u8(CUtensorMap *map, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_cols,
                     uint32_t box_rows)
{
    const DriverFns &fns = driver();
    if (!fns.ok) return GEMM_ERR_CUDA;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fns.encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_CUDA;
}

int encode_codes_u4(CUtensorMap *map, const void *ptr, int64_t rows, int64_t K, uint32_t box_rows)
{
    const DriverFns &fns = driver();
    if (!fns.ok) return GEMM_ERR_CUDA;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>((K + 1) / 2), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(mx4_row_bytes(K))};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fns.encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_CUDA;
}

int encode_scale_tiles(CUtensorMap *map, const void *ptr, int64_t rows, int64_t K, uint32_t box_k, uint32_t box_rows)
{
    const DriverFns &fns = driver();
    if (!fns.ok) return GEMM_ERR_CUDA;
    const cuuint64_t kt = static_cast<cuuint64_t>(mx4_k_tiles(K));
    cuuint64_t dims[3] = {kMx4TileBytes / 4, kt, static_cast<cuuint64_t>(mx4_row_tiles(rows))};
    cuuint64_t strides[2] = {kMx4TileBytes, kt * kMx4TileBytes};
    cuuint32_t box[3] = {kMx4TileBytes / 4, box_k, box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fns.encode(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_CUDA;
}

// (batch * heads, seq, dim) fp16 tensor, dims innermost first: dim, seq,
// batch * heads; boxes of 64 x 128 x 1 with 128-byte swizzle.  A box never
// crosses into another head's rows: rows past seq read as zero.
int encode_bhsd(CUtensorMap *map, const void *ptr, uint64_t bh, uint64_t seq, uint64_t dim)
{
    const DriverFns &fns = driver();
    if (!fns.ok) return GEMM_ERR_CUDA;
    cuuint64_t dims[3] = {dim, seq, bh};
    cuuint64_t strides[2] = {dim * 2, seq * dim * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fns.encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(ptr), dims, strides, box,
                            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_CUDA;
}

// Optional rasterisation panel height (in work units) for tuning sweeps.
int group_m_override()
{
    static int v = [] {
        const char *e = std::getenv("GEMM_F16_GROUP_M");
        const int x = e ? std::atoi(e) : 0;
        return x > 0 && x <= 4096 ? x : 0;
    }();
    return v;
}

}  // namespace gemm_sm103

namespace {

// ---------------------------------------------------------------- configuration choice

int pick_config(int64_t M, int64_t N, int64_t K, int sm_count)
{
    const int64_t pairs = sm_count / 2;
    const int64_t tiles_256x512 = ((M + 255) / 256) * ((N + 511) / 512);
    // At least one full wave of 256x512 pair tiles and a long K loop: the wide
    // tile needs the fewest operand bytes per flop.  Its tail is left whole:
    // a split tail runs 256-column MMAs on half the operand reuse.
    if (tiles_256x512 >= pairs && K >= 2048) return 5 | GEMM_F16_NO_SPLIT;
    const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256);
    // Enough 256x256 tiles to keep every SM pair busy: the CTA-pair kernel.
    if (pair_tiles >= pairs) return 3;
    const int64_t tiles256 = ((M + 127) / 128) * ((N + 255) / 256);
    if (tiles256 >= sm_count / 2) return 1;
    // Few tiles: narrower tiles put more SMs to work.
    return 2;
}

// ---------------------------------------------------------------- tuned selection

#if __has_include("gemm_f16_tuned.inc")
#include "gemm_f16_tuned.inc"
#define GEMM_F16_HAVE_TUNED 1
#else
#define GEMM_F16_HAVE_TUNED 0
#endif

int config_info(int cfg, int64_t M, int64_t N, bool split, const DeviceInfo &dev, int *grid_ctas, int *cluster_size,
                int *tiles)
{
    switch (cfg) {
        case 1: return launch_info_config_1(M, N, split, dev, grid_ctas, cluster_size, tiles);
        case 2: return launch_info_config_2(M, N, split, dev, grid_ctas, cluster_size, tiles);
        case 3: return launch_info_config_3(M, N, split, dev, grid_ctas, cluster_size, tiles);
        case 4: return launch_info_config_4(M, N, split, dev, grid_ctas, cluster_size, tiles);
        case 5: return launch_info_config_5(M, N, split, dev, grid_ctas, cluster_size, tiles);
        case 6: return launch_info_config_6(M, N, split, dev, grid_ctas, cluster_size, tiles);
        default: return GEMM_ERR_INVALID_ARG;
    }
}

// Resident CTAs (or clusters) of configuration `cfg` on this device: the grid
// of a problem large enough to fill every slot.
int64_t config_slots(int cfg, const DeviceInfo &dev)
{
    int grid = 0, cluster = 1, tiles = 0;
    if (config_info(cfg, int64_t{1} << 16, int64_t{1} << 16, false, dev, &grid, &cluster, &tiles) != GEMM_OK ||
        cluster <= 0)
        return 0;
    return grid / cluster;
}

// The slice count of GEMM_F16_KSPLIT_AUTO for configuration `cfg` (1: none):
// if its tiles are fewer than its CTA slots, as many slices as fill the slots
// once, at least 16 K blocks each, at most 16.
int rule_k_splits(int cfg, int64_t M, int64_t N, int64_t K, const DeviceInfo &dev)
{
    int grid = 0, cluster = 1, tiles = 0;
    if (config_info(cfg, M, N, false, dev, &grid, &cluster, &tiles) != GEMM_OK || cluster <= 0) return 1;
    const int64_t slots = config_slots(cfg, dev);
    const int64_t k_blocks = (K + 63) / 64;
    if (tiles <= 0 || tiles >= slots) return 1;
    int64_t n = slots / tiles;
    if (n > k_blocks / 16) n = k_blocks / 16;
    if (n > 16) n = 16;
    return n >= 2 ? static_cast<int>(n) : 1;
}

double wave_eff(int id, int64_t M, int64_t N, bool split, const DeviceInfo &dev)
{
    switch (id) {
        case 1: return wave_eff_config_1(M, N, split, dev);
        case 2: return wave_eff_config_2(M, N, split, dev);
        case 3: return wave_eff_config_3(M, N, split, dev);
        case 4: return wave_eff_config_4(M, N, split, dev);
        case 5: return wave_eff_config_5(M, N, split, dev);
        case 6: return wave_eff_config_6(M, N, split, dev);
        default: return 0.0;
    }
}

// Cluster size request of a config word for the cluster K split configuration:
// GEMM_F16_KSPLIT(n) asks for n CTAs per cluster, GEMM_F16_NO_KSPLIT for one,
// anything else for the size rule (0).
int ck_request_of(int word)
{
    const int n = (word & GEMM_F16_KSPLIT_MASK) >> GEMM_F16_KSPLIT_SHIFT;
    if (n >= 2) return n;
    if (word & GEMM_F16_NO_KSPLIT) return 1;
    return 0;
}

// The automatic choice.  The offline sweep (tune.py) measured every candidate
// (configuration x tail policy, and the cluster K split's sizes) on a grid of
// shapes.  None of the candidates allocates memory: a workspace K split is
// taken only on an explicit request (gemm_f16_ex with the K-split bits).  For a problem, take the
// nearest measured shape in log2 space (K weighted by half: it changes the
// per-tile work but not the wave count), scale each candidate's measured
// throughput by its wave efficiency here over its wave efficiency there, and
// take the best.  `any_layout`: only configurations with transposed-layout
// kernels qualify.  Without a table, the size rule above.
int select_config(int64_t M, int64_t N, int64_t K, bool any_layout, const DeviceInfo &dev)
{
#if GEMM_F16_HAVE_TUNED
    // The last choices are kept per thread (callers often repeat a few shapes).
    struct Last {
        int64_t M = -1, N = -1, K = -1;
        int device = -1, any_layout = -1, choice = 0;
    };
    constexpr int kCached = 64;
    thread_local Last cache[kCached];
    thread_local int next_slot = 0;
    for (const Last &c : cache)
        if (c.M == M && c.N == N && c.K == K && c.device == dev.device && c.any_layout == (any_layout ? 1 : 0))
            return c.choice;
    const double lm = std::log2(static_cast<double>(M > 0 ? M : 1));
    const double ln = std::log2(static_cast<double>(N > 0 ? N : 1));
    const double lk = std::log2(static_cast<double>(K > 0 ? K : 1));
    int row = 0;
    double best_d = 1e300;
    for (int r = 0; r < GEMM_F16_TUNED_ROWS; ++r) {
        const TunedRow &t = kTunedRows[r];
        const double d = std::fabs(lm - std::log2(static_cast<double>(t.M))) +
                         std::fabs(ln - std::log2(static_cast<double>(t.N))) +
                         0.5 * std::fabs(lk - std::log2(static_cast<double>(t.K)));
        if (d < best_d) {
            best_d = d;
            row = r;
        }
    }
    const TunedRow &t = kTunedRows[row];
    int choice = 0;
    double best = 0.0;
    for (int i = 0; i < GEMM_F16_TUNED_CANDIDATES; ++i) {
        const int c = kTunedCandidates[i];
        const int id = c & GEMM_F16_CONFIG_ID_MASK;
        if (id < 1 || id > kNumConfigs || (any_layout && !kConfigs[id].all_layouts)) continue;
        const bool split = (c & GEMM_F16_NO_SPLIT) == 0;
        const bool ck = id == kClusterKConfig;
        // The automatic choice allocates nothing: no workspace K split.
        if (!ck && (c & (GEMM_F16_KSPLIT_AUTO | GEMM_F16_KSPLIT_TAIL | GEMM_F16_KSPLIT_MASK)) != 0) continue;
        const double here = ck ? ck_wave_eff_config_6(M, N, K, ck_request_of(c), dev) : wave_eff(id, M, N, split, dev);
        const double there =
            ck ? ck_wave_eff_config_6(t.M, t.N, t.K, ck_request_of(c), dev) : wave_eff(id, t.M, t.N, split, dev);
        if (here <= 0.0 || there <= 0.0) continue;
        // (ratio first: exactly 1 on a measured shape, so ties keep table order)
        const double predicted = static_cast<double>(t.tflops[i]) * (here / there);
        if (predicted > best) {
            best = predicted;
            choice = c;
        }
    }
    if (choice != 0) {
        cache[next_slot] = Last{M, N, K, dev.device, any_layout ? 1 : 0, choice};
        next_slot = (next_slot + 1) % kCached;
        return choice;
    }
#endif
    (void)any_layout;
    return pick_config(M, N, K, dev.sm_count);
}

// K-split requests of a config word (parse_config's *k_request).
constexpr int kKsplitNever = -1;   // GEMM_F16_NO_KSPLIT (0: no K-split bit set)
constexpr int kKsplitRule = -2;    // GEMM_F16_KSPLIT_AUTO
constexpr int kKsplitTail = -3;    // GEMM_F16_KSPLIT_TAIL
                                   // n >= 2: GEMM_F16_KSPLIT(n)

// Splits a config argument into the configuration id and its flag bits;
// false for an unknown id or flag or contradictory K-split bits.
bool parse_config(int config, int *id, bool *allow_split, int *k_request = nullptr)
{
    constexpr int kKnown = GEMM_F16_CONFIG_ID_MASK | GEMM_F16_NO_SPLIT | GEMM_F16_NO_KSPLIT | GEMM_F16_KSPLIT_AUTO |
                           GEMM_F16_KSPLIT_TAIL | GEMM_F16_KSPLIT_MASK;
    if (config < 0 || (config & ~kKnown) != 0) return false;
    const int n = (config & GEMM_F16_KSPLIT_MASK) >> GEMM_F16_KSPLIT_SHIFT;
    const bool never = (config & GEMM_F16_NO_KSPLIT) != 0;
    const bool rule = (config & GEMM_F16_KSPLIT_AUTO) != 0;
    const bool tail = (config & GEMM_F16_KSPLIT_TAIL) != 0;
    if (n == 1 || n > 16 ||
        static_cast<int>(never) + static_cast<int>(rule) + static_cast<int>(tail) + static_cast<int>(n != 0) > 1)
        return false;
    *id = config & GEMM_F16_CONFIG_ID_MASK;
    *allow_split = (config & GEMM_F16_NO_SPLIT) == 0;
    if (k_request) *k_request = never ? kKsplitNever : rule ? kKsplitRule : tail ? kKsplitTail : n;
    return *id <= kNumConfigs;
}

// Workspace slice count for a parsed request on configuration `cfg` (the
// automatic choice never asks for one).
int k_splits_for(int k_request, int cfg, int64_t M, int64_t N, int64_t K, const DeviceInfo &dev)
{
    if (k_request >= 2) return k_request;
    if (k_request == kKsplitRule) return rule_k_splits(cfg, M, N, K, dev);
    return 1;
}

// ---------------------------------------------------------------- launch path

int run_gemm(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K, int transa, int transb,
             int relu, int config, void *stream, const LaunchHook &hook, bool noalloc = false)
{
    int st = check_sizes(M, N, K, relu);
    if (st != GEMM_OK) return st;
    if ((transa != 0 && transa != 1) || (transb != 0 && transb != 1))
        return reject(GEMM_ERR_INVALID_ARG, "transa / transb is not 0 or 1");
    int id = 0, k_request = 0;
    bool allow_split = true;
    if (!parse_config(config, &id, &allow_split, &k_request))
        return reject(GEMM_ERR_INVALID_ARG, "unknown configuration id or flag");
    if ((transa || transb) && !kConfigs[id].all_layouts)
        return reject(GEMM_ERR_INVALID_ARG, "this configuration has no transposed-layout kernels");
    if (M == 0 || N == 0) return GEMM_OK;

    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint64_t c_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * 2u;
    if ((st = check_device_buffer(C, c_bytes, dev.device)) != GEMM_OK) return st;

    if (K == 0) {
        // Empty sum: every output is R(+0) = +0.
        if (cudaMemsetAsync(C, 0, c_bytes, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    // Row pitches of the stored matrices must be multiples of 16 bytes.
    const int64_t lda = transa ? M : K, ldb = transb ? K : N;
    if ((lda % 8) != 0 || (ldb % 8) != 0 || (N % 8) != 0)
        return reject(GEMM_ERR_ALIGNMENT, "a row pitch (leading dimension) is not a multiple of 8 elements");
    const uint64_t a_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(K) * 2u;
    const uint64_t b_bytes = static_cast<uint64_t>(K) * static_cast<uint64_t>(N) * 2u;
    if ((st = check_device_buffer(A, a_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(B, b_bytes, dev.device)) != GEMM_OK) return st;
    if (ranges_overlap(C, c_bytes, A, a_bytes) || ranges_overlap(C, c_bytes, B, b_bytes))
        return reject(GEMM_ERR_INVALID_ARG, "C overlaps A or B");

    LaunchArgs a;
    a.A = A;
    a.B = B;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    a.relu = relu;
    a.transa = transa;
    a.transb = transb;
    a.dev = dev;
    a.stream = s;
    a.hook = hook;
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;

    int cfg = id, picked = 0;
    if (id == 0) {
        picked = select_config(M, N, K, transa || transb, dev);
        cfg = picked & GEMM_F16_CONFIG_ID_MASK;
        a.allow_split = allow_split && (picked & GEMM_F16_NO_SPLIT) == 0;
    } else {
        a.allow_split = allow_split;
    }
    if (cfg == kClusterKConfig) {
        // The K split runs across the cluster: its size from the config word
        // (or from the automatic choice's word), no workspace.
        if (k_request == kKsplitTail)
            return reject(GEMM_ERR_INVALID_ARG, "the cluster K split configuration has no tail split");
        a.ck_request = id == 0 ? ck_request_of(picked)
                       : k_request >= 2 ? k_request
                       : k_request == kKsplitNever ? 1 : 0;
        if (a.ck_request != 0 && a.ck_request != 1 && a.ck_request != 2 && a.ck_request != 4 && a.ck_request != 8)
            return reject(GEMM_ERR_INVALID_ARG, "a cluster K split takes 2, 4 or 8 CTAs per cluster");
        a.k_splits = 1;
        a.k_split_tail = false;
    } else {
        a.k_splits = k_splits_for(k_request, cfg, M, N, K, dev);
        a.k_split_tail = k_request == kKsplitTail;
    }
    if (hook.producer_off) {
        // the timeout self-test never writes C
        a.k_splits = 1;
        a.k_split_tail = false;
    }
    // K-slice partials of a noalloc call go to the library's fixed scratch;
    // the launch rejects a split that does not fit before it enqueues anything.
    a.noalloc = noalloc;
    switch (cfg) {
        case 1: st = launch_config_1(a); break;
        case 2: st = launch_config_2(a); break;
        case 3: st = launch_config_3(a); break;
        case 4: st = launch_config_4(a); break;
        case 5: st = launch_config_5(a); break;
        case 6: st = launch_config_6(a); break;
        default: return GEMM_ERR_INVALID_ARG;
    }
    if (st == GEMM_ERR_INVALID_ARG)
        return reject(st, noalloc ? "the K-slice partials exceed the 16 MiB scratch of gemm_f16_ex_noalloc"
                                  : "the problem has too many work units");
    return st;
}

thread_local uint64_t t_last_timeout_record = 0;

}  // namespace

// ==================================================================== C ABI

extern "C" int gemm_f16_tx(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K, int transa,
                           int transb, int relu, int config, void *stream)
{
    return run_gemm(A, B, C, M, N, K, transa, transb, relu, config, stream, LaunchHook());
}

extern "C" int gemm_f16_ex(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K, int relu,
                           int config, void *stream)
{
    return run_gemm(A, B, C, M, N, K, 0, 0, relu, config, stream, LaunchHook());
}

extern "C" int gemm_f16_ex_noalloc(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K, int relu,
                                   int config, void *stream)
{
    return run_gemm(A, B, C, M, N, K, 0, 0, relu, config, stream, LaunchHook{}, true);
}

extern "C" int gemm_f16(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K, int relu,
                        void *stream)
{
    return run_gemm(A, B, C, M, N, K, 0, 0, relu, 0, stream, LaunchHook());
}

extern "C" int gemm_f16_selftest_timeout(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K,
                                         int config, uint64_t timeout_cycles, void *stream)
{
    if (K == 0 || M == 0 || N == 0) return reject(GEMM_ERR_INVALID_ARG, "an empty problem launches no kernel");
    if (timeout_cycles < (1ull << 16) || timeout_cycles > (1ull << 32))
        return reject(GEMM_ERR_INVALID_ARG, "timeout_cycles outside 2^16 .. 2^32");
    LaunchHook hook;
    hook.producer_off = 1;
    hook.timeout_cycles = timeout_cycles;
    return run_gemm(A, B, C, M, N, K, 0, 0, 1, config, stream, hook);
}

namespace gemm_sm103 {
int tma_box_image_launch(const void *X, int64_t rows, int64_t cols, int box_rows, int x, int y, void *out,
                         unsigned long long *status, cudaStream_t stream);
}

extern "C" int gemm_f16_tma_box_image(const void *X, int64_t rows, int64_t cols, int64_t box_rows, int64_t x,
                                      int64_t y, void *out, void *stream)
{
    if (rows < 1 || cols < 1 || rows > INT32_MAX || cols > INT32_MAX)
        return reject(GEMM_ERR_INVALID_ARG, "rows and cols must be 1 .. INT32_MAX");
    if (box_rows < 1 || box_rows > 256) return reject(GEMM_ERR_INVALID_ARG, "box_rows must be 1 .. 256");
    if (x < INT32_MIN || x > INT32_MAX || y < INT32_MIN || y > INT32_MAX)
        return reject(GEMM_ERR_INVALID_ARG, "a box coordinate is outside the 32-bit range");
    if ((cols % 8) != 0) return reject(GEMM_ERR_ALIGNMENT, "cols (the row pitch) is not a multiple of 8 elements");
    if ((x % 8) != 0)
        return reject(GEMM_ERR_ALIGNMENT, "x is not a multiple of 8 elements (a box starts on a 16-byte boundary)");
    DeviceInfo dev;
    int st = current_device_info(&dev);
    if (st != GEMM_OK) return st;
    const uint64_t x_bytes = static_cast<uint64_t>(rows) * static_cast<uint64_t>(cols) * 2u;
    const uint64_t out_bytes = static_cast<uint64_t>(box_rows) * 128u;
    if ((st = check_device_buffer(X, x_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(out, out_bytes, dev.device)) != GEMM_OK) return st;
    if (ranges_overlap(out, out_bytes, X, x_bytes)) return reject(GEMM_ERR_INVALID_ARG, "out overlaps X");
    unsigned long long *status = status_word(dev.device);
    if (status == nullptr) return GEMM_ERR_CUDA;
    return tma_box_image_launch(X, rows, cols, static_cast<int>(box_rows), static_cast<int>(x), static_cast<int>(y),
                                out, status, static_cast<cudaStream_t>(stream));
}

namespace gemm_sm103 {
int relu_backward_launch(const void *dC, const void *C, void *dZ, int64_t n, int sm_count, cudaStream_t stream);
}

extern "C" int gemm_f16_relu_backward(const void *dC, const void *C, void *dZ, int64_t n, void *stream)
{
    if (n < 0) return reject(GEMM_ERR_INVALID_ARG, "n is negative");
    if (n == 0) return GEMM_OK;
    DeviceInfo dev;
    int st = current_device_info(&dev);
    if (st != GEMM_OK) return st;
    const uint64_t bytes = static_cast<uint64_t>(n) * 2u;
    if ((st = check_device_buffer(dC, bytes, dev.device, 2)) != GEMM_OK) return st;
    if ((st = check_device_buffer(C, bytes, dev.device, 2)) != GEMM_OK) return st;
    if ((st = check_device_buffer(dZ, bytes, dev.device, 2)) != GEMM_OK) return st;
    // In place over dC (or C) is fine element by element; a partial overlap is not.
    if ((dZ != dC && ranges_overlap(dZ, bytes, dC, bytes)) || (dZ != C && ranges_overlap(dZ, bytes, C, bytes)))
        return reject(GEMM_ERR_INVALID_ARG, "dZ partly overlaps dC or C");
    return relu_backward_launch(dC, C, dZ, n, dev.sm_count, static_cast<cudaStream_t>(stream));
}

extern "C" int gemm_fp8_block_scaled(const void *A, const float *SA, const void *W, const float *SW, void *C,
                                     int64_t M, int64_t N, int64_t K, int relu, void *stream)
{
    int st = check_sizes(M, N, K, relu);
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint64_t c_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * 2u;
    if ((st = check_device_buffer(C, c_bytes, dev.device)) != GEMM_OK) return st;
    if (K == 0) {
        // Empty sum in every block: every output is R(+0) = +0.
        if (cudaMemsetAsync(C, 0, c_bytes, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    if ((K % 16) != 0)
        return reject(GEMM_ERR_ALIGNMENT, "K is not a multiple of 16 (the E4M3 row pitch of A and W is K bytes)");
    if ((N % 8) != 0) return reject(GEMM_ERR_ALIGNMENT, "N is not a multiple of 8 (the fp16 row pitch of C)");
    const uint64_t KB = static_cast<uint64_t>((K + 127) / 128), NB = static_cast<uint64_t>((N + 127) / 128);
    const uint64_t a_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(K);
    const uint64_t w_bytes = static_cast<uint64_t>(N) * static_cast<uint64_t>(K);
    const uint64_t sa_bytes = static_cast<uint64_t>(M) * KB * 4u, sw_bytes = NB * KB * 4u;
    if ((st = check_device_buffer(A, a_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(W, w_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(SA, sa_bytes, dev.device, 4)) != GEMM_OK) return st;
    if ((st = check_device_buffer(SW, sw_bytes, dev.device, 4)) != GEMM_OK) return st;
    if (ranges_overlap(C, c_bytes, A, a_bytes) || ranges_overlap(C, c_bytes, W, w_bytes) ||
        ranges_overlap(C, c_bytes, SA, sa_bytes) || ranges_overlap(C, c_bytes, SW, sw_bytes))
        return reject(GEMM_ERR_INVALID_ARG, "C overlaps an input");
    Fp8LaunchArgs a;
    a.A = A;
    a.SA = SA;
    a.W = W;
    a.SW = SW;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    a.relu = relu;
    a.dev = dev;
    a.stream = s;
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;
    return launch_fp8(a);
}

extern "C" int gemm_mxfp8_block_scaled(const void *A, const uint8_t *SA, const void *W, const uint8_t *SW, void *C,
                                       int64_t M, int64_t N, int64_t K, int relu, void *stream)
{
    int st = check_sizes(M, N, K, relu);
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint64_t c_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * 2u;
    if ((st = check_device_buffer(C, c_bytes, dev.device)) != GEMM_OK) return st;
    if (K == 0) {
        // Empty sum in every block: every output is R(+0) = +0.
        if (cudaMemsetAsync(C, 0, c_bytes, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    if ((K % 16) != 0)
        return reject(GEMM_ERR_ALIGNMENT, "K is not a multiple of 16 (the E4M3 row pitch of A and W is K bytes)");
    if ((N % 8) != 0) return reject(GEMM_ERR_ALIGNMENT, "N is not a multiple of 8 (the fp16 row pitch of C)");
    const uint64_t KB = static_cast<uint64_t>((K + 127) / 128), NB = static_cast<uint64_t>((N + 127) / 128);
    const uint64_t a_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(K);
    const uint64_t w_bytes = static_cast<uint64_t>(N) * static_cast<uint64_t>(K);
    const uint64_t sa_bytes = static_cast<uint64_t>(M) * KB, sw_bytes = NB * KB;
    if ((st = check_device_buffer(A, a_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(W, w_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(SA, sa_bytes, dev.device, 1)) != GEMM_OK) return st;
    if ((st = check_device_buffer(SW, sw_bytes, dev.device, 1)) != GEMM_OK) return st;
    if (ranges_overlap(C, c_bytes, A, a_bytes) || ranges_overlap(C, c_bytes, W, w_bytes) ||
        ranges_overlap(C, c_bytes, SA, sa_bytes) || ranges_overlap(C, c_bytes, SW, sw_bytes))
        return reject(GEMM_ERR_INVALID_ARG, "C overlaps an input");
    MxLaunchArgs a;
    a.A = A;
    a.SA = SA;
    a.W = W;
    a.SW = SW;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    a.relu = relu;
    a.dev = dev;
    a.stream = s;
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;
    return launch_mxfp8(a);
}

namespace {

// Bytes of an element of a gemm_f16_type, 0 for an unknown type.
uint32_t type_bytes(int type)
{
    switch (type) {
    case GEMM_TYPE_F16:
    case GEMM_TYPE_BF16: return 2;
    case GEMM_TYPE_F32: return 4;
    default: return 0;
    }
}

}  // namespace

extern "C" int mxfp4_quantize(const void *X, int type, uint8_t *Q, uint8_t *S, void *V, int64_t rows, int64_t K,
                              int trans, void *stream)
{
    int st = check_sizes(rows, 0, K, 0);
    if (st != GEMM_OK) return st;
    const uint32_t el = type_bytes(type);
    if (el == 0) return reject(GEMM_ERR_INVALID_ARG, "type is not a gemm_f16_type");
    if (trans != 0 && trans != 1) return reject(GEMM_ERR_INVALID_ARG, "trans is not 0 or 1");
    if (rows == 0 || K == 0) return GEMM_OK;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const uint64_t x_bytes = static_cast<uint64_t>(rows) * static_cast<uint64_t>(K) * el;
    const uint64_t q_bytes = mx4_code_bytes(rows, K), s_bytes = mx4_scale_bytes(rows, K);
    if ((st = check_device_buffer_fast(X, x_bytes, dev.device, el)) != GEMM_OK) return st;
    if ((st = check_device_buffer_fast(Q, q_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer_fast(S, s_bytes, dev.device)) != GEMM_OK) return st;
    if (V != nullptr && (st = check_device_buffer_fast(V, x_bytes, dev.device, el)) != GEMM_OK) return st;
    if (ranges_overlap(Q, q_bytes, X, x_bytes) || ranges_overlap(S, s_bytes, X, x_bytes) ||
        ranges_overlap(Q, q_bytes, S, s_bytes) ||
        (V != nullptr && (ranges_overlap(V, x_bytes, X, x_bytes) || ranges_overlap(V, x_bytes, Q, q_bytes) ||
                          ranges_overlap(V, x_bytes, S, s_bytes))))
        return reject(GEMM_ERR_INVALID_ARG, "Q, S or V overlaps another buffer");
    Mx4QuantArgs a;
    a.X = X;
    a.Q = Q;
    a.S = S;
    a.V = V;
    a.rows = rows;
    a.K = K;
    a.type = type;
    a.trans = trans;
    a.sm_count = dev.sm_count;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_mxfp4_quantize(a);
}

namespace {

int run_mxfp4(const void *A, const uint8_t *SA, const void *W, const uint8_t *SW, void *C, int64_t M, int64_t N,
              int64_t K, int relu, void *stream, int withhold, uint64_t timeout_cycles)
{
    int st = check_sizes(M, N, K, relu);
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint64_t c_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * 2u;
    if ((st = check_device_buffer_fast(C, c_bytes, dev.device)) != GEMM_OK) return st;
    if (K == 0) {
        // Empty sum: every output is R(+0) = +0.
        if (cudaMemsetAsync(C, 0, c_bytes, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    if ((N % 8) != 0) return reject(GEMM_ERR_ALIGNMENT, "N is not a multiple of 8 (the fp16 row pitch of C)");
    const uint64_t a_bytes = mx4_code_bytes(M, K), w_bytes = mx4_code_bytes(N, K);
    const uint64_t sa_bytes = mx4_scale_bytes(M, K), sw_bytes = mx4_scale_bytes(N, K);
    if ((st = check_device_buffer_fast(A, a_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer_fast(W, w_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer_fast(SA, sa_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer_fast(SW, sw_bytes, dev.device)) != GEMM_OK) return st;
    if (ranges_overlap(C, c_bytes, A, a_bytes) || ranges_overlap(C, c_bytes, W, w_bytes) ||
        ranges_overlap(C, c_bytes, SA, sa_bytes) || ranges_overlap(C, c_bytes, SW, sw_bytes))
        return reject(GEMM_ERR_INVALID_ARG, "C overlaps an input");
    Mx4LaunchArgs a;
    a.A = A;
    a.SA = SA;
    a.W = W;
    a.SW = SW;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    a.relu = relu;
    a.dev = dev;
    a.stream = s;
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;
    a.withhold = withhold;
    a.timeout_cycles = timeout_cycles;
    return launch_mxfp4(a);
}

}  // namespace

extern "C" int gemm_mxfp4(const void *A, const uint8_t *SA, const void *W, const uint8_t *SW, void *C, int64_t M,
                          int64_t N, int64_t K, int relu, void *stream)
{
    return run_mxfp4(A, SA, W, SW, C, M, N, K, relu, stream, 0, 0);
}

extern "C" int gemm_mxfp4_selftest_timeout(const void *A, const uint8_t *SA, const void *W, const uint8_t *SW, void *C,
                                           int64_t M, int64_t N, int64_t K, int withhold, uint64_t timeout_cycles,
                                           void *stream)
{
    if (K == 0 || M == 0 || N == 0) return reject(GEMM_ERR_INVALID_ARG, "an empty problem launches no kernel");
    if (withhold != 1 && withhold != 2) return reject(GEMM_ERR_INVALID_ARG, "withhold is not 1 or 2");
    if (timeout_cycles < (1ull << 16) || timeout_cycles > (1ull << 32))
        return reject(GEMM_ERR_INVALID_ARG, "timeout_cycles outside 2^16 .. 2^32");
    return run_mxfp4(A, SA, W, SW, C, M, N, K, 0, stream, withhold, timeout_cycles);
}

namespace {

int check_norm_args(int64_t rows, int64_t dim, int xtype, int wtype)
{
    const int st = check_sizes(rows, dim, 0, 0);
    if (st != GEMM_OK) return st;
    if (type_bytes(xtype) == 0 || type_bytes(wtype) == 0)
        return reject(GEMM_ERR_INVALID_ARG, "xtype or wtype is not a gemm_f16_type");
    if (wtype != xtype && wtype != GEMM_TYPE_F32)
        return reject(GEMM_ERR_INVALID_ARG, "wtype is neither xtype nor GEMM_TYPE_F32");
    return GEMM_OK;
}

struct NormBuffer {
    const void *p;
    uint64_t bytes;
    uintptr_t align;
    bool written;
};

// Checks every buffer that is given and that what is written overlaps nothing
// else.
int check_norm_buffers(const NormBuffer *b, int n, int dev)
{
    for (int i = 0; i < n; ++i) {
        if (b[i].p == nullptr) continue;
        const int st = check_device_buffer_fast(b[i].p, b[i].bytes, dev, b[i].align);
        if (st != GEMM_OK) return st;
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (i == j || !b[i].written || b[i].p == nullptr || b[j].p == nullptr) continue;
            if (ranges_overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return reject(GEMM_ERR_INVALID_ARG, "an output overlaps another buffer");
        }
    return GEMM_OK;
}

}  // namespace

extern "C" int layer_norm_fwd(const void *X, const void *gamma, const void *beta, void *Y, float *mean, float *rstd,
                              int64_t rows, int64_t dim, float eps, int xtype, int wtype, void *stream)
{
    int st = check_norm_args(rows, dim, xtype, wtype);
    if (st != GEMM_OK) return st;
    if (!std::isfinite(eps) || eps < 0.0f) return reject(GEMM_ERR_INVALID_ARG, "eps is negative or not finite");
    if (rows == 0 || dim == 0) return GEMM_OK;
    if (X == nullptr || Y == nullptr) return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const uint64_t x_bytes = static_cast<uint64_t>(rows) * static_cast<uint64_t>(dim) * type_bytes(xtype);
    const uint64_t w_bytes = static_cast<uint64_t>(dim) * type_bytes(wtype);
    const uint64_t r_bytes = static_cast<uint64_t>(rows) * sizeof(float);
    const NormBuffer b[] = {{X, x_bytes, type_bytes(xtype), false},    {gamma, w_bytes, type_bytes(wtype), false},
                            {beta, w_bytes, type_bytes(wtype), false}, {Y, x_bytes, type_bytes(xtype), true},
                            {mean, r_bytes, 4, true},                  {rstd, r_bytes, 4, true}};
    if ((st = check_norm_buffers(b, 6, dev.device)) != GEMM_OK) return st;
    LayerNormArgs a;
    a.X = X;
    a.gamma = gamma;
    a.beta = beta;
    a.Y = Y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.dim = dim;
    a.eps = eps;
    a.xtype = xtype;
    a.wtype = wtype;
    a.sm_count = dev.sm_count;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_layer_norm_fwd(a);
}

extern "C" int64_t layer_norm_bwd_workspace(int64_t rows, int64_t dim)
{
    int st = check_sizes(rows, dim, 0, 0);
    if (st != GEMM_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    return 2 * layer_norm_parts(rows, dim, dev.sm_count) * dim * static_cast<int64_t>(sizeof(float));
}

namespace {

int run_layer_norm_bwd(const void *dY, const void *X, const void *gamma, const float *mean, const float *rstd, void *dX,
                       void *dgamma, void *dbeta, int64_t rows, int64_t dim, int xtype, int wtype, void *workspace,
                       int64_t workspace_bytes, void *stream, int withhold, uint64_t timeout_cycles)
{
    int st = check_norm_args(rows, dim, xtype, wtype);
    if (st != GEMM_OK) return st;
    if ((dgamma == nullptr) != (dbeta == nullptr))
        return reject(GEMM_ERR_INVALID_ARG, "one of dgamma and dbeta is NULL and the other is not");
    if (dim == 0) return GEMM_OK;
    if (rows > 0 && (dY == nullptr || X == nullptr || mean == nullptr || rstd == nullptr || dX == nullptr))
        return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    if (rows == 0 && dgamma == nullptr) return GEMM_OK;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint64_t x_bytes = static_cast<uint64_t>(rows) * static_cast<uint64_t>(dim) * type_bytes(xtype);
    const uint64_t w_bytes = static_cast<uint64_t>(dim) * type_bytes(wtype);
    const uint64_t r_bytes = static_cast<uint64_t>(rows) * sizeof(float);
    if (rows == 0) {
        // Empty sums.
        const NormBuffer b[] = {{dgamma, w_bytes, type_bytes(wtype), true}, {dbeta, w_bytes, type_bytes(wtype), true}};
        if ((st = check_norm_buffers(b, 2, dev.device)) != GEMM_OK) return st;
        if (cudaMemsetAsync(dgamma, 0, w_bytes, s) != cudaSuccess ||
            cudaMemsetAsync(dbeta, 0, w_bytes, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    const uint64_t need =
        dgamma ? 2 * static_cast<uint64_t>(layer_norm_parts(rows, dim, dev.sm_count)) * static_cast<uint64_t>(dim) * 4u
               : 0u;
    if (dgamma && (workspace == nullptr || workspace_bytes < 0 || static_cast<uint64_t>(workspace_bytes) < need))
        return reject(GEMM_ERR_INVALID_ARG, "the workspace is smaller than layer_norm_bwd_workspace says");
    const NormBuffer b[] = {{dY, x_bytes, type_bytes(xtype), false},
                            {X, x_bytes, type_bytes(xtype), false},
                            {gamma, w_bytes, type_bytes(wtype), false},
                            {mean, r_bytes, 4, false},
                            {rstd, r_bytes, 4, false},
                            {dX, x_bytes, type_bytes(xtype), true},
                            {dgamma, w_bytes, type_bytes(wtype), true},
                            {dbeta, w_bytes, type_bytes(wtype), true},
                            {dgamma ? workspace : nullptr, need, 16, true}};
    if ((st = check_norm_buffers(b, 9, dev.device)) != GEMM_OK) return st;
    LayerNormArgs a;
    a.dY = dY;
    a.X = X;
    a.gamma = gamma;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.Y = dX;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.workspace = static_cast<float *>(workspace);
    a.rows = rows;
    a.dim = dim;
    a.xtype = xtype;
    a.wtype = wtype;
    a.sm_count = dev.sm_count;
    a.device = dev.device;
    a.stream = s;
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;
    a.withhold = withhold;
    a.timeout_cycles = timeout_cycles;
    return launch_layer_norm_bwd(a);
}

}  // namespace

extern "C" int layer_norm_bwd(const void *dY, const void *X, const void *gamma, const float *mean, const float *rstd,
                              void *dX, void *dgamma, void *dbeta, int64_t rows, int64_t dim, int xtype, int wtype,
                              void *workspace, int64_t workspace_bytes, void *stream)
{
    return run_layer_norm_bwd(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, rows, dim, xtype, wtype, workspace,
                              workspace_bytes, stream, 0, 0);
}

extern "C" int layer_norm_bwd_selftest_timeout(const void *dY, const void *X, const float *mean, const float *rstd,
                                               void *dX, int64_t rows, int64_t dim, int xtype,
                                               uint64_t timeout_cycles, void *stream)
{
    if (rows == 0 || dim == 0) return reject(GEMM_ERR_INVALID_ARG, "an empty problem launches no kernel");
    if (timeout_cycles < (1ull << 16) || timeout_cycles > (1ull << 32))
        return reject(GEMM_ERR_INVALID_ARG, "timeout_cycles outside 2^16 .. 2^32");
    return run_layer_norm_bwd(dY, X, nullptr, mean, rstd, dX, nullptr, nullptr, rows, dim, xtype, xtype, nullptr, 0,
                              stream, 1, timeout_cycles);
}

namespace {

// An output that may take the place of one of the call's inputs: the same
// address, or no overlap.
bool in_place_or_apart(const void *out, uint64_t out_bytes, const void *in, uint64_t in_bytes)
{
    return in == nullptr || out == in || !ranges_overlap(out, out_bytes, in, in_bytes);
}

// What rms_norm_fwd and rms_norm_fp8 share: with Q the output is FP8.
int run_rms_norm_fwd(const void *X, const void *R, const void *gamma, void *H, void *Y, void *Q, void *S, float *rstd,
                     int64_t rows, int64_t dim, float eps, int xtype, int wtype, int pow2, void *stream)
{
    int st = check_norm_args(rows, dim, xtype, wtype);
    if (st != GEMM_OK) return st;
    if (!std::isfinite(eps) || eps < 0.0f) return reject(GEMM_ERR_INVALID_ARG, "eps is negative or not finite");
    if (pow2 != 0 && pow2 != 1) return reject(GEMM_ERR_INVALID_ARG, "pow2 is not 0 or 1");
    if ((R == nullptr) != (H == nullptr))
        return reject(GEMM_ERR_INVALID_ARG, "one of R and H is NULL and the other is not");
    if (rows == 0 || dim == 0) return GEMM_OK;
    if (X == nullptr || (Y == nullptr && Q == nullptr) || (Q != nullptr && S == nullptr))
        return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const uint32_t el = type_bytes(xtype);
    const uint64_t n = static_cast<uint64_t>(rows) * static_cast<uint64_t>(dim), x_bytes = n * el;
    const uint64_t s_bytes = static_cast<uint64_t>(rows) * static_cast<uint64_t>((dim + 127) / 128) * (pow2 ? 1u : 4u);
    // H takes the place of X or R, or overlaps nothing: left out here where it does.
    const bool in_place = H != nullptr && (H == X || H == R);
    const NormBuffer b[] = {{X, x_bytes, el, in_place && H == X},
                            {R, x_bytes, el, in_place && H == R},
                            {gamma, static_cast<uint64_t>(dim) * type_bytes(wtype), type_bytes(wtype), false},
                            {in_place ? nullptr : H, x_bytes, el, true},
                            {Y, x_bytes, el, true},
                            {Q, n, 1, true},
                            {S, s_bytes, pow2 ? 1u : 4u, true},
                            {rstd, static_cast<uint64_t>(rows) * sizeof(float), 4, true}};
    if (in_place && X == R) {
        // The stream doubled in place: X and R are one buffer, written.
        const NormBuffer one[] = {{X, x_bytes, el, true}, b[2], b[4], b[5], b[6], b[7]};
        if ((st = check_norm_buffers(one, 6, dev.device)) != GEMM_OK) return st;
    } else if ((st = check_norm_buffers(b, 8, dev.device)) != GEMM_OK) {
        return st;
    }
    RmsNormArgs a;
    a.X = X;
    a.R = R;
    a.gamma = gamma;
    a.H = H;
    a.Y = Y;
    a.Q = Q;
    a.S = S;
    a.rstd = rstd;
    a.rows = rows;
    a.dim = dim;
    a.eps = eps;
    a.xtype = xtype;
    a.wtype = wtype;
    a.pow2 = pow2;
    a.sm_count = dev.sm_count;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_rms_norm_fwd(a);
}

uint64_t rms_norm_bwd_bytes(int64_t rows, int64_t dim, int sm_count)
{
    return static_cast<uint64_t>(layer_norm_parts(rows, dim, sm_count)) * static_cast<uint64_t>(dim) * sizeof(float);
}

int run_rms_norm_bwd(const void *dY, const void *H, const void *gamma, const float *rstd, const void *dH, void *dX,
                     void *dgamma, int64_t rows, int64_t dim, int xtype, int wtype, void *workspace,
                     int64_t workspace_bytes, void *stream, int withhold, uint64_t timeout_cycles)
{
    int st = check_norm_args(rows, dim, xtype, wtype);
    if (st != GEMM_OK) return st;
    if (dim == 0) return GEMM_OK;
    if (rows > 0 && (dY == nullptr || H == nullptr || rstd == nullptr || dX == nullptr))
        return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    if (rows == 0 && dgamma == nullptr) return GEMM_OK;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const uint32_t el = type_bytes(xtype), wel = type_bytes(wtype);
    const uint64_t x_bytes = static_cast<uint64_t>(rows) * static_cast<uint64_t>(dim) * el;
    const uint64_t w_bytes = static_cast<uint64_t>(dim) * wel;
    if (rows == 0) {
        // Empty sums.
        const NormBuffer b[] = {{dgamma, w_bytes, wel, true}};
        if ((st = check_norm_buffers(b, 1, dev.device)) != GEMM_OK) return st;
        if (cudaMemsetAsync(dgamma, 0, w_bytes, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    const uint64_t need = dgamma ? rms_norm_bwd_bytes(rows, dim, dev.sm_count) : 0u;
    if (dgamma && (workspace == nullptr || workspace_bytes < 0 || static_cast<uint64_t>(workspace_bytes) < need))
        return reject(GEMM_ERR_INVALID_ARG, "the workspace is smaller than rms_norm_bwd_workspace says");
    const NormBuffer b[] = {{dY, x_bytes, el, false},
                            {H, x_bytes, el, false},
                            {gamma, w_bytes, wel, false},
                            {rstd, static_cast<uint64_t>(rows) * sizeof(float), 4, false},
                            {dH, x_bytes, el, false},
                            {dX, x_bytes, el, true},
                            {dgamma, w_bytes, wel, true},
                            {dgamma ? workspace : nullptr, need, 16, true}};
    if ((st = check_norm_buffers(b, 8, dev.device)) != GEMM_OK) return st;
    RmsNormArgs a;
    a.dY = dY;
    a.X = H;
    a.gamma = gamma;
    a.rstd = const_cast<float *>(rstd);
    a.dH = dH;
    a.dX = dX;
    a.dgamma = dgamma;
    a.workspace = static_cast<float *>(workspace);
    a.rows = rows;
    a.dim = dim;
    a.xtype = xtype;
    a.wtype = wtype;
    a.sm_count = dev.sm_count;
    a.device = dev.device;
    a.stream = static_cast<cudaStream_t>(stream);
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;
    a.withhold = withhold;
    a.timeout_cycles = timeout_cycles;
    return launch_rms_norm_bwd(a);
}

}  // namespace

extern "C" int rms_norm_fwd(const void *X, const void *R, const void *gamma, void *H, void *Y, float *rstd,
                            int64_t rows, int64_t dim, float eps, int xtype, int wtype, void *stream)
{
    if (Y == nullptr && rows > 0 && dim > 0) return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    return run_rms_norm_fwd(X, R, gamma, H, Y, nullptr, nullptr, rstd, rows, dim, eps, xtype, wtype, 0, stream);
}

extern "C" int rms_norm_fp8(const void *X, const void *R, const void *gamma, void *H, void *Q, void *S, float *rstd,
                            int64_t rows, int64_t dim, float eps, int xtype, int wtype, int pow2, void *stream)
{
    if (Q == nullptr && rows > 0 && dim > 0) return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    return run_rms_norm_fwd(X, R, gamma, H, nullptr, Q, S, rstd, rows, dim, eps, xtype, wtype, pow2, stream);
}

extern "C" int64_t rms_norm_bwd_workspace(int64_t rows, int64_t dim)
{
    int st = check_sizes(rows, dim, 0, 0);
    if (st != GEMM_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    return static_cast<int64_t>(rms_norm_bwd_bytes(rows, dim, dev.sm_count));
}

extern "C" int rms_norm_bwd(const void *dY, const void *H, const void *gamma, const float *rstd, const void *dH,
                            void *dX, void *dgamma, int64_t rows, int64_t dim, int xtype, int wtype, void *workspace,
                            int64_t workspace_bytes, void *stream)
{
    return run_rms_norm_bwd(dY, H, gamma, rstd, dH, dX, dgamma, rows, dim, xtype, wtype, workspace, workspace_bytes,
                            stream, 0, 0);
}

extern "C" int rms_norm_bwd_selftest_timeout(const void *dY, const void *H, const float *rstd, void *dX, int64_t rows,
                                             int64_t dim, int xtype, uint64_t timeout_cycles, void *stream)
{
    if (rows == 0 || dim == 0) return reject(GEMM_ERR_INVALID_ARG, "an empty problem launches no kernel");
    if (timeout_cycles < (1ull << 16) || timeout_cycles > (1ull << 32))
        return reject(GEMM_ERR_INVALID_ARG, "timeout_cycles outside 2^16 .. 2^32");
    return run_rms_norm_bwd(dY, H, nullptr, rstd, nullptr, dX, nullptr, rows, dim, xtype, xtype, nullptr, 0, stream, 1,
                            timeout_cycles);
}

extern "C" int fp8_quantize(const void *X, int type, void *Q, void *S, int64_t rows, int64_t K, int block_rows,
                            int pow2, void *stream)
{
    int st = check_sizes(rows, 0, K, 0);
    if (st != GEMM_OK) return st;
    const uint32_t el = type_bytes(type);
    if (el == 0) return reject(GEMM_ERR_INVALID_ARG, "type is not a gemm_f16_type");
    if (block_rows != 1 && block_rows != 128) return reject(GEMM_ERR_INVALID_ARG, "block_rows is not 1 or 128");
    if (pow2 != 0 && pow2 != 1) return reject(GEMM_ERR_INVALID_ARG, "pow2 is not 0 or 1");
    if (rows == 0 || K == 0) return GEMM_OK;
    const int64_t blocks = (rows + block_rows - 1) / block_rows * ((K + 127) / 128);
    if (blocks > INT32_MAX) return reject(GEMM_ERR_INVALID_ARG, "more than INT32_MAX blocks");
    if (X == nullptr || Q == nullptr || S == nullptr) return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const uint64_t n = static_cast<uint64_t>(rows) * static_cast<uint64_t>(K);
    const uint32_t sel = pow2 ? 1u : 4u;
    const NormBuffer b[] = {{X, n * el, el, false}, {Q, n, 1, true}, {S, static_cast<uint64_t>(blocks) * sel, sel, true}};
    if ((st = check_norm_buffers(b, 3, dev.device)) != GEMM_OK) return st;
    Fp8QuantArgs a;
    a.X = X;
    a.Q = Q;
    a.S = S;
    a.rows = rows;
    a.K = K;
    a.type = type;
    a.block_rows = block_rows;
    a.pow2 = pow2;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_fp8_quantize(a);
}

extern "C" int dropout_philox(const void *X, const void *R, void *Y, int64_t n, int type, double p, uint64_t seed,
                              uint64_t offset, const void *offset_ptr, void *stream)
{
    const uint32_t el = type_bytes(type);
    if (n < 0) return reject(GEMM_ERR_INVALID_ARG, "a size is negative");
    if (el == 0) return reject(GEMM_ERR_INVALID_ARG, "type is not a gemm_f16_type");
    if (!(p >= 0.0 && p < 1.0)) return reject(GEMM_ERR_INVALID_ARG, "p is not in [0, 1)");
    if (n == 0) return GEMM_OK;
    if (n > INT64_MAX / 8) return reject(GEMM_ERR_INVALID_ARG, "n is beyond any memory");
    if (X == nullptr || Y == nullptr) return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    DeviceInfo dev;
    int st = current_device_info(&dev);
    if (st != GEMM_OK) return st;
    const uint64_t bytes = static_cast<uint64_t>(n) * el;
    const NormBuffer b[] = {{X, bytes, el, false}, {R, bytes, el, false}, {Y, bytes, el, false}, {offset_ptr, 8, 8, false}};
    if ((st = check_norm_buffers(b, 4, dev.device)) != GEMM_OK) return st;
    if (!in_place_or_apart(Y, bytes, X, bytes) || !in_place_or_apart(Y, bytes, R, bytes) ||
        (offset_ptr != nullptr && ranges_overlap(Y, bytes, offset_ptr, 8)))
        return reject(GEMM_ERR_INVALID_ARG, "Y overlaps another buffer without being X or R");
    DropoutArgs a;
    a.X = X;
    a.R = R;
    a.Y = Y;
    a.n = n;
    a.type = type;
    a.p = p;
    a.seed = seed;
    a.offset = offset;
    a.offset_ptr = static_cast<const uint64_t *>(offset_ptr);
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_dropout(a);
}

namespace {

int check_w4_args(int64_t N, int64_t K, int group, int stype)
{
    const int st = check_sizes(N, 0, K, 0);
    if (st != GEMM_OK) return st;
    if (group != 32 && group != 64 && group != 128) return reject(GEMM_ERR_INVALID_ARG, "group is not 32, 64 or 128");
    if (stype != GEMM_TYPE_F16 && stype != GEMM_TYPE_BF16)
        return reject(GEMM_ERR_INVALID_ARG, "the scales' type is not a 16-bit gemm_f16_type");
    return GEMM_OK;
}

}  // namespace

extern "C" int w4_quantize(const void *W, int type, void *Q, void *S, uint8_t *Z, int64_t N, int64_t K, int group,
                           int stype, int trans, void *stream)
{
    int st = check_w4_args(N, K, group, stype);
    if (st != GEMM_OK) return st;
    const uint32_t el = type_bytes(type);
    if (el == 0) return reject(GEMM_ERR_INVALID_ARG, "type is not a gemm_f16_type");
    if (trans != 0 && trans != 1) return reject(GEMM_ERR_INVALID_ARG, "trans is not 0 or 1");
    if (N == 0 || K == 0) return GEMM_OK;
    if (W == nullptr || Q == nullptr || S == nullptr) return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const uint64_t values = static_cast<uint64_t>(w4_group_values(N, K, group));
    const NormBuffer b[] = {{W, static_cast<uint64_t>(N) * static_cast<uint64_t>(K) * el, el, false},
                            {Q, static_cast<uint64_t>(w4_code_bytes(N, K)), 16, true},
                            {S, values * 2u, 16, true},
                            {Z, values, 16, true}};
    if ((st = check_norm_buffers(b, 4, dev.device)) != GEMM_OK) return st;
    W4QuantArgs a;
    a.W = W;
    a.Q = Q;
    a.S = S;
    a.Z = Z;
    a.N = N;
    a.K = K;
    a.type = type;
    a.stype = stype;
    a.group = group;
    a.trans = trans;
    a.stream = static_cast<cudaStream_t>(stream);
    return launch_w4_quantize(a);
}

static int run_linear_w4(const void *X, int type, const void *Q, const void *S, const uint8_t *Z, void *C, int64_t M,
                         int64_t N, int64_t K, int group, int relu, void *stream, int withhold, uint64_t timeout_cycles)
{
    int st = check_w4_args(N, K, group, type);
    if (st != GEMM_OK) return st;
    if ((st = check_sizes(M, N, K, relu)) != GEMM_OK) return st;
    if (M > GEMM_W4_MAX_ROWS) return reject(GEMM_ERR_INVALID_ARG, "M is above GEMM_W4_MAX_ROWS");
    if (M == 0 || N == 0) return GEMM_OK;
    if (C == nullptr || (K > 0 && (X == nullptr || Q == nullptr || S == nullptr)))
        return reject(GEMM_ERR_INVALID_ARG, "a buffer pointer is NULL");
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const uint64_t c_bytes = static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * 2u;
    if (K == 0) {
        // Empty sum: every output is R(+0) = +0.
        if ((st = check_device_buffer_fast(C, c_bytes, dev.device, 2)) != GEMM_OK) return st;
        if (cudaMemsetAsync(C, 0, c_bytes, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    const uint64_t values = static_cast<uint64_t>(w4_group_values(N, K, group));
    const NormBuffer b[] = {{X, static_cast<uint64_t>(M) * static_cast<uint64_t>(K) * 2u, 2, false},
                            {Q, static_cast<uint64_t>(w4_code_bytes(N, K)), 16, false},
                            {S, values * 2u, 16, false},
                            {Z, values, 16, false},
                            {C, c_bytes, 2, true}};
    if ((st = check_norm_buffers(b, 5, dev.device)) != GEMM_OK) return st;
    W4LinearArgs a;
    a.X = X;
    a.Q = Q;
    a.S = S;
    a.Z = Z;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    a.type = type;
    a.group = group;
    a.relu = relu;
    a.sm_count = dev.sm_count;
    a.device = dev.device;
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;
    a.withhold = withhold;
    a.timeout_cycles = timeout_cycles;
    a.stream = static_cast<cudaStream_t>(stream);
    if (group == 32) return launch_linear_w4_g32(a);
    return group == 64 ? launch_linear_w4_g64(a) : launch_linear_w4_g128(a);
}

extern "C" int linear_w4(const void *X, int type, const void *Q, const void *S, const uint8_t *Z, void *C, int64_t M,
                         int64_t N, int64_t K, int group, int relu, void *stream)
{
    return run_linear_w4(X, type, Q, S, Z, C, M, N, K, group, relu, stream, 0, 0);
}

static int w4_selftest_timeout(const void *X, int type, const void *Q, const void *S, const uint8_t *Z, void *C,
                               int64_t M, int64_t N, int64_t K, int group, uint64_t timeout_cycles, void *stream)
{
    if (timeout_cycles < (1ull << 16) || timeout_cycles > (1ull << 32))
        return reject(GEMM_ERR_INVALID_ARG, "timeout_cycles outside 2^16 .. 2^32");
    return run_linear_w4(X, type, Q, S, Z, C, M, N, K, group, 0, stream, 1, timeout_cycles);
}

extern "C" int linear_w4_selftest_timeout(const void *X, int type, const void *Q, const void *S, const uint8_t *Z,
                                          void *C, int64_t M, int64_t N, int64_t K, int group, uint64_t timeout_cycles,
                                          void *stream)
{
    if (M <= 32 || N == 0 || K == 0) return reject(GEMM_ERR_INVALID_ARG, "this hook takes more than 32 rows of X");
    return w4_selftest_timeout(X, type, Q, S, Z, C, M, N, K, group, timeout_cycles, stream);
}

extern "C" int linear_w4_few_selftest_timeout(const void *X, int type, const void *Q, const void *S, const uint8_t *Z,
                                              void *C, int64_t M, int64_t N, int64_t K, int group,
                                              uint64_t timeout_cycles, void *stream)
{
    if (check_sizes(M, N, K, 0) != GEMM_OK || M > 32 || !w4_by_tmem(M, N, K))
        return reject(GEMM_ERR_INVALID_ARG, "these sizes' kernel has no waits, or more than 32 rows of X");
    return w4_selftest_timeout(X, type, Q, S, Z, C, M, N, K, group, timeout_cycles, stream);
}

extern "C" int gemm_fp8_launch_info(int64_t M, int64_t N, int64_t K, int *grid_ctas, int *tiles)
{
    int st = check_sizes(M, N, K, 0);
    if (st != GEMM_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    return fp8_launch_info(M, N, dev, grid_ctas, tiles);
}

extern "C" int attention_fwd_f16(const void *Q, const void *K, const void *V, void *O, int64_t batch,
                                 int64_t heads, int64_t seq, int64_t dim, float sm_scale, int causal, void *stream)
{
    return attention_fwd_f16_queue(Q, K, V, O, batch, heads, seq, dim, sm_scale, causal, nullptr, stream);
}

extern "C" int attention_fwd_f16_queue(const void *Q, const void *K, const void *V, void *O, int64_t batch,
                                       int64_t heads, int64_t seq, int64_t dim, float sm_scale, int causal,
                                       unsigned int *queue, void *stream)
{
    if (batch < 0 || heads < 0 || seq < 0) return reject(GEMM_ERR_INVALID_ARG, "a size is negative");
    if (dim != 64 && dim != 128) return reject(GEMM_ERR_INVALID_ARG, "dim is not 64 or 128");
    if (causal != 0 && causal != 1) return reject(GEMM_ERR_INVALID_ARG, "causal is not 0 or 1");
    if (!std::isfinite(sm_scale)) return reject(GEMM_ERR_INVALID_ARG, "sm_scale is not finite");
    if (batch > 65535 || heads > 65535 || seq > INT32_MAX)
        return reject(GEMM_ERR_INVALID_ARG, "batch or heads above 65535, or seq above INT32_MAX");
    if (batch == 0 || heads == 0 || seq == 0) return GEMM_OK;
    DeviceInfo dev;
    int st = current_device_info(&dev);
    if (st != GEMM_OK) return st;
    const uint64_t bytes = static_cast<uint64_t>(batch) * static_cast<uint64_t>(heads) * static_cast<uint64_t>(seq) *
                           static_cast<uint64_t>(dim) * 2u;
    if ((st = check_device_buffer(Q, bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(K, bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(V, bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(O, bytes, dev.device)) != GEMM_OK) return st;
    if (ranges_overlap(O, bytes, Q, bytes) || ranges_overlap(O, bytes, K, bytes) || ranges_overlap(O, bytes, V, bytes))
        return reject(GEMM_ERR_INVALID_ARG, "O overlaps Q, K or V");
    if (causal && queue != nullptr) {
        const uint64_t qb = 2 * sizeof(unsigned int);
        if ((st = check_device_buffer(queue, qb, dev.device, 4)) != GEMM_OK) return st;
        if (ranges_overlap(queue, qb, O, bytes) || ranges_overlap(queue, qb, Q, bytes) ||
            ranges_overlap(queue, qb, K, bytes) || ranges_overlap(queue, qb, V, bytes))
            return reject(GEMM_ERR_INVALID_ARG, "queue overlaps Q, K, V or O");
    }
    AttnLaunchArgs a;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.batch = batch;
    a.heads = heads;
    a.seq = seq;
    a.dim = dim;
    a.sm_scale = sm_scale;
    a.causal = causal;
    a.dev = dev;
    a.stream = static_cast<cudaStream_t>(stream);
    a.status = status_word(dev.device);
    if (a.status == nullptr) return GEMM_ERR_CUDA;
    a.queue = causal ? queue : nullptr;
    return launch_attention(a);
}

extern "C" int gemm_f16_num_configs(void) { return kNumConfigs; }

extern "C" const char *gemm_f16_config_name(int config)
{
    int id = 0;
    bool allow_split = true;
    if (!parse_config(config, &id, &allow_split)) return nullptr;
    return kConfigs[id].name;
}

extern "C" int gemm_f16_config_layouts(int config)
{
    int id = 0;
    bool allow_split = true;
    if (!parse_config(config, &id, &allow_split))
        return reject(GEMM_ERR_INVALID_ARG, "unknown configuration id or flag");
    return kConfigs[id].all_layouts ? 0xF : 0x1;
}

extern "C" int gemm_f16_config_cluster_k(int config)
{
    int id = 0;
    bool allow_split = true;
    if (!parse_config(config, &id, &allow_split))
        return reject(GEMM_ERR_INVALID_ARG, "unknown configuration id or flag");
    return id == kClusterKConfig ? 1 : 0;
}

extern "C" int gemm_f16_auto_config(int64_t M, int64_t N, int64_t K)
{
    int st = check_sizes(M, N, K, 0);
    if (st != GEMM_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    const int picked = select_config(M, N, K, false, dev);
    const int cfg = picked & GEMM_F16_CONFIG_ID_MASK;
    if (cfg == kClusterKConfig) {
        // The cluster size resolved for this problem.
        int cluster = 1;
        ck_launch_info_config_6(M, N, K, ck_request_of(picked), dev, nullptr, &cluster, nullptr);
        return cfg | (cluster >= 2 ? GEMM_F16_KSPLIT(cluster) : GEMM_F16_NO_KSPLIT);
    }
    return picked;
}

extern "C" int gemm_f16_launch_info(int64_t M, int64_t N, int64_t K, int config, int *grid_ctas,
                                    int *cluster_size, int *tiles)
{
    int st = check_sizes(M, N, K, 0);
    if (st != GEMM_OK) return st;
    int id = 0, k_request = 0;
    bool split = true;
    if (!parse_config(config, &id, &split, &k_request))
        return reject(GEMM_ERR_INVALID_ARG, "unknown configuration id or flag");
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    int cfg = id, picked = 0;
    if (id == 0) {
        picked = select_config(M, N, K, false, dev);
        cfg = picked & GEMM_F16_CONFIG_ID_MASK;
        split = split && (picked & GEMM_F16_NO_SPLIT) == 0;
    }
    if (cfg == kClusterKConfig) {
        const int request = id == 0 ? ck_request_of(picked)
                            : k_request >= 2 ? k_request
                            : k_request == kKsplitNever ? 1 : 0;
        return ck_launch_info_config_6(M, N, K, request, dev, grid_ctas, cluster_size, tiles);
    }
    const int k_req = k_splits_for(k_request, cfg, M, N, K, dev);
    const bool tail = k_request == kKsplitTail;
    int grid = 0, cluster = 1, n_tiles = 0;
    if ((st = config_info(cfg, M, N, split && k_req <= 1 && !tail, dev, &grid, &cluster, &n_tiles)) != GEMM_OK)
        return st;
    const int64_t slots = config_slots(cfg, dev);
    const KPlan kp = plan_k_split(n_tiles, slots, (K + 63) / 64, k_req, tail);
    if (kp.ks.count > 1) {
        // Whole tiles, then K slices, on at most one CTA (cluster) per slot.
        const int64_t units = kp.units(n_tiles);
        grid = static_cast<int>((units < slots ? units : slots) * cluster);
    }
    if (grid_ctas) *grid_ctas = grid;
    if (cluster_size) *cluster_size = cluster;
    if (tiles) *tiles = n_tiles;
    return GEMM_OK;
}

namespace {

// Per device: the two streams the host-buffer entry point moves data on
// (uploads, downloads), created by its first call on that device.
struct CopyStreams {
    cudaStream_t in = nullptr, out = nullptr;
    int status = GEMM_ERR_CUDA;
};
CopyStreams g_copy_streams[kMaxDevices];
std::once_flag g_copy_once[kMaxDevices];

int copy_streams(int dev, CopyStreams **out)
{
    if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_CUDA;
    std::call_once(g_copy_once[dev], [dev]() {
        CopyStreams &c = g_copy_streams[dev];
        if (cudaStreamCreateWithFlags(&c.in, cudaStreamNonBlocking) == cudaSuccess &&
            cudaStreamCreateWithFlags(&c.out, cudaStreamNonBlocking) == cudaSuccess) {
            c.status = GEMM_OK;
        } else {
            cudaGetLastError();
        }
    });
    *out = &g_copy_streams[dev];
    return g_copy_streams[dev].status;
}

// Events of one call, destroyed once enqueued (they are released when the
// work they mark completes).
struct EventSet {
    cudaEvent_t ev[2 * kMaxFromHostPanels + 2] = {};
    int n = 0;
    bool make(int count)
    {
        for (n = 0; n < count; ++n) {
            if (cudaEventCreateWithFlags(&ev[n], cudaEventDisableTiming) != cudaSuccess) {
                cudaGetLastError();
                return false;
            }
        }
        return true;
    }
    ~EventSet()
    {
        for (int i = 0; i < n; ++i) cudaEventDestroy(ev[i]);
    }
};

}  // namespace

extern "C" int gemm_f16_from_host(const void *A_host, const void *B_host, void *C_host, void *A_dev, void *B_dev,
                                  void *C_dev, int64_t M, int64_t N, int64_t K, int relu, void *stream)
{
    int st = check_sizes(M, N, K, relu);
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    if (C_host == nullptr || (K > 0 && (A_host == nullptr || B_host == nullptr)))
        return reject(GEMM_ERR_INVALID_ARG, "a host buffer pointer is NULL");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t a_bytes = static_cast<size_t>(M) * static_cast<size_t>(K) * 2u;
    const size_t b_bytes = static_cast<size_t>(K) * static_cast<size_t>(N) * 2u;
    const size_t c_bytes = static_cast<size_t>(M) * static_cast<size_t>(N) * 2u;
    if (K == 0) {
        if ((st = gemm_f16(A_dev, B_dev, C_dev, M, N, K, relu, stream)) != GEMM_OK) return st;
        if (cudaMemcpyAsync(C_host, C_dev, c_bytes, cudaMemcpyDeviceToHost, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_OK;
    }
    // Validate the device side before anything is enqueued.
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != GEMM_OK) return st;
    if ((N % 8) != 0 || (K % 8) != 0)
        return reject(GEMM_ERR_ALIGNMENT, "a row pitch (leading dimension) is not a multiple of 8 elements");
    if ((st = check_device_buffer(A_dev, a_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(B_dev, b_bytes, dev.device)) != GEMM_OK) return st;
    if ((st = check_device_buffer(C_dev, c_bytes, dev.device)) != GEMM_OK) return st;
    if (ranges_overlap(C_dev, c_bytes, A_dev, a_bytes) || ranges_overlap(C_dev, c_bytes, B_dev, b_bytes))
        return reject(GEMM_ERR_INVALID_ARG, "C overlaps A or B");
    CopyStreams *cs = nullptr;
    if ((st = copy_streams(dev.device, &cs)) != GEMM_OK) return st;

    // Row panels of A and C (multiples of 256 rows, at least 1024 each, at
    // most kMaxFromHostPanels): B goes up first, then panel i of A; the GEMM
    // of panel i runs on `stream` once its rows are up; panel i of C comes
    // down while later panels are uploaded and computed.
    int64_t panels = M / 1024;
    if (panels < 1) panels = 1;
    if (panels > kMaxFromHostPanels) panels = kMaxFromHostPanels;
    const int64_t rows = ((M + panels - 1) / panels + 255) / 256 * 256;
    panels = (M + rows - 1) / rows;
    const int np = static_cast<int>(panels);
    EventSet evs;
    if (!evs.make(2 * np + 2)) return GEMM_ERR_CUDA;
    cudaEvent_t e_start = evs.ev[0], e_done = evs.ev[1];
    auto ea = [&](int i) { return evs.ev[2 + i]; };        // panel i of A is up
    auto ec = [&](int i) { return evs.ev[2 + np + i]; };   // panel i of C is computed
    auto fail = []() {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    };
    // The copy streams start after everything already enqueued on `stream`
    // (which may still use A_dev, B_dev or C_dev).
    if (cudaEventRecord(e_start, s) != cudaSuccess || cudaStreamWaitEvent(cs->in, e_start, 0) != cudaSuccess ||
        cudaStreamWaitEvent(cs->out, e_start, 0) != cudaSuccess)
        return fail();
    if (cudaMemcpyAsync(B_dev, B_host, b_bytes, cudaMemcpyHostToDevice, cs->in) != cudaSuccess) return fail();
    for (int i = 0; i < np; ++i) {
        const int64_t r0 = i * rows, mi = (M - r0 < rows) ? M - r0 : rows;
        const size_t off = static_cast<size_t>(r0) * static_cast<size_t>(K) * 2u;
        if (cudaMemcpyAsync(static_cast<char *>(A_dev) + off, static_cast<const char *>(A_host) + off,
                            static_cast<size_t>(mi) * static_cast<size_t>(K) * 2u, cudaMemcpyHostToDevice,
                            cs->in) != cudaSuccess ||
            cudaEventRecord(ea(i), cs->in) != cudaSuccess)
            return fail();
    }
    for (int i = 0; i < np; ++i) {
        const int64_t r0 = i * rows, mi = (M - r0 < rows) ? M - r0 : rows;
        if (cudaStreamWaitEvent(s, ea(i), 0) != cudaSuccess) return fail();
        st = gemm_f16(static_cast<const char *>(A_dev) + static_cast<size_t>(r0) * static_cast<size_t>(K) * 2u,
                      B_dev, static_cast<char *>(C_dev) + static_cast<size_t>(r0) * static_cast<size_t>(N) * 2u, mi,
                      N, K, relu, stream);
        if (st != GEMM_OK) return st;
        if (cudaEventRecord(ec(i), s) != cudaSuccess || cudaStreamWaitEvent(cs->out, ec(i), 0) != cudaSuccess)
            return fail();
        const size_t off = static_cast<size_t>(r0) * static_cast<size_t>(N) * 2u;
        if (cudaMemcpyAsync(static_cast<char *>(C_host) + off, static_cast<const char *>(C_dev) + off,
                            static_cast<size_t>(mi) * static_cast<size_t>(N) * 2u, cudaMemcpyDeviceToHost,
                            cs->out) != cudaSuccess)
            return fail();
    }
    // `stream` covers the downloads: synchronising it is enough to read C_host.
    if (cudaEventRecord(e_done, cs->out) != cudaSuccess || cudaStreamWaitEvent(s, e_done, 0) != cudaSuccess)
        return fail();
    return GEMM_OK;
}

extern "C" int gemm_f16_check(void *stream)
{
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    unsigned long long v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gemm_f16_status, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    if (v != 0) {
        t_last_timeout_record = v;
        const unsigned long long zero = 0;
        if (cudaMemcpyToSymbol(g_gemm_f16_status, &zero, sizeof(zero)) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        return GEMM_ERR_TIMEOUT;
    }
    return GEMM_OK;
}

extern "C" uint64_t gemm_f16_last_timeout_record(void) { return t_last_timeout_record; }

extern "C" const char *gemm_f16_last_error_detail(void) { return t_last_detail; }

extern "C" const char *gemm_f16_strerror(int status)
{
    switch (status) {
        case GEMM_OK: return "success";
        case GEMM_ERR_INVALID_ARG: return "invalid argument";
        case GEMM_ERR_ALIGNMENT: return "misaligned pointer, or a row pitch not a multiple of 8 elements";
        case GEMM_ERR_UNSUPPORTED_DEVICE: return "current device is not compute capability 10.3 (GB300)";
        case GEMM_ERR_LAUNCH: return "kernel launch failed";
        case GEMM_ERR_TIMEOUT: return "a kernel wait exceeded its limit; the output is incomplete";
        case GEMM_ERR_CUDA: return "CUDA runtime or driver call failed";
        default: return "unknown status";
    }
}

extern "C" int gemm_f16_version(void) { return GEMM_F16_VERSION; }
