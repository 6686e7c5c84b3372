// feed_forward_launch.cuh -- arguments of the operators around a feed-forward
// block that are not norms: FP8 quantisation (fp8_quantize.cu), dropout
// (dropout.cu) and products with 4-bit weights (w4_quantize.cu, linear_w4_g*.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gemm_sm103 {

struct Fp8QuantArgs {
    const void *X = nullptr;
    void *Q = nullptr, *S = nullptr;
    int64_t rows = 0, K = 0;
    int type = 0, block_rows = 1, pow2 = 0;
    cudaStream_t stream = nullptr;
};
int launch_fp8_quantize(const Fp8QuantArgs &a);

struct DropoutArgs {
    const void *X = nullptr, *R = nullptr;
    void *Y = nullptr;
    int64_t n = 0;
    int type = 0;
    double p = 0.0;
    uint64_t seed = 0, offset = 0;
    const uint64_t *offset_ptr = nullptr;   // given: read by the kernel in place of `offset`
    cudaStream_t stream = nullptr;
};
int launch_dropout(const DropoutArgs &a);

// Packed 4-bit weights (N, K): tiles of 16 rows x 64 columns in 512 bytes; one
// scale (and zero point) per row and `group` columns, 16 rows side by side.
constexpr int kW4Rows = 16, kW4Cols = 64, kW4TileBytes = 512;
inline int64_t w4_strips(int64_t N) { return (N + kW4Rows - 1) / kW4Rows; }
inline int64_t w4_code_bytes(int64_t N, int64_t K)
{
    return w4_strips(N) * ((K + kW4Cols - 1) / kW4Cols) * kW4TileBytes;
}
inline int64_t w4_group_values(int64_t N, int64_t K, int group)
{
    return w4_strips(N) * ((K + group - 1) / group) * kW4Rows;
}

struct W4QuantArgs {
    const void *W = nullptr;
    void *Q = nullptr, *S = nullptr;
    uint8_t *Z = nullptr;   // NULL: symmetric
    int64_t N = 0, K = 0;
    int type = 0, stype = 0, group = 0, trans = 0;
    cudaStream_t stream = nullptr;
};
int launch_w4_quantize(const W4QuantArgs &a);

// Which products go through tensor memory (both sides' times: linear_w4_launch.cuh).
inline bool w4_by_tmem(int64_t M, int64_t N, int64_t K) { return M > 32 || (M > 16 && K % 8 == 0 && N * K >= 1 << 24); }

struct W4LinearArgs {
    const void *X = nullptr, *Q = nullptr, *S = nullptr;
    const uint8_t *Z = nullptr;
    void *C = nullptr;
    int64_t M = 0, N = 0, K = 0;
    int type = 0, group = 0, relu = 0;
    int sm_count = 0, device = 0;
    cudaStream_t stream = nullptr;
    unsigned long long *status = nullptr;       // device status word
    int withhold = 0;                           // test hook (linear_w4_selftest_timeout, ..._few_...)
    uint64_t timeout_cycles = 0;                // 0: the normal budget
};
// One scale group width each.
int launch_linear_w4_g32(const W4LinearArgs &a);
int launch_linear_w4_g64(const W4LinearArgs &a);
int launch_linear_w4_g128(const W4LinearArgs &a);

}  // namespace gemm_sm103
