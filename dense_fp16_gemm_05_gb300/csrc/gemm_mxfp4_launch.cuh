// gemm_mxfp4_launch.cuh -- internal interface between the C ABI (gemm_f16.cu)
// and the 4-bit microscaled kernels (gemm_mxfp4.cu, mxfp4_quantize.cu).
#pragma once

#include "gemm_launch.cuh"

namespace gemm_sm103 {

constexpr int64_t kMx4Block = 32;        // elements per scale
constexpr int64_t kMx4TileRows = 128;    // rows of a scale tile
constexpr int64_t kMx4TileBytes = 512;   // 128 rows x 4 blocks

// Bytes of the packed form of a (rows, K) matrix.
inline int64_t mx4_row_bytes(int64_t K) { return (K + kMx4Block - 1) / kMx4Block * (kMx4Block / 2); }
inline int64_t mx4_k_tiles(int64_t K) { return (K + 4 * kMx4Block - 1) / (4 * kMx4Block); }
inline int64_t mx4_row_tiles(int64_t rows) { return (rows + kMx4TileRows - 1) / kMx4TileRows; }
inline uint64_t mx4_code_bytes(int64_t rows, int64_t K)
{
    return static_cast<uint64_t>(rows) * static_cast<uint64_t>(mx4_row_bytes(K));
}
inline uint64_t mx4_scale_bytes(int64_t rows, int64_t K)
{
    return static_cast<uint64_t>(mx4_row_tiles(rows)) * static_cast<uint64_t>(mx4_k_tiles(K)) * kMx4TileBytes;
}

// Codes of a (rows, K) matrix: rows of ceil(K/2) bytes, 16 ceil(K/32) bytes
// apart, boxes of 128 bytes x box_rows with 128-byte swizzle (gemm_f16.cu).
int encode_codes_u4(CUtensorMap *map, const void *ptr, int64_t rows, int64_t K, uint32_t box_rows);
// Scale tiles of a (rows, K) matrix: 128 words x tiles along K x row blocks,
// boxes of one tile's words x box_k x box_rows (gemm_f16.cu).
int encode_scale_tiles(CUtensorMap *map, const void *ptr, int64_t rows, int64_t K, uint32_t box_k, uint32_t box_rows);

// Everything one launch of the 4-bit GEMM needs, already validated by the C ABI.
struct Mx4LaunchArgs {
    const void *A = nullptr;      // (M,K) E2M1 codes
    const uint8_t *SA = nullptr;  // scale tiles
    const void *W = nullptr;      // (N,K) E2M1 codes
    const uint8_t *SW = nullptr;  // scale tiles
    void *C = nullptr;            // (M,N) fp16
    int64_t M = 0, N = 0, K = 0;
    int relu = 1;
    DeviceInfo dev;
    cudaStream_t stream = nullptr;
    unsigned long long *status = nullptr;
    int withhold = 0;              // test hook: loads that are not issued (Mx4Params)
    uint64_t timeout_cycles = 0;   // 0: the normal budget
};

int launch_mxfp4(const Mx4LaunchArgs &a);

// X (rows, K), or (K, rows) if trans, of type `type` -> codes, scale tiles and
// (V not NULL) the values they stand for, (rows, K) of X's type.
struct Mx4QuantArgs {
    const void *X = nullptr;
    uint8_t *Q = nullptr;
    uint8_t *S = nullptr;
    void *V = nullptr;
    int64_t rows = 0, K = 0;
    int type = 0, trans = 0;
    int sm_count = 0;
    cudaStream_t stream = nullptr;
};

int launch_mxfp4_quantize(const Mx4QuantArgs &a);

}  // namespace gemm_sm103
