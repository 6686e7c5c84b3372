// rms_norm.cuh -- arguments of the RMS norm kernels (rms_norm_fwd.cu,
// rms_norm_bwd.cu), whose pieces they share with layer norm's.
#pragma once

#include "layer_norm.cuh"

namespace gemm_sm103 {

struct RmsNormArgs {
    const void *X = nullptr, *R = nullptr, *gamma = nullptr;
    void *Y = nullptr, *H = nullptr;            // Y: type xtype (NULL with Q)
    void *Q = nullptr, *S = nullptr;            // FP8 output: codes and scales
    float *rstd = nullptr;                      // written forward, read backward
    const void *dY = nullptr, *dH = nullptr;    // backward; X is the kept stream there
    void *dX = nullptr, *dgamma = nullptr;
    float *workspace = nullptr;                 // parts x dim floats (backward)
    int64_t rows = 0, dim = 0;
    float eps = 0.0f;
    int xtype = 0, wtype = 0, pow2 = 0;
    int sm_count = 0, device = 0;
    cudaStream_t stream = nullptr;
    unsigned long long *status = nullptr;       // device status word
    int withhold = 0;                           // test hook (rms_norm_bwd_selftest_timeout)
    uint64_t timeout_cycles = 0;                // 0: the normal budget
};

int launch_rms_norm_fwd(const RmsNormArgs &a);
int launch_rms_norm_bwd(const RmsNormArgs &a);

}  // namespace gemm_sm103
