// linear_w4_g128.cu -- linear_w4's kernels for scale groups of 128 columns.
#include "linear_w4_launch.cuh"

namespace gemm_sm103 {

int launch_linear_w4_g128(const W4LinearArgs &a)
{
    return a.type == GEMM_TYPE_F16 ? launch_w4<__half, 128>(a) : launch_w4<__nv_bfloat16, 128>(a);
}

}  // namespace gemm_sm103
