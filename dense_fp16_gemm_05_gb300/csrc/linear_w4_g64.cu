// linear_w4_g64.cu -- linear_w4's kernels for scale groups of 64 columns.
#include "linear_w4_launch.cuh"

namespace gemm_sm103 {

int launch_linear_w4_g64(const W4LinearArgs &a)
{
    return a.type == GEMM_TYPE_F16 ? launch_w4<__half, 64>(a) : launch_w4<__nv_bfloat16, 64>(a);
}

}  // namespace gemm_sm103
