// linear_w4_launch.cuh -- which kernel takes a product with 4-bit weights.
#pragma once

#include "linear_w4_kernel.cuh"
#include "linear_w4_tmem.cuh"

namespace gemm_sm103 {

// Calls of one scale group width (linear_w4_g32.cu, ...: a translation unit each).
template <class T, int G>
int launch_w4(const W4LinearArgs &a)
{
    W4Params<T> p{};
    p.X = static_cast<const T *>(a.X);
    p.Q = static_cast<const uint8_t *>(a.Q);
    p.S = static_cast<const uint8_t *>(a.S);
    p.Z = a.Z;
    p.C = static_cast<T *>(a.C);
    p.M = static_cast<int32_t>(a.M);
    p.N = a.N;
    p.K = a.K;
    p.strips = static_cast<int32_t>(w4_strips(a.N));
    p.k_tiles = static_cast<int32_t>((a.K + kW4Cols - 1) / kW4Cols);
    p.groups = static_cast<int32_t>((a.K + G - 1) / G);
    p.units = (p.k_tiles + 1) / 2;
    p.relu = a.relu;
    p.vec = (reinterpret_cast<uintptr_t>(p.X) & 15u) == 0 && p.K % 8 == 0;
    // By mma.sync, 8 rows of X to an instruction, or from tensor memory, whose MMAs take up
    // to 64 in the time of 8: 64 x 8192 x 8192 39 and 26 us, 40 x 4096 x 4096 28 and 11.  Up
    // to 32 rows only if the weight is large and X's rows can lie on the 16-byte grid
    // (32 x 8192 x 8192 23.6 and 22.8 us, 24 x 4096 x 4096 10.3 and 9.4, 32 x 4096 x 11008 29.0
    // and 17.2, but 24 x 1024 x 8192 8.7 and 9.8, 24 x 2048 x 4096 7.5 and 8.7, 32 x 16383 x 8191
    // 53.5 and 62.7), up to 16 not at all (16 x 8192 x 8192 14.5 and 16.8).  By K and not by X's
    // address, so that equal values give equal bits wherever X lies: one element off the grid
    // 32 x 16384 x 8192 takes 54 and 64 us, 32 x 4096 x 11008 33 and 21.
    if (p.M <= 8) return launch_w4_kernel<T, 1, G>(p, a);
    if (p.M <= 16) return launch_w4_kernel<T, 2, G>(p, a);
    if (p.M > 32) return launch_w4_tmem<T, 64, G>(p, a);
    return w4_by_tmem(p.M, p.N, p.K) ? launch_w4_tmem<T, 32, G>(p, a) : launch_w4_kernel<T, 4, G>(p, a);
}

}  // namespace gemm_sm103
