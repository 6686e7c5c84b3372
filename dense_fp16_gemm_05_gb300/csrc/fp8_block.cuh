// fp8_block.cuh -- E4M3 elements and the scale that a block of them shares, as
// the block-scaled FP8 products take them (rms_norm_fwd.cu, fp8_quantize.cu).
// With a = max |x| over the block:
//
//   fp32 scales         S = a / 448,                Q = e4m3(448 x / a)
//   power-of-two scales S = 2^e with the least e that keeps a / S <= 448,
//                       given as the E8M0 byte e + 127, Q = e4m3(x 2^-e)
//
// and S = 1 for a block of zeros.  A block that holds an infinity or a NaN gets
// a NaN scale and NaN codes, so that it does not vanish from a product.
#pragma once

#include <cstdint>
#include <type_traits>

#include "sm103_ptx.cuh"

namespace gemm_sm103 {

constexpr int kFp8Block = 128;   // columns that share a scale

// Two values to E4M3, nearest even, the first in the low byte; beyond 448 to 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t fp8_magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
// The largest of |m|, |x.x| and |x.y|, NaN if one of them is, in one instruction.
__device__ __forceinline__ float fp8_largest(float m, float2 x)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(x.x), "f"(x.y));
    return r;
}

// Scale of a block whose largest |x| has the bit pattern `amax` (NaN above
// infinity), and what its elements are converted with.
struct Fp8Block {
    float inv, rest;   // 448 / (a k) as the sum of two numbers, or 1 / S
    float k;           // a power of two
    bool pow2, near_limits;

    __device__ __forceinline__ Fp8Block(uint32_t amax, bool pow2_)
    {
        pow2 = pow2_;
        near_limits = false;
        k = 1.0f;
        rest = 0.0f;
        if (amax >= 0x7F800000u) {
            inv = __uint_as_float(0x7FC00000u);
        } else if (pow2) {
            inv = __uint_as_float((254u - byte_of(amax)) << 23);
        } else if (amax == 0u) {
            inv = 1.0f;
        } else {
            float a = __uint_as_float(amax);
            // The quotient and what it lacks stay clear of fp32's limits.
            near_limits = a < 0x1p-100f || a > 0x1p100f;
            if (near_limits) k = a < 1.0f ? 0x1p100f : 0x1p-100f;
            a *= k;
            inv = 448.0f / a;
            rest = fmaf(-inv, a, 448.0f) * inv * (1.0f / 448.0f);   // the remainder is exact
        }
    }

    // amax = 1.m 2^x against 448 = 1.75 2^8; anything below 2^-119 to the least byte.
    __device__ __forceinline__ static uint32_t byte_of(uint32_t amax)
    {
        if (amax == 0u) return 127u;
        const int b = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        return b < 0 ? 0u : static_cast<uint32_t>(b);
    }
    // The stored scale: fp32 bits, or the E8M0 byte.
    __device__ __forceinline__ static void store(void *S, int64_t at, uint32_t amax, bool pow2)
    {
        if (pow2) {
            static_cast<uint8_t *>(S)[at] = static_cast<uint8_t>(amax >= 0x7F800000u ? 255u : byte_of(amax));
        } else {
            float s = __uint_as_float(amax) / 448.0f;
            if (amax == 0u) s = 1.0f;
            if (amax >= 0x7F800000u) s = __uint_as_float(0x7FC00000u);
            static_cast<float *>(S)[at] = s;
        }
    }

    // Calls f(std::integral_constant<int, way>{}) for the way that the block's elements are
    // converted: decided once for all of them.
    template <class F>
    __device__ __forceinline__ void by_way(F f) const
    {
        if (pow2) f(std::integral_constant<int, 0>{});
        else if (!near_limits) f(std::integral_constant<int, 1>{});
        else f(std::integral_constant<int, 2>{});
    }

    // Two elements' codes.  448 x / a is x inv + x rest with one rounding of note: a
    // quotient half way between two codes, which 16-bit elements often give, stays there
    // (the product with a rounded 448 / a alone put one in thirteen of them on either side).
    template <int kWay>
    __device__ __forceinline__ uint32_t codes(float2 x) const
    {
        const float2 inv2 = make_float2(inv, inv);
        if constexpr (kWay == 2) x = mul_f32x2(x, make_float2(k, k));
        float2 q;
        if constexpr (kWay == 0) q = mul_f32x2(x, inv2);
        else q = fma_f32x2(x, inv2, mul_f32x2(x, make_float2(rest, rest)));
        return e4m3x2(q.x, q.y);
    }
};

}  // namespace gemm_sm103
