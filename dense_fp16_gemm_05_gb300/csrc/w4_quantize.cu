// w4_quantize.cu -- a weight to 4 bits with a 16-bit scale, and optionally a zero
// point, per row and group of 32, 64 or 128 columns, in linear_w4's layout:
//
//   symmetric    s = max|w| / 7 rounded to the scales' type,
//                q = 8 + w / s rounded to nearest even, kept in 0 .. 15
//   zero points  s = (max(w, 0) - min(w, 0)) / 15 rounded, z = -min(w, 0) / s
//                rounded and kept in 0 .. 15, q = z + w / s rounded, kept in 0 .. 15
//
// A group of zeros (or of values whose scale rounds to zero) has s = 0; a group
// that holds an infinity or a NaN has a NaN scale; scales beyond the type's
// largest number are that number.  A weight is quantised once, so this kernel is
// plain: a block takes 16 rows x 128 columns through shared memory.
#include "feed_forward_launch.cuh"
#include "layer_norm.cuh"

namespace {

using namespace gemm_sm103;

template <class T, class S>
struct W4QuantParams {
    const T *W;
    uint32_t *Q;   // words
    S *scale;
    uint8_t *Z;
    int64_t N, K;
    int64_t k_tiles, groups;
    int32_t group, trans;
};

template <class S>
__device__ __forceinline__ float w4_largest();
template <>
__device__ __forceinline__ float w4_largest<__half>() { return 65504.0f; }
template <>
__device__ __forceinline__ float w4_largest<__nv_bfloat16>() { return 3.3895314e38f; }

template <class T, class S>
__global__ void __launch_bounds__(128) w4_quantize_kernel(W4QuantParams<T, S> p)
{
    __shared__ float w[16][129];
    __shared__ uint8_t code[16][128];
    griddep_wait();
    griddep_launch_dependents();
    const int t = static_cast<int>(threadIdx.x);
    const int64_t units = (p.k_tiles + 1) / 2;   // of 128 columns
    const int64_t strip = blockIdx.x / units, unit = blockIdx.x % units;
    const int64_t n0 = strip * kW4Rows, k0 = unit * 128;
    for (int i = t; i < 16 * 128; i += 128) {
        // Neighbouring threads read neighbouring elements.
        const int r = p.trans ? i % 16 : i / 128, c = p.trans ? i / 16 : i % 128;
        const int64_t n = n0 + r, k = k0 + c;
        w[r][c] = n < p.N && k < p.K ? ln_float(p.W[p.trans ? k * p.N + n : n * p.K + k]) : 0.0f;
    }
    __syncthreads();
    // Eight threads of a row, 16 columns each; a group belongs to group / 16 of them.
    const int r = t / 8, c0 = t % 8 * 16;
    float lo = 0.0f, hi = 0.0f;
    uint32_t top = 0;
    for (int i = 0; i < 16; ++i) {
        const float v = w[r][c0 + i];
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
        top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);
    }
    for (int o = 1; o < p.group / 16; o *= 2) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    // The halves' difference: the whole one may be beyond fp32.
    float s = p.Z ? (hi * (1.0f / 16.0f) - lo * (1.0f / 16.0f)) * (16.0f / 15.0f) : __uint_as_float(top) / 7.0f;
    const S stored = ln_round<S>(top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fminf(s, w4_largest<S>()));
    s = ln_float(stored);
    const float z = p.Z ? (s > 0.0f ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 0.0f) : 8.0f;
    for (int i = 0; i < 16; ++i) {
        const float v = s > 0.0f ? rintf(w[r][c0 + i] / s) : 0.0f;
        const bool in = n0 + r < p.N && k0 + c0 + i < p.K;
        code[r][c0 + i] = in ? static_cast<uint8_t>(fminf(fmaxf(v + z, 0.0f), 15.0f)) : uint8_t{0};
    }
    if (c0 % p.group == 0 && k0 + c0 < p.K) {
        const int64_t at = (strip * p.groups + (k0 + c0) / p.group) * kW4Rows + r;
        const bool in = n0 + r < p.N;
        p.scale[at] = in ? stored : ln_round<S>(0.0f);
        if (p.Z) p.Z[at] = in ? static_cast<uint8_t>(z) : uint8_t{0};
    }
    __syncthreads();
    // Word `t` of either tile: lane t / 4 of the product, its word j.
    const int lane = t / 4, j = t % 4, g = lane / 4, c = 32 * (j / 2) + 8 * (lane % 4) + 4 * (j % 2);
    for (int h = 0; h < 2; ++h) {
        const int64_t tile = 2 * unit + h;
        if (tile >= p.k_tiles) continue;
        uint32_t word = 0;
        for (int nib = 0; nib < 8; ++nib)
            word |= static_cast<uint32_t>(code[g + 8 * (nib & 1)][64 * h + c + 2 * (nib >> 1 & 1) + (nib >> 2)]) << (4 * nib);
        p.Q[(strip * p.k_tiles + tile) * (kW4TileBytes / 4) + t] = word;
    }
}

template <class T, class S>
int quantize(const W4QuantArgs &a)
{
    W4QuantParams<T, S> p{};
    p.W = static_cast<const T *>(a.W);
    p.Q = static_cast<uint32_t *>(a.Q);
    p.scale = static_cast<S *>(a.S);
    p.Z = a.Z;
    p.N = a.N;
    p.K = a.K;
    p.k_tiles = (a.K + kW4Cols - 1) / kW4Cols;
    p.groups = (a.K + a.group - 1) / a.group;
    p.group = a.group;
    p.trans = a.trans;
    const int64_t blocks = w4_strips(a.N) * ((p.k_tiles + 1) / 2);
    return ln_launch(w4_quantize_kernel<T, S>, dim3(static_cast<unsigned>(blocks), 1, 1), 128, a.stream, p);
}

template <class T>
int quantize(const W4QuantArgs &a)
{
    return a.stype == GEMM_TYPE_F16 ? quantize<T, __half>(a) : quantize<T, __nv_bfloat16>(a);
}

}  // namespace

namespace gemm_sm103 {

int launch_w4_quantize(const W4QuantArgs &a)
{
    if (a.type == GEMM_TYPE_F32) return quantize<float>(a);
    if (a.type == GEMM_TYPE_F16) return quantize<__half>(a);
    return quantize<__nv_bfloat16>(a);
}

}  // namespace gemm_sm103
