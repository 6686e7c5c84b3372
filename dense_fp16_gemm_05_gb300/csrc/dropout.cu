// dropout.cu -- dropout whose mask is made on the fly, forward and backward:
//
//   y = r + x / (1 - p) for a kept element, r (0 without a residual) for another
//
// Element e is kept if word e % 4 of Philox4x32-10 (J. K. Salmon, M. A. Moraes,
// R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011)
// with counter (e / 4, offset), 64 bits each, and key seed is at least
// floor(p 2^32).  The gradient is the same call on dY without a residual: the
// mask is made again from seed and offset and never stored.  Ten rounds for four
// elements are some 19 instructions for each beside 4 to 6 bytes: with a residual the
// pass is bound by memory (16384 x 4096 fp16 58 us, 6.9 TB/s), without one by its
// instructions, most of all those that multiply whole numbers (54 us, 4.9 TB/s, their
// pipe busy for 77 % of the cycles and issue slots for 65 %).
#include "feed_forward_launch.cuh"
#include "layer_norm.cuh"

namespace {

using namespace gemm_sm103;

template <class T>
struct DropoutParams {
    const T *X, *R;   // R NULL: none
    T *Y;
    int64_t n;
    uint32_t key[20];   // the ten rounds' keys
    uint32_t threshold;
    float scale;
    uint64_t offset;
    const uint64_t *offset_ptr;   // NULL: offset
};

struct Words {
    uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t index, uint64_t offset, const uint32_t (&key)[20])
{
    uint32_t c0 = static_cast<uint32_t>(index), c1 = static_cast<uint32_t>(index >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ key[2 * i];
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ key[2 * i + 1];
        c1 = static_cast<uint32_t>(p1);
        c3 = static_cast<uint32_t>(p0);
    }
    return {{c0, c1, c2, c3}};
}

// Packs of a thread, a block's threads apart: the keys and the offset's products are
// the same for all of them.  Two, in registers that let eight blocks run on an SM: one
// pack 73 us and 65 us (with and without a residual), four on five blocks 57 and 58.
constexpr int kPacks = 2;

// V elements at a time: 16 bytes, or the four of one counter one by one.
template <class T, int V, bool kPacked>
__global__ void __launch_bounds__(256, 8) dropout_kernel(DropoutParams<T> p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (256 * kPacks) + threadIdx.x) * V;
    const uint64_t offset = p.offset_ptr ? __ldg(p.offset_ptr) : p.offset;
    LnPack<T, V> x[kPacks], r[kPacks];
    auto whole = [&](int64_t e) { return kPacked && e + V <= p.n; };
#pragma unroll
    for (int u = 0; u < kPacks; ++u) {
        const int64_t e = first + u * (256 * V);
        // Y may be X or R, so not through the read-only path.
        if (whole(e)) {
            x[u].load_shared(p.X + e);
            if (p.R) r[u].load_shared(p.R + e);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (e + j >= p.n) continue;
                x[u].e[j] = p.X[e + j];
                if (p.R) r[u].e[j] = p.R[e + j];
            }
        }
    }
    const float2 scale = make_float2(p.scale, p.scale);
#pragma unroll
    for (int u = 0; u < kPacks; ++u) {
        const int64_t e = first + u * (256 * V);
        if (e >= p.n) continue;
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const Words words = philox(static_cast<uint64_t>(e / 4 + i), offset, p.key);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                // A dropped element's value does not matter, infinite or not.
                float2 v = mul_f32x2(x[u].pair(2 * i + j / 2), scale);
                v.x = words.w[j] >= p.threshold ? v.x : 0.0f;
                v.y = words.w[j + 1] >= p.threshold ? v.y : 0.0f;
                if (p.R) v = add_f32x2(r[u].pair(2 * i + j / 2), v);
                x[u].set_pair(2 * i + j / 2, v);
            }
        }
        if (whole(e)) {
            x[u].store(p.Y + e);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e + j < p.n) p.Y[e + j] = x[u].e[j];
        }
    }
}

template <class T>
int dropout(const DropoutArgs &a)
{
    DropoutParams<T> p{};
    p.X = static_cast<const T *>(a.X);
    p.R = static_cast<const T *>(a.R);
    p.Y = static_cast<T *>(a.Y);
    p.n = a.n;
    uint32_t k0 = static_cast<uint32_t>(a.seed), k1 = static_cast<uint32_t>(a.seed >> 32);
    for (int i = 0; i < 10; ++i) {
        p.key[2 * i] = k0;
        p.key[2 * i + 1] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    p.threshold = static_cast<uint32_t>(a.p * 4294967296.0);   // p < 1
    p.scale = static_cast<float>(1.0 / (1.0 - a.p));
    p.offset = a.offset;
    p.offset_ptr = a.offset_ptr;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.R) |
                           reinterpret_cast<uintptr_t>(a.Y);
    constexpr int V = 16 / sizeof(T);
    const bool packed = (bits & 15u) == 0;
    const int64_t per = 256 * kPacks * (packed ? V : 4);
    const dim3 grid(static_cast<unsigned>((a.n + per - 1) / per), 1, 1);
    return packed ? ln_launch(dropout_kernel<T, V, true>, grid, 256, a.stream, p)
                  : ln_launch(dropout_kernel<T, 4, false>, grid, 256, a.stream, p);
}

}  // namespace

namespace gemm_sm103 {

int launch_dropout(const DropoutArgs &a)
{
    if (a.type == GEMM_TYPE_F32) return dropout<float>(a);
    if (a.type == GEMM_TYPE_F16) return dropout<__half>(a);
    return dropout<__nv_bfloat16>(a);
}

}  // namespace gemm_sm103
