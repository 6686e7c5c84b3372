// dropout.cu -- dropout whose mask is made on the fly, forward and backward:
//
//   y = r + x / (1 - p) for a kept element, r (0 without a residual) for another
//
// Element e is kept if word e % 4 of Philox4x32-10 (J. K. Salmon, M. A. Moraes,
// R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011)
// with counter (e / 4, offset), 64 bits each, and key seed is at least
// floor(p 2^32).  The gradient is the same call on dY without a residual: the
// mask is made again from seed and offset and never stored.
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

// V elements of a thread at a time: 16 bytes, or the four of one counter one by one.
template <class T, int V, bool kPacked>
__global__ void __launch_bounds__(256) dropout_kernel(DropoutParams<T> p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
    if (e >= p.n) return;
    const bool full = e + V <= p.n;
    LnPack<T, V> x, r;
    if (kPacked && full) {
        // Y may be X or R, so not through the read-only path.
        x.load_shared(p.X + e);
        if (p.R) r.load_shared(p.R + e);
    } else {
        x.fill(0.0f);
        r.fill(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (e + j >= p.n) continue;
            x.e[j] = p.X[e + j];
            if (p.R) r.e[j] = p.R[e + j];
        }
    }
    const uint64_t offset = p.offset_ptr ? __ldg(p.offset_ptr) : p.offset;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const Words words = philox(static_cast<uint64_t>(e / 4 + i), offset, p.key);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // A dropped element's value does not matter, infinite or not.
            const float v = words.w[j] >= p.threshold ? x[4 * i + j] * p.scale : 0.0f;
            x.e[4 * i + j] = ln_round<T>(p.R ? r[4 * i + j] + v : v);
        }
    }
    if (kPacked && full) {
        x.store(p.Y + e);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e + j < p.n) p.Y[e + j] = x.e[j];
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
    const int64_t per = 256 * (packed ? V : 4);
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
