// layer_norm_fwd.cu -- layer norm over the last dimension:
//
//   mean = sum x / dim,  rstd = 1 / sqrt(sum (x - mean)^2 / dim + eps),
//   y = (x - mean) rstd gamma + beta,
//
// sums in fp32, the second one over deviations of the row that is still in
// registers (not sum x^2 - mean^2, which cancels).  The mean is the quotient
// correctly rounded: the product with 1 / dim is one step off for a quarter of
// all sums, which rstd magnifies in rows of nearly equal elements (57600
// everywhere, dim 1000, eps 1e-5: y = -0.78 instead of 0).  Bound by memory: X is
// read once and Y written once.  A row belongs to a warp or to one block, chosen
// so that a thread holds at most 32 elements; longer rows are read again from L2.
#include "layer_norm.cuh"

#include <type_traits>

namespace {

using namespace gemm_sm103;

template <class T, class W>
struct FwdParams {
    const T *X;
    const W *gamma;   // NULL: ones
    const W *beta;    // NULL: zeros
    T *Y;
    float *mean, *rstd;   // NULL: not kept
    int64_t rows;
    int32_t dim;
    float n, inv_dim, eps;   // n = dim
};

// Threads of a block (its bound, where the launch chooses).
__host__ __device__ constexpr int fwd_threads(int tpr) { return tpr < 0 ? -tpr : (tpr < 128 ? 128 : tpr); }

// Blocks per SM that the registers are held to, where the compiler's own choice
// is one block too few (4096 x 16384 fp32: 108 us, and 80 us so); 0: its choice.
__host__ __device__ constexpr int fwd_blocks(int tpr, int per)
{
    if (tpr == 512 || tpr == -512) return per > 8 ? 2 : 0;
    return tpr == -1024 && per == 8 ? 2 : 0;
}

// tpr threads per row, NV packs of V elements per thread, pack i of thread t at
// element (i tpr + t) V.
// kInner: every pack but a thread's last lies inside the row whatever the thread.
template <class T, class W, int V, int NV, int TPR, bool kInner, bool kGamma, bool kBeta>
__global__ void __launch_bounds__(fwd_threads(TPR), fwd_blocks(TPR, V * NV)) layer_norm_fwd_kernel(FwdParams<T, W> p)
{
    constexpr int R = TPR > 0 ? fwd_threads(TPR) / TPR : 1;   // rows of a block
    __shared__ float sh[2][ln_warps(TPR)];
    griddep_wait();   // X may come from the kernel just before
    griddep_launch_dependents();
    const int tpr = ln_threads<TPR>();
    const int t = TPR > 0 ? static_cast<int>(threadIdx.x) % tpr : static_cast<int>(threadIdx.x);
    int64_t row = static_cast<int64_t>(blockIdx.x) * R + (R > 1 ? static_cast<int>(threadIdx.x) / tpr : 0);
    // Lanes without a row take the last one along, for the sake of the shuffles.
    const bool in = row < p.rows;
    if (!in) row = p.rows - 1;
    const T *x = p.X + row * p.dim;
    auto inside = [&](int i) { return (kInner && i < NV - 1) || (i * tpr + t) * V < p.dim; };
    // On pairs, two fp32 operations per instruction: element by element the
    // narrow variants are bound by instructions.
    constexpr int P = V * NV / 2;
    float2 x2[P];
    {
        LnPack<T, V> px[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (inside(i)) px[i].load(x + (i * tpr + t) * V);
            else px[i].fill(0.0f);
        }
#pragma unroll
        for (int m = 0; m < P; ++m) x2[m] = ln_pair_of(px, m);
    }
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int m = 0; m < P; ++m) s = add_f32x2(s, x2[m]);
    const float mean = ln_quotient(ln_row_sum<TPR>(s.x + s.y, sh[0]), p.n, p.inv_dim);
    const float2 neg_mean = make_float2(-mean, -mean);
    s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int m = 0; m < P; ++m) {
        x2[m] = add_f32x2(x2[m], neg_mean);
        // A pair of packs one of which may lie outside the row (V = 1), or a pack.
        const int i0 = 2 * m / V, i1 = (2 * m + 1) / V;
        float2 d = x2[m];
        if (!inside(i0)) d.x = 0.0f;
        if (!inside(i1)) d.y = 0.0f;
        s = fma_f32x2(d, d, s);
    }
    const float var = ln_row_sum<TPR>(s.x + s.y, sh[1]) * p.inv_dim;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (!in) return;
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    // The weights pack by pack: all of a thread's 32 at once cost 24 registers
    // more and with them a block per SM (16384 x 4096 fp16: 46 us against 40 us).
    T *y = p.Y + row * p.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!inside(i)) continue;
        const int k = (i * tpr + t) * V;
        LnPack<W, V> g, b;
        if constexpr (kGamma) g.load(p.gamma + k);
        if constexpr (kBeta) b.load(p.beta + k);
        LnPack<T, V> out;
        if constexpr (V == 1) {
            float v = ln_half(x2[i / 2], i) * rstd;
            if constexpr (kGamma && kBeta) v = fmaf(v, g[0], b[0]);
            else if constexpr (kGamma) v *= g[0];
            else if constexpr (kBeta) v += b[0];
            out.e[0] = ln_round<T>(v);
        } else {
            const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                float2 v = mul_f32x2(x2[i * (V / 2) + j], rstd2);
                if constexpr (kGamma && kBeta) v = fma_f32x2(v, g.pair(j), b.pair(j));
                else if constexpr (kGamma) v = mul_f32x2(v, g.pair(j));
                else if constexpr (kBeta) v = add_f32x2(v, b.pair(j));
                out.e[2 * j] = ln_round<T>(v.x);
                out.e[2 * j + 1] = ln_round<T>(v.y);
            }
        }
        out.store(y + k);
    }
}

// Rows longer than a block holds: three passes over the row.
template <class T, class W>
__global__ void __launch_bounds__(1024) layer_norm_fwd_long(FwdParams<T, W> p)
{
    __shared__ float sh[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = p.X + row * p.dim;
    float s = 0.0f;
    for (int64_t k = threadIdx.x; k < p.dim; k += 1024) s += ln_float(x[k]);
    const float mean = ln_quotient(ln_row_sum<1024>(s, sh[0]), p.n, p.inv_dim);
    s = 0.0f;
    for (int64_t k = threadIdx.x; k < p.dim; k += 1024) {
        const float d = ln_float(x[k]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(ln_row_sum<1024>(s, sh[1]) * p.inv_dim + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    T *y = p.Y + row * p.dim;
    for (int64_t k = threadIdx.x; k < p.dim; k += 1024) {
        const float g = p.gamma ? ln_float(p.gamma[k]) : 1.0f, b = p.beta ? ln_float(p.beta[k]) : 0.0f;
        y[k] = ln_round<T>(fmaf((ln_float(x[k]) - mean) * rstd, g, b));
    }
}

template <class T, class W, int V, int NV, int TPR>
int launch_one(const FwdParams<T, W> &p, cudaStream_t stream)
{
    // Threads: those of the template, or the whole warps that NV packs each need.
    const int packs = (p.dim + V - 1) / V;
    const int BT = TPR > 0 ? fwd_threads(TPR) : ((packs + NV - 1) / NV + 31) / 32 * 32;
    constexpr int R = TPR > 0 ? fwd_threads(TPR) / TPR : 1;
    // The usual case, both weights, has its own kernel: a branch on each pointer
    // at every element is a tenth of the narrow variants' instructions.
    const dim3 grid(static_cast<unsigned>((p.rows + R - 1) / R), 1, 1);
    auto launch = [&](auto inner) {
        constexpr bool I = decltype(inner)::value;
        if (p.gamma && p.beta) return ln_launch(layer_norm_fwd_kernel<T, W, V, NV, TPR, I, true, true>, grid, BT, stream, p);
        if (p.gamma) return ln_launch(layer_norm_fwd_kernel<T, W, V, NV, TPR, I, true, false>, grid, BT, stream, p);
        if (p.beta) return ln_launch(layer_norm_fwd_kernel<T, W, V, NV, TPR, I, false, true>, grid, BT, stream, p);
        return ln_launch(layer_norm_fwd_kernel<T, W, V, NV, TPR, I, false, false>, grid, BT, stream, p);
    };
    if constexpr (V <= 2 && TPR < 0)
        if (static_cast<int64_t>(NV - 1) * BT * V <= p.dim) return launch(std::true_type{});
    return launch(std::false_type{});
}

template <class T, class W, int V>
int launch_packs(const FwdParams<T, W> &p, cudaStream_t stream)
{
    const int packs = (p.dim + V - 1) / V;
    constexpr int N = 8 / V;   // packs of 8 elements
    if constexpr (V > 2) {
        // Short rows (a head's width) share a warp: 262144 x 128 fp16 66 -> 34 us.
        if (packs <= 8 * N) return launch_one<T, W, V, N, 8>(p, stream);
        if (packs <= 16 * N) return launch_one<T, W, V, N, 16>(p, stream);
    }
    if (packs <= 32 * N) return launch_one<T, W, V, N, 32>(p, stream);
    if constexpr (V > 2) {
        if (packs <= 32 * 2 * N) return launch_one<T, W, V, 2 * N, 32>(p, stream);
        if (packs <= 32 * 4 * N) return launch_one<T, W, V, 4 * N, 32>(p, stream);
        // 32 elements per thread and a power of 2 of threads, whose sums are the
        // shorter, where at least two thirds of them have work (8192 x 7168 fp16:
        // 41.6 us, 44.9 us with as many warps as the row needs; 16384 x 5120, five
        // eighths: 65.7 us and 58.0 us).
        auto mostly = [&](int threads) { return 3 * packs >= 2 * threads * 4 * N && packs <= threads * 4 * N; };
        if (packs <= 128 * 2 * N) return launch_one<T, W, V, 2 * N, 128>(p, stream);
        if (packs <= 128 * 4 * N) return launch_one<T, W, V, 4 * N, 128>(p, stream);
        if (mostly(256)) return launch_one<T, W, V, 4 * N, 256>(p, stream);
        if (mostly(512)) return launch_one<T, W, V, 4 * N, 512>(p, stream);
        if (packs <= 512 * 4 * N) return launch_one<T, W, V, 4 * N, -512>(p, stream);
    } else {
        // Narrow loads are bound by instructions, so no more threads than eight
        // elements each take (16384 x 4097 fp16: 148 us with the next power of 2,
        // 104 us this way, with two blocks per SM).
        if (packs <= 512 * N) return launch_one<T, W, V, N, -512>(p, stream);
        if (packs <= 1024 * N) return launch_one<T, W, V, N, -1024>(p, stream);
        if (packs <= 1024 * 2 * N) return launch_one<T, W, V, 2 * N, -1024>(p, stream);
    }
    return ln_launch(layer_norm_fwd_long<T, W>, dim3(static_cast<unsigned>(p.rows), 1, 1), 1024, stream, p);
}

template <class T, class W>
int forward(const LayerNormArgs &a)
{
    FwdParams<T, W> p{};
    p.X = static_cast<const T *>(a.X);
    p.gamma = static_cast<const W *>(a.gamma);
    p.beta = static_cast<const W *>(a.beta);
    p.Y = static_cast<T *>(a.Y);
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.rows = a.rows;
    p.dim = static_cast<int32_t>(a.dim);
    p.n = static_cast<float>(a.dim);
    p.inv_dim = 1.0f / p.n;
    p.eps = a.eps;
    const uintptr_t x_bits = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.Y) |
                             (static_cast<uintptr_t>(a.dim) * sizeof(T));
    const uintptr_t w_bits = reinterpret_cast<uintptr_t>(a.gamma) | reinterpret_cast<uintptr_t>(a.beta);
    constexpr int V = 16 / sizeof(T);
    const int pack = ln_pack_elements<T, W>(x_bits, w_bits);
    if (pack == V) return launch_packs<T, W, V>(p, a.stream);
    if constexpr (V > 4)
        if (pack == V / 4) return launch_packs<T, W, V / 4>(p, a.stream);
    return launch_packs<T, W, 1>(p, a.stream);
}

}  // namespace

namespace gemm_sm103 {

int launch_layer_norm_fwd(const LayerNormArgs &a)
{
    return ln_dispatch(a.xtype, a.wtype, [&](auto t, auto w) { return forward<decltype(t), decltype(w)>(a); });
}

}  // namespace gemm_sm103
