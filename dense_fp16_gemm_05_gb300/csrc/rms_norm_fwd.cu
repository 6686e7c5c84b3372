// rms_norm_fwd.cu -- root-mean-square norm over the last dimension, with the
// residual's addition in front of it:
//
//   h = x + r (rounded to the type: the residual stream as it is kept; x alone
//   without a residual),  rstd = 1 / sqrt(sum h^2 / dim + eps),  y = h rstd gamma
//
// in fp32; y is rounded to the type or quantised to E4M3 with one scale per 128
// columns straight from fp32.  The norm is taken of the rounded stream, which the
// backward pass has again.  Bound by memory: X and R are read once, H and Y
// written once.  A row belongs to some lanes, a warp or a block, chosen so that a
// thread holds at most 32 elements; longer rows are read again from L2.  16384 x 4096
// fp16 with a residual takes 78.5 us, 6.8 TB/s.
#include <type_traits>

#include "fp8_block.cuh"
#include "rms_norm.cuh"

namespace {

using namespace gemm_sm103;

template <class T, class W>
struct RmsParams {
    const T *X, *R;   // R NULL: no residual
    const W *gamma;   // NULL: ones
    T *H;             // written if R is given; may be X or R itself
    T *Y;
    uint8_t *Q;
    void *S;
    float *rstd;      // NULL: not kept
    int64_t rows;
    int32_t dim, blocks;   // blocks of 128 columns
    float inv_dim, eps;
    int32_t pow2;
};

__host__ __device__ constexpr int rms_threads(int tpr) { return tpr < 0 ? -tpr : (tpr < 128 ? 128 : tpr); }

// Lanes that take neighbouring packs, and the packs of each that follow at once: of
// narrow packs, a warp's 128 columns; for FP8 output, 128 columns of eight lanes, so
// that a scale is worked out once for 16 elements of a lane (8192 x 8192 bf16 with a
// residual: 82 us with 16 lanes and eight elements, 71.5 us so; 70.7 us, 6.7 TB/s, since
// the way of conversion is decided once per block.  Without a residual, fp16, 44.4 us).
__host__ __device__ constexpr int rms_lanes(int tpr, int v, bool fp8) { return tpr > 0 && tpr < 32 ? tpr : (v >= 4 && fp8 ? 8 : 32); }
__host__ __device__ constexpr int rms_run(int tpr, int v, bool fp8)
{
    if (tpr > 0 && tpr < 32) return 1;
    return v >= 4 && !fp8 ? 1 : 128 / (rms_lanes(tpr, v, fp8) * v);
}

// A pack of X, R or H: H may be either of them, so not through the read-only path.
template <class T, int V>
__device__ __forceinline__ void rms_load(LnPack<T, V> &p, const T *src) { p.load_shared(src); }

// Elements above 10^18 have squares whose sum is beyond fp32: such rows' squares are
// summed again, scaled down.  (A row that holds an infinity has rstd 0 either way.)
constexpr float kDown = 0x1p-100f;
// Squares of elements below 2^-63 are subnormal or vanish, which counts where eps does
// not hide it: where mean and eps are below 2^-110 together, the row's elements (below
// 2^-39 then, whatever its length) are scaled up and their squares summed again, which
// stay above 2^-118 and below 2^102.  (The scaled elements in the place of the row's own
// from there on, for rows whose rstd is beyond fp32, cost 8192 x 8192 to FP8 20 us.)
constexpr float kUp = 0x1p90f, kSmall = 0x1p-110f;

__device__ __forceinline__ bool rms_beyond(float sum) { return !(sum <= 3.4028235e38f); }
__device__ __forceinline__ bool rms_below(float sum, float inv_dim, float eps) { return fmaf(sum, inv_dim, eps) < kSmall; }
__device__ __forceinline__ float rms_rstd(float sum, float inv_dim, float eps) { return 1.0f / sqrtf(sum * inv_dim + eps); }

// kShift: a row that is not whole 16-byte pieces is taken with the pieces that it lies
// in, from the first one on; of the first and the last the neighbours' elements count
// as zeros and the row's own are stored one by one.
template <class T, class W, int V, int NV, int TPR, bool kFp8, bool kShift>
__global__ void __launch_bounds__(rms_threads(TPR)) rms_norm_fwd_kernel(RmsParams<T, W> p)
{
    static_assert(!kShift || (TPR > 32 || TPR < 0), "a block's rows begin at one place");
    constexpr int R = TPR > 0 ? rms_threads(TPR) / TPR : 1;   // rows of a block
    constexpr int C = rms_run(TPR, V, kFp8), RL = rms_lanes(TPR, V, kFp8);
    static_assert(NV % C == 0 || !kFp8, "whole blocks of columns");
    __shared__ float sh[2][ln_warps(TPR)];
    griddep_wait();   // X may come from the kernel just before
    griddep_launch_dependents();
    const int tpr = ln_threads<TPR>();
    const int t = TPR > 0 ? static_cast<int>(threadIdx.x) % tpr : static_cast<int>(threadIdx.x);
    int64_t row = static_cast<int64_t>(blockIdx.x) * R + (R > 1 ? static_cast<int>(threadIdx.x) / tpr : 0);
    // Lanes without a row take the last one along, for the sake of the shuffles.
    const bool in = row < p.rows;
    if (!in) row = p.rows - 1;
    const int64_t at = row * p.dim;
    // Elements in front of the row in its first piece.
    const int shift = kShift ? static_cast<int>((reinterpret_cast<uint64_t>(p.X + at) & 15u) / sizeof(T)) : 0;
    auto column = [&](int i) {
        if constexpr (C == 1) return (i * tpr + t) * V - shift;
        else return (((i / C) * (tpr / RL) + t / RL) * (RL * C) + (i % C) * RL + t % RL) * V;
    };
    auto whole = [&](int k) { return !kShift || (k >= 0 && k + V <= p.dim); };
    auto own = [&](int k) { return k >= 0 && k < p.dim; };
    // A pack of a row at column k < dim, with the neighbours' elements that its piece
    // holds; one by one where the piece reaches past the tensor's ends.
    const int64_t total = p.rows * p.dim;
    auto load = [&](LnPack<T, V> &pack, const T *src, int k) {
        if (!kShift || (at + k >= 0 && at + k + V <= total)) {
            rms_load(pack, src + at + k);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) pack.e[j] = own(k + j) ? src[at + k + j] : ln_round<T>(0.0f);
        }
    };
    auto store = [&](const LnPack<T, V> &pack, T *dst, int k) {
        if (whole(k)) {
            pack.store(dst + k);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (own(k + j)) dst[k + j] = pack.e[j];
        }
    };
    constexpr int P = V * NV / 2;
    float2 h[P];
    {
        LnPack<T, V> px[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (column(i) < p.dim) load(px[i], p.X, column(i));
            else px[i].fill(0.0f);
        }
        if (p.R) {
            LnPack<T, V> pr[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (column(i) < p.dim) load(pr[i], p.R, column(i));
                else pr[i].fill(0.0f);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (V == 1) {
                    px[i].e[0] = ln_round<T>(px[i][0] + pr[i][0]);
                } else {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) px[i].set_pair(j, add_f32x2(px[i].pair(j), pr[i].pair(j)));
                }
                if (in && column(i) < p.dim) store(px[i], p.H + at, column(i));
            }
        }
        if constexpr (kShift) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (whole(column(i))) continue;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (!own(column(i) + j)) px[i].e[j] = ln_round<T>(0.0f);
            }
        }
#pragma unroll
        for (int m = 0; m < P; ++m) h[m] = ln_pair_of(px, m);
    }
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int m = 0; m < P; ++m) s = fma_f32x2(h[m], h[m], s);
    const float sum = ln_row_sum<TPR>(s.x + s.y, sh[0]);
    float rstd = rms_rstd(sum, p.inv_dim, p.eps);
    // The same answer for all lanes that take part in the sum.
    const bool beyond = rms_beyond(sum), below = rms_below(sum, p.inv_dim, p.eps);
    if (TPR > 0 && TPR < 32 ? __any_sync(0xffffffffu, beyond || below) : beyond || below) {
        const float by = beyond ? kDown : kUp;
        const float2 by2 = make_float2(by, by);
        s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int m = 0; m < P; ++m) {
            const float2 d = mul_f32x2(h[m], by2);
            s = fma_f32x2(d, d, s);
        }
        const float again = ln_row_sum<TPR>(s.x + s.y, sh[1]);
        if (beyond || below) rstd = by * rms_rstd(again, p.inv_dim, p.eps * by * by);
    }
    if (t == 0 && in && p.rstd) p.rstd[row] = rstd;
    const float2 rstd2 = make_float2(rstd, rstd);
    if constexpr (!kFp8) {
        if (!in) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = column(i);
            if (k >= p.dim) continue;
            LnPack<W, V> g;
            g.fill(1.0f);
            if constexpr (kShift) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (p.gamma && own(k + j)) g.e[j] = __ldg(p.gamma + k + j);
            } else if (p.gamma) {
                g.load(p.gamma + k);
            }
            LnPack<T, V> out;
            if constexpr (V == 1) {
                out.e[0] = ln_round<T>(ln_half(h[i / 2], i) * rstd * g[0]);
            } else {
#pragma unroll
                for (int j = 0; j < V / 2; ++j)
                    out.set_pair(j, mul_f32x2(mul_f32x2(h[i * (V / 2) + j], rstd2), g.pair(j)));
            }
            store(out, p.Y + at, k);
        }
    } else {
        // h becomes y; what lies past the row's end is zero.
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            LnPack<W, V> g;
            if (p.gamma && column(i) < p.dim) g.load(p.gamma + column(i));
            else g.fill(1.0f);
            if constexpr (V == 1) {
                float &v = (i & 1) ? h[i / 2].y : h[i / 2].x;
                v = v * rstd * g[0];
            } else {
#pragma unroll
                for (int j = 0; j < V / 2; ++j)
                    h[i * (V / 2) + j] = mul_f32x2(mul_f32x2(h[i * (V / 2) + j], rstd2), g.pair(j));
            }
        }
        // G packs and L lanes make up a block of columns.
        constexpr bool kOne = TPR > 0 && TPR < 32;   // rows of up to 128 columns
        constexpr int G = kOne ? NV : C;
        constexpr int L = RL;
#pragma unroll
        for (int i0 = 0; i0 < NV; i0 += G) {
            static_assert(G * V % 2 == 0, "pairs");
            float largest = 0.0f;
#pragma unroll
            for (int e = i0 * V / 2; e < (i0 + G) * V / 2; ++e) largest = fp8_largest(largest, h[e]);
            uint32_t m = __float_as_uint(largest);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int k0 = column(i0);
            if (!in) continue;
            if ((t & (L - 1)) == 0 && k0 < p.dim)
                Fp8Block::store(p.S, row * p.blocks + (kOne ? 0 : k0 / kFp8Block), m, p.pow2 != 0);
            const Fp8Block b(m, p.pow2 != 0);
            b.by_way([&](auto way) {
                constexpr int W8 = decltype(way)::value;
#pragma unroll
                for (int i = i0; i < i0 + G; ++i) {
                    const int k = column(i);
                    if (k >= p.dim) continue;
                    uint8_t *q = p.Q + at + k;
                    if constexpr (V == 1) {
                        *q = static_cast<uint8_t>(b.template codes<W8>(make_float2(ln_half(h[i / 2], i), 0.0f)));
                    } else if constexpr (V == 2) {
                        *reinterpret_cast<uint16_t *>(q) = static_cast<uint16_t>(b.template codes<W8>(h[i]));
                    } else {
                        uint32_t c[V / 4];
#pragma unroll
                        for (int j = 0; j < V / 4; ++j)
                            c[j] = b.template codes<W8>(h[i * (V / 2) + 2 * j]) |
                                   (b.template codes<W8>(h[i * (V / 2) + 2 * j + 1]) << 16);
                        if constexpr (V == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(c[0], c[1]);
                        else *reinterpret_cast<uint32_t *>(q) = c[0];
                    }
                }
            });
        }
    }
}

// Rows longer than a block holds, and elements that no pack fits: three passes
// over the row, each thread the same four columns of a block in each.
template <class T, class W, bool kFp8>
__global__ void __launch_bounds__(1024) rms_norm_fwd_long(RmsParams<T, W> p)
{
    __shared__ float sh[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x, at = row * p.dim;
    const int lane = threadIdx.x & 31;
    const T *h = p.R ? p.H : p.X;
    float s = 0.0f;
    const int64_t first = static_cast<int64_t>(threadIdx.x >> 5) * kFp8Block;
    for (int64_t k0 = first; k0 < p.dim; k0 += 32 * kFp8Block)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = k0 + j * 32 + lane;
            if (k >= p.dim) continue;
            T v = p.X[at + k];
            if (p.R) {
                v = ln_round<T>(ln_float(v) + ln_float(p.R[at + k]));
                p.H[at + k] = v;
            }
            s = fmaf(ln_float(v), ln_float(v), s);
        }
    const float sum = ln_row_sum<1024>(s, sh[0]);
    float rstd = rms_rstd(sum, p.inv_dim, p.eps);
    const bool beyond = rms_beyond(sum);
    if (beyond || rms_below(sum, p.inv_dim, p.eps)) {
        const float by = beyond ? kDown : kUp;
        s = 0.0f;
        for (int64_t k0 = first; k0 < p.dim; k0 += 32 * kFp8Block)
            for (int j = 0; j < 4; ++j) {
                const int64_t k = k0 + j * 32 + lane;
                const float d = k < p.dim ? ln_float(h[at + k]) * by : 0.0f;
                s = fmaf(d, d, s);
            }
        rstd = by * rms_rstd(ln_row_sum<1024>(s, sh[1]), p.inv_dim, p.eps * by * by);
    }
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    for (int64_t k0 = first; k0 < p.dim; k0 += 32 * kFp8Block) {
        float y[4];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = k0 + j * 32 + lane;
            y[j] = 0.0f;
            if (k < p.dim) {
                y[j] = ln_float(h[at + k]) * rstd * (p.gamma ? ln_float(p.gamma[k]) : 1.0f);
                if constexpr (!kFp8) p.Y[at + k] = ln_round<T>(y[j]);
            }
            m = max(m, fp8_magnitude(y[j]));
        }
        if constexpr (kFp8) {
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) Fp8Block::store(p.S, row * p.blocks + k0 / kFp8Block, m, p.pow2 != 0);
            const Fp8Block b(m, p.pow2 != 0);
            b.by_way([&](auto way) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t k = k0 + j * 32 + lane;
                    if (k < p.dim) p.Q[at + k] = static_cast<uint8_t>(b.template codes<decltype(way)::value>(make_float2(y[j], 0.0f)));
                }
            });
        }
    }
}

template <class T, class W, bool kFp8, int V, int NV, int TPR, bool kShift = false>
int launch_one(const RmsParams<T, W> &p, cudaStream_t stream)
{
    // Threads: those of the template, or the whole warps that NV packs each need.
    constexpr int C = rms_run(TPR, V, kFp8);
    const int64_t runs = (static_cast<int64_t>(p.dim) + (kShift ? V - 1 : 0) + V * C - 1) / (V * C);   // C packs each
    const int BT = TPR > 0 ? rms_threads(TPR) : static_cast<int>(((runs + NV / C - 1) / (NV / C) + 31) / 32 * 32);
    constexpr int R = TPR > 0 ? rms_threads(TPR) / TPR : 1;
    return ln_launch(rms_norm_fwd_kernel<T, W, V, NV, TPR, kFp8, kShift>,
                     dim3(static_cast<unsigned>((p.rows + R - 1) / R), 1, 1), BT, stream, p);
}

template <class T, class W, bool kFp8, int V>
int launch_packs(const RmsParams<T, W> &p, cudaStream_t stream)
{
    const int64_t packs = (static_cast<int64_t>(p.dim) + V - 1) / V;
    constexpr int N = 8 / V;   // packs of 8 elements
    if constexpr (V > 2) {
        if (packs <= 8 * N) return launch_one<T, W, kFp8, V, N, 8>(p, stream);
        if (packs <= 16 * N) return launch_one<T, W, kFp8, V, N, 16>(p, stream);
    }
    if constexpr (V <= 2 || !kFp8)
        if (packs <= 32 * N) return launch_one<T, W, kFp8, V, N, 32>(p, stream);
    if constexpr (V > 2) {
        if (packs <= 32 * 2 * N) return launch_one<T, W, kFp8, V, 2 * N, 32>(p, stream);
        if (packs <= 32 * 4 * N) return launch_one<T, W, kFp8, V, 4 * N, 32>(p, stream);
        if (packs <= 128 * 2 * N) return launch_one<T, W, kFp8, V, 2 * N, 128>(p, stream);
        if (packs <= 128 * 4 * N) return launch_one<T, W, kFp8, V, 4 * N, 128>(p, stream);
        if (packs <= 512 * 4 * N) return launch_one<T, W, kFp8, V, 4 * N, -512>(p, stream);
    } else {
        if (packs <= 512 * N) return launch_one<T, W, kFp8, V, N, -512>(p, stream);
        if (packs <= 1024 * N) return launch_one<T, W, kFp8, V, N, -1024>(p, stream);
        if (packs <= 1024 * 2 * N) return launch_one<T, W, kFp8, V, 2 * N, -1024>(p, stream);
    }
    return ln_launch(rms_norm_fwd_long<T, W, kFp8>, dim3(static_cast<unsigned>(p.rows), 1, 1), 1024, stream, p);
}

template <class T, class W, bool kFp8>
int forward(const RmsNormArgs &a)
{
    RmsParams<T, W> p{};
    p.X = static_cast<const T *>(a.X);
    p.R = static_cast<const T *>(a.R);
    p.gamma = static_cast<const W *>(a.gamma);
    p.H = static_cast<T *>(a.H);
    p.Y = static_cast<T *>(a.Y);
    p.Q = static_cast<uint8_t *>(a.Q);
    p.S = a.S;
    p.rstd = a.rstd;
    p.rows = a.rows;
    p.dim = static_cast<int32_t>(a.dim);
    p.blocks = static_cast<int32_t>((a.dim + kFp8Block - 1) / kFp8Block);
    p.inv_dim = 1.0f / static_cast<float>(a.dim);
    p.eps = a.eps;
    p.pow2 = a.pow2;
    const uintptr_t x_bits = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.R) |
                             reinterpret_cast<uintptr_t>(a.R ? a.H : nullptr) | reinterpret_cast<uintptr_t>(a.Y) |
                             (static_cast<uintptr_t>(a.dim) * sizeof(T));
    const uintptr_t w_bits = reinterpret_cast<uintptr_t>(a.gamma);
    constexpr int V = 16 / sizeof(T);
    int pack = ln_pack_elements<T, W>(x_bits, w_bits);
    // Q is stored a pack at a time, a byte per element.
    if (kFp8 && (reinterpret_cast<uintptr_t>(a.Q) & static_cast<uintptr_t>(pack - 1)) != 0) pack = 1;
    if (pack == V) return launch_packs<T, W, kFp8, V>(p, a.stream);
    if constexpr (!kFp8) {
        // All arrays' rows begin at the same place of a 16-byte piece and fit a block, and
        // there is enough to stream to pay for the edges: 16384 x 4097 fp16 88 us, 150 us
        // by elements; 65536 x 1023 93 and 104; but 65536 x 513 75 and 71, 1 x 4097 3.4
        // and 2.2, 2000 x 3001 fp32 21.1 and 18.9.  Pairs: 16384 x 4098 87 and 99, but
        // 16384 x 2050 49 and 47.
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.X), y = reinterpret_cast<uintptr_t>(a.Y);
        const uintptr_t r = a.R ? reinterpret_cast<uintptr_t>(a.R) : x, h = a.R ? reinterpret_cast<uintptr_t>(a.H) : x;
        constexpr int N = 8 / V;   // packs of 8 elements
        const int64_t packs = (static_cast<int64_t>(p.dim) + 2 * V - 2) / V;
        if ((((x ^ y) | (x ^ r) | (x ^ h)) & 15u) == 0 && p.dim >= (pack == 1 ? 768 : 2560) &&
            p.rows * p.dim >= (sizeof(T) == 2 ? 1 << 22 : 1 << 23)) {
            if (packs <= 128 * 2 * N) return launch_one<T, W, false, V, 2 * N, -128, true>(p, a.stream);
            if (packs <= 512 * 4 * N) return launch_one<T, W, false, V, 4 * N, -512, true>(p, a.stream);
        }
    }
    if constexpr (V > 4)
        if (pack == V / 4) return launch_packs<T, W, kFp8, V / 4>(p, a.stream);
    return launch_packs<T, W, kFp8, 1>(p, a.stream);
}

}  // namespace

namespace gemm_sm103 {

int launch_rms_norm_fwd(const RmsNormArgs &a)
{
    return ln_dispatch(a.xtype, a.wtype, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        return a.Q ? forward<T, W, true>(a) : forward<T, W, false>(a);
    });
}

}  // namespace gemm_sm103
