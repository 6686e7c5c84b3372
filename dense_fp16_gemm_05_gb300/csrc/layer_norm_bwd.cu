// layer_norm_bwd.cu -- gradients of layer norm.  With z = (x - mean) rstd and
// g = dy gamma,
//
//   dx     = rstd (g - sum(g) / dim - z sum(g z) / dim)      (sums over a row)
//   dgamma = sum dy z,   dbeta = sum dy                      (sums over all rows)
//
// Bound by memory: dY and X are read once and dX written once.  A block walks
// rows; a thread always has the same columns, so the columns' sums stay in its
// registers (fp32) until the block's last row, and only then one partial sum
// per block and column goes to the workspace.  A second kernel adds the blocks'
// partial sums in a fixed order and keeps what the additions lose: no atomics, the
// same bits every time.
#include "layer_norm.cuh"

#include <atomic>

#include "gemm_kernel.cuh"

namespace {

using namespace gemm_sm103;

template <class T, class W>
struct BwdParams {
    const T *dY, *X;
    const W *gamma;   // NULL: ones
    const float *mean, *rstd;
    T *dX;
    float *part;      // (2, parts, dim): dgamma's, then dbeta's; NULL: not wanted
    int64_t rows;
    int32_t dim;
    int32_t parts;    // blocks
    float inv_dim;
    int32_t stages;   // rows under way per block (the ring kernel)
    int32_t withhold; // test hook: 1 = the ring's rows are not loaded; 0 in every normal call
    uint64_t limit;   // SM clocks of a wait (the ring kernel)
    unsigned long long *status;
    W *dgamma, *dbeta;
    int32_t sm_count;
};

// Threads of a block, and blocks per SM: some 1024 threads, so that the loads of
// one block run while another waits for its row's sum.
__host__ __device__ constexpr int bwd_threads(int tpr) { return tpr < 0 ? -tpr : (tpr <= 32 ? 256 : tpr); }
__host__ __device__ constexpr int bwd_blocks(int tpr, int v, int per)
{
    if (tpr < 0) return 1;
    if (tpr <= 32) return per <= 8 ? (v > 2 ? 4 : 2) : 2;
    return 1024 / tpr;
}

// kInner: every pack but a thread's last lies inside the row whatever the thread.
template <class T, class W, int V, int NV, int TPR, bool kInner>
__global__ void __launch_bounds__(bwd_threads(TPR), bwd_blocks(TPR, V, V * NV)) layer_norm_bwd_kernel(BwdParams<T, W> p)
{
    constexpr int R = TPR > 0 ? bwd_threads(TPR) / TPR : 1;   // rows at a time
    static_assert(TPR <= 32 || R == 1, "lanes of a warp or a block per row");
    // Rows of lanes without one: a warp holds several.
    constexpr bool kShared = TPR > 0 && TPR < 32;
    __shared__ float2 sh[2][ln_warps(TPR)];
    extern __shared__ float comb[];   // R > 1: (R, dim)
    griddep_wait();
    griddep_launch_dependents();
    const int tpr = ln_threads<TPR>();
    const int t = R > 1 ? static_cast<int>(threadIdx.x) % tpr : static_cast<int>(threadIdx.x);
    const int sub = R > 1 ? static_cast<int>(threadIdx.x) / tpr : 0;
    // The arithmetic is done on pairs (two fp32 operations per instruction): with
    // 16-bit elements the pass is as much a matter of instructions as of bytes
    // (16384 x 4096 fp16: 90 us one by one, 83 us in pairs).
    constexpr int P = V * NV / 2;   // pair m: elements 2m, 2m + 1 of the packs in order
    // What a thread keeps is weighed against registers: fp32 rows and 16 elements
    // per thread read gamma again for every row (from L1), and 16 elements in a
    // block of 1024 threads, which has 64 registers for each, also neither
    // prefetch nor keep z and g.
    constexpr bool kReload = sizeof(T) == 4 || V * NV > 8;
    constexpr bool kLean = (TPR == 1024 || TPR == -1024) && V * NV > 8;
    float2 dg[P], db[P], gm[P];
    auto inside = [&](int i) { return (kInner && i < NV - 1) || (i * tpr + t) * V < p.dim; };
    auto load_gamma = [&]() {
        LnPack<W, V> pg[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (p.gamma && inside(i)) pg[i].load(p.gamma + k);
            else pg[i].fill(1.0f);
        }
#pragma unroll
        for (int m = 0; m < P; ++m) gm[m] = ln_pair_of(pg, m);
    };
    if constexpr (!kReload) load_gamma();
#pragma unroll
    for (int m = 0; m < P; ++m) dg[m] = db[m] = make_float2(0.0f, 0.0f);
    // The next row's loads are under way while a row's sums are taken.
    LnPack<T, V> nx[NV], nd[NV];
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto load = [&](int64_t row) {
        const T *x = p.X + row * p.dim;
        const T *dy = p.dY + row * p.dim;
        const bool in = !kShared || row < p.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (in && inside(i)) {
                nx[i].load(x + k);
                nd[i].load(dy + k);
            } else {
                nx[i].fill(0.0f);
                nd[i].fill(0.0f);   // adds nothing to any sum
            }
        }
        next_mean = in ? __ldg(p.mean + row) : 0.0f;
        next_rstd = in ? __ldg(p.rstd + row) : 0.0f;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * R;
    int64_t row = static_cast<int64_t>(blockIdx.x) * R + sub;
    // Lanes of a warp with several rows stay together for the shuffles: `lead`
    // is the warp's first row, and a lane without a row adds zeros.
    int64_t lead = row - (kShared ? sub % (32 / (TPR > 0 ? TPR : 32)) : 0);
    // A row that is not there is loaded as the last one, and not used: loads
    // without a condition can be issued ahead.
    auto there = [&](int64_t r) { return kShared || r < p.rows ? r : p.rows - 1; };
    if constexpr (!kLean) load(there(row));
    for (int it = 0; lead < p.rows; lead += step, row += step, it ^= 1) {
        LnPack<T, V> px[NV], pd[NV];
        if constexpr (kLean) load(row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            px[i] = nx[i];
            pd[i] = nd[i];
        }
        const float mean = next_mean, rstd = next_rstd;
        if constexpr (!kLean) load(there(row + step));
        if constexpr (kReload) load_gamma();
        // z and g stay in registers for the second use.
        float2 z[P], g[P];
        float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
        const float2 neg_mean = make_float2(-mean, -mean), rstd2 = make_float2(rstd, rstd);
#pragma unroll
        for (int m = 0; m < P; ++m) {
            const float2 d = ln_pair_of(pd, m);
            // Past the row's end d = 0, so that z does not matter there.
            z[m] = mul_f32x2(add_f32x2(ln_pair_of(px, m), neg_mean), rstd2);
            g[m] = mul_f32x2(d, gm[m]);
            s1 = add_f32x2(s1, g[m]);
            s2 = fma_f32x2(g[m], z[m], s2);
            dg[m] = fma_f32x2(d, z[m], dg[m]);
            db[m] = add_f32x2(db[m], d);
        }
        const float2 sum = ln_row_sum2<TPR>(s1.x + s1.y, s2.x + s2.y, sh[it]);
        const float rc1 = rstd * (sum.x * p.inv_dim), rc2 = rstd * (sum.y * p.inv_dim);
        const float2 neg_rc1 = make_float2(-rc1, -rc1), neg_rc2 = make_float2(-rc2, -rc2);
        if constexpr (kLean) {
            // From the packed elements again; the barrier keeps the compiler from
            // holding (and spilling) the first values instead.
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                px[i].opaque();
                pd[i].opaque();
            }
            load_gamma();
#pragma unroll
            for (int m = 0; m < P; ++m) {
                z[m] = mul_f32x2(add_f32x2(ln_pair_of(px, m), neg_mean), rstd2);
                g[m] = mul_f32x2(ln_pair_of(pd, m), gm[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < P; ++m) z[m] = fma_f32x2(z[m], neg_rc2, fma_f32x2(rstd2, g[m], neg_rc1));
        T *dx = p.dX + row * p.dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (!inside(i) || (kShared && row >= p.rows)) continue;
            LnPack<T, V> out;
#pragma unroll
            for (int j = 0; j < V; ++j) out.e[j] = ln_round<T>(ln_half(z[(i * V + j) / 2], i * V + j));
            out.store(dx + k);
        }
    }
    if (p.part == nullptr) return;
    // The block's partial sums, first dgamma's and then dbeta's.
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *out = p.part + (static_cast<int64_t>(which) * p.parts + blockIdx.x) * p.dim;
        if constexpr (R == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int k = (i * tpr + t) * V;
                if (k >= p.dim) continue;
#pragma unroll
                for (int j = 0; j < V; ++j) out[k + j] = ln_half(which == 0 ? dg[(i * V + j) / 2] : db[(i * V + j) / 2], i * V + j);
            }
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int k = (i * tpr + t) * V;
                if (k >= p.dim) continue;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    comb[sub * p.dim + k + j] = ln_half(which == 0 ? dg[(i * V + j) / 2] : db[(i * V + j) / 2], i * V + j);
            }
            __syncthreads();
            for (int k = threadIdx.x; k < p.dim; k += static_cast<int>(blockDim.x)) {
                float s = comb[k];
#pragma unroll
                for (int r = 1; r < R; ++r) s += comb[r * p.dim + k];
                out[k] = s;
            }
        }
    }
}

// Rows of 16-byte pieces, a block per row at a time: the rows come through a
// ring of bulk copies in shared memory, `stages` rows of X and dY ahead, so that
// the bytes under way are not bounded by registers (16384 x 4096 fp16: 82 us with
// one row prefetched in registers, 79 us with four in the ring; 75 us, 5.4 TB/s,
// since both row sums share their shuffles and full rows have no bounds).  What
// bounds it by counters is issue slots (55-60 % busy) and the two dependent
// chains of shuffles around the row's barrier, not DRAM.  A ring slot is
// free once every thread has its pieces in registers, which the row sum's
// barrier says; with 16 elements in each of 1024 threads (kReread) z and g are
// taken from shared memory a second time instead of being kept, and the slot is
// refilled one row later.  Every wait is bounded: on expiry the site is recorded in the
// device status word and the block leaves.
constexpr int kRingStages = 4;

// Packs that do not make up 16-byte pieces: rows of other lengths and
// alignments, copied with the whole 16-byte pieces that they lie in.
template <class T, int V>
constexpr bool kRingAny = V * sizeof(T) < 16;

// Bytes of a row's place in the ring.
template <class T, int V>
__host__ __device__ __forceinline__ uint32_t ring_row_bytes(int dim)
{
    const uint32_t bytes = static_cast<uint32_t>(dim) * static_cast<uint32_t>(sizeof(T));
    return kRingAny<T, V> ? (bytes + 15u) / 16u * 16u + 16u : bytes;
}

// The 16-byte pieces of global memory that hold `bytes` bytes at `src`, and what
// of them lies inside the tensor [lo, hi): the rest is not read.
struct RingWindow {
    uint64_t first, begin, end, src, last;

    __device__ __forceinline__ RingWindow(uint64_t src_, uint32_t bytes, uint64_t lo, uint64_t hi)
    {
        src = src_;
        last = src + bytes;
        first = src & ~15ull;
        begin = first < lo ? first + 16 : first;
        end = (last + 15ull) & ~15ull;
        if (end > hi) end -= 16;
        if (end < begin) end = begin;
    }
};

// Blocks per SM that the registers are held to.
__host__ __device__ constexpr int ring_blocks(int tpr, int per)
{
    if (tpr > 0) return 1024 / tpr;
    return per > 8 && tpr != -320 ? 1 : 2;
}

// TPR > 0: the row is exactly the threads' elements, no bounds to check.
// kInner: every pack but a thread's last lies inside the row whatever the thread.
template <class T, class W, int V, int NV, int TPR, bool kInner>
__global__ void __launch_bounds__(bwd_threads(TPR), ring_blocks(TPR, V * NV)) layer_norm_bwd_ring(BwdParams<T, W> p)
{
    constexpr bool kFull = TPR > 0;
    constexpr bool kReread = V * NV > 8 && (TPR == 1024 || TPR == -1024);
    constexpr bool kReload = sizeof(T) == 4 || V * NV > 8;   // gamma again for every row, from L1
    constexpr int P = V * NV / 2;
    extern __shared__ uint4 ring[];   // (stages, 2, dim) elements
    __shared__ float2 sh[2][ln_warps(TPR)];
    __shared__ uint64_t full_mem[kRingStages];
    __shared__ volatile int failed[2];
    const int t = static_cast<int>(threadIdx.x), tpr = ln_threads<TPR>();
    const uint32_t row_bytes = ring_row_bytes<T, V>(p.dim);
    const uint32_t ring_base = smem_addr(ring), full0 = smem_addr(full_mem);
    if (t == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(full0 + 8u * s, 1);
        failed[0] = failed[1] = 0;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    auto fetch = [&](uint32_t row, int s) {
        const uint32_t bar = full0 + 8u * static_cast<uint32_t>(s);
        const uint32_t dst = ring_base + 2u * static_cast<uint32_t>(s) * row_bytes;
        if constexpr (kRingAny<T, V>) {
            const uint32_t bytes = static_cast<uint32_t>(p.dim) * static_cast<uint32_t>(sizeof(T));
            const uint64_t size = static_cast<uint64_t>(p.rows) * bytes, at = static_cast<uint64_t>(row) * bytes;
            const uint64_t bx = reinterpret_cast<uint64_t>(p.X), bd = reinterpret_cast<uint64_t>(p.dY);
            const RingWindow w[2] = {RingWindow(bx + at, bytes, bx, bx + size), RingWindow(bd + at, bytes, bd, bd + size)};
            uint8_t *to = reinterpret_cast<uint8_t *>(ring) + (dst - ring_base);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // Elements in pieces that reach past the tensor's ends, one by one;
                // the arrival below releases them to the waiting threads, and the
                // fence orders them before the copies of the slot's later rows.
                auto edge = [&](uint64_t a, uint64_t b) {
                    for (; a < b; a += sizeof(T))
                        *reinterpret_cast<T *>(to + h * row_bytes + (a - w[h].first)) = *reinterpret_cast<const T *>(a);
                    fence_proxy_async_smem();
                };
                if (w[h].begin > w[h].src) edge(w[h].src, w[h].begin < w[h].last ? w[h].begin : w[h].last);
                if (w[h].end < w[h].last) edge(w[h].end > w[h].src ? w[h].end : w[h].src, w[h].last);
            }
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(w[0].end - w[0].begin + w[1].end - w[1].begin));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (w[h].end > w[h].begin)
                    bulk_load(dst + static_cast<uint32_t>(h) * row_bytes + static_cast<uint32_t>(w[h].begin - w[h].first),
                              reinterpret_cast<const void *>(w[h].begin),
                              static_cast<uint32_t>(w[h].end - w[h].begin), bar);
            return;
        }
        mbar_arrive_expect_tx(bar, 2u * row_bytes);
        bulk_load(dst, p.X + static_cast<int64_t>(row) * p.dim, row_bytes, bar);
        bulk_load(dst + row_bytes, p.dY + static_cast<int64_t>(row) * p.dim, row_bytes, bar);
    };
    // Rows as unsigned 32-bit numbers: the ones past the end may pass 2^31.
    const uint32_t step = gridDim.x, rows = static_cast<uint32_t>(p.rows);
    uint32_t row = blockIdx.x;
    if (t == 0 && p.withhold == 0)
        for (int s = 0; s < p.stages && row + static_cast<uint32_t>(s) * step < rows; ++s)
            fetch(row + static_cast<uint32_t>(s) * step, s);

    auto inside = [&](int i) { return kFull || (kInner && i < NV - 1) || (i * tpr + t) * V < p.dim; };
    float2 dg[P], db[P], gm[P];
    auto load_gamma = [&]() {
        LnPack<W, V> pg[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (p.gamma && inside(i)) pg[i].load(p.gamma + k);
            else pg[i].fill(1.0f);
        }
#pragma unroll
        for (int m = 0; m < P; ++m) gm[m] = ln_pair_of(pg, m);
    };
    if constexpr (!kReload) load_gamma();
#pragma unroll
    for (int m = 0; m < P; ++m) dg[m] = db[m] = make_float2(0.0f, 0.0f);
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (row < rows) {
        next_mean = __ldg(p.mean + row);
        next_rstd = __ldg(p.rstd + row);
    }
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; row < rows; row += step, it ^= 1) {
        const float mean = next_mean, rstd = next_rstd;
        if (row + step < rows) {
            next_mean = __ldg(p.mean + row + step);
            next_rstd = __ldg(p.rstd + row + step);
        }
        if constexpr (kReload) load_gamma();
        if (!mbar_try_wait(full0 + 8u * static_cast<uint32_t>(s), ph)) {
            const long long t0 = clock64();
            while (!mbar_try_wait(full0 + 8u * static_cast<uint32_t>(s), ph))
                if (static_cast<uint64_t>(clock64() - t0) > p.limit) {
                    failed[it] = 1;
                    break;
                }
        }
        const T *x = reinterpret_cast<const T *>(reinterpret_cast<const uint8_t *>(ring) +
                                                 2ull * static_cast<uint32_t>(s) * row_bytes);
        const T *dy = reinterpret_cast<const T *>(reinterpret_cast<const uint8_t *>(x) + row_bytes);
        if constexpr (kRingAny<T, V>) {
            const int64_t at = static_cast<int64_t>(row) * p.dim;
            x += (reinterpret_cast<uint64_t>(p.X + at) & 15u) / sizeof(T);
            dy += (reinterpret_cast<uint64_t>(p.dY + at) & 15u) / sizeof(T);
        }
        LnPack<T, V> px[NV], pd[NV];
        auto pieces = [&]() {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int k = (i * tpr + t) * V;
                if (inside(i)) {
                    px[i].load_shared(x + k);
                    pd[i].load_shared(dy + k);
                } else {
                    px[i].fill(0.0f);
                    pd[i].fill(0.0f);   // adds nothing to any sum
                }
            }
        };
        pieces();
        float2 z[P], g[P];
        float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
        const float2 neg_mean = make_float2(-mean, -mean), rstd2 = make_float2(rstd, rstd);
#pragma unroll
        for (int m = 0; m < P; ++m) {
            const float2 d = ln_pair_of(pd, m);
            z[m] = mul_f32x2(add_f32x2(ln_pair_of(px, m), neg_mean), rstd2);
            g[m] = mul_f32x2(d, gm[m]);
            s1 = add_f32x2(s1, g[m]);
            s2 = fma_f32x2(g[m], z[m], s2);
            dg[m] = fma_f32x2(d, z[m], dg[m]);
            db[m] = add_f32x2(db[m], d);
        }
        const float2 sum = ln_row_sum2<TPR>(s1.x + s1.y, s2.x + s2.y, sh[it]);
        if (failed[it]) {   // the same answer for every thread: set before the barrier
            ok = false;
            break;
        }
        if (t == 0) {
            // This row's slot, or (kReread) the one before's, which every thread
            // had left when it came to this row's barrier.
            if constexpr (kReread) {
                const uint32_t next = row + static_cast<uint32_t>(p.stages - 1) * step;
                if (row != blockIdx.x && next < rows) fetch(next, s == 0 ? p.stages - 1 : s - 1);
            } else {
                const uint32_t next = row + static_cast<uint32_t>(p.stages) * step;
                if (next < rows) fetch(next, s);
            }
        }
        const float rc1 = rstd * (sum.x * p.inv_dim), rc2 = rstd * (sum.y * p.inv_dim);
        const float2 neg_rc1 = make_float2(-rc1, -rc1), neg_rc2 = make_float2(-rc2, -rc2);
        if constexpr (kReread) {
            pieces();
            load_gamma();
#pragma unroll
            for (int m = 0; m < P; ++m) {
                z[m] = mul_f32x2(add_f32x2(ln_pair_of(px, m), neg_mean), rstd2);
                g[m] = mul_f32x2(ln_pair_of(pd, m), gm[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < P; ++m) z[m] = fma_f32x2(z[m], neg_rc2, fma_f32x2(rstd2, g[m], neg_rc1));
        T *dx = p.dX + static_cast<int64_t>(row) * p.dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (!inside(i)) continue;
            LnPack<T, V> out;
#pragma unroll
            for (int j = 0; j < V; ++j) out.e[j] = ln_round<T>(ln_half(z[(i * V + j) / 2], i * V + j));
            out.store(dx + k);
        }
        if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
        }
    }
    if (!ok) {
        if (t == 0) {
            atomicCAS(p.status, 0ull,
                      static_cast<unsigned long long>(kSiteNormRow) | (static_cast<unsigned long long>(blockIdx.x) << 8));
            // Give the copies in flight a bounded time to land before the block exits.
            const long long t0 = clock64();
            while (static_cast<uint64_t>(clock64() - t0) < 1000000ull) {
            }
        }
        __syncthreads();
        return;
    }
    if (p.part == nullptr) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *out = p.part + (static_cast<int64_t>(which) * p.parts + blockIdx.x) * p.dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (!inside(i)) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) out[k + j] = ln_half(which == 0 ? dg[(i * V + j) / 2] : db[(i * V + j) / 2], i * V + j);
        }
    }
}

// Rows longer than a block holds: dX in two passes over the row ...
template <class T, class W>
__global__ void __launch_bounds__(1024) layer_norm_bwd_long(BwdParams<T, W> p)
{
    __shared__ float2 sh[2][32];
    griddep_wait();
    griddep_launch_dependents();
    int it = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, it ^= 1) {
        const T *x = p.X + row * p.dim;
        const T *dy = p.dY + row * p.dim;
        T *dx = p.dX + row * p.dim;
        const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t k = threadIdx.x; k < p.dim; k += 1024) {
            const float g = ln_float(dy[k]) * (p.gamma ? ln_float(p.gamma[k]) : 1.0f);
            s1 += g;
            s2 = fmaf(g, (ln_float(x[k]) - mean) * rstd, s2);
        }
        const float2 sum = ln_row_sum2<1024>(s1, s2, sh[it]);
        const float c1 = sum.x * p.inv_dim, c2 = sum.y * p.inv_dim;
        for (int64_t k = threadIdx.x; k < p.dim; k += 1024) {
            const float g = ln_float(dy[k]) * (p.gamma ? ln_float(p.gamma[k]) : 1.0f);
            dx[k] = ln_round<T>(rstd * (g - c1 - (ln_float(x[k]) - mean) * rstd * c2));
        }
    }
}

// ... and the columns' partial sums, a thread per column, rows blockIdx.y,
// blockIdx.y + parts, ...
template <class T, class W>
__global__ void __launch_bounds__(256) layer_norm_bwd_columns(BwdParams<T, W> p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (k >= p.dim) return;
    for (int64_t part = blockIdx.y; part < p.parts; part += gridDim.y) {
        float dg = 0.0f, db = 0.0f;
        for (int64_t row = part; row < p.rows; row += p.parts) {
            const float d = ln_float(p.dY[row * p.dim + k]);
            const float z = (ln_float(p.X[row * p.dim + k]) - __ldg(p.mean + row)) * __ldg(p.rstd + row);
            dg = fmaf(d, z, dg);
            db += d;
        }
        p.part[part * p.dim + k] = dg;
        p.part[(static_cast<int64_t>(p.parts) + part) * p.dim + k] = db;
    }
}

// Adds x to s and what the addition loses to c (Knuth's exact error of a sum): s + c
// then has the terms' sum but for errors of second order.
__device__ __forceinline__ void ln_add_exact(float &s, float &c, float x)
{
    const float t = s + x;
    const float b = t - s;
    c += (s - (t - b)) + (x - b);
    s = t;
}

// Adds the parts of 32 columns: NW warps take every NW-th part, then their sums
// are added in a tree of fixed order.  There are hundreds of parts of both signs,
// so what their additions lose is kept and added last: the result is the parts'
// sum rounded once.  (Both kernels, with plain sums one after another and so:
// 16384 x 4096 fp16 75.0 us and 74.7, 8192 x 768 19.3 and 19.9, 4096 x 5000 fp32
// 45.0 and 45.5; in fp64 the additions alone would be 4 us at 16384 x 4096.)
template <class W, int NW>
__global__ void __launch_bounds__(NW * 32) layer_norm_bwd_finish(const float *__restrict__ part, W *__restrict__ dgamma,
                                                             W *__restrict__ dbeta, int parts, int dim)
{
    __shared__ float sh[NW][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const float *src = part + static_cast<int64_t>(blockIdx.y) * parts * dim;
    float s = 0.0f, c = 0.0f;
    if (k < dim) {
        auto at = [&](int r) { return src[static_cast<int64_t>(r) * dim + k]; };
        constexpr int B = 8;   // loads under way
        int r = w;
        for (; r + (B - 1) * NW < parts; r += B * NW) {
            float x[B];
#pragma unroll
            for (int i = 0; i < B; ++i) x[i] = at(r + i * NW);
#pragma unroll
            for (int i = 0; i < B; ++i) ln_add_exact(s, c, x[i]);
        }
#pragma unroll 4
        for (; r < parts; r += NW) ln_add_exact(s, c, at(r));
    }
    // NW neighbouring lanes take a column's sums.  One array for both: with two
    // these blocks started later (1000 x 1023 fp32: 11.3 us, 8.7 us so), likely for
    // another split of the SM between L1 and shared memory than the main kernel's.
    const int column = threadIdx.x / NW, from = threadIdx.x % NW;
    sh[w][lane] = s;
    __syncthreads();
    s = sh[from][column];
    __syncthreads();
    sh[w][lane] = c;
    __syncthreads();
    c = sh[from][column];
#pragma unroll
    for (int o = NW / 2; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, s, o);
        const float other_lost = __shfl_xor_sync(0xffffffffu, c, o);
        ln_add_exact(s, c, other);
        c += other_lost;
    }
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + column;
    // Of a sum that is infinite or NaN the errors are NaN.
    if (from == 0 && out < dim) (blockIdx.y == 0 ? dgamma : dbeta)[out] = ln_round<W>(c == c ? s + c : s);
}

// The second kernel, if the weights' gradients are wanted.  More than two parts
// per SM come with short rows, so few columns for the SMs to share: 32 warps each
// (8192 x 768 fp16, both kernels: 21.4 us with 16 warps, 19.8 us); with fewer parts
// the smaller blocks start sooner (64 x 4096: 8.0 us, 12.5 us with 32 warps).
template <class T, class W>
int finish(const BwdParams<T, W> &p, cudaStream_t stream)
{
    if (p.part == nullptr) return GEMM_OK;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.dim) + 31) / 32), 2, 1);
    const float *part = p.part;
    if (p.parts > 2 * p.sm_count)
        return ln_launch(layer_norm_bwd_finish<W, 32>, grid, 1024, stream, part, p.dgamma, p.dbeta, p.parts, p.dim);
    return ln_launch(layer_norm_bwd_finish<W, 16>, grid, 512, stream, part, p.dgamma, p.dbeta, p.parts, p.dim);
}

template <class T, class W, int V, int NV, int TPR>
int launch_one(const BwdParams<T, W> &p, cudaStream_t stream)
{
    // Threads: those of the template, or the whole warps that NV packs each need.
    const int packs = (p.dim + V - 1) / V;
    const int BT = TPR > 0 ? bwd_threads(TPR) : ((packs + NV - 1) / NV + 31) / 32 * 32;
    constexpr int R = TPR > 0 ? bwd_threads(TPR) / TPR : 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(p.parts), 1, 1);
    lc.blockDim = dim3(BT, 1, 1);
    lc.dynamicSmemBytes = R > 1 ? static_cast<size_t>(R) * p.dim * sizeof(float) : 0;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    cudaError_t e;
    if constexpr (V <= 2 && TPR < 0)
        e = static_cast<int64_t>(NV - 1) * BT * V <= p.dim
                ? cudaLaunchKernelEx(&lc, layer_norm_bwd_kernel<T, W, V, NV, TPR, true>, p)
                : cudaLaunchKernelEx(&lc, layer_norm_bwd_kernel<T, W, V, NV, TPR, false>, p);
    else
        e = cudaLaunchKernelEx(&lc, layer_norm_bwd_kernel<T, W, V, NV, TPR, false>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return finish<T, W>(p, stream);
}

template <class T, class W, int V, int NV, int TPR, bool kInner>
int launch_ring_kernel(const BwdParams<T, W> &p, int device, int threads, int64_t stage, cudaStream_t stream)
{
    auto kern = layer_norm_bwd_ring<T, W, V, NV, TPR, kInner>;
    static std::atomic<int> prepared[kMaxDevices];
    if (!prepared[device].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        prepared[device].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(p.parts), 1, 1);
    lc.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    lc.dynamicSmemBytes = static_cast<size_t>(p.stages) * static_cast<size_t>(stage);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaLaunchKernelEx(&lc, kern, p) != cudaSuccess) {
        cudaGetLastError();
        prepared[device].store(0, std::memory_order_release);
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// The ring kernel, where at least two rows fit a block's share of the shared
// memory, else the register kernel.
template <class T, class W, int V, int NV, int TPR>
int launch_ring(BwdParams<T, W> p, int device, int sm_count, cudaStream_t stream)
{
    const int packs = (p.dim + V - 1) / V;
    const int threads = TPR > 0 ? TPR : ((packs + NV - 1) / NV + 31) / 32 * 32;
    // Blocks per SM: those of the launch bound, or more where they are small.
    const int fit_blocks = V * NV > 8 ? ring_blocks(TPR, V * NV) : 1024 / threads;
    const int budget = (227 * 1024 - fit_blocks * 2048) / fit_blocks;
    const int64_t stage = 2 * static_cast<int64_t>(ring_row_bytes<T, V>(p.dim));
    const int64_t fit = budget / stage;
    // Two rows always fit but in fp32 rows of 16 elements in each of 1024 threads:
    // others have eight elements per thread and 1024 threads share the SM, or are
    // at most 8192 long, or of 16-bit elements.
    if constexpr (sizeof(T) == 4 && V * NV > 8 && (TPR == 1024 || TPR == -1024))
        if (fit < 2) return launch_one<T, W, V, NV, TPR>(p, stream);
    p.stages = static_cast<int32_t>(fit < kRingStages ? fit : kRingStages);
    const int64_t wave = static_cast<int64_t>(fit_blocks) * sm_count;
    if (p.parts > wave) p.parts = static_cast<int32_t>(wave);
    int st;
    if constexpr (kRingAny<T, V>)
        st = static_cast<int64_t>(NV - 1) * threads * V <= p.dim
                 ? launch_ring_kernel<T, W, V, NV, TPR, true>(p, device, threads, stage, stream)
                 : launch_ring_kernel<T, W, V, NV, TPR, false>(p, device, threads, stage, stream);
    else
        st = launch_ring_kernel<T, W, V, NV, TPR, false>(p, device, threads, stage, stream);
    return st != GEMM_OK ? st : finish<T, W>(p, stream);
}

template <class T, class W, int V>
int launch_packs(const BwdParams<T, W> &p, int device, int sm_count, cudaStream_t stream)
{
    const int packs = (p.dim + V - 1) / V;
    constexpr int N = 8 / V;   // packs of 8 elements
    if constexpr (V > 2) {
        // Short rows (a head's width) share a warp.
        if (packs <= 8 * N) return launch_one<T, W, V, N, 8>(p, stream);
        if (packs <= 16 * N) return launch_one<T, W, V, N, 16>(p, stream);
    }
    // Up to 512 elements a warp per row; layer_norm_parts counts on it.
    if (packs <= 32 * N) return launch_one<T, W, V, N, 32>(p, stream);
    if (packs <= 32 * 2 * N) return launch_one<T, W, V, 2 * N, 32>(p, stream);
    if constexpr (V > 2) {
        // Rows that fill a power of 2 of threads, eight elements each (16 in the
        // longest), and then any others: as many warps as the row needs, two blocks
        // of some 300 threads with 16 elements rather than one of some 600
        // (16384 x 4104 fp16: 137 us with the next power of 2, 79 us this way).
        if (packs == 128 * N) return launch_ring<T, W, V, N, 128>(p, device, sm_count, stream);
        if (packs == 256 * N) return launch_ring<T, W, V, N, 256>(p, device, sm_count, stream);
        if (packs == 512 * N) return launch_ring<T, W, V, N, 512>(p, device, sm_count, stream);
        if (packs == 1024 * N) return launch_ring<T, W, V, N, 1024>(p, device, sm_count, stream);
        if (packs == 1024 * 2 * N) return launch_ring<T, W, V, 2 * N, 1024>(p, device, sm_count, stream);
        if (packs <= 512 * N) return launch_ring<T, W, V, N, -512>(p, device, sm_count, stream);
        if (packs <= 320 * 2 * N) return launch_ring<T, W, V, 2 * N, -320>(p, device, sm_count, stream);
        if (packs <= 512 * 2 * N) return launch_ring<T, W, V, 2 * N, -512>(p, device, sm_count, stream);
        if (packs <= 1024 * 2 * N) return launch_ring<T, W, V, 2 * N, -1024>(p, device, sm_count, stream);
    } else {
        // No more threads than eight elements each take (16384 x 4097 fp16: 347 us
        // with the next power of 2, 171 us this way).  Such rows too go through the
        // ring, which leaves registers for a second block per SM (16384 x 3001
        // fp16: 118 us without, 99 us; 16384 x 7001: 311 us, 195 us), unless rows are
        // short (65536 x 1023: 117 us without, 124 us).
        if (packs <= 128 * N) return launch_one<T, W, V, N, -512>(p, stream);
        if (packs <= 512 * N) return launch_ring<T, W, V, N, -512>(p, device, sm_count, stream);
        if (packs <= 320 * 2 * N) return launch_ring<T, W, V, 2 * N, -320>(p, device, sm_count, stream);
        if (packs <= 512 * 2 * N) return launch_ring<T, W, V, 2 * N, -512>(p, device, sm_count, stream);
        if (packs <= 1024 * 2 * N) return launch_one<T, W, V, 2 * N, -1024>(p, stream);
    }
    int st = ln_launch(layer_norm_bwd_long<T, W>, dim3(static_cast<unsigned>(p.parts), 1, 1), 1024, stream, p);
    if (st != GEMM_OK || p.part == nullptr) return st;
    st = ln_launch(layer_norm_bwd_columns<T, W>,
                   dim3(static_cast<unsigned>((static_cast<int64_t>(p.dim) + 255) / 256),
                        static_cast<unsigned>(p.parts), 1),
                   256, stream, p);
    return st != GEMM_OK ? st : finish<T, W>(p, stream);
}

template <class T, class W>
int backward(const LayerNormArgs &a)
{
    BwdParams<T, W> p{};
    p.dY = static_cast<const T *>(a.dY);
    p.X = static_cast<const T *>(a.X);
    p.gamma = static_cast<const W *>(a.gamma);
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.dX = static_cast<T *>(a.Y);
    p.part = a.dgamma ? a.workspace : nullptr;
    p.rows = a.rows;
    p.dim = static_cast<int32_t>(a.dim);
    p.parts = static_cast<int32_t>(layer_norm_parts(a.rows, a.dim, a.sm_count));
    p.inv_dim = 1.0f / static_cast<float>(a.dim);
    p.withhold = a.withhold;
    p.limit = a.timeout_cycles ? a.timeout_cycles : 1ull << 31;   // about a second
    p.status = a.status;
    p.dgamma = static_cast<W *>(a.dgamma);
    p.dbeta = static_cast<W *>(a.dbeta);
    p.sm_count = a.sm_count;
    const uintptr_t x_bits = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.dY) |
                             reinterpret_cast<uintptr_t>(a.Y) |
                             (static_cast<uintptr_t>(a.dim) * sizeof(T));
    const uintptr_t w_bits = reinterpret_cast<uintptr_t>(a.gamma);
    constexpr int V = 16 / sizeof(T);
    const int pack = ln_pack_elements<T, W>(x_bits, w_bits);
    if (pack == V) return launch_packs<T, W, V>(p, a.device, a.sm_count, a.stream);
    if constexpr (V > 4)
        if (pack == V / 4) return launch_packs<T, W, V / 4>(p, a.device, a.sm_count, a.stream);
    return launch_packs<T, W, 1>(p, a.device, a.sm_count, a.stream);
}

}  // namespace

namespace gemm_sm103 {

// The most parts, one per block of the row kernels, that a call writes.  Rows
// of up to 512 elements go eight or more at a time, longer ones one at a time,
// with the block's threads taking eight elements each: so many blocks that an
// SM holds some 1024 threads, but no more than two per SM or one per eight
// rows, whichever is more, for a part costs as much as a row's writes.
int64_t layer_norm_parts(int64_t rows, int64_t dim, int sm_count)
{
    const int64_t per = dim <= 512 ? 8 : 1;
    const int64_t blocks = dim <= 512 ? 4 : (dim > 5120 ? 1 : (8192 / dim > 2 ? 8192 / dim : 2));
    const int64_t sms = sm_count;
    int64_t parts = (rows + per - 1) / per;
    if (parts > blocks * sms) parts = blocks * sms;
    const int64_t enough = rows / 8 > 2 * sms ? rows / 8 : 2 * sms;
    return parts < enough ? parts : enough;
}

int launch_layer_norm_bwd(const LayerNormArgs &a)
{
    return ln_dispatch(a.xtype, a.wtype, [&](auto t, auto w) { return backward<decltype(t), decltype(w)>(a); });
}

}  // namespace gemm_sm103
