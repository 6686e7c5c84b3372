// rms_norm_bwd.cu -- gradients of the RMS norm.  With h the stream that the
// forward pass kept, z = h rstd and g = dy gamma,
//
//   dx     = dh + rstd (g - z sum(g z) / dim)      (sum over a row)
//   dgamma = sum dy z                              (sum over all rows)
//
// where dh is the gradient that reaches the stream past the norm (absent: 0); dx
// is the gradient of both of the forward pass's summands.  Bound by memory: dY, H
// and dH are read once and dX written once.  As in layer norm's backward pass a
// block walks rows, a thread always has the same columns and keeps their sums in
// registers, one partial sum per block and column goes to the workspace, and a
// second kernel adds those in a fixed order without loss: no atomics, the same
// bits every time.
#include "norm_bwd.cuh"
#include "rms_norm.cuh"

namespace {

using namespace gemm_sm103;

template <class T, class W>
struct RmsBwdParams {
    const T *dY, *H;
    const T *dH;      // NULL: none
    const W *gamma;   // NULL: ones
    const float *rstd;
    T *dX;
    float *part;      // (parts, dim); NULL: dgamma is not wanted
    int64_t rows;
    int32_t dim;
    int32_t parts;    // blocks
    float inv_dim;
    int32_t stages;   // rows under way per block (the ring kernel)
    int32_t arrays;   // of a row: 3 with dH, else 2 (the ring kernel)
    int32_t withhold; // test hook: 1 = the ring's rows are not loaded; 0 in every normal call
    uint64_t limit;   // SM clocks of a wait (the ring kernel)
    unsigned long long *status;
    W *dgamma;
    int32_t sm_count;
};

__host__ __device__ constexpr int rms_bwd_threads(int tpr) { return tpr < 0 ? -tpr : (tpr <= 32 ? 256 : tpr); }

// Rows in registers, the next row's loads under way while a row's sum is taken.
template <class T, class W, int V, int NV, int TPR>
__global__ void __launch_bounds__(rms_bwd_threads(TPR)) rms_norm_bwd_kernel(RmsBwdParams<T, W> p)
{
    constexpr int R = TPR > 0 ? rms_bwd_threads(TPR) / TPR : 1;   // rows at a time
    static_assert(TPR <= 32 || R == 1, "lanes of a warp or a block per row");
    // Rows of lanes without one: a warp holds several.
    constexpr bool kShared = TPR > 0 && TPR < 32;
    __shared__ float sh[2][ln_warps(TPR)];
    extern __shared__ float comb[];   // R > 1: (R, dim)
    griddep_wait();
    griddep_launch_dependents();
    const int tpr = ln_threads<TPR>();
    const int t = R > 1 ? static_cast<int>(threadIdx.x) % tpr : static_cast<int>(threadIdx.x);
    const int sub = R > 1 ? static_cast<int>(threadIdx.x) / tpr : 0;
    constexpr int P = V * NV / 2;   // pair m: elements 2m, 2m + 1 of the packs in order
    constexpr bool kReload = sizeof(T) == 4 || V * NV > 8;   // gamma again for every row, from L1
    float2 dg[P], gm[P];
    auto inside = [&](int i) { return (i * tpr + t) * V < p.dim; };
    auto load_gamma = [&]() {
        LnPack<W, V> pg[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.gamma && inside(i)) pg[i].load(p.gamma + (i * tpr + t) * V);
            else pg[i].fill(1.0f);
        }
#pragma unroll
        for (int m = 0; m < P; ++m) gm[m] = ln_pair_of(pg, m);
    };
    if constexpr (!kReload) load_gamma();
#pragma unroll
    for (int m = 0; m < P; ++m) dg[m] = make_float2(0.0f, 0.0f);
    LnPack<T, V> nh[NV], nd[NV], ns[NV];
    float next_rstd = 0.0f;
    auto load = [&](int64_t row) {
        const bool in = !kShared || row < p.rows;
        const int64_t at = row * p.dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (in && inside(i)) {
                nh[i].load(p.H + at + k);
                nd[i].load(p.dY + at + k);
            } else {
                nh[i].fill(0.0f);
                nd[i].fill(0.0f);   // adds nothing to any sum
            }
            if (p.dH && in && inside(i)) ns[i].load(p.dH + at + k);
            else ns[i].fill(0.0f);
        }
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
    load(there(row));
    for (int it = 0; lead < p.rows; lead += step, row += step, it ^= 1) {
        LnPack<T, V> ph[NV], pd[NV], ps[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ph[i] = nh[i];
            pd[i] = nd[i];
            ps[i] = ns[i];
        }
        const float rstd = next_rstd;
        load(there(row + step));
        if constexpr (kReload) load_gamma();
        float2 z[P], g[P];
        float2 s = make_float2(0.0f, 0.0f);
        const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
        for (int m = 0; m < P; ++m) {
            const float2 d = ln_pair_of(pd, m);
            z[m] = mul_f32x2(ln_pair_of(ph, m), rstd2);
            g[m] = mul_f32x2(d, gm[m]);
            s = fma_f32x2(g[m], z[m], s);
            dg[m] = fma_f32x2(d, z[m], dg[m]);
        }
        const float c = ln_row_sum<TPR>(s.x + s.y, sh[it]) * p.inv_dim;
        T *dx = p.dX + row * p.dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (!inside(i) || (kShared && row >= p.rows)) continue;
            LnPack<T, V> out;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int m = (i * V + j) / 2;
                const float v = rstd * fmaf(ln_half(z[m], i * V + j), -c, ln_half(g[m], i * V + j));
                out.e[j] = ln_round<T>(ps[i][j] + v);
            }
            out.store(dx + k);
        }
    }
    if (p.part == nullptr) return;
    float *out = p.part + static_cast<int64_t>(blockIdx.x) * p.dim;
    if constexpr (R == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (k >= p.dim) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) out[k + j] = ln_half(dg[(i * V + j) / 2], i * V + j);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * tpr + t) * V;
            if (k >= p.dim) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) comb[sub * p.dim + k + j] = ln_half(dg[(i * V + j) / 2], i * V + j);
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

// Rows through a ring of bulk copies in shared memory, `stages` rows ahead, a
// block per row at a time.  A slot is free once every thread has its pieces in
// registers, which the row sum's barrier says; with 16 elements in each of 1024
// threads (kReread) they are read a second time instead of being kept, and the slot is
// refilled one row later.  Every wait is bounded: on expiry
// the site is recorded in the device status word and the block leaves.
//
// Rows that are not whole 16-byte pieces (kShift) are taken with the whole pieces that
// they lie in, from the first one on: a block's rows lie a multiple of a piece's elements
// apart, so that all of them begin at the same place in their first piece, a thread's
// columns are the same in each and only the first and the last piece of a row have
// elements that are not its own (16384 x 4097 fp16 88 us; 262 us element by element).
// Blocks per SM that the registers are held to.
__host__ __device__ constexpr int rms_ring_blocks(int tpr, int per)
{
    if (tpr > 0) return 1024 / tpr;
    return per > 8 && tpr != -320 ? 1 : 2;
}

template <class T>
constexpr int kPiece = 16 / static_cast<int>(sizeof(T));   // elements

// Bytes of a row's place in the ring.
template <class T, bool kShift>
__host__ __device__ __forceinline__ uint32_t rms_row_bytes(int dim)
{
    const uint32_t bytes = static_cast<uint32_t>(dim) * static_cast<uint32_t>(sizeof(T));
    return kShift ? (bytes + 15u) / 16u * 16u + 16u : bytes;
}

// TPR > 0: the row is exactly the threads' elements, no bounds to check.
template <class T, class W, int NV, int TPR, bool kShift>
__global__ void __launch_bounds__(rms_bwd_threads(TPR), rms_ring_blocks(TPR, kPiece<T> * NV)) rms_norm_bwd_ring(RmsBwdParams<T, W> p)
{
    constexpr int V = kPiece<T>;
    constexpr bool kFull = TPR > 0;
    constexpr bool kReload = kShift || sizeof(T) == 4 || V * NV > 8;   // gamma again for every row, from L1
    // 16 elements in each of 1024 threads, which have 64 registers each.
    constexpr bool kReread = V * NV > 8 && (TPR == 1024 || TPR == -1024);
    constexpr int P = V * NV / 2;
    extern __shared__ uint4 ring[];   // (stages, arrays, dim) elements: H, dY, dH
    __shared__ float sh[2][ln_warps(TPR)];
    __shared__ uint64_t full_mem[kRingStages];
    __shared__ volatile int failed[2];
    __shared__ uint4 edge_mask[2];   // kShift: of the row's first and last piece
    // kShift: the first and the last warp have the edges to see to.
    constexpr int kIssuer = kShift ? 32 : 0;
    const int t = static_cast<int>(threadIdx.x), tpr = ln_threads<TPR>();
    // Elements in front of the row in its first piece: the same number for all rows of
    // the block.
    const int shift = kShift ? static_cast<int>((reinterpret_cast<uint64_t>(p.H + static_cast<int64_t>(blockIdx.x) * p.dim) & 15u) / sizeof(T)) : 0;
    auto column = [&](int i) { return (i * tpr + t) * V - shift; };   // of pack i's first element
    auto inside = [&](int i) { return kFull || column(i) < p.dim; };
    auto whole = [&](int i) { return !kShift || (column(i) >= 0 && column(i) + V <= p.dim); };
    auto own = [&](int k) { return k >= 0 && k < p.dim; };
    const uint32_t row_bytes = rms_row_bytes<T, kShift>(p.dim), slot_bytes = static_cast<uint32_t>(p.arrays) * row_bytes;
    const uint32_t ring_base = smem_addr(ring), full0 = smem_addr(full_mem);
    if (t == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(full0 + 8u * s, 1);
        failed[0] = failed[1] = 0;
        fence_mbar_init();
    }
    if (kShift && t < 2) {
        const int tail = (p.dim + shift) % V;   // elements in the last piece, 0: all
        T keep[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool in = t == 0 ? j >= shift : (tail == 0 || j < tail);
            memset(&keep[j], in ? 0xFF : 0, sizeof(T));
        }
        memcpy(&edge_mask[t], keep, 16);
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    auto source = [&](int h) { return h == 0 ? p.H : (h == 1 ? p.dY : p.dH); };
    auto fetch = [&](uint32_t row, int s) {
        const uint32_t bar = full0 + 8u * static_cast<uint32_t>(s);
        const uint32_t dst = ring_base + static_cast<uint32_t>(s) * slot_bytes;
        if constexpr (kShift) {
            // The arrays' rows begin alike: one window for all.
            const uint32_t bytes = static_cast<uint32_t>(p.dim) * static_cast<uint32_t>(sizeof(T));
            const uint64_t size = static_cast<uint64_t>(p.rows) * bytes, at = static_cast<uint64_t>(row) * bytes;
            const uint64_t base = reinterpret_cast<uint64_t>(p.H);
            const RingWindow w(base + at, bytes, base, base + size);
            const uint32_t n = static_cast<uint32_t>(w.end - w.begin);
            // Elements in pieces that reach past the tensor's ends, one by one; the
            // arrival below releases them to the waiting threads, and the fence orders
            // them before the copies of the slot's later rows.
            if (w.begin > w.src || w.end < w.last) {
                uint8_t *to = reinterpret_cast<uint8_t *>(ring) + (dst - ring_base);
                for (int h = 0; h < p.arrays; ++h) {
                    const uint64_t from = reinterpret_cast<uint64_t>(source(h)) - base;
                    auto edge = [&](uint64_t a, uint64_t b) {
                        for (; a < b; a += sizeof(T))
                            *reinterpret_cast<T *>(to + h * row_bytes + (a - w.first)) = *reinterpret_cast<const T *>(from + a);
                    };
                    if (w.begin > w.src) edge(w.src, w.begin);
                    if (w.end < w.last) edge(w.end, w.last);
                }
                fence_proxy_async_smem();
            }
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.arrays) * n);
            for (int h = 0; h < p.arrays; ++h)
                bulk_load(dst + static_cast<uint32_t>(h) * row_bytes + static_cast<uint32_t>(w.begin - w.first),
                          reinterpret_cast<const uint8_t *>(source(h)) + (w.begin - base), n, bar);
            return;
        }
        mbar_arrive_expect_tx(bar, slot_bytes);
        const int64_t at = static_cast<int64_t>(row) * p.dim;
        bulk_load(dst, p.H + at, row_bytes, bar);
        bulk_load(dst + row_bytes, p.dY + at, row_bytes, bar);
        if (p.dH) bulk_load(dst + 2u * row_bytes, p.dH + at, row_bytes, bar);
    };
    // Rows as unsigned 32-bit numbers: the ones past the end may pass 2^31.
    const uint32_t step = gridDim.x, rows = static_cast<uint32_t>(p.rows);
    uint32_t row = blockIdx.x;
    if (t == kIssuer && p.withhold == 0)
        for (int s = 0; s < p.stages && row + static_cast<uint32_t>(s) * step < rows; ++s)
            fetch(row + static_cast<uint32_t>(s) * step, s);
    // kShift: gamma behind the ring, with the rows' columns.
    constexpr bool kGammaShared = kShift && sizeof(T) == 2 && !kReread;
    W *gamma_row = reinterpret_cast<W *>(reinterpret_cast<uint8_t *>(ring) + static_cast<size_t>(p.stages) * slot_bytes);
    if constexpr (kGammaShared) {
        W w[V * NV];   // all loads under way at once
#pragma unroll
        for (int u = 0; u < V * NV; ++u) {
            const int k = u * tpr + t - shift;
            w[u] = p.gamma && own(k) ? __ldg(p.gamma + k) : ln_round<W>(1.0f);
        }
#pragma unroll
        for (int u = 0; u < V * NV; ++u) {
            const int k = u * tpr + t;
            if (k < (p.dim + 2 * V - 1) / V * V) gamma_row[k] = w[u];
        }
        __syncthreads();
    }

    float2 dg[P], gm[P];
    auto load_gamma = [&]() {
        LnPack<W, V> pg[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            pg[i].fill(1.0f);
            if ((!kGammaShared && !p.gamma) || !inside(i)) continue;
            if constexpr (kGammaShared) {
                pg[i].load_shared(gamma_row + (i * tpr + t) * V);
            } else if constexpr (kShift) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (own(column(i) + j)) pg[i].e[j] = __ldg(p.gamma + column(i) + j);
            } else {
                pg[i].load(p.gamma + column(i));
            }
        }
#pragma unroll
        for (int m = 0; m < P; ++m) gm[m] = ln_pair_of(pg, m);
    };
    // gamma of elements j and j + 1 of pack i, from L1.
    auto gamma_of = [&](int i, int j) {
        const int k = column(i) + j;
        if (!p.gamma || !inside(i)) return make_float2(1.0f, 1.0f);
        if constexpr (kShift) {
            return make_float2(own(k) ? ln_float(__ldg(p.gamma + k)) : 0.0f, own(k + 1) ? ln_float(__ldg(p.gamma + k + 1)) : 0.0f);
        } else {
            LnPack<W, 2> w;
            w.load(p.gamma + k);
            return w.pair(0);
        }
    };
    if constexpr (!kReload) load_gamma();
#pragma unroll
    for (int m = 0; m < P; ++m) dg[m] = make_float2(0.0f, 0.0f);
    float next_rstd = row < rows ? __ldg(p.rstd + row) : 0.0f;
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; row < rows; row += step, it ^= 1) {
        const float rstd = next_rstd;
        if (row + step < rows) next_rstd = __ldg(p.rstd + row + step);
        if (!mbar_try_wait(full0 + 8u * static_cast<uint32_t>(s), ph)) {
            const long long t0 = clock64();
            while (!mbar_try_wait(full0 + 8u * static_cast<uint32_t>(s), ph))
                if (static_cast<uint64_t>(clock64() - t0) > p.limit) {
                    failed[it] = 1;
                    break;
                }
        }
        const uint8_t *slot = reinterpret_cast<const uint8_t *>(ring) + static_cast<size_t>(s) * slot_bytes;
        // Pack i of array h of the row; of H and dY zeros for what is not the row's own,
        // which add nothing to any sum.
        auto piece = [&](LnPack<T, V> &pack, int h, int i) {
            if (!inside(i)) {
                pack.fill(0.0f);
                return;
            }
            pack.load_shared(reinterpret_cast<const T *>(slot + static_cast<size_t>(h) * row_bytes) + (i * tpr + t) * V);
            if (kShift && h < 2 && !whole(i)) {
                const uint4 mask = edge_mask[column(i) < 0 ? 0 : 1];
                uint4 raw;
                memcpy(&raw, pack.e, 16);
                raw = make_uint4(raw.x & mask.x, raw.y & mask.y, raw.z & mask.z, raw.w & mask.w);
                memcpy(pack.e, &raw, 16);
            }
        };
        T *dx = p.dX + static_cast<int64_t>(row) * p.dim;
        auto put = [&](const LnPack<T, V> &pack, int i) {
            if (whole(i)) {
                pack.store(dx + column(i));
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (own(column(i) + j)) dx[column(i) + j] = pack.e[j];
            }
        };
        float2 z[P];   // in the end dX
        float2 sum2 = make_float2(0.0f, 0.0f);
        const float2 rstd2 = make_float2(rstd, rstd);
        if constexpr (kReread) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                LnPack<T, V> px, pd;
                piece(px, 0, i);
                piece(pd, 1, i);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float2 d = pd.pair(j), zz = mul_f32x2(px.pair(j), rstd2);
                    float2 &acc = dg[i * (V / 2) + j];
                    acc = fma_f32x2(d, zz, acc);
                    sum2 = fma_f32x2(mul_f32x2(d, gamma_of(i, 2 * j)), zz, sum2);
                }
            }
            const float c = ln_row_sum<TPR>(sum2.x + sum2.y, sh[it]) * p.inv_dim;
            if (failed[it]) {   // the same answer for every thread: set before the barrier
                ok = false;
                break;
            }
            // The slot of the row before, which every thread has left.
            if (t == kIssuer && p.stages > 1) {
                const uint32_t next = row + static_cast<uint32_t>(p.stages - 1) * step;
                if (row != blockIdx.x && next < rows) fetch(next, s == 0 ? p.stages - 1 : s - 1);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!inside(i)) continue;
                LnPack<T, V> px, pd, ps, out;
                piece(px, 0, i);
                piece(pd, 1, i);
                if (p.dH) piece(ps, 2, i);
                else ps.fill(0.0f);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float2 zz = mul_f32x2(px.pair(j), rstd2), gz = mul_f32x2(pd.pair(j), gamma_of(i, 2 * j));
                    out.set_pair(j, fma_f32x2(fma_f32x2(zz, make_float2(-c, -c), gz), rstd2, ps.pair(j)));
                }
                put(out, i);
            }
            if (p.stages == 1) {
                __syncthreads();   // the one slot is read
                if (t == kIssuer && row + step < rows) fetch(row + step, 0);
            }
        } else {
            if constexpr (kReload) load_gamma();
            LnPack<T, V> px[NV], pd[NV], ps[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                piece(px[i], 0, i);
                piece(pd[i], 1, i);
            }
            if (p.dH) {
#pragma unroll
                for (int i = 0; i < NV; ++i) piece(ps[i], 2, i);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) ps[i].fill(0.0f);
            }
            float2 g[P];
#pragma unroll
            for (int m = 0; m < P; ++m) {
                const float2 d = ln_pair_of(pd, m);
                z[m] = mul_f32x2(ln_pair_of(px, m), rstd2);
                g[m] = mul_f32x2(d, gm[m]);
                sum2 = fma_f32x2(g[m], z[m], sum2);
                dg[m] = fma_f32x2(d, z[m], dg[m]);
            }
            const float c = ln_row_sum<TPR>(sum2.x + sum2.y, sh[it]) * p.inv_dim;
            if (failed[it]) {   // the same answer for every thread: set before the barrier
                ok = false;
                break;
            }
            if (t == kIssuer) {
                const uint32_t next = row + static_cast<uint32_t>(p.stages) * step;
                if (next < rows) fetch(next, s);
            }
            const float2 neg_c2 = make_float2(-c, -c);
#pragma unroll
            for (int m = 0; m < P; ++m)
                z[m] = fma_f32x2(fma_f32x2(z[m], neg_c2, g[m]), rstd2, ln_pair_of(ps, m));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!inside(i)) continue;
                LnPack<T, V> out;
#pragma unroll
                for (int j = 0; j < V / 2; ++j) out.set_pair(j, z[i * (V / 2) + j]);
                put(out, i);
            }
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
    float *out = p.part + static_cast<int64_t>(blockIdx.x) * p.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int k = column(i);
        if (!inside(i)) continue;
        if constexpr (!kShift) {   // dim is a multiple of V, the workspace on the 16-byte grid
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float2 a = dg[(i * V + j) / 2], b = dg[(i * V + j) / 2 + 1];
                *reinterpret_cast<float4 *>(out + k + j) = make_float4(a.x, a.y, b.x, b.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (own(k + j)) out[k + j] = ln_half(dg[(i * V + j) / 2], i * V + j);
        }
    }
}

// Rows longer than a block holds: dX in two passes over the row ...
template <class T, class W>
__global__ void __launch_bounds__(1024) rms_norm_bwd_long(RmsBwdParams<T, W> p)
{
    __shared__ float sh[2][32];
    griddep_wait();
    griddep_launch_dependents();
    int it = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, it ^= 1) {
        const int64_t at = row * p.dim;
        const float rstd = __ldg(p.rstd + row);
        float s = 0.0f;
        for (int64_t k = threadIdx.x; k < p.dim; k += 1024) {
            const float g = ln_float(p.dY[at + k]) * (p.gamma ? ln_float(p.gamma[k]) : 1.0f);
            s = fmaf(g, ln_float(p.H[at + k]) * rstd, s);
        }
        const float c = ln_row_sum<1024>(s, sh[it]) * p.inv_dim;
        for (int64_t k = threadIdx.x; k < p.dim; k += 1024) {
            const float g = ln_float(p.dY[at + k]) * (p.gamma ? ln_float(p.gamma[k]) : 1.0f);
            const float v = fmaf(ln_float(p.H[at + k]) * rstd, -c, g);
            p.dX[at + k] = ln_round<T>(fmaf(v, rstd, p.dH ? ln_float(p.dH[at + k]) : 0.0f));
        }
    }
}

// ... and the columns' partial sums, a thread per column, rows blockIdx.y,
// blockIdx.y + parts, ...
template <class T, class W>
__global__ void __launch_bounds__(256) rms_norm_bwd_columns(RmsBwdParams<T, W> p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (k >= p.dim) return;
    for (int64_t part = blockIdx.y; part < p.parts; part += gridDim.y) {
        float dg = 0.0f;
        for (int64_t row = part; row < p.rows; row += p.parts)
            dg = fmaf(ln_float(p.dY[row * p.dim + k]), ln_float(p.H[row * p.dim + k]) * __ldg(p.rstd + row), dg);
        p.part[part * p.dim + k] = dg;
    }
}

// The second kernel, if dgamma is wanted: 32 warps per block for short rows, whose few
// columns few blocks share, and for many parts.
template <class T, class W>
int finish(const RmsBwdParams<T, W> &p, cudaStream_t stream)
{
    if (p.part == nullptr) return GEMM_OK;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.dim) + 31) / 32), 1, 1);
    const float *part = p.part;
    if (p.parts > 2 * p.sm_count || (p.parts > p.sm_count && p.dim <= 32 * p.sm_count))
        return ln_launch(norm_bwd_finish<W, 32>, grid, 1024, stream, part, p.dgamma, p.dgamma, p.parts, p.dim);
    return ln_launch(norm_bwd_finish<W, 16>, grid, 512, stream, part, p.dgamma, p.dgamma, p.parts, p.dim);
}

template <class T, class W>
int launch(void (*kern)(RmsBwdParams<T, W>), const RmsBwdParams<T, W> &p, int threads, size_t smem, cudaStream_t stream)
{
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(p.parts), 1, 1);
    lc.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaLaunchKernelEx(&lc, kern, p) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

template <class T, class W, int V, int NV, int TPR>
int launch_one(const RmsBwdParams<T, W> &p, cudaStream_t stream)
{
    // Threads: those of the template, or the whole warps that NV packs each need.
    const int64_t packs = (static_cast<int64_t>(p.dim) + V - 1) / V;
    const int BT = TPR > 0 ? rms_bwd_threads(TPR) : static_cast<int>(((packs + NV - 1) / NV + 31) / 32 * 32);
    constexpr int R = TPR > 0 ? rms_bwd_threads(TPR) / TPR : 1;
    const int st = launch(rms_norm_bwd_kernel<T, W, V, NV, TPR>, p, BT,
                          R > 1 ? static_cast<size_t>(R) * p.dim * sizeof(float) : 0, stream);
    return st != GEMM_OK ? st : finish<T, W>(p, stream);
}

// The ring kernel, where one row fits a block's share of the shared memory.
template <class T, class W, int NV, int TPR, bool kShift>
int launch_ring(RmsBwdParams<T, W> p, int device, cudaStream_t stream, bool *done)
{
    constexpr int V = kPiece<T>;
    const int64_t packs = (static_cast<int64_t>(p.dim) + (kShift ? 2 * V - 2 : V - 1)) / V;
    const int threads = TPR > 0 ? TPR : static_cast<int>(((packs + NV - 1) / NV + 31) / 32 * 32);
    // Blocks per SM: those of the launch bound, or more where they are small.
    const int fit_blocks = V * NV > 8 ? rms_ring_blocks(TPR, V * NV) : 1024 / threads;
    const int budget = (227 * 1024 - fit_blocks * 2048) / fit_blocks;
    p.arrays = p.dH ? 3 : 2;
    const int64_t stage = p.arrays * static_cast<int64_t>(rms_row_bytes<T, kShift>(p.dim));
    constexpr bool kGammaShared = kShift && sizeof(T) == 2 && TPR != -1024;
    const int64_t gamma_bytes = kGammaShared ? (static_cast<int64_t>(p.dim) + 2 * V - 1) / V * V * static_cast<int64_t>(sizeof(W)) : 0;
    const int64_t fit = (budget - gamma_bytes) / stage;
    *done = fit >= 1;
    if (fit < 1) return GEMM_OK;
    p.stages = static_cast<int32_t>(fit < kRingStages ? fit : kRingStages);
    const int64_t wave = static_cast<int64_t>(fit_blocks) * p.sm_count;
    if (p.parts > wave) p.parts = static_cast<int32_t>(wave);
    if (kShift && p.parts < p.rows) {   // a block's rows begin alike
        p.parts = p.parts / V * V;
        *done = p.parts > 0;
        if (p.parts == 0) return GEMM_OK;
    }
    auto kern = rms_norm_bwd_ring<T, W, NV, TPR, kShift>;
    static std::atomic<int> prepared[kMaxDevices];
    if (!prepared[device].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        prepared[device].store(1, std::memory_order_release);
    }
    const int st = launch(kern, p, threads, static_cast<size_t>(p.stages * stage + gamma_bytes), stream);
    if (st != GEMM_OK) {
        prepared[device].store(0, std::memory_order_release);
        return st;
    }
    return finish<T, W>(p, stream);
}

template <class T, class W>
int launch_long(const RmsBwdParams<T, W> &p, cudaStream_t stream)
{
    int st = ln_launch(rms_norm_bwd_long<T, W>, dim3(static_cast<unsigned>(p.parts), 1, 1), 1024, stream, p);
    if (st != GEMM_OK || p.part == nullptr) return st;
    st = ln_launch(rms_norm_bwd_columns<T, W>,
                   dim3(static_cast<unsigned>((static_cast<int64_t>(p.dim) + 255) / 256),
                        static_cast<unsigned>(p.parts), 1),
                   256, stream, p);
    return st != GEMM_OK ? st : finish<T, W>(p, stream);
}

// Rows of more than 512 elements through the ring.
template <class T, class W, bool kShift>
int launch_rows(const RmsBwdParams<T, W> &p, int device, cudaStream_t stream)
{
    constexpr int V = kPiece<T>, N = 8 / V;   // packs of 8 elements
    const int64_t packs = (static_cast<int64_t>(p.dim) + (kShift ? 2 * V - 2 : V - 1)) / V;
    bool done = false;
    int st = GEMM_OK;
    // Thread counts as for layer norm: rows that fill a power of 2 of threads, then
    // any others, with as many warps as the row needs.
    if constexpr (!kShift) {
        if (packs == 128 * N) st = launch_ring<T, W, N, 128, false>(p, device, stream, &done);
        else if (packs == 256 * N) st = launch_ring<T, W, N, 256, false>(p, device, stream, &done);
        else if (packs == 512 * N) st = launch_ring<T, W, N, 512, false>(p, device, stream, &done);
        else if (packs == 1024 * N) st = launch_ring<T, W, N, 1024, false>(p, device, stream, &done);
        if (done || st != GEMM_OK) return st;
    }
    if (packs <= 512 * N) st = launch_ring<T, W, N, -512, kShift>(p, device, stream, &done);
    else if (packs <= 320 * 2 * N) st = launch_ring<T, W, 2 * N, -320, kShift>(p, device, stream, &done);
    else if (packs <= 512 * 2 * N) st = launch_ring<T, W, 2 * N, -512, kShift>(p, device, stream, &done);
    else if (packs <= 1024 * 2 * N) st = launch_ring<T, W, 2 * N, -1024, kShift>(p, device, stream, &done);
    return done || st != GEMM_OK ? st : launch_long<T, W>(p, stream);
}

// Rows of up to 512 elements by lanes of a warp, V elements at a time; layer_norm_parts
// counts on it.
template <class T, class W, int V>
int launch_short(const RmsBwdParams<T, W> &p, cudaStream_t stream)
{
    const int64_t packs = (static_cast<int64_t>(p.dim) + V - 1) / V;
    constexpr int N = 8 / V;   // packs of 8 elements
    if constexpr (V > 2) {
        // Short rows (a head's width) share a warp.
        if (packs <= 8 * N) return launch_one<T, W, V, N, 8>(p, stream);
        if (packs <= 16 * N) return launch_one<T, W, V, N, 16>(p, stream);
    }
    if (packs <= 32 * N) return launch_one<T, W, V, N, 32>(p, stream);
    return launch_one<T, W, V, 2 * N, 32>(p, stream);
}

template <class T, class W>
int backward(const RmsNormArgs &a)
{
    RmsBwdParams<T, W> p{};
    p.dY = static_cast<const T *>(a.dY);
    p.H = static_cast<const T *>(a.X);
    p.dH = static_cast<const T *>(a.dH);
    p.gamma = static_cast<const W *>(a.gamma);
    p.rstd = a.rstd;
    p.dX = static_cast<T *>(a.dX);
    p.part = a.dgamma ? a.workspace : nullptr;
    p.rows = a.rows;
    p.dim = static_cast<int32_t>(a.dim);
    p.parts = static_cast<int32_t>(layer_norm_parts(a.rows, a.dim, a.sm_count));
    p.inv_dim = 1.0f / static_cast<float>(a.dim);
    p.withhold = a.withhold;
    p.limit = a.timeout_cycles ? a.timeout_cycles : 1ull << 31;   // about a second
    p.status = a.status;
    p.dgamma = static_cast<W *>(a.dgamma);
    p.sm_count = a.sm_count;
    const uintptr_t all[] = {reinterpret_cast<uintptr_t>(a.X), reinterpret_cast<uintptr_t>(a.dY),
                             reinterpret_cast<uintptr_t>(a.dX), reinterpret_cast<uintptr_t>(a.dH ? a.dH : a.X)};
    const uintptr_t x_bits = all[0] | all[1] | all[2] | all[3] | (static_cast<uintptr_t>(a.dim) * sizeof(T));
    const uintptr_t w_bits = reinterpret_cast<uintptr_t>(a.gamma);
    constexpr int V = kPiece<T>;
    const int pack = ln_pack_elements<T, W>(x_bits, w_bits);
    if (a.dim <= 512) {
        if (pack == V) return launch_short<T, W, V>(p, a.stream);
        if constexpr (V > 4)
            if (pack == V / 4) return launch_short<T, W, V / 4>(p, a.stream);
        return launch_short<T, W, 1>(p, a.stream);
    }
    if (pack == V) return launch_rows<T, W, false>(p, a.device, a.stream);
    // All arrays' rows begin at the same place of a 16-byte piece, or their elements are
    // taken one by one, as are a few short rows, for which the ring is not worth its
    // setting up (300 x 2047 bf16 9.6 us with it, 7.5 us without; 1000 x 1023 fp32 8.5 and
    // 8.1; 4000 x 2047 fp16 22 and 33).
    const bool few = a.dim * static_cast<int64_t>(sizeof(T)) <= 4096 && a.rows <= 4 * static_cast<int64_t>(p.parts);
    if (!few && (((all[0] ^ all[1]) | (all[0] ^ all[2]) | (all[0] ^ all[3])) & 15u) == 0)
        return launch_rows<T, W, true>(p, a.device, a.stream);
    if (a.dim <= 512 * 8) return launch_one<T, W, 1, 8, -512>(p, a.stream);
    if (a.dim <= 512 * 16) return launch_one<T, W, 1, 16, -512>(p, a.stream);
    return launch_long<T, W>(p, a.stream);
}

}  // namespace

namespace gemm_sm103 {

int launch_rms_norm_bwd(const RmsNormArgs &a)
{
    return ln_dispatch(a.xtype, a.wtype, [&](auto t, auto w) { return backward<decltype(t), decltype(w)>(a); });
}

}  // namespace gemm_sm103
