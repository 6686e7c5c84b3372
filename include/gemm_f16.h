/*
 * gemm_f16.h -- C ABI of the GB300 (sm_103a) half-precision GEMM with a fused
 * ReLU epilogue.
 *
 * Operation.  C = R(A @ B) for dense row-major IEEE binary16 matrices
 * A (M,K), B (K,N) and C (M,N), products accumulated in fp32, R(x) = max(x, 0)
 * when relu = 1 (every x <= 0, -0 and NaN give +0) and R(x) = x when relu = 0,
 * then one round-to-nearest-even cast to binary16.  This is the kernel of
 * "Writing High-Performance Kernels in TileLang, from GEMM to MLA"
 * (atlascloud.ai), section "Let's write a GEMM": float16 A, B and C, a float
 * accumulator cleared per output tile, ReLU on the accumulator, one copy back
 * to float16.  relu = 0 is the plain GEMM of the TileLang-MUSA lesson
 * (7yue.com, section 3) and of the nxmr.cn A100 benchmark (section 2.2).
 *
 * Layout.  Leading dimensions are implied: K for A, N for B and N for C (no
 * stride arguments, as in the pages' T.Tensor((M,K)) ... declarations).
 *
 * Ownership.  The caller owns every buffer.  gemm_f16 (and every automatic
 * choice, configuration 0) allocates nothing per call.  Only an explicit
 * request for a workspace K split (the K-split bits of gemm_f16_ex or
 * gemm_f16_tx on a configuration whose split uses a workspace) takes that
 * workspace from the stream-ordered allocator on `stream` and returns it there;
 * gemm_f16_ex_noalloc uses a fixed scratch instead.  The library's device
 * state is one status word per GPU (a __device__ variable of the library's
 * module) that the kernels set when a bounded wait expires, the 16 MiB
 * scratch of gemm_f16_ex_noalloc, and the two copy streams per device that
 * the first gemm_f16_from_host call creates.  C must not overlap A or B.
 *
 * Asynchrony.  gemm_f16 and gemm_f16_ex only enqueue work on `stream` (a
 * cudaStream_t; NULL is the legacy default stream) and return without
 * synchronising.  Argument errors are reported synchronously by the return
 * value and launch nothing.  A device-side timeout is reported later, by
 * gemm_f16_check.  Every kernel of this library is launched as a
 * programmatic dependent of the kernel before it on the stream: its set-up
 * (barriers, tensor memory, descriptor prefetch) may run while that kernel
 * finishes, but it reads and writes no global memory before that kernel has
 * completed and its writes are visible, so the results are those of plain
 * stream order (also inside a CUDA graph capture).
 *
 * Thread safety.  All entry points may be called from several host threads.
 * Tensor-map descriptors are built on the host per call and passed by value
 * as kernel parameters; there is no cache to race on.
 *
 * Device.  Requires a compute capability 10.3 GPU (GB300) as the current
 * device; any other device gives GEMM_ERR_UNSUPPORTED_DEVICE.
 */
#ifndef GEMM_F16_H_
#define GEMM_F16_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_F16_VERSION 11

/* Return codes.  0 is success; every error is negative. */
enum gemm_f16_status {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = -1,        /* negative size, size > INT32_MAX, relu not 0/1,
                                         NULL or non-device pointer, buffer smaller than
                                         its matrix, C overlapping A or B, bad config id */
    GEMM_ERR_ALIGNMENT = -2,          /* a pointer not 16-byte aligned, or a row pitch
                                         (N or K for gemm_f16) not a multiple of 8 (the
                                         16-byte row-pitch rule of the tensor-memory-access
                                         unit) */
    GEMM_ERR_UNSUPPORTED_DEVICE = -3, /* current device is not compute capability 10.3 */
    GEMM_ERR_LAUNCH = -4,             /* the CUDA launch itself failed */
    GEMM_ERR_TIMEOUT = -5,            /* a kernel's bounded wait expired (gemm_f16_check) */
    GEMM_ERR_CUDA = -6                /* another CUDA runtime/driver call failed */
};

/*
 * gemm_f16 -- C = R(A @ B) on the current device, enqueued on `stream`.
 *
 *   A       device pointer, M*K binary16 values, row-major (leading dim K)
 *   B       device pointer, K*N binary16 values, row-major (leading dim N)
 *   C       device pointer, M*N binary16 values, row-major (leading dim N), written
 *   M,N,K   sizes, 0 <= M,N,K <= INT32_MAX
 *   relu    1: fused ReLU epilogue; 0: plain product
 *   stream  cudaStream_t (NULL: legacy default stream)
 *
 * Degenerate sizes: M == 0 or N == 0 is a no-op returning GEMM_OK (no pointer
 * is touched or checked).  K == 0 fills C with +0 (the empty sum; R(+0) = +0).
 * Alignment: A, B, C 16-byte aligned and N % 8 == 0, K % 8 == 0, else
 * GEMM_ERR_ALIGNMENT.  M is unrestricted; ragged edges in M, N and K are
 * handled in the kernel (out-of-range operand elements read as zero,
 * out-of-range C elements are never written).
 */
int gemm_f16(const void *A, const void *B, void *C,
             int64_t M, int64_t N, int64_t K, int relu, void *stream);

/*
 * Configuration arguments.  The low byte is a configuration id: 0 for the
 * automatic choice, 1..gemm_f16_num_configs() for a fixed tiling.  Flag bits
 * above it change how the persistent schedule treats the last, partly filled
 * wave of tiles:
 *
 *   GEMM_F16_NO_SPLIT  keep every work unit a whole tile.  Without it, the
 *                      tiles of a partly filled last wave may be split along
 *                      N into 2, 4 ... narrower units so that more SMs share
 *                      the tail.  Either way every output element is the same
 *                      K-ordered fp32 sum, so the results do not change.
 *
 * The K-split bits below may also be set; no other bit may be set
 * (GEMM_ERR_INVALID_ARG).  This tail policy is an
 * implementation choice of this library; the tile GEMM of the pages has no
 * persistent schedule and no tail split.
 */
#define GEMM_F16_CONFIG_ID_MASK 0xFF
#define GEMM_F16_NO_SPLIT 0x100

/*
 * K split (bits 9-11 and 12-16 of a config word).  The K loop of a tile can
 * be cut into slices that run on different SMs: when a problem has fewer
 * output tiles than the GPU has SMs (or SM pairs) for them, or for the tiles
 * of a partly filled last wave.  Each slice writes its fp32 partial product to
 * a workspace taken from the stream-ordered allocator (cudaMallocAsync /
 * cudaFreeAsync on `stream`: private to the call, ordered with its kernels,
 * legal inside a stream capture), and a second kernel adds the slices in
 * ascending order, applies the ReLU and rounds once to fp16.  Each such output
 * is then the fp32 sum of per-slice fp32 sums, a different order of the same
 * terms than without a split (results may differ in the last bits; ReLU is
 * still exactly max(plain, +0)).  The workspace holds slices x (split tiles)
 * x (tile area) floats.  With a K split every work unit is a whole tile or a
 * slice of one (GEMM_F16_NO_SPLIT is implied).
 *
 *   GEMM_F16_KSPLIT(n)    n = 2 .. 16: cut K into at most n slices of whole
 *                         64-element blocks (fewer if K has fewer blocks; none
 *                         for K <= 64).
 *   GEMM_F16_KSPLIT_AUTO  the slice count of a rule: if the configuration's
 *                         tiles are fewer than its CTA slots (one per SM, or
 *                         per SM pair or cluster), as many slices as fill the
 *                         slots once, at least 16 K blocks each, at most 16;
 *                         none if that is fewer than 2.
 *   GEMM_F16_KSPLIT_TAIL  only the tiles of a partly filled last wave, into as
 *                         many slices as fill the CTA slots once (at most 8, at
 *                         least 8 K blocks each); whole tiles before them.
 *   GEMM_F16_NO_KSPLIT    never split K.
 *
 * Configuration 0 takes whatever the offline-measured table chose for the
 * nearest measured shape among schedules that allocate nothing: whole tiles,
 * the tail split along N, and the cluster K split below; it never takes a
 * workspace K split.  A fixed configuration id without these bits does not
 * split K.  If the workspace cannot be allocated the call runs without a K
 * split.  The pages' tile GEMM keeps each tile's K loop in one block; this is
 * a scheduling choice of this library.
 */
#define GEMM_F16_NO_KSPLIT 0x200
#define GEMM_F16_KSPLIT_AUTO 0x400
#define GEMM_F16_KSPLIT_TAIL 0x800
#define GEMM_F16_KSPLIT_SHIFT 12
#define GEMM_F16_KSPLIT_MASK 0x1F000
#define GEMM_F16_KSPLIT(n) ((n) << GEMM_F16_KSPLIT_SHIFT)

/*
 * Cluster K split.  One configuration (gemm_f16_config_cluster_k(id) == 1;
 * "1sm_128x128_ck_s6") splits the K loop of each 128 x 128 output tile over
 * the CTAs of a cluster instead: CTA r of a cluster of S = 1, 2, 4 or 8 runs
 * the r-th slice, writes its fp32 partial tile to its own shared memory, and
 * then adds rows [r * 128/S, (r+1) * 128/S) of all S partials in rank order,
 * reading the other CTAs' shared memory through the cluster; it applies R,
 * rounds once to fp16 and stores C.  Nothing is allocated and no second
 * kernel runs.  The sums are those of the workspace K split with the same
 * slices (bit for bit).  For this configuration the K-split bits mean:
 * GEMM_F16_KSPLIT(n), n in {2, 4, 8}: clusters of n CTAs (halved while a
 * slice would be empty; any other n is GEMM_ERR_INVALID_ARG);
 * GEMM_F16_NO_KSPLIT: clusters of one CTA; no bit or GEMM_F16_KSPLIT_AUTO: the
 * size rule (the largest size up to 8 whose clusters hold every tile at once
 * and leave each CTA at least two 64-element K blocks);
 * GEMM_F16_KSPLIT_TAIL: GEMM_ERR_INVALID_ARG.  NN layout only.
 *
 * gemm_f16_ex -- gemm_f16 with an explicit kernel configuration.
 *
 *   config  0: automatic choice (what gemm_f16 uses); 1..gemm_f16_num_configs():
 *           a fixed tiling, see gemm_f16_config_name(); either may carry the
 *           flag bits above.  Every configuration computes the same function;
 *           they differ in tile shape and in the number of SMs that cooperate
 *           on one tile.  Unknown id or flag: GEMM_ERR_INVALID_ARG.
 */
int gemm_f16_ex(const void *A, const void *B, void *C,
                int64_t M, int64_t N, int64_t K, int relu, int config, void *stream);

/*
 * gemm_f16_ex_noalloc -- gemm_f16_ex that allocates nothing.  For callers that
 * may not allocate device memory while they run: a serving process that
 * reserved its memory budget up front (its own pool holds the GPU's memory,
 * so a stream-ordered allocation from the default pool can fail or push it
 * over budget), a plug-in whose host framework forbids allocation during its
 * execute step, or a latency-bound loop that must not enter the allocator.
 * When the call splits K through a workspace (GEMM_F16_KSPLIT(n),
 * GEMM_F16_KSPLIT_AUTO or GEMM_F16_KSPLIT_TAIL on a workspace configuration),
 * the fp32 slice partials go to a fixed scratch array of this library on the
 * current device (16 MiB, a file-scope device array that every device using
 * the library keeps until the process exits) instead of a stream-ordered
 * allocation; any other call (configuration 0, whose choices never use a
 * workspace, the cluster K split, no split) is exactly gemm_f16_ex.  The pages
 * have no counterpart: their tile GEMM has no K split and no workspace.
 *
 * Arguments, layouts, ownership and checks as for gemm_f16_ex.  In addition:
 *  - slices x (split tiles) x (tile area) x 4 bytes must fit the 16 MiB (e.g.
 *    1024 x 1024 in 128 x 128 tiles with 4 slices); a larger split is rejected
 *    (GEMM_ERR_INVALID_ARG) before anything is launched;
 *  - the scratch's address is looked up once per device, by the first call
 *    that splits K: make that call before any stream capture;
 *  - nothing in the scratch has to start at zero: every element the reduction
 *    reads was written by the GEMM kernel of the same call, and the scratch
 *    keeps whatever the last call left;
 *  - calls that overlap in time on one device (other streams, other threads,
 *    graph replays running concurrently) share the one scratch and race, with
 *    undefined results: serialise them (one stream, or events).
 */
int gemm_f16_ex_noalloc(const void *A, const void *B, void *C,
                        int64_t M, int64_t N, int64_t K, int relu, int config, void *stream);

/*
 * gemm_f16_tx -- C = R(op(A) @ op(B)) with transposed operand layouts (the
 * transpose_A / transpose_B options of the tile GEMM in "Writing
 * High-Performance Kernels in TileLang, from GEMM to MLA", section "Let's
 * write a GEMM"; the backward pair of the autograd wrapper in the TileLang-MUSA
 * lesson, section 6, needs op(B) = B^T for dA = dC @ B^T and op(A) = A^T for
 * dB = A^T @ dC).  op(A) is M x K and op(B) is K x N:
 *
 *   transa  0: A stored (M,K) row-major (leading dim K); 1: A stored (K,M)
 *           row-major (leading dim M) and op(A) = A^T
 *   transb  0: B stored (K,N) row-major (leading dim N); 1: B stored (N,K)
 *           row-major (leading dim K) and op(B) = B^T
 *
 * C is always (M,N) row-major.  Every stored row pitch (leading dimension)
 * must be a multiple of 8 elements, else GEMM_ERR_ALIGNMENT.  config as for
 * gemm_f16_ex; a configuration without transposed-layout kernels
 * (gemm_f16_config_layouts) returns GEMM_ERR_INVALID_ARG for transa or transb.
 * Everything else as gemm_f16.
 */
int gemm_f16_tx(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K,
                int transa, int transb, int relu, int config, void *stream);

/*
 * gemm_f16_relu_backward -- gradient through the fused ReLU epilogue:
 * dZ[i] = dC[i] if C[i] > 0 else +0, for i < n, where C is the stored output
 * of gemm_f16(..., relu = 1) and dC the gradient arriving at it.  "C[i] > 0"
 * means a positive, nonzero, non-NaN binary16 value (+inf included); the
 * pre-activation A @ B is not kept, so its sign is read from C (a product that
 * rounds to +0 in binary16 gets gradient 0).  The autograd wrapper of the
 * TileLang-MUSA lesson (7yue.com, section 6) then applies dA = dZ @ B^T and
 * dB = A^T @ dZ (gemm_f16_tx with transb = 1 and transa = 1).
 *
 *   dC, C, dZ  device pointers to n binary16 values, 2-byte aligned (16-byte
 *              alignment of all three selects the vectorised path)
 *   n          number of elements, >= 0 (0: no-op)
 *
 * dZ may be the same buffer as dC or C (in place); any other overlap is
 * GEMM_ERR_INVALID_ARG.  Asynchronous on `stream`, like gemm_f16.
 */
int gemm_f16_relu_backward(const void *dC, const void *C, void *dZ, int64_t n, void *stream);

/*
 * gemm_fp8_block_scaled -- FP8 block-scaled GEMM (a linear layer on an FP8
 * weight with per-block scales: fp8_block_scaled_linear(x, w_fp8, scale_w,
 * block=128) in the TileLang-MUSA lesson, 7yue.com, section 8.2; the
 * per-block scaling strategy named in the nxmr.cn TileLang article, section 7):
 *
 *   C[i,j] = R( sum_b SA[i,b] * SW[j/128, b] * sum_{k in block b, k < K} A[i,k] * W[j,k] )
 *
 * with blocks of 128 along K, accumulated in fp32 and rounded once to fp16
 * (R as for gemm_f16).  All pointers are device pointers on the current
 * device, owned by the caller:
 *
 *   A   (M,K) OCP FP8 E4M3 codes, row-major (leading dimension K bytes)
 *   SA  (M, ceil(K/128)) float32, row-major: one scale per row of A per K block
 *   W   (N,K) E4M3 codes, row-major: the weight as a linear layer stores it
 *       (out-features x in-features), so C = A @ W^T
 *   SW  (ceil(N/128), ceil(K/128)) float32, row-major: one scale per 128 x 128
 *       block of W
 *   C   (M,N) IEEE binary16, row-major, written in place
 *
 * A partial last block (K or N not a multiple of 128) keeps its own scale.
 * Checks before any launch, as for gemm_f16: sizes and relu
 * (GEMM_ERR_INVALID_ARG), K % 16 == 0 and N % 8 == 0 and 16-byte aligned A, W,
 * C, 4-byte aligned SA, SW (GEMM_ERR_ALIGNMENT), every buffer inside one
 * allocation of the current device, C overlapping no input
 * (GEMM_ERR_INVALID_ARG).  M == 0 or N == 0: no-op; K == 0: C = +0.  Only
 * enqueues on `stream`; device timeouts are reported by gemm_f16_check.
 */
int gemm_fp8_block_scaled(const void *A, const float *SA, const void *W, const float *SW, void *C,
                          int64_t M, int64_t N, int64_t K, int relu, void *stream);

/*
 * gemm_mxfp8_block_scaled -- the FP8 block-scaled GEMM of gemm_fp8_block_scaled
 * with every scale a power of two, given as an E8M0 byte (the scale type of
 * the OCP microscaling formats: value 2^(byte - 127), byte 0xFF is NaN):
 *
 *   C[i,j] = R( sum_b 2^(SA[i,b]-127) * 2^(SW[j/128,b]-127) * sum_{k in block b} A[i,k] * W[j,k] )
 *
 * Same blocks of 128, layouts and checks as gemm_fp8_block_scaled, except
 *
 *   SA  (M, ceil(K/128)) uint8 E8M0, row-major: one exponent per row of A per K block
 *   SW  (ceil(N/128), ceil(K/128)) uint8 E8M0, row-major: one per 128 x 128 block of W
 *
 * (no alignment requirement on SA and SW).  Restricting the scales to powers of
 * two lets the tensor core apply them inside the MMA (the block-scaled MMA
 * multiplies each 32-element product group by its two scales), so every K
 * block accumulates into one fp32 accumulator in tensor memory.  Quantizers
 * that round each block's scale up to a power of two produce such scales.
 * The sums are exact where the fp32 one of gemm_fp8_block_scaled is (small
 * integer operands); otherwise the two may differ in the last bits.
 */
int gemm_mxfp8_block_scaled(const void *A, const uint8_t *SA, const void *W, const uint8_t *SW, void *C,
                            int64_t M, int64_t N, int64_t K, int relu, void *stream);

/* Element types of the entry points that take one. */
enum gemm_f16_type {
    GEMM_TYPE_F16 = 0,    /* IEEE binary16 */
    GEMM_TYPE_BF16 = 1,   /* bfloat16 */
    GEMM_TYPE_F32 = 2     /* IEEE binary32 */
};

/*
 * MXFP4 matrices (OCP microscaling formats, version 1.0: E2M1 elements, one
 * E8M0 scale of value 2^(byte - 127) per 32 elements along K).  The packed
 * form of a (rows, K) matrix is two device buffers:
 *
 *   Q  codes, (rows, 16 ceil(K/32)) bytes row-major: element 2i of a row in
 *      the low half of byte i, element 2i + 1 in the high half.  Codes past K
 *      are zero.  16-byte aligned.
 *   S  scales, (ceil(rows/128), ceil(K/128), 512) bytes: the byte of row r and
 *      block b (elements 32 b .. 32 b + 31) at tile [r / 128][b / 4], byte
 *      (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4.  Bytes of blocks past K are
 *      zero (any value but 0xFF, NaN, serves); bytes of rows past `rows` are
 *      not used.  16-byte aligned.
 *
 * The scale order is the one the tensor core's scale memory is filled from:
 * a tile is 32 rows of 16 bytes, four words for rows r, r + 32, r + 64, r + 96.
 *
 * mxfp4_quantize -- X -> (Q, S).  Per block: e = floor(log2 max|x|) - 2, kept
 * within -127 .. 127, scale byte e + 127; element = x 2^-e rounded to the
 * nearest E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives), ties to even,
 * magnitudes above 6 to 6.  A block of zeros gets scale byte 0.  A block that
 * holds an infinity or a NaN gets scale byte 0xFF (NaN) and zero codes.
 *
 *   X      device pointer, elements of type `type` (enum gemm_f16_type),
 *          row-major: (rows, K) for trans = 0; (K, rows) for trans = 1, whose
 *          columns become the rows of the packed form (the weight of a linear
 *          layer stored in-features x out-features).  Aligned to its element.
 *   V      NULL, or a buffer like the (rows, K) matrix of X's type, row-major,
 *          that receives the values the codes stand for, rounded once to that
 *          type (exact in bfloat16 and binary32): what the product will see,
 *          for a quantisation error or a straight-through gradient
 *   rows, K  0 .. INT32_MAX; either 0: no-op
 *
 * Q, S and V overlap neither X nor each other.  Only enqueues on `stream`.
 * The pages name per-block scaling as the FP8 layer's preparation (nxmr.cn,
 * section 7; 7yue.com, section 8.2); the 4-bit form is this library's.
 */
int mxfp4_quantize(const void *X, int type, uint8_t *Q, uint8_t *S, void *V, int64_t rows, int64_t K, int trans,
                   void *stream);

/*
 * gemm_mxfp4 -- C = R(A @ W^T) from MXFP4 operands, fp16 C:
 *
 *   C[i,j] = R( sum_b 2^(sa[i,b]-127) * 2^(sw[j,b]-127) * sum_{k in block b} A[i,k] * W[j,k] )
 *
 * accumulated in fp32 by the block-scaled 4-bit MMA and rounded once to fp16
 * (R as for gemm_f16; a NaN scale gives NaN without ReLU, +0 with it).  The
 * choice of tiles, and over how many CTAs a tile's K range is divided (few rows
 * of A: up to 8), depends on the sizes and the GPU alone and every sum has a
 * fixed order, so equal calls give equal bits.
 * A, SA: the packed form of a (M,K) matrix; W, SW: of a (N,K) matrix (a linear
 * layer's weight, out-features x in-features); C (M,N) row-major.
 *
 * Checks as for gemm_mxfp8_block_scaled, with any K and N a
 * multiple of 8 (GEMM_ERR_ALIGNMENT), SA and SW 16-byte aligned.  M == 0 or
 * N == 0: no-op; K == 0: C = +0.  Only enqueues on `stream`, allocates
 * nothing; device timeouts are reported by gemm_f16_check.
 */
int gemm_mxfp4(const void *A, const uint8_t *SA, const void *W, const uint8_t *SW, void *C,
               int64_t M, int64_t N, int64_t K, int relu, void *stream);

/*
 * gemm_mxfp4_selftest_timeout -- exercises the bounded waits of gemm_mxfp4's
 * kernels (a test hook as gemm_f16_selftest_timeout; it computes nothing).  The
 * kernel of the problem is launched with a wait budget of `timeout_cycles` SM
 * clocks (2^16 .. 2^32) and its producer issues no load (withhold = 1), or the
 * operands' loads and not the scale tiles' (withhold = 2): the waits for them run
 * out, every role leaves its loop, the loads in flight land, the tensor memory
 * is freed and the kernel exits without writing C.  The next gemm_f16_check
 * returns GEMM_ERR_TIMEOUT.  Buffers and sizes are validated as for gemm_mxfp4.
 */
int gemm_mxfp4_selftest_timeout(const void *A, const uint8_t *SA, const void *W, const uint8_t *SW, void *C,
                                int64_t M, int64_t N, int64_t K, int withhold, uint64_t timeout_cycles,
                                void *stream);

/*
 * layer_norm_fwd -- layer norm over rows of `dim` elements (the norm in front of
 * a feed-forward or attention block; the TileLang-MUSA lesson, 7yue.com, has
 * its backward pass on its roadmap):
 *
 *   mean = sum x / dim,  rstd = 1 / sqrt(sum (x - mean)^2 / dim + eps)
 *   Y = (X - mean) rstd gamma + beta
 *
 * in fp32, rounded once to X's type.
 *
 *   X, Y         device pointers, (rows, dim) row-major, type xtype (enum
 *                gemm_f16_type)
 *   gamma, beta  NULL (ones, zeros) or dim elements of type wtype: xtype, or
 *                GEMM_TYPE_F32
 *   mean, rstd   NULL (not kept) or rows floats, written, for layer_norm_bwd
 *   eps          finite, >= 0
 *
 * Buffers are aligned to their element (16-byte alignment of all of them, the
 * weights too, and rows of a multiple of 16 bytes select the vectorised path;
 * 16-bit rows and weights on the grid of two elements go by pairs, anything
 * else element by element); outputs overlap neither
 * inputs nor each other.  rows == 0 or dim == 0: no-op.  Only enqueues on `stream`.
 */
int layer_norm_fwd(const void *X, const void *gamma, const void *beta, void *Y, float *mean, float *rstd,
                   int64_t rows, int64_t dim, float eps, int xtype, int wtype, void *stream);

/*
 * layer_norm_bwd -- gradients of layer_norm_fwd.  With z = (X - mean) rstd and
 * g = dY gamma:
 *
 *   dX = rstd (g - mean_row(g) - z mean_row(g z)),  dgamma = sum_rows dY z,  dbeta = sum_rows dY
 *
 * in fp32, each output rounded once; the sums over rows are taken in a fixed
 * order (equal calls give equal bits on one GPU model): a block's rows in fp32,
 * then the blocks' sums without loss, rounded once.
 *
 *   dY, X, gamma, mean, rstd  as given to and kept by layer_norm_fwd
 *   dX             (rows, dim) of type xtype
 *   dgamma, dbeta  dim elements of type wtype each, or both NULL (not wanted)
 *   workspace      layer_norm_bwd_workspace(rows, dim) bytes, 16-byte aligned,
 *                  written before it is read; may be NULL if dgamma is.  Calls
 *                  that may run at the same time need one each.
 *
 * Outputs and the workspace overlap neither inputs nor each other.  rows == 0:
 * dgamma and dbeta are filled with zeros; dim == 0: no-op.
 */
int layer_norm_bwd(const void *dY, const void *X, const void *gamma, const float *mean, const float *rstd, void *dX,
                   void *dgamma, void *dbeta, int64_t rows, int64_t dim, int xtype, int wtype, void *workspace,
                   int64_t workspace_bytes, void *stream);

/* Bytes of workspace layer_norm_bwd needs for these sizes on the current
 * device, or a negative status. */
int64_t layer_norm_bwd_workspace(int64_t rows, int64_t dim);

/*
 * layer_norm_bwd_selftest_timeout -- exercises the bounded wait of the kernel
 * that takes rows through a ring of bulk copies, rows of more than 512 elements
 * (1024 where they are not on the 16-byte grid) up to about 16384 (a test hook as
 * gemm_f16_selftest_timeout).  No row is loaded and a wait may take
 * `timeout_cycles` SM clocks (2^16 .. 2^32): every block records the site (9) and
 * leaves without writing dX.  The next gemm_f16_check returns GEMM_ERR_TIMEOUT.
 * Other rows wait for nothing: there the call computes dX.  Arguments are
 * validated as for layer_norm_bwd without weights.
 */
int layer_norm_bwd_selftest_timeout(const void *dY, const void *X, const float *mean, const float *rstd, void *dX,
                                    int64_t rows, int64_t dim, int xtype, uint64_t timeout_cycles, void *stream);

/*
 * rms_norm_fwd -- root-mean-square norm over rows of `dim` elements, after the
 * residual's addition (the norm in front of a feed-forward or attention block;
 * "Writing High-Performance Kernels in TileLang, from GEMM to MLA" has an RMS
 * norm among its kernels):
 *
 *   H = X + R (X itself without a residual),  rstd = 1 / sqrt(sum H^2 / dim + eps),  Y = H rstd gamma
 *
 * in fp32.  H is rounded to X's type, the norm is taken of the rounded H, and Y
 * is rounded once to X's type.  Squares beyond fp32 or below it are no matter; an
 * rstd beyond fp32 (eps = 0 and a root mean square below 2^-128) is an infinity.
 *
 *   X, R, H, Y  device pointers, (rows, dim) row-major, type xtype (enum
 *               gemm_f16_type).  R and H are both given or both NULL; H may be
 *               X or R itself (the residual stream updated in place)
 *   gamma       NULL (ones) or dim elements of type wtype: xtype, or
 *               GEMM_TYPE_F32
 *   rstd        NULL (not kept) or rows floats, written, for rms_norm_bwd
 *   eps         finite, >= 0
 *
 * Alignment, overlap and sizes as for layer_norm_fwd.  Only enqueues on `stream`.
 */
int rms_norm_fwd(const void *X, const void *R, const void *gamma, void *H, void *Y, float *rstd,
                 int64_t rows, int64_t dim, float eps, int xtype, int wtype, void *stream);

/*
 * rms_norm_fp8 -- rms_norm_fwd with Y quantised to E4M3 straight from fp32, as
 * the A operand of gemm_fp8_block_scaled or gemm_mxfp8_block_scaled:
 *
 *   Q  device pointer, (rows, dim) E4M3 codes, row-major
 *   S  (rows, ceil(dim/128)) scales: floats (pow2 = 0) or E8M0 bytes (pow2 = 1);
 *      see fp8_quantize
 *
 * dim may be any number (the products take multiples of 16).  Q and S overlap
 * nothing else.  Everything else as for rms_norm_fwd.
 */
int rms_norm_fp8(const void *X, const void *R, const void *gamma, void *H, void *Q, void *S, float *rstd,
                 int64_t rows, int64_t dim, float eps, int xtype, int wtype, int pow2, void *stream);

/*
 * rms_norm_bwd -- gradients of rms_norm_fwd.  With z = H rstd and g = dY gamma:
 *
 *   dX = dH + rstd (g - z mean_row(g z)),  dgamma = sum_rows dY z
 *
 * in fp32, each output rounded once; dX is the gradient of X and of R alike.
 * Sums over rows are taken in a fixed order (equal calls give equal bits on one
 * GPU model; how the buffers lie on the 16-byte grid is part of a call): a block's
 * rows in fp32, then the blocks' sums without loss, rounded once.
 *
 *   dY, H, gamma, rstd  as given to and kept by rms_norm_fwd (H: X itself where
 *                  there was no residual)
 *   dH             NULL (0) or the gradient that reaches H past the norm, like H
 *   dX             (rows, dim) of type xtype
 *   dgamma         dim elements of type wtype, or NULL (not wanted)
 *   workspace      rms_norm_bwd_workspace(rows, dim) bytes, 16-byte aligned,
 *                  written before it is read; may be NULL if dgamma is.  Calls
 *                  that may run at the same time need one each.
 *
 * Outputs and the workspace overlap neither inputs nor each other.  rows == 0:
 * dgamma is filled with zeros; dim == 0: no-op.
 */
int rms_norm_bwd(const void *dY, const void *H, const void *gamma, const float *rstd, const void *dH, void *dX,
                 void *dgamma, int64_t rows, int64_t dim, int xtype, int wtype, void *workspace,
                 int64_t workspace_bytes, void *stream);

/* Bytes of workspace rms_norm_bwd needs for these sizes on the current device,
 * or a negative status. */
int64_t rms_norm_bwd_workspace(int64_t rows, int64_t dim);

/*
 * rms_norm_bwd_selftest_timeout -- exercises the bounded wait of rms_norm_bwd's
 * ring of bulk copies, as layer_norm_bwd_selftest_timeout does (a test hook; the
 * same site, 9).
 */
int rms_norm_bwd_selftest_timeout(const void *dY, const void *H, const float *rstd, void *dX, int64_t rows,
                                  int64_t dim, int xtype, uint64_t timeout_cycles, void *stream);

/*
 * fp8_quantize -- X -> (Q, S) for the block-scaled FP8 products: E4M3 codes with
 * one scale per block of block_rows x 128 elements (block_rows = 1: the A operand;
 * 128: a weight).  With a = max |x| over a block:
 *
 *   pow2 = 0  S = a / 448, fp32;  Q = 448 x / a to the nearest E4M3, ties to even
 *   pow2 = 1  S = 2^e with the least e >= -127 for which a <= 448 2^e, stored as
 *             the E8M0 byte e + 127;  Q = x 2^-e to the nearest E4M3
 *
 * and S = 1 for a block of zeros.  A block that holds an infinity or a NaN gets
 * a NaN scale (E8M0 0xFF) and NaN codes.
 *
 *   X  device pointer, (rows, K) row-major, type `type` (enum gemm_f16_type)
 *   Q  (rows, K) codes;  S  (ceil(rows/block_rows), ceil(K/128)), row-major
 *
 * Buffers are aligned to their element (16-byte aligned rows of X take the
 * vectorised path) and do not overlap.  At most INT32_MAX blocks.  rows == 0 or
 * K == 0: no-op.  Only enqueues on `stream`.
 */
int fp8_quantize(const void *X, int type, void *Q, void *S, int64_t rows, int64_t K, int block_rows, int pow2,
                 void *stream);

/*
 * dropout_philox -- dropout: Y = R + X / (1 - p) where an element is kept, R where not (R NULL:
 * 0), rounded once to the type.  Element e of n is kept if word e % 4 of
 * Philox4x32-10 with the 64-bit counter halves (e / 4, offset) and the key `seed`
 * is at least floor(p 2^32): the mask is a function of seed, offset and e, and is
 * not stored.  Its gradient with respect to X is the same call on dY without R.
 *
 *   X, R, Y     device pointers, n elements of type `type` (enum gemm_f16_type);
 *               Y may be X or R itself, and overlaps nothing else
 *   p           0 <= p < 1
 *   offset_ptr  NULL, or a device pointer to a 64-bit offset, 8-byte aligned, read
 *               by the kernel in place of `offset`: a captured graph that advances
 *               it draws another mask at every replay
 *
 * A dropped element's value does not matter (an infinity or NaN of X is dropped
 * too); a -0 of R comes out as +0 there.  n == 0: no-op.  Only enqueues on `stream`.
 */
int dropout_philox(const void *X, const void *R, void *Y, int64_t n, int type, double p, uint64_t seed,
                   uint64_t offset, const void *offset_ptr, void *stream);

/*
 * Weights in 4 bits with group scales, for products with a few rows of 16-bit
 * activations.  The packed form of a weight W (N, K), W[n, k] = s (q - z) with
 * a 16-bit scale s and optionally a zero point z (else 8) per row and `group`
 * (32, 64 or 128) columns:
 *
 *   Q  (ceil(N/16), ceil(K/64), 512) bytes.  In the 512 bytes of 16 rows and 64
 *      columns the little-endian word 4 (4 g + t) + j holds rows g and g + 8
 *      (g < 8) and columns 32 (j / 2) + 8 t + 4 (j % 2) + c, c = 0 .. 3
 *      (t < 4, j < 4): nibbles 0 .. 3 are (g, c = 0), (g + 8, 0), (g, 2), (g + 8, 2),
 *      nibbles 4 .. 7 the same with c = 1 and 3
 *   S  (ceil(N/16), ceil(K/group), 16) scales, one per group and row
 *   Z  NULL, or as S in bytes, of which the low four bits count
 *
 * All three are 16-byte aligned.  Codes, scales and zero points of rows and columns
 * that W does not have may be anything; w4_quantize writes zeros.
 *
 * w4_quantize -- W -> (Q, S, Z).  Without Z: s = max|w| / 7 over the group rounded
 * to the scales' type, q = 8 + w / s; with Z: s = (max(w, 0) - min(w, 0)) / 15,
 * z = -min(w, 0) / s, q = z + w / s; z and q rounded to nearest even and kept in
 * 0 .. 15.  s is at most the type's largest number; a group whose scale rounds to
 * zero has s = 0; one that holds an infinity or a NaN has a NaN scale.
 *
 *   W      device pointer, elements of type `type`, (N, K) row-major for trans = 0,
 *          (K, N) for trans = 1 (a weight stored in-features x out-features)
 *   stype  the scales' type, GEMM_TYPE_F16 or GEMM_TYPE_BF16: the activations'
 *
 * W is aligned to its element; buffers do not overlap.
 * N == 0 or K == 0: no-op.  Only enqueues on `stream`.
 */
int w4_quantize(const void *W, int type, void *Q, void *S, uint8_t *Z, int64_t N, int64_t K, int group, int stype,
                int trans, void *stream);

/* Most rows of X that linear_w4 takes: it is made for tokens being generated. */
#define GEMM_W4_MAX_ROWS 64

/*
 * linear_w4 -- C = R(X @ W^T) from a packed 4-bit weight (R as for gemm_f16):
 *
 *   C[m,n] = R( sum_groups s[n] * sum_{k in group} X[m,k] (q[n,k] - z[n]) )
 *
 * q - z is exact, sums are fp32, the result is rounded once to X's type.
 *
 *   X  device pointer, (M, K) row-major, GEMM_TYPE_F16 or GEMM_TYPE_BF16, M up to
 *      GEMM_W4_MAX_ROWS; the scales have its type
 *   C  (M, N) row-major of X's type, overlapping no input
 *
 * Any N and K.  X and C are aligned to their element; rows of X on the 16-byte
 * grid take the vectorised path.  The division of K among blocks depends on the
 * sizes and the GPU alone and every sum has a fixed order, so equal values give
 * equal bits, wherever X lies.  M == 0 or N == 0: no-op; K == 0: C = +0.
 * Only enqueues on `stream`, allocates nothing.
 */
int linear_w4(const void *X, int type, const void *Q, const void *S, const uint8_t *Z, void *C, int64_t M, int64_t N,
              int64_t K, int group, int relu, void *stream);

/*
 * linear_w4_selftest_timeout -- exercises the bounded waits of linear_w4's tensor
 * memory kernel, here for more than 32 rows of X (a test hook as
 * gemm_f16_selftest_timeout; C is left alone).  Of the blocks that share K, the last
 * hands none of W's operands to the tensor core, the others do; a wait may take
 * timeout_cycles (2^16 .. 2^32) SM clocks; gemm_f16_check then returns
 * GEMM_ERR_TIMEOUT (site 3).
 */
int linear_w4_selftest_timeout(const void *X, int type, const void *Q, const void *S, const uint8_t *Z, void *C,
                               int64_t M, int64_t N, int64_t K, int group, uint64_t timeout_cycles, void *stream);

/*
 * linear_w4_few_selftest_timeout -- the same for 17 to 32 rows of X beside a weight
 * of at least 2^24 elements, K a multiple of 8: what that kernel takes of them.
 */
int linear_w4_few_selftest_timeout(const void *X, int type, const void *Q, const void *S, const uint8_t *Z, void *C,
                                   int64_t M, int64_t N, int64_t K, int group, uint64_t timeout_cycles, void *stream);

/* Launch geometry of gemm_fp8_block_scaled for this problem on the current
 * device: persistent grid in CTAs (CTA pairs over 256 x 256 output tiles) and
 * the number of tiles.  Either pointer may be NULL.  Launches nothing. */
int gemm_fp8_launch_info(int64_t M, int64_t N, int64_t K, int *grid_ctas, int *tiles);

/*
 * attention_fwd_f16 -- attention forward (the FlashAttention loop of the
 * TileLang-MUSA lesson, 7yue.com, section 5, "FlashAttention skeleton"; the
 * same loop in "Writing High-Performance Kernels in TileLang, from GEMM to
 * MLA", MLA section):
 *
 *   O[b,h,i,:] = sum_j softmax_j(sm_scale * Q[b,h,i,:] . K[b,h,j,:]) V[b,h,j,:]
 *
 * over keys j < seq, or j <= i when causal = 1.  Q, K, V, O: device pointers
 * to (batch, heads, seq, dim) row-major IEEE binary16 tensors on the current
 * device, owned by the caller; O is written in place and must not overlap Q,
 * K or V.  dim is 64 or 128.  sm_scale: the softmax temperature (the pages'
 * skeletons do not show one; 1/sqrt(dim) is the usual value).  Scores and
 * the running row sums are fp32, the probabilities are rounded to fp16 for
 * the second product, the output is rounded once to fp16.  Checks before any
 * launch: sizes >= 0, batch and heads <= 65535, dim, causal and a finite
 * sm_scale (GEMM_ERR_INVALID_ARG); 16-byte aligned buffers inside one
 * allocation of the current device.  Any size 0: no-op.  Only enqueues on
 * `stream`; device timeouts are reported by gemm_f16_check.
 */
int attention_fwd_f16(const void *Q, const void *K, const void *V, void *O, int64_t batch, int64_t heads,
                      int64_t seq, int64_t dim, float sm_scale, int causal, void *stream);

/*
 * attention_fwd_f16_queue -- attention_fwd_f16 with a work queue for the
 * causal case.  Same operation, arguments, checks and results (bit for bit:
 * the queue changes which SM computes a query block, not how).  With the
 * causal mask the query blocks have unequal work; attention_fwd_f16 gives
 * every SM a fixed share, this entry lets the SMs take the next block pair
 * from a queue, so they finish together.
 *
 * `queue`: device pointer to two 32-bit words, 4-byte aligned, on the current
 * device, owned by the caller, zero when the launch starts; the kernel leaves
 * them zero when it completes, so one queue serves any number of launches
 * that run one after another (on one stream).  Two launches that may run at
 * the same time (other streams, graphs) need separate queues: a shared one
 * gives wrong results.  NULL: the fixed shares of attention_fwd_f16.  Not
 * used when causal = 0 (every block pair has the same work).  Non-zero words
 * at launch make the launch skip work items (results undefined; no error).
 */
int attention_fwd_f16_queue(const void *Q, const void *K, const void *V, void *O, int64_t batch, int64_t heads,
                            int64_t seq, int64_t dim, float sm_scale, int causal, unsigned int *queue,
                            void *stream);

/* Operand layouts a configuration supports: bit (transa * 2 + transb) is set
 * for each supported (transa, transb); 0xF = all four, 0x1 = only (0,0).
 * GEMM_ERR_INVALID_ARG for an unknown id.  config 0 (automatic) supports all. */
int gemm_f16_config_layouts(int config);

/* 1 if configuration `config` splits K across the CTAs of a cluster (the
 * K-split bits then name the cluster size, see gemm_f16_ex), 0 if its K split
 * uses a workspace, GEMM_ERR_INVALID_ARG for an unknown id. */
int gemm_f16_config_cluster_k(int config);

/* Number of fixed configurations accepted by gemm_f16_ex (ids 1..n). */
int gemm_f16_num_configs(void);

/* Short name of a configuration id ("auto" for 0; flag bits are ignored), or
 * NULL for an unknown id or flag.  The string is static; the caller must not
 * free it. */
const char *gemm_f16_config_name(int config);

/* Configuration that gemm_f16 picks for this problem size on the current
 * device: a nonzero id, possibly with flag bits (GEMM_F16_NO_SPLIT,
 * GEMM_F16_KSPLIT(n)), which gemm_f16_ex accepts as it is; or a negative
 * status for invalid sizes. */
int gemm_f16_auto_config(int64_t M, int64_t N, int64_t K);

/*
 * gemm_f16_launch_info -- launch geometry gemm_f16_ex would use on the current
 * device for this problem and configuration (0 = automatic): the persistent
 * grid in CTAs (a multiple of the cluster size, at most one CTA per SM), the
 * CTAs per cluster (2 for the CTA-pair configurations), and the number of
 * output tiles.  Any output pointer may be NULL.  Launches nothing.
 */
int gemm_f16_launch_info(int64_t M, int64_t N, int64_t K, int config, int *grid_ctas, int *cluster_size,
                         int *tiles);

/*
 * gemm_f16_from_host -- end-to-end call on host buffers.
 *
 * Computes what gemm_f16(A_dev, B_dev, C_dev, ...) computes from A_host and
 * B_host and leaves the result in C_host: B is copied up, then A in row
 * panels (multiples of 256 rows, at least 1024, at most 8 panels); the GEMM of
 * each panel runs on `stream` as soon as its rows are on the device, and the
 * panel's rows of C are copied down while later panels are uploaded and
 * computed.  The copies run on two streams of this library per device
 * (created by the first call on that device; make it outside any stream
 * capture), ordered after the work already on `stream` and joined back into
 * it: synchronising `stream` is enough before reading C_host.  All six buffers
 * belong to the caller (host ones page-locked for asynchronous copies; device
 * ones sized as for gemm_f16); A_dev, B_dev and C_dev are overwritten.
 * Returns after enqueueing.  Errors as gemm_f16, plus GEMM_ERR_INVALID_ARG for
 * a NULL host pointer and GEMM_ERR_CUDA when a copy, event or stream cannot be
 * created or enqueued (work enqueued before that point still runs).
 * Calls on one stream run one after the other (each overwrites its device
 * buffers).  Calls on different streams with different device buffers may
 * overlap: a caller streaming independent problems through two streams and
 * two buffer sets gets one call's uploads started as soon as the previous
 * call's uploads are done (the uploads of all calls share one copy stream,
 * in call order).
 */
int gemm_f16_from_host(const void *A_host, const void *B_host, void *C_host,
                       void *A_dev, void *B_dev, void *C_dev,
                       int64_t M, int64_t N, int64_t K, int relu, void *stream);

/*
 * gemm_f16_check -- synchronises `stream`, then reads and clears the device
 * status word of the current device.  Returns GEMM_OK, GEMM_ERR_TIMEOUT if any
 * kernel launched on this device since the last check hit its wait limit (its
 * output is then incomplete), or GEMM_ERR_CUDA if the stream reported an
 * error.  The status word is shared by all launches on the device.
 */
int gemm_f16_check(void *stream);

/*
 * gemm_f16_selftest_timeout -- exercises the kernels' bounded waits (a test
 * hook; it computes nothing).  Launches the kernel of `config` (0 = automatic)
 * for the given problem with its TMA producer switched off and a wait budget
 * of `timeout_cycles` SM clocks (2^16 .. 2^32), so that the MMA thread's first
 * wait for operand data runs out: the kernel records the wait site, every role
 * leaves its loop, the tensor memory is freed and the kernel exits without
 * writing C.  The next gemm_f16_check on `stream` returns GEMM_ERR_TIMEOUT and
 * gemm_f16_last_timeout_record() holds the site (3: MMA waiting for operand
 * data; 4: epilogue waiting for an accumulator, in a CTA whose MMA thread
 * aborted first).  Buffers and sizes are validated as for gemm_f16; no copy,
 * MMA or store is in flight when the waits give up.  Nothing in the product
 * path calls this.
 */
int gemm_f16_selftest_timeout(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K,
                              int config, uint64_t timeout_cycles, void *stream);

/*
 * gemm_f16_tma_box_image -- layout diagnostic (nothing in the GEMM calls it).
 * Loads one box of box_rows x 64 binary16 values (128 bytes per row) at column
 * x, row y of the row-major matrix X (rows x cols) into shared memory exactly
 * as the GEMM loads its operand tiles -- the same tensor-map encoding (128-byte
 * swizzle, elements outside X read as zero) and the same TMA instruction --
 * and copies the raw shared-memory image, box_rows * 128 bytes, to `out`.
 * With the 128-byte swizzle, element (y + r, x + c) of X sits at byte
 * r * 128 + ((c / 8) ^ (r % 8)) * 16 + (c % 8) * 2 of the image, the layout
 * the GEMM's MMA descriptors read.  The pages discuss shared-memory tile
 * layout and bank conflicts ("Writing High-Performance Kernels in TileLang,
 * from GEMM to MLA"; the nxmr.cn A100 article, sections 3.3 and 6.2, where a
 * layout that disagrees with the copy's swizzle misplaces data by 16 bytes);
 * this call lets a test check that layout directly.
 *
 *   X         device pointer, rows * cols binary16 values, 16-byte aligned
 *   rows,cols 1 .. INT32_MAX; cols % 8 == 0 (GEMM_ERR_ALIGNMENT)
 *   box_rows  1 .. 256
 *   x, y      box origin (column, row); may lie partly or wholly outside X
 *             (negative too); x % 8 == 0 (a box starts on a 16-byte
 *             boundary, GEMM_ERR_ALIGNMENT)
 *   out       device pointer to box_rows * 128 bytes, 16-byte aligned, not
 *             overlapping X; written
 *
 * Asynchronous on `stream`; a load that does not land within its wait bound
 * is reported by gemm_f16_check (GEMM_ERR_TIMEOUT, site 7) and leaves `out`
 * unwritten.
 */
int gemm_f16_tma_box_image(const void *X, int64_t rows, int64_t cols, int64_t box_rows, int64_t x, int64_t y,
                           void *out, void *stream);

/* Raw value of the last timeout record read by gemm_f16_check on this thread
 * (0 if none): bits 0-7 the wait site, bits 8-31 the block index. */
uint64_t gemm_f16_last_timeout_record(void);

/* Why the last call on this thread that returned GEMM_ERR_INVALID_ARG or
 * GEMM_ERR_ALIGNMENT was rejected (static storage; "" if none yet). */
const char *gemm_f16_last_error_detail(void);

/* Human-readable text for a status code (static storage). */
const char *gemm_f16_strerror(int status);

/* GEMM_F16_VERSION of the built library. */
int gemm_f16_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F16_H_ */
