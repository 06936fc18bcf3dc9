/*
 * gemm_gb300.h -- C ABI of a GEMM library for one NVIDIA GB300 GPU (sm_103a).
 *
 * Every entry point computes the general matrix product of the copecc.github.io "GEMM"
 * page (section "核心问题与运算特征"):
 *
 *     C = alpha * op(A) * op(B) + beta * C          op(A): M x K, op(B): K x N, C: M x N
 *
 * with each C[i][j] the dot product of row i of op(A) and column j of op(B) (the same
 * section; also yekq.top "LeetGPU 第二题", section "题目描述").
 *
 * Layout.  All matrices are ROW-MAJOR.  A leading dimension is the element distance
 * between the first elements of two consecutive stored rows, and may exceed the logical
 * row length when rows are padded (copecc "GEMM" page, section "Leading Dimension (lda,
 * ldb, ldc)").  The transpose flags choose how a buffer is read (the role the op
 * arguments play in cublasSgemm on the ssxxe.cn page, section "三、cuBLAS 实现方式探究",
 * restated for row-major storage):
 *     opA = GEMM_OP_N: A stored M x K, op(A)[i][k] = A[i*lda + k], lda >= max(1, K)
 *     opA = GEMM_OP_T: A stored K x M, op(A)[i][k] = A[k*lda + i], lda >= max(1, M)
 *     opB = GEMM_OP_N: B stored K x N, op(B)[k][j] = B[k*ldb + j], ldb >= max(1, N)
 *     opB = GEMM_OP_T: B stored N x K, op(B)[k][j] = B[j*ldb + k], ldb >= max(1, K)
 *     C stored M x N, C[i][j] at C[i*ldc + j], ldc >= max(1, N)
 *
 * Ownership.  A, B and C are device memory owned by the caller (host memory for the
 * *_host entry points); the library never frees or retains them.  C must not overlap A or
 * B.  The library keeps scratch per (device, stream): a split-K workspace (64 MB and 8192
 * counters), two buffers for transposed fp32 operands and, for the *_host entry points, a
 * staging area; each is allocated when first needed, grown when a larger problem needs it
 * (after the stream's earlier work), kept until exit, and never allocated while the stream
 * is being captured (a call then takes a path that needs no new scratch, except where host
 * matrices must be staged).  At most 16 streams per device hold each kind: calls on further
 * streams run without split-K or transposition (same results within the stated bounds,
 * slower), and a *_host call on a further stream first synchronises the device and releases
 * the other streams' staging areas.  The *_host calls enqueue their work one host thread at
 * a time.
 *
 * Asynchrony.  A call validates its arguments on the host, launches on `stream` (a
 * cudaStream_t passed as void*; NULL means the legacy default stream of the current
 * device) and returns without waiting.  The return value reports argument errors and
 * launch errors only; gemm_get_device_status() reports errors raised inside a kernel.
 * Nothing aborts or exits the process.
 *
 * BLAS conventions.  M == 0 or N == 0: nothing is launched and GEMM_OK is returned.
 * K == 0 or alpha == 0: C = beta * C.  beta == 0: C is written without being read, so
 * NaN or Inf already in C does not propagate.  alpha and beta are host values.
 *
 * Thread safety.  Calls may come from several host threads.  Calls on one stream from
 * different threads must not overlap in time (a call may grow that stream's scratch while
 * the other enqueues work that uses it); calls that write the same C concurrently race, as
 * with any BLAS.
 */
#ifndef GEMM_GB300_H
#define GEMM_GB300_H

#include <stdint.h>

/* Symbols of this header are the only ones the shared library exports. */
#if defined(__GNUC__)
#define GEMM_API __attribute__((visibility("default")))
#else
#define GEMM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_OP_N = 0, GEMM_OP_T = 1 } gemm_op_t;

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_VALUE = 1,  /* bad size, op, leading dimension or NULL pointer */
    GEMM_ERR_MISALIGNED = 2,     /* pointer or leading dimension breaks the alignment rule */
    GEMM_ERR_UNSUPPORTED = 3,    /* size beyond the library's limits (see each call) */
    GEMM_ERR_LAUNCH = 4,         /* the CUDA runtime refused the launch */
    GEMM_ERR_DEVICE_TIMEOUT = 5, /* a kernel gave up waiting on a barrier (bounded wait) */
    GEMM_ERR_NO_DEVICE = 6       /* no usable sm_103 device is current */
} gemm_status_t;

/*
 * Strict-FP32 GEMM (SGEMM) on the CUDA cores: every product and sum is an IEEE fp32
 * fused multiply-add, never TF32 and never a reduced-precision tensor operation.
 * A, B, C: 4-byte aligned fp32 device pointers; any leading dimension is accepted (the
 * 16-byte vector paths are used only where pointer and leading dimension allow them).
 * Above 1e10 flops, an operand whose rows run along K (op(A) = N, op(B) = T) may first be
 * transposed into this stream's scratch buffer (8 bytes of traffic per element) so that
 * the kernel reads it with 16-byte copies; the result does not depend on it.
 * Limits: M, N, K < 2^31.
 */
GEMM_API gemm_status_t gemm_sgemm_f32(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K,
                             float alpha, const float *A, int64_t lda, const float *B,
                             int64_t ldb, float beta, float *C, int64_t ldc, void *stream);

/*
 * fp16-input GEMM with fp32 accumulation and fp32 output on the tcgen05 tensor cores
 * (the mixed-precision mode of the copecc "GEMM" page, section "Batched 执行与混合精度", and
 * of the dandandamowang.xyz "GEMM优化（二）" page): products of IEEE binary16 inputs are
 * summed in fp32, then C = alpha * sum + beta * C in fp32.
 * A, B: IEEE binary16 bit patterns (uint16_t), 2-byte aligned, any lda, ldb; an odd byte
 * address gives GEMM_ERR_MISALIGNED.  The tensor-memory-access unit reads rows only from a
 * 16-byte aligned base with a leading dimension that is a multiple of 8 elements; an operand
 * laid out otherwise is read by loader warps of the same kernel instead (each row copied as
 * the aligned 16-byte blocks that cover it, then shifted into place in shared memory; rows
 * at the ends of the operand's storage or cut by the matrix edge element by element), with
 * no extra launch and no scratch memory, at a fraction of the TMA path's rate.
 * C: fp32, 4-byte aligned, any ldc.
 * Limits: M, N, K < 2^31; lda, ldb < 2^35 elements.
 */
GEMM_API gemm_status_t gemm_hgemm_f16f32(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N,
                                int64_t K, float alpha, const uint16_t *A, int64_t lda,
                                const uint16_t *B, int64_t ldb, float beta, float *C,
                                int64_t ldc, void *stream);

/*
 * bfloat16-input GEMM with fp32 accumulation and fp32 output on the tcgen05 tensor cores:
 * the BF16 case of the mixed-precision mode of the copecc "GEMM" page, section "Batched 执行与
 * 混合精度" (FP16/BF16 inputs, FP32 accumulation).  Same rules as gemm_hgemm_f16f32, with
 * A and B holding bfloat16 bit patterns (the upper halves of IEEE binary32 values).
 */
GEMM_API gemm_status_t gemm_bgemm_bf16f32(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N,
                                          int64_t K, float alpha, const uint16_t *A, int64_t lda,
                                          const uint16_t *B, int64_t ldb, float beta, float *C,
                                          int64_t ldc, void *stream);

/*
 * Strided-batched forms (copecc "GEMM" page, section "Batched 执行与混合精度": one call runs
 * `batch` GEMMs of the same M, N, K whose operands sit strideA, strideB and strideC elements
 * apart).  Problem b computes
 *     C_b = alpha * op(A_b) * op(B_b) + beta * C_b,   X_b = X + b * strideX,
 * with the row-major rules of the single calls.  A stride of 0 shares that operand between
 * all problems; strideC must keep the outputs apart: strideC >= (M - 1) * ldc + N when
 * batch > 1 (else GEMM_ERR_INVALID_VALUE).  batch == 0 launches nothing.  A 16-bit
 * operand whose batch stride is not a multiple of 8 elements is read by the loader warps,
 * like one with an unaligned leading dimension (see gemm_hgemm_f16f32).
 * Limits: batch <= 2^31.
 */
GEMM_API gemm_status_t gemm_sgemm_f32_strided_batched(gemm_op_t opA, gemm_op_t opB, int64_t M,
                                                      int64_t N, int64_t K, float alpha,
                                                      const float *A, int64_t lda, int64_t strideA,
                                                      const float *B, int64_t ldb, int64_t strideB,
                                                      float beta, float *C, int64_t ldc,
                                                      int64_t strideC, int64_t batch, void *stream);

GEMM_API gemm_status_t gemm_hgemm_f16f32_strided_batched(gemm_op_t opA, gemm_op_t opB, int64_t M,
                                                         int64_t N, int64_t K, float alpha,
                                                         const uint16_t *A, int64_t lda,
                                                         int64_t strideA, const uint16_t *B,
                                                         int64_t ldb, int64_t strideB, float beta,
                                                         float *C, int64_t ldc, int64_t strideC,
                                                         int64_t batch, void *stream);

GEMM_API gemm_status_t gemm_bgemm_bf16f32_strided_batched(gemm_op_t opA, gemm_op_t opB, int64_t M,
                                                          int64_t N, int64_t K, float alpha,
                                                          const uint16_t *A, int64_t lda,
                                                          int64_t strideA, const uint16_t *B,
                                                          int64_t ldb, int64_t strideB, float beta,
                                                          float *C, int64_t ldc, int64_t strideC,
                                                          int64_t batch, void *stream);

/*
 * The three products on matrices in HOST memory: same arguments, layouts, leading-dimension
 * rules, results and errors as gemm_sgemm_f32, gemm_hgemm_f16f32 and gemm_bgemm_bf16f32,
 * but A, B and C are host pointers (page-locked, from cudaHostAlloc / cudaHostRegister /
 * torch pin_memory, for the call to stay asynchronous; pageable memory works too, with the
 * copies then synchronising as cudaMemcpyAsync does for it).  The source pages have no
 * counterpart: they copy operands in and results out around the kernel by hand.
 *
 * In order on `stream`, the call copies each stored operand -- and C when beta != 0 -- to a
 * device staging area of this (device, stream) pair as one contiguous copy that keeps the
 * caller's leading dimension, runs the device GEMM there, and copies the M x N elements of
 * C back into the caller's C (the row padding of an ldc > N matrix is neither read when
 * beta == 0 nor ever written).  It returns after enqueueing: A, B and C must stay alive and
 * unchanged until the stream has passed the call (cudaStreamSynchronize, or an event), and
 * C holds the result only then.  Calls on different streams overlap on the GPU (the copies
 * of one with the GEMM of another); calls on one stream run one after the other.
 *
 * The staging area is allocated by the first call on a stream and reallocated -- after
 * synchronising that stream -- when a larger problem arrives; it is kept until the process
 * exits (see Thread safety above for calls sharing a stream).  Returns GEMM_ERR_UNSUPPORTED without enqueueing anything when the area would have
 * to be (re)allocated while the stream is being captured, when device memory for it cannot
 * be had, or when a matrix spans more than 2^40 elements; GEMM_ERR_LAUNCH when a copy
 * cannot be enqueued (after the input copies, C may then be partly written or not at all).
 */
GEMM_API gemm_status_t gemm_sgemm_f32_host(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N,
                                           int64_t K, float alpha, const float *A, int64_t lda,
                                           const float *B, int64_t ldb, float beta, float *C,
                                           int64_t ldc, void *stream);
GEMM_API gemm_status_t gemm_hgemm_f16f32_host(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N,
                                              int64_t K, float alpha, const uint16_t *A, int64_t lda,
                                              const uint16_t *B, int64_t ldb, float beta, float *C,
                                              int64_t ldc, void *stream);
GEMM_API gemm_status_t gemm_bgemm_bf16f32_host(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N,
                                               int64_t K, float alpha, const uint16_t *A, int64_t lda,
                                               const uint16_t *B, int64_t ldb, float beta, float *C,
                                               int64_t ldc, void *stream);

/*
 * Allocation-free variant of gemm_sgemm_f32, for callers that must not allocate device
 * memory while they run: a framework whose own allocator owns the device memory and
 * forbids other cudaMalloc calls, or a latency-critical caller that cannot afford the
 * blocking, device-wide synchronisation or late failure of an allocation.  The source
 * pages have no counterpart to this entry point.
 *
 * Same arguments, rules and result as gemm_sgemm_f32 (strict FP32, row-major, caller-owned
 * A, B, C), computed by the split-K kernel (64 x 64 tiles, K split over up to 16 CTAs whose
 * partial tiles are added in a fixed order).  Its scratch -- arrival counters and partial
 * tiles -- lives in one statically sized device array of 16 MiB + 16 KiB that the library
 * holds on every GPU that loads it, until the process exits; the call itself never calls
 * cudaMalloc, cudaFree or any allocating routine.
 *
 * The K split count S is reduced until the split's scratch fits the array: at most 4096
 * tiles of 64 x 64 and tiles * S <= 1024 partial tiles.  S = 1 uses no scratch, so problems
 * too large to split still run (unsplit).
 * Limits: M, N, K < 2^31; larger sizes return GEMM_ERR_UNSUPPORTED without launching anything.
 * The first call on a device looks up the device address of the scratch array (with that
 * device current); make that first call before capturing the stream into a graph.
 * Every call shares the one array, whose contents persist between calls: the call clears
 * the counters it needs on `stream` before its kernel, but two calls whose work overlaps on
 * the GPU (e.g. on different streams) race on the array and corrupt each other's results.
 */
GEMM_API gemm_status_t gemm_sgemm_f32_noalloc(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N,
                                              int64_t K, float alpha, const float *A, int64_t lda,
                                              const float *B, int64_t ldb, float beta, float *C,
                                              int64_t ldc, void *stream);

/*
 * Waits for `stream`, then returns and clears the error word that kernels of this library
 * set on the current device when a bounded barrier wait expires (GEMM_ERR_DEVICE_TIMEOUT),
 * or GEMM_OK.  A kernel that sets the word leaves its output tile unwritten.  After a
 * timeout it also synchronises every stream of the current device that owns a split-K
 * workspace and zeroes that workspace's arrival counters, which an abandoned wait may have
 * left raised.
 */
GEMM_API gemm_status_t gemm_get_device_status(void *stream);

/* Static, human-readable name of a status code. */
GEMM_API const char *gemm_status_string(gemm_status_t status);

/* Library version as 10000 * major + 100 * minor + patch. */
GEMM_API int gemm_version(void);

/*
 * Number of kernels this process has launched through the library so far, on every device
 * and stream (GEMM kernels and the operand re-layout and scaling kernels).  For accounting:
 * the difference across a region counts the library's launches in it.  Needs no GPU.
 */
GEMM_API uint64_t gemm_kernel_launches(void);

/*
 * Measured FP32 fused multiply-add throughput of the current device, in TFLOP/s (2 flops
 * per multiply-add), written to *tflops: the strict-FP32 path's roofline denominator, next
 * to the figure derived from SM count x 128 FP32 lanes x 2 x clock.  A kernel of
 * independent packed multiply-add chains (fma.rn.f32x2) fills every SM; one untimed launch,
 * then the best of three launches timed with CUDA events on `stream` (synchronises it;
 * about a millisecond of GPU time).  Returns GEMM_ERR_INVALID_VALUE for a NULL output,
 * GEMM_ERR_NO_DEVICE without a current device, GEMM_ERR_LAUNCH when a launch or an event
 * fails (then *tflops is 0).
 */
GEMM_API gemm_status_t gemm_measure_fp32_fma_peak(void *stream, double *tflops);

/*
 * The tile configurations of the strict-FP32 path (a host function: needs no GPU), for
 * tools and tests.  Configuration `index` (0, 1, ... in the order the planner considers
 * them) is written to *out: its one-letter name, block tile BM x BN, K slice BK, thread tile
 * TM x TN, ring stages, threads per CTA, the CTAs per SM it is compiled for, the padding of
 * each [k][x] stage row in floats (0: XOR-swizzled rows), and its dynamic shared memory,
 * STAGES * BK * (BM + BN + 2 * pad) * 4 bytes -- the footprint arithmetic of the ssxxe.cn
 * GEMM page, section "2.1 矩阵分块利用Shared Memory", BK * (BM + BN) * 4 bytes per stage,
 * plus the padding.  Returns GEMM_ERR_INVALID_VALUE for an index past the last
 * configuration or a NULL output.
 */
typedef struct {
    char name;
    int bm, bn, bk, tm, tn, stages, threads, ctas_per_sm, row_pad, smem_bytes;
} gemm_sgemm_config_t;
GEMM_API gemm_status_t gemm_sgemm_config(int index, gemm_sgemm_config_t *out);

/*
 * Tile raster used by the kernels (a host function: needs no GPU).  It maps the t-th tile
 * of a tiles_m x tiles_n grid of output tiles to (tile_m, tile_n) so that consecutive
 * tiles sweep a group of 2^log_group tile rows column by column, which keeps the operand
 * tiles they share resident in L2 (copecc "GEMM" page, section "线程块网格重排 (Thread Block
 * Swizzling)"; with tiles_m = 2^log_group this is exactly that section's mapping).  The
 * last group may be shorter.  Returns GEMM_ERR_INVALID_VALUE for t outside the grid,
 * non-positive grid sizes, log_group outside [0, 16] or NULL outputs.
 */
GEMM_API gemm_status_t gemm_tile_raster(int64_t t, int64_t tiles_m, int64_t tiles_n, int log_group,
                               int64_t *tile_m, int64_t *tile_n);

/* ------------------------------------------------------------------------------------------
 * Routed products: linear layers whose weights differ from row to row, because a router gave
 * each token its experts or because each request brings an adapter of its own, and what decides
 * which rows meet which weights.  The source pages have no counterpart; rows, leading dimensions,
 * streams, statuses and asynchrony are those of the GEMM calls above.
 *
 * Every array is device memory owned by the caller, index arrays are int32, and no call keeps
 * anything from one call for the next: no scratch memory is allocated, so every call may be
 * captured into a graph.  Index values are checked on the device: an expert, adapter, row or
 * position outside its range counts as "none" and is skipped, never followed.
 *
 * Vocabulary.  T tokens, E experts, k experts per token.  SLOT t * k + j is the j-th choice of
 * token t.  The plan orders the slots by expert (stable: slots of one expert in ascending order)
 * and calls a slot's place in that order its POSITION: expert e owns positions
 * offsets[e] .. offsets[e + 1] - 1, tokens[position] is the slot's token, where[slot] its
 * position.  Slots without an expert (-1) have no position (where = -1); arrays of T * k
 * positions are then used only up to offsets[E].
 */
typedef enum { GEMM_TYPE_F32 = 0, GEMM_TYPE_F16 = 1, GEMM_TYPE_BF16 = 2 } gemm_type_t;
typedef enum { GEMM_SCORE_SOFTMAX = 0, GEMM_SCORE_SIGMOID = 1 } gemm_score_t;

/*
 * Routing to experts.  For each row x of logits (T x E, leading dimension ld, fp32 or 16-bit,
 * computed in fp32):
 *     s = softmax(x) or 1 / (1 + exp(-x)),   c = s + bias   (bias: E floats, or NULL)
 *     groups > 1: the E experts form `groups` runs of E / groups; a run's value is the sum of its
 *       group_top (1 or 2) largest c, and only the groups_kept runs of largest value stay
 *     ids[t]     = the top_k experts of largest c that stay, largest first
 *     weights[t] = scale * s[ids], divided by their sum first when renormalise is not 0
 * The bias (a load-balancing term) takes part in the choice only.  Without a bias the choice goes
 * by the logit, whose order is that of s.  Ties go to the lowest index, of experts and of runs.
 *
 * Masks: a logit of -inf or NaN, or a c of -inf or NaN, takes its expert out of the choice (and a
 * masked logit out of the softmax); +inf counts as the largest finite value.  Where fewer than
 * top_k experts are left the remaining ids are -1 with weight 0; a row with none is all -1.
 * Weights whose sum is 0 are 0.
 *
 * With offsets (E + 1), tokens (T * top_k) and where (T * top_k) the call also writes the plan;
 * all three NULL leaves it out.
 * Limits: 1 <= E <= 1024, 1 <= top_k <= min(32, E / groups * groups_kept), groups <= 32 dividing
 * E, T * max(E, top_k) < 2^31.  T == 0 writes offsets only.
 */
GEMM_API gemm_status_t gemm_moe_route(gemm_type_t type, int64_t T, int64_t E, const void *logits,
                                      int64_t ld, const float *bias, gemm_score_t score, int groups,
                                      int groups_kept, int group_top, int top_k, int renormalise,
                                      float scale, int32_t *ids, float *weights, int32_t *offsets,
                                      int32_t *tokens, int32_t *where, void *stream);

/*
 * Gradient of the weights of gemm_moe_route with respect to the logits, the choice held fixed:
 * dlogits (T x E, leading dimension ldd, the type of the logits) from dweights (T x top_k), the
 * logits and the ids of the forward call, with the same score, renormalise and scale.  With
 * s, S = sum over the row's ids of s[id]:
 *     ds[id_j] = scale * dw_j,  or renormalised  scale / S * (dw_j - sum_i dw_i s[id_i] / S)
 *     dx = s * (ds - sum(ds * s))  (softmax)     dx = ds * s * (1 - s)  (sigmoid)
 * Every element of dlogits is written; masked logits and rows without an expert get 0.
 */
GEMM_API gemm_status_t gemm_moe_route_backward(gemm_type_t type, int64_t T, int64_t E,
                                               const float *dweights, const void *logits, int64_t ld,
                                               const int32_t *ids, gemm_score_t score, int top_k,
                                               int renormalise, float scale, void *dlogits,
                                               int64_t ldd, void *stream);

/*
 * The plan of given choices ids (T x top_k, -1 or out of range: none; a token may name an expert
 * twice).  Limits: 1 <= E <= 1024, 1 <= top_k <= 1024, T * top_k < 2^31.
 */
GEMM_API gemm_status_t gemm_moe_plan(int64_t T, int64_t E, int top_k, const int32_t *ids,
                                     int32_t *offsets, int32_t *tokens, int32_t *where, void *stream);

/*
 * Rows out to their positions: out[where[t * k + j]] = w[t * k + j] * x[t], for all slots that have
 * a position below `positions`; weights NULL: 1.  x is T x H, out positions x H, both of `type`.
 */
GEMM_API gemm_status_t gemm_moe_dispatch(gemm_type_t type, int64_t T, int64_t H, int top_k,
                                         const void *x, int64_t ldx, const int32_t *where,
                                         const float *weights, int64_t positions, void *out,
                                         int64_t ldo, void *stream);

/*
 * Rows back to their tokens: y[t] = sum over j of weights[t * k + j] * rows[where[t * k + j]]
 * (weights NULL: 1), summed in fp32 in the order of j.  rows is positions x H of rows_type, y
 * T x H of y_type.  A token without a position gets 0.
 */
GEMM_API gemm_status_t gemm_moe_combine(gemm_type_t rows_type, gemm_type_t y_type, int64_t T, int64_t H,
                                        int top_k, const void *rows, int64_t ldr, int64_t positions,
                                        const int32_t *where, const float *weights, void *y,
                                        int64_t ldy, void *stream);

/*
 * Gradient of gemm_moe_combine: drows[where[slot]] = weights[slot] * dy[t] (drows and dy of `type`)
 * and dweights[slot] = the dot product of dy[t] and rows[where[slot]] in fp32 (0 for a slot without
 * a position).
 */
GEMM_API gemm_status_t gemm_moe_combine_backward(gemm_type_t type, gemm_type_t rows_type, int64_t T,
                                                 int64_t H, int top_k, const void *dy, int64_t lddy,
                                                 const void *rows, int64_t ldr, int64_t positions,
                                                 const int32_t *where, const float *weights,
                                                 void *drows, int64_t lddr, float *dweights,
                                                 void *stream);

/*
 * Gradient of the gated activation h = silu(gate) * up, pre = [gate | up] (rows x 2 I):
 *     dgate = dh * up * g (1 + gate (1 - g)),   dup = dh * gate * g,   g = 1 / (1 + exp(-gate))
 * pre and dpre (rows x 2 I) are of `type`, dh (rows x I) of dh_type (`type` or fp32); computed in
 * fp32.  dpre may be pre.
 */
GEMM_API gemm_status_t gemm_gated_silu_backward(gemm_type_t type, gemm_type_t dh_type, int64_t rows,
                                                int64_t I, const void *pre, int64_t ldp, const void *dh,
                                                int64_t lddh, void *dpre, int64_t lddp, void *stream);

/*
 * Grouped linear layer: for every group g and every position p of offsets[g] .. offsets[g + 1] - 1
 *     Y[p] = X[r(p)] * op(W_g),   r(p) = rows[p], or p when rows is NULL,
 * fp16 or bf16 inputs (`type`, not fp32), fp32 accumulation on the tensor cores, Y of y_type (fp32
 * or `type`), N columns.  W_g = W + g * strideW; opW = GEMM_OP_T reads it as stored N x K (a linear
 * layer's weight: Y = X W^T), opW = GEMM_OP_N as stored K x N (the layer's input gradient
 * dX = dY W).  X has x_rows rows; a position whose row is outside [0, x_rows) is computed as if its
 * row were zeros.  Y has y_rows rows; positions at or beyond it are not written.
 *
 * gated (opW = GEMM_OP_T only): W_g holds 2 N rows, N gate rows and then N up rows, and
 *     Y[p] = silu(gate) * up,   gate = X[r(p)] * W_gate^T,   up = X[r(p)] * W_up^T,
 * with both factors in fp32.  pre (y_rows x 2 N of `type`, or NULL) receives [gate | up], which
 * gemm_gated_silu_backward needs.
 *
 * offsets (groups + 1 values) must not decrease; values are clamped to [0, y_rows].  Y must not
 * overlap the inputs.  K == 0 writes zeros.
 *
 * work: y_rows * (K rounded up to a multiple of 64) elements of `type` for the call to use, or NULL.
 * With it, gathered rows (rows not NULL) of more than 64 positions per group on average are laid
 * out contiguously first, which is faster than gathering them in the product; the result is the
 * same.
 * Alignment: X, W, pre and work 16-byte aligned, ldx, ldw, strideW and ldp multiples of 8 elements, Y
 * 16-byte aligned with ldy a multiple of 8 (else GEMM_ERR_MISALIGNED); N and K are free.
 * Limits: groups <= 1024, y_rows and x_rows < 2^31, N and K < 2^24.
 */
GEMM_API gemm_status_t gemm_grouped_linear(gemm_type_t type, gemm_type_t y_type, int64_t groups,
                                           const int32_t *offsets, gemm_op_t opW, int gated,
                                           int64_t N, int64_t K, const void *X, int64_t ldx,
                                           int64_t x_rows, const int32_t *rows, const void *W,
                                           int64_t ldw, int64_t strideW, void *Y, int64_t ldy,
                                           int64_t y_rows, void *pre, int64_t ldp, void *work,
                                           void *stream);

/*
 * Weight gradient of the grouped linear layer: for every group
 *     dW_g = sum over positions p of the group of dY[p]^T * X[p]       (N x K, leading dimension lddw)
 * dY (positions x N) and X (positions x K) of `type` (fp16 or bf16), fp32 accumulation, dW of
 * dw_type (fp32 or `type`).  A group without positions gets zeros.  Where X's rows were gathered,
 * gemm_moe_dispatch lays them out first.
 * Alignment: dY, X, dW 16-byte aligned, all leading dimensions and strideDW multiples of 8
 * elements.  Limits as above.
 */
GEMM_API gemm_status_t gemm_grouped_weight_grad(gemm_type_t type, gemm_type_t dw_type, int64_t groups,
                                                const int32_t *offsets, int64_t N, int64_t K,
                                                const void *dY, int64_t lddy, const void *X,
                                                int64_t ldx, int64_t positions, void *dW,
                                                int64_t lddw, int64_t strideDW, void *stream);

/*
 * A shared linear layer with the low-rank adapters of many requests beside it:
 *     Y[t] = X[t] W^T + scales[a] * (X[t] A_a^T) B_a^T,     a = the adapter of token t,
 * X (T x K), W (N x K), A_a = A + a * strideA (R x K) and B_a = B + a * strideB (N x R) of `type`
 * (fp16 or bf16), Y (T x N) of y_type (fp32 or `type`).  Tokens lie request by request: request q
 * owns tokens segments[q] .. segments[q + 1] - 1 (requests + 1 values that do not decrease,
 * clamped to [0, T]) and uses adapter adapters[q]; an adapter outside [0, n_adapters) means none,
 * as does lying in no request.  scales: n_adapters floats, NULL: 1.  An adapter of a rank below R
 * is padded with zero rows of A_a.  An infinity or NaN in an adapter or in a token's row of X reaches
 * the tokens that use it only.
 *
 * The inner products scales[a] * X A^T are summed in fp32.  For many tokens they enter the second
 * product as sums of 16-bit parts: of bf16 to 16 bits (24 when Y is fp32); of fp16 to 22 bits from
 * 2^-3 up, and to 2^-25 below it, where the second part's own spacing is 2^-24 whatever the value (12 bits
 * are left at 2^-13: inner products that small want a larger A and a smaller B); those that the parts
 * cannot hold (beyond 65504) stay in fp32.
 *
 * work: gemm_lora_work_bytes(T, N, K, requests, R) bytes for the call to use (not kept; NULL when
 * there are no requests, no adapters, or R or K is 0).  That function gives the bytes for the current
 * device.
 * Alignment: X, W, A, B, Y and work 16-byte aligned; ldx, ldw, lda, ldb, ldy, strideA, strideB
 * multiples of 8 elements.  Limits: R <= 128, T < 2^24, requests < 2^24, N and K < 2^24, and
 * (T / 32 + requests) * 32 * 6 < 2^31.
 */
GEMM_API int64_t gemm_lora_work_bytes(int64_t T, int64_t N, int64_t K, int64_t requests, int64_t R);
GEMM_API gemm_status_t gemm_lora_linear(gemm_type_t type, gemm_type_t y_type, int64_t T, int64_t N,
                                        int64_t K, const void *X, int64_t ldx, const void *W,
                                        int64_t ldw, int64_t requests, const int32_t *segments,
                                        const int32_t *adapters, int64_t n_adapters, int64_t R,
                                        const void *A, int64_t lda, int64_t strideA, const void *B,
                                        int64_t ldb, int64_t strideB, const float *scales, void *Y,
                                        int64_t ldy, void *work, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_GB300_H */
