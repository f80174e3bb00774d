/*
 * sam.h -- C ABI of the shape-adaptive GEMM library for MI355X (gfx950).
 *
 * Operation (page "Scale coverage exposes a remaining GEMM gap", section
 * "Measurement contract and evidence"): C = A*B with compact row-major
 * A[M][K], B[K][N], C[M][N] (leading dimensions K, N, N), alpha one, beta
 * zero: C is write-only and its old contents are never read. Operands are
 * FP32, or bfloat16 / IEEE binary16 passed as raw 16-bit patterns; products
 * are accumulated in FP32 and C is always FP32 (the 16-bit operand runs of
 * page "Measured data point on fixed-tile vs shape-adaptive GEMM", section
 * "One more result that surprised us", there on other hardware).
 *
 * Shape adaptivity (same page, sections "The wall, and why we think it's
 * structural" and "The actual question"; page "Post-mortem: a GPU stack
 * without nvcc, cuBLAS, or LLVM", section 2.1): a dispatcher picks one of
 * several macro-tile / schedule variants from (M, N, K, dtype) alone, through
 * a frozen, source-controlled table. No timing happens at run time.
 *
 * Determinism (page "Measured data point ...", question 2; page
 * "Post-mortem ...", section 7): no atomics anywhere; the K sum of every
 * output runs in a fixed order per variant, and split-K partials are added
 * in split order 0, 1, ..., S-1 by a separate kernel. The same (M, N, K,
 * dtype) on the same library build gives the same plan and the same bits.
 *
 * Conventions shared by every entry point:
 *   - All pointers to operands, C and workspace are DEVICE pointers of the
 *     current HIP device; `stream` is a hipStream_t (NULL = default stream).
 *   - Calls are asynchronous: work is enqueued on `stream` and the call
 *     returns. The library never synchronises the host and keeps no pointer
 *     after returning; buffers must live until the stream work completes.
 *   - The caller owns and allocates everything (A, B, C, workspace). The
 *     library never allocates device memory on these paths.
 *   - Errors found before enqueueing (arguments, workspace size, device,
 *     launch) are returned as a negative sam_status; detail text is in
 *     sam_last_error() (per thread). Faults inside kernels surface at the
 *     caller's next synchronisation. No C++ exception crosses this ABI.
 *   - Sizes: M, N, K >= 0. M == 0 or N == 0 is a no-op returning SAM_OK.
 *     K == 0 writes +0.0f to every element of C. M*N, M*K and K*N must fit
 *     in int64 and every index below 2^31 elements per operand.
 *   - A, B, C, workspace base addresses must be 16-byte aligned, else
 *     SAM_ERR_MISALIGNED. Odd K or N are fine: such shapes take load paths
 *     that never form an unaligned vector address.
 *   - C must not overlap A, B or the workspace (SAM_ERR_INVALID_ARG).
 *   - Thread-safe: the variant table is immutable and module state is
 *     initialised once.
 */
#ifndef SAM_H
#define SAM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* SAM_MXFP8 / SAM_MXFP4 name block-scaled 8-bit / 4-bit operands
 * (sam_gemm_mxfp8, sam_gemm_mxfp4) in plan queries; the other entry points
 * take the first three. */
typedef enum { SAM_F32 = 0, SAM_BF16 = 1, SAM_F16 = 2, SAM_MXFP8 = 3, SAM_MXFP4 = 4 } sam_dtype;

typedef enum {
    SAM_OK = 0,
    SAM_ERR_INVALID_ARG = -1,        /* bad size, null or overlapping pointer */
    SAM_ERR_MISALIGNED = -2,         /* a base pointer not 16-byte aligned   */
    SAM_ERR_WORKSPACE = -3,          /* workspace smaller than the plan needs */
    SAM_ERR_UNSUPPORTED = -4,        /* forced variant cannot take this case  */
    SAM_ERR_UNSUPPORTED_DEVICE = -5, /* no gfx950 device / kernels not loadable */
    SAM_ERR_LAUNCH = -6,             /* the HIP runtime refused a launch      */
    SAM_ERR_INTERNAL = -7
} sam_status;

/* One dispatch decision. Plain old data; struct_size is set by the library
 * to sizeof(sam_plan) for ABI versioning. */
typedef struct {
    uint32_t struct_size;
    int32_t variant_id;        /* stable index into the variant table        */
    char name[64];             /* e.g. "f32_t256x256_w2x2_b32" + "_s4" ...    */
    int32_t dtype;             /* sam_dtype                                   */
    int32_t tile_m, tile_n, tile_k; /* macro tile; tile_k = K per LDS stage  */
    int32_t waves_m, waves_n;  /* wave grid inside a workgroup               */
    int32_t mfma_m;            /* MFMA block edge: 32 or 16                   */
    int32_t split_k;           /* 1 = single pass; >1 = partials + ordered sum;
                                  -1 = stream-K: grid_wgs persistent workgroups
                                  share the tiles' K iterations evenly, shared
                                  tiles are summed in a fixed order after */
    int32_t group_m;           /* grouped-raster height in tiles             */
    int32_t xcd_remap;         /* 1 = workgroup ids remapped per XCD          */
    int32_t a_vector, b_vector;/* 1 = 16-byte loads of A / B rows            */
    int64_t grid_wgs;          /* workgroups of the main kernel              */
    uint64_t workspace_bytes;  /* device workspace the call needs (0 if none) */
    double est_us;             /* the dispatcher's cost estimate, microseconds */
    int32_t raster_n;          /* 0: groups of group_m tile rows sweep the tile
                                  columns (M-major); 1: groups of group_m tile
                                  columns sweep the rows (N-major)           */
    int32_t operand_swap;      /* 1: the MFMA takes B's fragment as its first
                                  operand, so accumulators hold the transposed
                                  block (stored 16 bytes per lane)           */
    int64_t sk_dp_tiles;       /* stream-K: leading tiles run one per
                                  workgroup before the shared ones (16-bit)  */
    int32_t tuned;             /* 0 cost model, 1 frozen table (this shape),
                                  2 frozen table (a measured shape in the same
                                  half-octave bucket)                        */
} sam_plan;

/* The plan sam_gemm_<dtype> would run for this shape. Host only: touches no
 * device state and needs no GPU. Returns SAM_ERR_INVALID_ARG for negative
 * sizes or a null `out`. */
sam_status sam_gemm_plan(int64_t M, int64_t N, int64_t K, sam_dtype dtype,
                         sam_plan* out);

/* C = A*B, FP32 operands. `workspace` may be NULL when the plan's
 * workspace_bytes is 0; otherwise it must hold at least that many bytes
 * (else SAM_ERR_WORKSPACE: the call never falls back to another plan). */
sam_status sam_gemm_f32(const float* A, const float* B, float* C, int64_t M,
                        int64_t N, int64_t K, void* workspace,
                        uint64_t workspace_bytes, void* stream);

/* C = A*B, bfloat16 operands as raw bit patterns, FP32 accumulate/output. */
sam_status sam_gemm_bf16(const uint16_t* A, const uint16_t* B, float* C,
                         int64_t M, int64_t N, int64_t K, void* workspace,
                         uint64_t workspace_bytes, void* stream);

/* C = A*B, IEEE binary16 operands as raw bit patterns, FP32 accumulate/out. */
sam_status sam_gemm_f16(const uint16_t* A, const uint16_t* B, float* C,
                        int64_t M, int64_t N, int64_t K, void* workspace,
                        uint64_t workspace_bytes, void* stream);

/* Element formats of block-scaled 8-bit operands (OCP Microscaling
 * specification v1.0): E4M3 (bias 7, 3 fraction bits, no infinity, largest
 * finite 448) and E5M2 (bias 15, 2 fraction bits, IEEE-style Inf/NaN). */
typedef enum { SAM_E4M3 = 0, SAM_E5M2 = 1 } sam_fp8_format;

/* Block-scaled 8-bit GEMM (the block-scaled low-precision operands whose
 * tile variants page "fix(fp4_gemm autotune) SM107 kernel family excluded
 * from autotune candidates and heuristics update - #4856" tunes; the page
 * fixes no format, this takes the OCP MX formats gfx950's matrix cores
 * implement):
 *   C[i][j] = sum over k of (2^(scale_a[i][k/32] - 127) * A[i][k])
 *                         * (2^(scale_b[j][k/32] - 127) * Bt[j][k])
 * with products accumulated in FP32 and C written in FP32.
 *   A       device, M rows of K element codes (format fmt_a), row stride K.
 *   Bt      device, N rows of K element codes (format fmt_b): B given
 *           K-contiguous, Bt[j][k] = B[k][j], row stride K.
 *   scale_a device, M rows of K/32 E8M0 codes (2^(code-127)), row stride K/32.
 *   scale_b device, N rows of K/32 E8M0 codes, row stride K/32.
 *   C       device, M rows of N floats, row stride N; write-only.
 * K must be a multiple of 32 (SAM_ERR_INVALID_ARG otherwise). A, Bt, C and
 * the workspace must be 16-byte aligned; the scale arrays may have any
 * alignment. Codes that encode NaN or Inf, and the scale code 255, are not
 * valid inputs: the elements of C they reach are then unspecified (no
 * fault). Workspace as for sam_gemm_f32 (sam_gemm_plan with SAM_MXFP8 gives
 * the plan and its workspace_bytes). Asynchronous on `stream`. */
sam_status sam_gemm_mxfp8(sam_fp8_format fmt_a, sam_fp8_format fmt_b,
                          const uint8_t* A, const uint8_t* scale_a,
                          const uint8_t* Bt, const uint8_t* scale_b, float* C,
                          int64_t M, int64_t N, int64_t K, void* workspace,
                          uint64_t workspace_bytes, void* stream);

/* The same with a forced block-scaled variant `id` and split (0 = the
 * variant's own choice; stream-K is not offered). SAM_ERR_UNSUPPORTED when
 * the variant is not a block-scaled one or the split is not admissible. */
sam_status sam_gemm_mxfp8_variant(int32_t id, int32_t split_k,
                                  sam_fp8_format fmt_a, sam_fp8_format fmt_b,
                                  const uint8_t* A, const uint8_t* scale_a,
                                  const uint8_t* Bt, const uint8_t* scale_b,
                                  float* C, int64_t M, int64_t N, int64_t K,
                                  void* workspace, uint64_t workspace_bytes,
                                  void* stream);

/* Block-scaled 4-bit GEMM (MXFP4, OCP Microscaling v1.0): the product of
 * sam_gemm_mxfp8 with E2M1 elements (1 sign, 2 exponent bits with bias 1, 1
 * fraction bit; values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) packed
 * two per byte: element k of a row is the low nibble of byte k/2 for even k
 * and the high nibble for odd k.
 *   A       device, M rows of K/2 bytes, row stride K/2.
 *   Bt      device, N rows of K/2 bytes (Bt[j] holds column j of B).
 *   scale_a, scale_b, C, K, alignment, workspace and errors as for
 *           sam_gemm_mxfp8 (sam_gemm_plan with SAM_MXFP4 gives the plan). */
sam_status sam_gemm_mxfp4(const uint8_t* A, const uint8_t* scale_a,
                          const uint8_t* Bt, const uint8_t* scale_b, float* C,
                          int64_t M, int64_t N, int64_t K, void* workspace,
                          uint64_t workspace_bytes, void* stream);

/* The same with a forced block-scaled variant `id` and split (0 = the
 * variant's own choice). */
sam_status sam_gemm_mxfp4_variant(int32_t id, int32_t split_k,
                                  const uint8_t* A, const uint8_t* scale_a,
                                  const uint8_t* Bt, const uint8_t* scale_b,
                                  float* C, int64_t M, int64_t N, int64_t K,
                                  void* workspace, uint64_t workspace_bytes,
                                  void* stream);

/* Operand forms of the general entry point. */
typedef enum { SAM_OP_N = 0, SAM_OP_T = 1 } sam_op;

/* General form C = alpha * op(A) * op(B) + beta * C, the usual BLAS
 * definition (the pages' GEMM is its alpha = 1, beta = 0, no-transpose
 * case: page "Scale coverage exposes a remaining GEMM gap", section
 * "Measurement contract and evidence"). Row-major storage with row strides:
 *   op(A) is M x K: SAM_OP_N reads A as M rows of K values (lda >= K),
 *                   SAM_OP_T reads A as K rows of M values (lda >= M);
 *   op(B) is K x N: SAM_OP_N reads K rows of N (ldb >= N), SAM_OP_T N rows of
 *                   K (ldb >= K);
 *   C is M rows of N values, ldc >= N.
 * Element types as for sam_gemm_<dtype>; alpha and beta are FP32. C is read
 * only when beta != 0 (with beta == 0 whatever C held never reaches the
 * result); A and B are not read when alpha == 0 or K == 0. The result is
 * fmaf(alpha, P, beta * C) with P the FP32 product of the GEMM path (alpha * P
 * when beta == 0).
 * How: a call with SAM_OP_N, SAM_OP_N, compact strides, alpha 1 and beta 0 is
 * exactly sam_gemm_<dtype>. Otherwise the plan for (M, N, K, dtype) decides:
 *  - ring plans (FP32 "f..." and 16-bit "r..." variants) read A and B rows
 *    with their strides in place when each row stays whole 16-byte pieces
 *    (or the plan reads that operand one value at a time, or copies it into
 *    padded rows anyway), and store C themselves with row stride ldc (a
 *    multiple of 4) and alpha / beta applied where C is written: in the
 *    kernel, the split-K reduce or the stream-K fix-up. 16-bit 16x16x32 ring
 *    plans also read transposed operands (SAM_OP_T) straight, when K, N and
 *    the transposed operand's leading dimension are multiples of 8 (a
 *    192-row tile hands a transposed A to its 256-row twin); FP32 ring plans
 *    with tiles up to 128 x 256 read a transposed B straight when K and ldb
 *    are multiples of 4, and those and the 256 x 256 tile a transposed A
 *    when N and lda are multiples of 4; FP32 with both operands transposed
 *    runs as the
 *    plain product B A of the operands as stored, whose ring plan stores C
 *    transposed;
 *  - whatever remains (a transposed operand the plan cannot read, other
 *    strides, other plan kinds) is copied into compact rows in the
 *    workspace first, the product goes to a workspace temporary unless the
 *    plan stores C itself or ldc == N and beta == 0, and a last pass applies
 *    alpha and beta; those copies cost extra HBM traffic.
 * Base pointers must be 16-byte aligned; the workspace must hold
 * sam_gemm_ex_workspace() bytes (SAM_ERR_WORKSPACE otherwise).
 * Asynchronous on `stream`, like the other entry points. */
sam_status sam_gemm_ex(sam_dtype dtype, sam_op trans_a, sam_op trans_b,
                       int64_t M, int64_t N, int64_t K, float alpha,
                       const void* A, int64_t lda, const void* B, int64_t ldb,
                       float beta, float* C, int64_t ldc, void* workspace,
                       uint64_t workspace_bytes, void* stream);

/* Workspace bytes sam_gemm_ex needs for these arguments (host only). */
sam_status sam_gemm_ex_workspace(sam_dtype dtype, sam_op trans_a,
                                 sam_op trans_b, int64_t M, int64_t N,
                                 int64_t K, int64_t lda, int64_t ldb,
                                 int64_t ldc, float alpha, float beta,
                                 uint64_t* bytes);

/* sam_gemm_ex with a forced plan: variant `id`, split_k and raster_n as for
 * sam_gemm_variant_r (SAM_ERR_UNSUPPORTED / SAM_ERR_INVALID_ARG likewise);
 * everything else as for sam_gemm_ex, with the workspace from
 * sam_gemm_ex_variant_workspace. For tests and tuning of the general forms. */
sam_status sam_gemm_ex_variant(int32_t id, int32_t split_k, int32_t raster_n,
                               sam_dtype dtype, sam_op trans_a,
                               sam_op trans_b, int64_t M, int64_t N,
                               int64_t K, float alpha, const void* A,
                               int64_t lda, const void* B, int64_t ldb,
                               float beta, float* C, int64_t ldc,
                               void* workspace, uint64_t workspace_bytes,
                               void* stream);

/* Workspace bytes sam_gemm_ex_variant needs for these arguments (host only). */
sam_status sam_gemm_ex_variant_workspace(int32_t id, int32_t split_k,
                                         int32_t raster_n, sam_dtype dtype,
                                         sam_op trans_a, sam_op trans_b,
                                         int64_t M, int64_t N, int64_t K,
                                         int64_t lda, int64_t ldb, int64_t ldc,
                                         float alpha, float beta,
                                         uint64_t* bytes);

/* Low-rank adapters of many requests beside a shared projection: every row
 * gets the shared weight and the adapter pair of its own request,
 *   Y[m] = X[m] W + scale[a] (X[m] A[a]^T) B[a],   a = ids[m],
 * and only X[m] W where ids[m] names no adapter (any value outside 0 ..
 * n_adapters - 1, -1 by custom). Rows may come in any order; rows of one
 * request next to each other cost least. What another request's adapter
 * holds (Inf and NaN too) never reaches a row. Inf and NaN of a row's own
 * operands go where the formulas take them and no further; an Inf of theirs
 * may come out as NaN, which depends on the sizes.
 *   dtype   SAM_BF16 or SAM_F16: X, W, A and B.
 *   X       device, M rows of K values, row stride ldx >= K.
 *   W       device, K rows of N values (trans_w SAM_OP_N, ldw >= N) or N rows
 *           of K values (SAM_OP_T, ldw >= K).
 *   A       device, n_adapters x rank rows of K values, compact.
 *   B       device, n_adapters x rank rows of N values, compact.
 *   ids     device, M int32. 4-byte aligned, like scale. With n_adapters 0
 *           not looked at (NULL).
 *   scale   device, n_adapters floats, or NULL for 1.
 *   out     the type of Y: SAM_F32 or dtype (rounded once, to nearest even).
 *   Y       device, M rows of N values, row stride ldy >= N; write-only.
 * rank 1 .. 128 (adapters of lower rank: zero rows); n_adapters 0 is the
 * plain projection; N, K >= 1; M == 0 is a no-op. Sums are FP32; the rank-r
 * intermediate is FP32 too, or kept to 22 bits (SAM_F16; 16 for SAM_BF16 with
 * a SAM_BF16 result) relative to its row's largest value. Other base
 * addresses must be 16-byte aligned; rows that are no whole 16-byte pieces (K
 * or N not a multiple of 8, or such a stride) are copied into the workspace
 * first, all but a W whose rows run along the result's columns (N here, K in
 * the gradients) with a stride that is a multiple of 8: it is read in place,
 * in aligned 16-byte pieces, up to 14 bytes behind a row's end with the last
 * of them. Y must not overlap anything else. Workspace:
 * sam_adapter_gemm_workspace() bytes, SAM_ERR_WORKSPACE when short. N, K and
 * strides up to 2.08 M values (a single row's stride may be any). Asynchronous on `stream`, no atomics on
 * results, fixed summation order. */
sam_status sam_adapter_gemm(sam_dtype dtype, sam_op trans_w, int64_t M,
                            int64_t N, int64_t K, int64_t n_adapters,
                            int64_t rank, const void* X, int64_t ldx,
                            const void* W, int64_t ldw, const void* A,
                            const void* B, const int32_t* ids,
                            const float* scale, sam_dtype out, void* Y,
                            int64_t ldy, void* workspace,
                            uint64_t workspace_bytes, void* stream);

/* Workspace bytes sam_adapter_gemm needs for these arguments (host only). */
sam_status sam_adapter_gemm_workspace(sam_dtype dtype, sam_op trans_w,
                                      int64_t M, int64_t N, int64_t K,
                                      int64_t n_adapters, int64_t rank,
                                      int64_t ldx, int64_t ldw,
                                      uint64_t* bytes);

/* Gradients of sam_adapter_gemm for a given gradient dY of Y (dtype, M rows
 * of N, row stride lddy); W is frozen. For the rows m of adapter a:
 *   dX[m] = dY[m] W^T + scale[a] (dY[m] B[a]^T) A[a]
 *   dA[a] = scale[a] sum_m (dY[m] B[a]^T)^T X[m]      (rank x K, FP32)
 *   dB[a] = scale[a] sum_m (X[m] A[a]^T)^T dY[m]      (rank x N, FP32)
 * and dX[m] = dY[m] W^T for rows without an adapter. dA and dB (compact,
 * n_adapters x rank rows) are written whole, zeros for adapters without
 * rows. dX (type `out`: SAM_F32 or dtype, row stride lddx >= K) may be NULL,
 * and so may dA and dB together; what is not wanted is not computed. Rows
 * are added up in row order in chunks of a fixed size, and these in a fixed
 * order: the same bits every time. dA and dB take the intermediate whole
 * (SAM_BF16) or to 22 bits of the largest value that its rank has in a chunk
 * (SAM_F16); Inf and NaN in one rank leave the others as they are. Everything else as for sam_adapter_gemm. With M ==
 * 0 dA and dB are zeros. */
sam_status sam_adapter_backward(sam_dtype dtype, sam_op trans_w, int64_t M,
                                int64_t N, int64_t K, int64_t n_adapters,
                                int64_t rank, const void* dY, int64_t lddy,
                                const void* X, int64_t ldx, const void* W,
                                int64_t ldw, const void* A, const void* B,
                                const int32_t* ids, const float* scale,
                                sam_dtype out, void* dX, int64_t lddx,
                                float* dA, float* dB, void* workspace,
                                uint64_t workspace_bytes, void* stream);

/* Workspace bytes sam_adapter_backward needs (host only). want_dx, want_dab:
 * whether dX, and dA with dB, will be asked for. */
sam_status sam_adapter_backward_workspace(sam_dtype dtype, sam_op trans_w,
                                          int64_t M, int64_t N, int64_t K,
                                          int64_t n_adapters, int64_t rank,
                                          int64_t lddy, int64_t ldx,
                                          int64_t ldw, int32_t want_dx,
                                          int32_t want_dab, uint64_t* bytes);

/* Distillation from a teacher's top logits: the student's logits z of a row
 * against the teacher's `top` largest ones t at the vocabulary entries
 * `index`, at temperature T:
 *   p = softmax(t / T) over the row's valid entries, q = softmax(z / T)
 *   loss = weight T^2 sum_j p_j (log p_j - log q_j)
 *   grad = weight T (q - p)      (its derivative with respect to z)
 *   dtype    SAM_F32, SAM_BF16 or SAM_F16: the type of logits and grad.
 *   logits   device, `rows` rows of V values, row stride ldz >= V, aligned to
 *            one value (rows that start on 16 bytes cost nothing extra).
 *   t_dtype, teacher  device, rows x top values, compact, any of the three types.
 *   index    device, rows x top int32, compact; a value outside 0 .. V - 1
 *            marks an empty entry. Entries with the same index each have
 *            their own term in the loss and add up in the gradient.
 *   weight   device, `rows` floats (the loss's own gradient and any mean's
 *            1 / n belong here), or NULL for 1.
 *   loss, lse  device, `rows` floats; lse = log sum exp(z / T) (-inf for a
 *            row of -inf).
 *   grad     device, `rows` rows of V, row stride ldg >= V; the logits
 *            themselves (same pointer and stride) or no part of them.
 * Logits of -inf are masked vocabulary entries: probability and gradient
 * contribution 0, loss +inf where the teacher's p is not 0. A row whose
 * weight is 0, whose entries are all empty or -inf, or whose logits are all
 * -inf has loss 0 and gradient 0 (with weight 0 also where its logits are
 * NaN). NaN elsewhere stays in its row. top 1 .. 1024, V up to 2^31 - 65536,
 * T from 2^-40 to 2^40; rows == 0 is a no-op. Sums are FP32; no atomics, a
 * fixed order. No workspace. Asynchronous on `stream`. */
sam_status sam_distill_loss(sam_dtype dtype, int64_t rows, int64_t V,
                            int64_t top, const void* logits, int64_t ldz,
                            sam_dtype t_dtype, const void* teacher,
                            const int32_t* index, const float* weight,
                            float temperature, float* loss, float* lse,
                            void* stream);

/* The gradient from the lse that sam_distill_loss wrote. q is as exact as
 * lse's rounding lets it be (2^-24 |lse|): a row whose logits all lie next to
 * a type's lowest value has lost its sum there; sam_distill has not. */
sam_status sam_distill_grad(sam_dtype dtype, int64_t rows, int64_t V,
                            int64_t top, const void* logits, int64_t ldz,
                            const float* lse, sam_dtype t_dtype,
                            const void* teacher, const int32_t* index,
                            const float* weight, float temperature, void* grad,
                            int64_t ldg, void* stream);

/* Loss and gradient together: the logits are read once. */
sam_status sam_distill(sam_dtype dtype, int64_t rows, int64_t V, int64_t top,
                       const void* logits, int64_t ldz, sam_dtype t_dtype,
                       const void* teacher, const int32_t* index,
                       const float* weight, float temperature, float* loss,
                       void* grad, int64_t ldg, void* stream);

/* MXFP4 tensors (the operands of sam_gemm_mxfp4) from values, and back. Of
 * every block of 32 values of a row (zeros behind the last ones when K is no
 * multiple of 32):
 *   s = floor(log2(max |x|)) - 2, at least -127 (-127 too for a block of zeros)
 *   code = E2M1(x / 2^s): the nearest value, ties to the even code, at most 6
 *   scale code = s + 127
 * A block that holds an Inf or NaN gets the scale code 255 and codes 0: it
 * stands for NaN throughout.
 *   dtype   SAM_F32, SAM_BF16 or SAM_F16: the values' type.
 *   trans   SAM_OP_N: X is `rows` rows of K values, ldx >= K. SAM_OP_T: X is K
 *           rows of `rows` values, ldx >= rows (a K x N weight becomes the N
 *           rows of K that the products take).
 *   X       device, aligned to one value (rows on 16 bytes cost least).
 *   codes   device, rows x ceil(K / 32) x 16 bytes, compact, 16-byte aligned:
 *           element k of a row in the low half of its byte k / 2 for even k.
 *   scales  device, rows x ceil(K / 32) bytes, compact, any alignment.
 * codes and scales overlap neither X nor each other. K >= 1, rows *
 * ceil(K / 32) up to 2^31 - 4096; rows == 0 is a no-op. Asynchronous on
 * `stream`. */
sam_status sam_quantize_mxfp4(sam_dtype dtype, sam_op trans, int64_t rows,
                              int64_t K, const void* X, int64_t ldx,
                              uint8_t* codes, uint8_t* scales, void* stream);

/* The values that codes and scales stand for, rounded to nearest even where
 * `dtype` cannot hold them (SAM_F16: under 2^-14 or over 65504; SAM_BF16 and
 * SAM_F32 hold all that sam_quantize_mxfp4 makes): X is `rows` rows of K
 * values, row stride ldx >= K, aligned to one value. Scale code 255 gives
 * NaN. */
sam_status sam_dequantize_mxfp4(sam_dtype dtype, int64_t rows, int64_t K,
                                const uint8_t* codes, const uint8_t* scales,
                                void* X, int64_t ldx, void* stream);

/* Projection by a weight kept in MXFP4, for single tokens, prompts and
 * training:
 *   Y = q(X) Wq^T
 * q(X) are the values of X's rows after sam_quantize_mxfp4, Wq the N rows of K
 * values that codes and scales stand for. Products and sums as in
 * sam_gemm_mxfp4, FP32, rounded once (to nearest even) where `out` is a 16-bit
 * type.
 *   dtype   SAM_F32, SAM_BF16 or SAM_F16: X.
 *   X       device, M rows of K values, row stride ldx >= K.
 *   codes   device, N x ceil(K / 32) x 16 bytes, 16-byte aligned.
 *   scales  device, N x ceil(K / 32) bytes, any alignment.
 *   out     the type of Y: SAM_F32 or dtype.
 *   Y       device, M rows of N values, row stride ldy >= N; write-only.
 * X and Y are aligned to one value. A block of X or of the weight that stands
 * for NaN makes the results of its row (of its column) NaN. N, K >= 1, they
 * and ldy up to 2.08 M, M * ceil(max(N, K) / 128) and N * ceil(K / 128) up to
 * 2^29 - 2^26; M == 0 is a no-op; a single row's stride may be any. Y overlaps
 * nothing else. Workspace: sam_linear_mxfp4_workspace() bytes,
 * SAM_ERR_WORKSPACE when short. Asynchronous on `stream`, no atomics, a fixed
 * order. */
sam_status sam_linear_mxfp4(sam_dtype dtype, int64_t M, int64_t N, int64_t K,
                            const void* X, int64_t ldx, const uint8_t* codes,
                            const uint8_t* scales, sam_dtype out, void* Y,
                            int64_t ldy, void* workspace,
                            uint64_t workspace_bytes, void* stream);

/* Workspace bytes sam_linear_mxfp4 needs for these sizes and types (host only). */
sam_status sam_linear_mxfp4_workspace(sam_dtype dtype, sam_dtype out, int64_t M,
                                      int64_t N, int64_t K, uint64_t* bytes);

/* Gradient of sam_linear_mxfp4 with respect to X for a given gradient dY of Y;
 * the weight is frozen and the rounding of X is passed through as it is:
 *   dX = dY Wq      (M rows of K)
 * dY (dtype, M rows of N, row stride lddy >= N) is not rounded; Wq is taken in
 * dtype, as sam_dequantize_mxfp4 gives it. dX (type `out`: SAM_F32 or dtype, row stride
 * lddx >= K) is written whole. dY and dX must be 16-byte aligned; strides up
 * to 2.08 M values (a single row's may be any). Everything else as for
 * sam_linear_mxfp4, the workspace by sam_linear_mxfp4_backward_workspace(). */
sam_status sam_linear_mxfp4_backward(sam_dtype dtype, int64_t M, int64_t N,
                                     int64_t K, const void* dY, int64_t lddy,
                                     const uint8_t* codes,
                                     const uint8_t* scales, sam_dtype out,
                                     void* dX, int64_t lddx, void* workspace,
                                     uint64_t workspace_bytes, void* stream);

/* Workspace bytes sam_linear_mxfp4_backward needs (host only): for any
 * strides, or (_strided) for these. In it lies the weight in dtype, N rows of K
 * values; beside it what the product takes, with strides that are no whole 16
 * bytes also a copy of dY and (FP32) one of dX. */
sam_status sam_linear_mxfp4_backward_workspace(sam_dtype dtype, sam_dtype out,
                                               int64_t M, int64_t N, int64_t K,
                                               uint64_t* bytes);
sam_status sam_linear_mxfp4_backward_workspace_strided(
    sam_dtype dtype, sam_dtype out, int64_t M, int64_t N, int64_t K,
    int64_t lddy, int64_t lddx, uint64_t* bytes);

/* Log probabilities of given tokens, with the entropy and the most likely
 * entries of every row of logits z at temperature T:
 *   m = max z,  L = log sum_j exp((z_j - m) / T)
 *   log p_j = (z_j - m) / T - L
 *   logprob = log p[token],  entropy = - sum_j p_j log p_j
 *   dtype    SAM_F32, SAM_BF16 or SAM_F16: the logits.
 *   logits   device, `rows` rows of V values, row stride ldz >= V, aligned to
 *            one value (rows that start on 16 bytes cost nothing extra).
 *   tokens   device, `rows` int32; a value outside 0 .. V - 1 names none: that
 *            row's logprob is 0.
 *   logprob, entropy  device, `rows` floats.
 *   norm     device, rows x 2 floats: m and L (log sum exp(z / T) = m / T + L;
 *            kept apart, so that nothing is lost far from zero).
 *   top      0 .. 128 and at most V: how many of the row's most likely entries
 *            are wanted.
 *   top_logprob, top_index  device, rows x top, compact: log p and index of
 *            those, the largest logit first, the lowest index first among
 *            equal ones (the two zeros are equal). NULL with top 0.
 * Logits of -inf are masked entries: probability 0, log probability -inf,
 * nothing in the entropy; as most likely entries they come last. A row
 * without any other has entropy 0, m = L = -inf and log probabilities -inf. A row that
 * holds NaN or +inf has NaN results, but its top_index are entries all the
 * same (NaN counts as the largest). V up to 2^31 - 65536, rows *
 * ceil(V / 16384) under 2^22, T from 2^-40 to 2^40; rows == 0 is a no-op. Sums are FP32 and kept without the largest entry's
 * own 1: log p, entropy and L near 0 are as exact as the probabilities beside
 * that entry. No atomics on results, a fixed order. Results overlap nothing
 * else. Workspace: sam_token_logprobs_workspace() bytes,
 * SAM_ERR_WORKSPACE when short. Asynchronous on `stream`. */
sam_status sam_token_logprobs(sam_dtype dtype, int64_t rows, int64_t V,
                              int64_t top, const void* logits, int64_t ldz,
                              const int32_t* tokens, float temperature,
                              float* logprob, float* entropy, float* norm,
                              float* top_logprob, int32_t* top_index,
                              void* workspace, uint64_t workspace_bytes,
                              void* stream);

/* Workspace bytes sam_token_logprobs needs for these arguments (host only). */
sam_status sam_token_logprobs_workspace(sam_dtype dtype, int64_t rows, int64_t V,
                                        int64_t top, uint64_t* bytes);

/* Gradient with respect to the logits for given gradients u of logprob and v
 * of entropy:
 *   dz_j = (u (1[j = token] - p_j) - v p_j (log p_j + entropy)) / T
 * norm and entropy are what sam_token_logprobs wrote for the same logits and
 * temperature; dlogprob and dentropy are `rows` floats or NULL for 0 (entropy
 * may be NULL where dentropy is). A row without a token takes no u. Masked
 * entries get 0 (a masked token u / T), and so do the rows of two zero gradients, whatever
 * their logits hold, and rows of -inf. grad: `rows` rows of V, of the logits'
 * type, row stride ldg >= V; the logits themselves (same pointer and stride)
 * or no part of them. */
sam_status sam_token_logprobs_grad(sam_dtype dtype, int64_t rows, int64_t V,
                                   const void* logits, int64_t ldz,
                                   const int32_t* tokens, float temperature,
                                   const float* norm, const float* entropy,
                                   const float* dlogprob, const float* dentropy,
                                   void* grad, int64_t ldg, void* stream);

/* Number of entries in the variant table (ids 0 .. count-1). */
int32_t sam_variant_count(void);

/* Static description of variant `id` (no shape: split_k = 1, grid 0). */
sam_status sam_variant_info(int32_t id, sam_plan* out);

/* The plan for a forced variant and split. split_k = 0 lets the dispatcher
 * pick the split for that variant, -1 asks for its stream-K form (FP32 ring
 * variants with tiles up to 128 x 256, when the shape has at least as many K
 * iterations as resident workgroups). SAM_ERR_UNSUPPORTED if the variant does
 * not take `dtype` or the split is not admissible for the shape;
 * SAM_ERR_INVALID_ARG for split_k < -1. The 16-bit 16x16x32 ring variants
 * have a stream-K form too: whole waves of tiles run one per workgroup and
 * the tiles of the last, partial wave share their K iterations. */
sam_status sam_variant_plan(int32_t id, int64_t M, int64_t N, int64_t K,
                            sam_dtype dtype, int32_t split_k, sam_plan* out);

/* The same with a forced raster order: raster_n = 0 (M-major), 1 (N-major)
 * or -1 (the one the cost model prefers for this variant and split; ties go
 * to M-major). The raster order decides which tiles run together and so how
 * much of each A and B panel the XCD's L2 serves to several of them (page
 * "fix(fp4_gemm autotune) SM107 kernel family excluded from autotune
 * candidates and heuristics update - #4856", section "Swap × raster
 * experiment: tile reuse root cause"). SAM_ERR_INVALID_ARG for other
 * raster_n; SAM_ERR_UNSUPPORTED where the variant has no tiles (the streaming
 * skinny kernels) and raster_n is 1. */
sam_status sam_variant_plan_r(int32_t id, int64_t M, int64_t N, int64_t K,
                              sam_dtype dtype, int32_t split_k, int32_t raster_n,
                              sam_plan* out);

/* The cost model's own plan for this shape, ignoring the frozen table of
 * measured shapes (host only; for calibration reports and tests). */
sam_status sam_gemm_plan_model(int64_t M, int64_t N, int64_t K, sam_dtype dtype,
                               sam_plan* out);

/* Run a forced variant (tests, profiling and calibration). Operands as for
 * sam_gemm_<dtype> (16-bit ones as uint16_t patterns). SAM_MXFP8 and
 * SAM_MXFP4 are refused with SAM_ERR_INVALID_ARG: block-scaled operands go
 * through sam_gemm_mxfp8_variant / sam_gemm_mxfp4_variant. */
sam_status sam_gemm_variant(int32_t id, sam_dtype dtype, int32_t split_k,
                            const void* A, const void* B, float* C, int64_t M,
                            int64_t N, int64_t K, void* workspace,
                            uint64_t workspace_bytes, void* stream);

/* Bytes of the device scratch array behind sam_gemm_noalloc (64 MiB per GPU). */
#define SAM_SCRATCH_BYTES (64ull << 20)

/* C = A*B exactly as sam_gemm_f32 / sam_gemm_bf16 / sam_gemm_f16 (`dtype`
 * SAM_F32, SAM_BF16 or SAM_F16; the same plan, kernels and bits) without a
 * caller workspace and without any allocation: for callers that cannot
 * allocate device memory (code under graph capture, tight serving loops,
 * harnesses that forbid hipMalloc). The plan's workspace (padded operand
 * copies, split-K partials, stream-K slots) goes to a file-scope device array of SAM_SCRATCH_BYTES that each GPU holds from
 * its first such call until the process ends. A plan whose workspace_bytes
 * exceeds SAM_SCRATCH_BYTES is refused with SAM_ERR_WORKSPACE (use
 * sam_gemm_<dtype> with a workspace for it). Nothing in the array needs to
 * start at zero: every plan writes each workspace value before reading it.
 * Every call on one GPU shares that GPU's array, so calls that overlap in
 * time on one GPU (on different streams, or from different threads without
 * ordering) race and may return wrong results; calls in order on one stream
 * are safe. Other arguments, alignment and errors as for sam_gemm_f32. */
sam_status sam_gemm_noalloc(sam_dtype dtype, const void* A, const void* B,
                            float* C, int64_t M, int64_t N, int64_t K,
                            void* stream);

/* sam_gemm_variant with a forced raster order (raster_n as for
 * sam_variant_plan_r). */
sam_status sam_gemm_variant_r(int32_t id, sam_dtype dtype, int32_t split_k,
                              int32_t raster_n, const void* A, const void* B,
                              float* C, int64_t M, int64_t N, int64_t K,
                              void* workspace, uint64_t workspace_bytes,
                              void* stream);

/* Checks once per process that the current device is gfx950 and that the
 * library's kernels are loadable on it. SAM_ERR_UNSUPPORTED_DEVICE if not. */
sam_status sam_device_check(void);

/* Static text for a status code. */
const char* sam_status_string(sam_status s);

/* Detail of the last failing call on this thread ("" if none). */
const char* sam_last_error(void);

/* Build stamp: library version, git revision, ROCm/HIP version, target. */
const char* sam_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* SAM_H */
