/*
 * tgemm_ops.h -- C ABI of libtgemm, the operators beside the GEMMs of tgemm.h: MXFP4 (4-bit
 * microscaled) matrices with their quantiser and products, the orthogonalisation of a weight's
 * update, the root-mean-square norm with the residual's addition, and an expert layer's routing
 * (tokens sorted by expert and back) and products. The same library and conventions (row-major
 * storage, device pointers owned by the caller, nothing allocated, enqueue-only calls on the given
 * stream, the TGEMM_E* codes of tgemm.h, C not overlapping an input).
 */
#ifndef TGEMM_OPS_H_
#define TGEMM_OPS_H_

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of operands that come in more than one. */
#define TGEMM_DTYPE_F16 0
#define TGEMM_DTYPE_F32 1

/*
 * MXFP4: microscaled 4-bit floating point (the OCP microscaling format's FP4). An MXFP4 matrix
 * of R x K values is two byte arrays:
 *   codes, ldq : R rows of KB = ceil(K/32) blocks of 16 bytes (ldq >= max(1, KB) * 16 bytes): 32
 *                E2M1 codes along k, two a byte, the even k in the low half. E2M1 has a sign, two
 *                exponent bits (bias 1) and a fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6. Codes past
 *                K in a row's last block are zero (mxfp4_quant writes them so; the products sum
 *                whole blocks);
 *   scale, lds : R rows of KB bytes (lds >= max(1, KB) bytes), one E8M0 scale per block: byte s
 *                stands for 2^(s - 127), 255 for NaN.
 * The fast kernels take codes and scales 16-byte aligned, with ldq and lds multiples of 16, at
 * most 2 * TGEMM_FAST_MAX_LD bytes (they read the scales of a row in 16-byte pieces, the last one
 * whole); the one for few rows takes scales of any alignment and lds. Other arguments take the
 * generic kernel with the same results (within float32 summation order). No size may exceed
 * TGEMM_MX_MAX_DIM. Device pointers, ownership, streams and errors as for gemm_f16.
 */
#define TGEMM_MX_MAX_DIM (TGEMM_MAX_DIM - 512)

/*
 * Quantiser: binary16 X (R x K, ldx elements) to MXFP4 along its rows (Q, scale: R x K) and / or
 * along its columns (QT, scale_t: X^T, K x R, blocks of 32 along R -- the operand a product over
 * R reads, as the gradient of a linear layer's weight does), in one pass over X. A pair of NULL
 * pointers is not wanted; one NULL of a pair, or both pairs NULL, is TGEMM_ENULL. For a block
 * whose largest magnitude is amax: scale 2^(floor(log2 amax) - 2) (1 for a block of zeros), codes
 * x / scale rounded to nearest, ties to the even code, saturated at 6. A block that holds an
 * infinity or a NaN gets scale byte 255 and zero codes. R == 0 or K == 0 is a no-op. X must be
 * 2-byte aligned; no other alignment is needed. R * ceil(K/32) may be at
 * most 2^31 - 128 (also of mxfp4_dequant).
 */
TGEMM_API int mxfp4_quant(int64_t R, int64_t K, const void* X, int64_t ldx,
                          void* Q, int64_t ldq, void* scale, int64_t lds,
                          void* QT, int64_t ldqt, void* scale_t, int64_t ldst, void* stream);

/*
 * The inverse: binary16 X (R x K, ldx elements, only the R x K values written) from an MXFP4
 * matrix, each value rounded to nearest even. Scales from 2^-23 to 2^13 decode exactly; above,
 * values past binary16's range become infinite; a scale byte of 255 gives NaN.
 */
TGEMM_API int mxfp4_dequant(int64_t R, int64_t K, const void* Q, int64_t ldq, const void* scale, int64_t lds,
                            void* X, int64_t ldx, void* stream);

/*
 * C = ReLU?(A @ B^T) of two MXFP4 matrices, A (M x K) and B (N x K, a linear layer's weight):
 *   C[i,j] = ReLU?( sum_kb 2^(sa + sb - 254) sum_{k in kb} a[i,k] * b[j,k] ),
 * accumulated in float32 and rounded to binary16 once. M == 0 or N == 0 is a no-op, K == 0 writes
 * C = 0. A NaN scale makes its row (A) or column (B) of C NaN (+0 with relu). A product of more
 * than 2^23 - 1 tiles (128 x 128 at the smallest but for up to 256 rows) is TGEMM_EINVAL_DIM.
 */
TGEMM_API int mxfp4_gemm(int64_t M, int64_t N, int64_t K,
                         const void* A, int64_t lda, const void* scale_a, int64_t ldsa,
                         const void* B, int64_t ldb, const void* scale_b, int64_t ldsb,
                         void* C, int64_t ldc, int relu, void* stream);

/*
 * C = ReLU?(A @ W^T) of binary16 A (M x K, lda elements) and an MXFP4 weight (N x K) decoded to
 * binary16 as mxfp4_dequant does, accumulated in float32. For few rows (single tokens, small
 * batches) a kernel reads the weight once for every 64 rows, with A of any alignment and K: up to
 * 32 rows always, up to 256 while ceil(M/64) * ceil(N/16) is at most 768 (1024 for an A or scales
 * that the others cannot take). The other fast kernels also need A 16-byte aligned, lda and K
 * multiples of 8 and lda at most TGEMM_FAST_MAX_LD: past those sizes a caller with other rows of A
 * copies them to ones padded with zeros (100 x 8192 x 4095: 47 us with that copy, 74 without).
 * Otherwise as mxfp4_gemm.
 */
TGEMM_API int mxfp4_gemm_f16(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                             const void* B, int64_t ldb, const void* scale_b, int64_t ldsb,
                             void* C, int64_t ldc, int relu, void* stream);

/*
 * Orthogonalisation of a weight's update by Newton-Schulz products: for each of `batch` matrices
 * G (R x C, row stride ldg, matrix stride stride_g, in elements; dtype TGEMM_DTYPE_F16 or
 * TGEMM_DTYPE_F32),
 *   X_0 = G / (|G|_F + 1e-7);  `steps` times  A = X X^T,  X <- a X + (b A + c A A) X;
 *   the result scale * X as binary16 (row stride ldx, matrix stride stride_x; only R x C values
 *   of each matrix written),
 * which leaves G's singular vectors and moves its singular values towards one (a, b, c = 3.4445,
 * -4.7750, 2.0315 with 5 steps: into about 0.7 .. 1.2). For R > C the products run on X^T X, which
 * gives the same X. The norm is summed in float64; A, the polynomial and the iterate are held to 22
 * bits (diagonals of the first two in float32) and multiplied to that, with float32 sums. Before its
 * rounding to binary16 (2e-4 of it in Frobenius norms) the result is as near the exact one as
 * float32 products bring it: 1e-6 of it on random matrices, with strong directions or without,
 * after 4 to 10 steps. Where one direction is 1e3 or 1e4 times the others, its roundings, which the
 * steps draw out, are up to 1e-4 of the result after 5 or 6 steps and 8e-4 after 10. Values past
 * binary16's range on the way (coefficients under which the iterate grows) end in NaN.
 *   workspace : caller-owned device memory, 256-byte aligned, at least
 *               orthogonalize_workspace_bytes(batch, R, C) bytes, nothing expected of its
 *               contents; calls that may overlap in time need different ones.
 * X may be G (same strides, binary16), no other overlap. min(R, C) is at most 32768, max(R, C) at
 * most TGEMM_FAST_MAX_LD, steps 1 .. 64 (else TGEMM_EINVAL_DIM, as for an unknown dtype); stride_x
 * is at least (R - 1) * ldx + C (TGEMM_EINVAL_LD). An empty batch or matrix is a no-op; a matrix of
 * zeros gives zeros; one that holds an infinity or a NaN gives NaN in that matrix. X must be
 * 2-byte and G aligned to its type.
 */
TGEMM_API int64_t orthogonalize_workspace_bytes(int64_t batch, int64_t R, int64_t C);
TGEMM_API int orthogonalize_f16(int64_t batch, int64_t R, int64_t C, int dtype,
                                const void* G, int64_t ldg, int64_t stride_g,
                                void* X, int64_t ldx, int64_t stride_x,
                                int steps, float a, float b, float c, float scale,
                                void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Root-mean-square norm with the residual's addition, for each row of X (R x K binary16):
 *   h = round(x + residual) to the residual's type (h = x without a residual),
 *   y = h * W / sqrt(mean(h^2) + eps),
 * with float32 sums, to any of
 *   Y, ldy           : y as binary16;
 *   Q, ldq and scale : y as E4M3 codes and float32 scales per 1 x 128 block, R x K codes and R x
 *                      ceil(K/128) scales, contiguous, as gemm_fp8_block takes them. They are made
 *                      from the float32 y (not from one rounded to binary16): s = amax / 448, q =
 *                      E4M3(y / s) to nearest even. A block of magnitudes below 2^-100 has codes 0
 *                      and scale 1; one that holds an infinity or a NaN codes 0 and scale NaN;
 *   residual_out     : h, in the residual's type (residual itself, with its stride, to update it in
 *                      place). Y may be X with its stride; no other overlap.
 * Each may be NULL, but not Y and Q both; Q and scale go together and residual_out needs a residual
 * (else TGEMM_ENULL). residual_dtype and w_dtype are TGEMM_DTYPE_F16 or TGEMM_DTYPE_F32 (residual
 * NULL: none, its type is not looked at). K is at most TGEMM_NORM_MAX_K, R times the threads of a row
 * (16 up to K = 128, 32 up to 256, 64 up to 1024, 256 up to 4096, 512 up to 8192, else 1024) at most
 * 2^32 - 2048, eps at least 0; else TGEMM_EINVAL_DIM. Pointers need the alignment of their type; no stride
 * or K needs more.
 * Rows at the ends of float32: the squares are summed before the division by K, so a row whose sum of
 * squares passes 3.4e38 (a root mean square of 1.8e19 / sqrt(K): 2.9e17 for K = 4096) gives y = 0, codes 0
 * and scale 1, and the gradient dX = dH. With eps = 0, rows of zeros give NaN, and rows whose squares fall
 * below 1.2e-38 (values below 1e-19) lose digits, down to infinities where all of them are 0 (values below
 * 2.6e-23).
 */
#define TGEMM_NORM_MAX_K 16384
TGEMM_API int rmsnorm_f16(int64_t R, int64_t K, const void* X, int64_t ldx,
                          const void* residual, int64_t ldr, int residual_dtype, const void* W, int w_dtype, float eps,
                          void* residual_out, int64_t ldro, void* Y, int64_t ldy,
                          void* Q, int64_t ldq, float* scale, void* stream);

/*
 * Its gradient, from dY (the gradient of y), H (h as it was stored: residual_out, or X where there
 * was no residual; h_dtype its type), W, eps and dH (the gradient of residual_out, of H's type;
 * NULL: none), with rstd = 1 / sqrt(mean(h^2) + eps) and xhat = h rstd:
 *   dX = rstd (W dY - xhat mean(W dY xhat)) + dH as binary16; dR the same in H's type (the
 *   residual's gradient; NULL: not wanted); dW = the sum over the rows of dY xhat in W's type (NULL:
 *   not wanted), float32 partial sums added in a fixed order.
 *   workspace : 256-byte aligned, rmsnorm_f16_backward_workspace_bytes(R, K) bytes, nothing expected
 *               of its contents (not needed without dW); calls that may overlap in time need
 *               different ones.
 * dX may be dY and dR may be dH or H, with their strides; no other overlap. R == 0 writes dW = 0.
 */
TGEMM_API int64_t rmsnorm_f16_backward_workspace_bytes(int64_t R, int64_t K);
TGEMM_API int rmsnorm_f16_backward(int64_t R, int64_t K, const void* dY, int64_t lddy,
                                   const void* H, int64_t ldh, int h_dtype, const void* W, int w_dtype,
                                   float eps, const void* dH, int64_t lddh, void* dX, int64_t lddx,
                                   void* dR, int64_t lddr, void* dW, void* workspace, int64_t workspace_bytes,
                                   void* stream);

/*
 * Tokens sorted by expert. Each of `tokens` tokens has k slots, slot t * k + j with an id in [0,
 * experts), or any other number for no expert (a padding token, an expert that lives elsewhere):
 *   ids, ldi : tokens x k ids, TGEMM_INDEX_I32 or _I64, row stride ldi >= max(1, k);
 *   offsets  : experts + 1 int32: how many slots have a smaller expert. Expert e owns the sorted rows
 *              offsets[e] .. offsets[e + 1], and offsets[experts] rows are in use;
 *   order    : tokens * k int32: the slot of each sorted row, in slot order inside an expert, -1 behind
 *              the last row in use;
 *   place    : tokens x k int32, contiguous: each slot's sorted row, -1 for a slot of no expert.
 *   workspace: 256-byte aligned, expert_sort_workspace_bytes(tokens, k, experts) bytes (0 up to 8192
 *              slots), nothing expected of its contents; calls that may overlap in time need different
 *              ones.
 * experts is 1 .. TGEMM_MAX_EXPERTS and tokens * k at most TGEMM_MAX_SLOTS (else TGEMM_EINVAL_DIM).
 * Deterministic; one launch up to 8192 slots, two beyond.
 */
#define TGEMM_INDEX_I32 0
#define TGEMM_INDEX_I64 1
#define TGEMM_MAX_EXPERTS 1024
#define TGEMM_MAX_SLOTS (((int64_t)1 << 26) - 1024)
TGEMM_API int64_t expert_sort_workspace_bytes(int64_t tokens, int64_t k, int64_t experts);
TGEMM_API int expert_sort(int64_t tokens, int64_t k, int64_t experts, const void* ids, int64_t ldi, int ids_type,
                          void* offsets, void* order, void* place, void* workspace, int64_t workspace_bytes,
                          void* stream);

/*
 * Rows out to their places: XS[place[t, j], :] = X[t, :] for every slot (X tokens x H, XS rows x H,
 * binary16). A place outside [0, rows) is skipped, two slots with one place leave one of their rows.
 * With offsets (experts + 1 int32, as expert_sort writes them) the rows of XS behind
 * offsets[experts] are set to zero; with NULL they are left as they were, as are rows before
 * offsets[experts] that no slot has. With k = 0 X and place are not read and may be NULL.
 */
TGEMM_API int expert_gather_f16(int64_t tokens, int64_t k, int64_t rows, int64_t H, const void* X, int64_t ldx,
                                const void* place, void* XS, int64_t ldxs, const void* offsets, int64_t experts,
                                void* stream);

/*
 * And back: OUT[t, :] = sum_j weights[t, j] * Y[place[t, j], :], summed in float32 in the order of j
 * and rounded to binary16 once; a slot without a place in [0, rows) adds nothing, a token without
 * any gives zeros. weights: tokens x k, contiguous, of w_dtype (NULL: ones, which makes this the
 * gradient of expert_gather_f16).
 */
TGEMM_API int expert_combine_f16(int64_t tokens, int64_t k, int64_t rows, int64_t H, const void* Y, int64_t ldy,
                                 const void* place, const void* weights, int w_dtype, void* OUT, int64_t ldo,
                                 void* stream);

/*
 * Its gradient: dY[place[t, j], :] = weights[t, j] * dOUT[t, :] and dweights[t, j] = <dOUT[t, :],
 * Y[place[t, j], :]> (of w_dtype; 0 for a slot of no place), either NULL where it is not wanted (Y is
 * read for dweights only). Rows of dY behind offsets[experts] as for expert_gather_f16; rows before it
 * that no slot has are left as they were.
 */
TGEMM_API int expert_combine_f16_backward(int64_t tokens, int64_t k, int64_t rows, int64_t H, const void* dOUT,
                                          int64_t lddo, const void* Y, int64_t ldy, const void* place,
                                          const void* weights, int w_dtype, void* dY, int64_t lddy, void* dweights,
                                          const void* offsets, int64_t experts, void* stream);

/*
 * The experts' products over sorted rows: gemm_f16_grouped where only the device knows the groups.
 * A (rows x K) and C (rows x N) binary16; expert e owns rows offsets[e] .. offsets[e + 1] (experts + 1
 * int32 in device memory, not decreasing; values outside [0, rows] are clamped) and the matrix at B +
 * e * stride_b (elements), N x K with trans_b (a linear layer's weight), else K x N:
 *   C[p, :] = ReLU?(A[p, :] op(B_e)),
 * accumulated in float32 and rounded to binary16 once. Rows of C that no expert owns are left as they
 * were, or, with zero_rest, those from offsets[experts] on are set to zero. K == 0 writes zeros to the
 * rows that are owned. The tile kernels need A and B 16-byte aligned, lda, ldb, stride_b and their
 * contiguous dimensions multiples of 8, lda and ldb at most TGEMM_FAST_MAX_LD; other arguments take the
 * generic kernel. A launch of 2^23 workgroups or more is TGEMM_EINVAL_DIM.
 */
TGEMM_API int expert_gemm_f16(int trans_b, int64_t rows, int64_t experts, int64_t N, int64_t K,
                              const void* A, int64_t lda, const void* offsets, const void* B, int64_t ldb,
                              int64_t stride_b, void* C, int64_t ldc, int relu, int zero_rest, void* stream);

/*
 * The products' gradient by the experts' matrices: C_e = A_e^T B_e for every expert, A (rows x M) and
 * B (rows x N), C_e (M x N binary16) at C + e * stride_c; zeros for an expert of no rows. (With C =
 * A B_e^T above: dA = dC B_e is expert_gemm_f16 without trans_b, dB_e = dC_e^T A_e.) stride_c is at
 * least (M - 1) * ldc + N.
 */
TGEMM_API int expert_gemm_f16_tn(int64_t rows, int64_t experts, int64_t M, int64_t N, const void* A, int64_t lda,
                                 const void* B, int64_t ldb, const void* offsets, void* C, int64_t ldc,
                                 int64_t stride_c, void* stream);

/* Tooling: the experts' products forced to kernel idx (TGEMM_EXPERT_*; TGEMM_EINVAL_CFG for an index
 * out of range or a kernel that cannot take the arguments), and the kernel a call takes (form 0: rows
 * with trans_b, 1: rows without, 2: the _tn product, K ignored; -100 for a call that launches nothing). */
#define TGEMM_EXPERT_GENERIC 0
#define TGEMM_EXPERT_32 1   /* 32 x 128 tiles; not of the _tn product */
#define TGEMM_EXPERT_128 2  /* TGEMM_EXPERT_TILES held to 128 x 128 tiles */
#define TGEMM_EXPERT_256 3  /* and to 256 x 256, but for edges of half of one or less */
#define TGEMM_EXPERT_TILES 4
#define TGEMM_EXPERT_64 5   /* 64 x 128 tiles; not of the _tn product */
TGEMM_API int expert_gemm_f16_cfg(int idx, int trans_b, int64_t rows, int64_t experts, int64_t N, int64_t K,
                                  const void* A, int64_t lda, const void* offsets, const void* B, int64_t ldb,
                                  int64_t stride_b, void* C, int64_t ldc, int relu, int zero_rest, void* stream);
TGEMM_API int expert_gemm_f16_tn_cfg(int idx, int64_t rows, int64_t experts, int64_t M, int64_t N,
                                     const void* A, int64_t lda, const void* B, int64_t ldb, const void* offsets,
                                     void* C, int64_t ldc, int64_t stride_c, void* stream);
TGEMM_API int expert_gemm_select_config(int form, int64_t rows, int64_t experts, int64_t M, int64_t N, int64_t K,
                                        const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b);

/* MXFP4 tooling: the two products forced to kernel idx (TGEMM_MX_*; TGEMM_EINVAL_CFG for an
 * index out of range, a fast kernel that cannot take the arguments, or the skinny kernel with M
 * > 256), and the kernel a call takes (-100 / -101 as for tgemm_select_config; f16_a: the
 * product with binary16 A, scale_a ignored). */
#define TGEMM_MX_GENERIC 0
#define TGEMM_MX_SKINNY 1
#define TGEMM_MX_128 2
#define TGEMM_MX_256 3
#define TGEMM_MX_64 4   /* 64 x 128 tiles; not with binary16 A */
TGEMM_API int mxfp4_gemm_cfg(int idx, int64_t M, int64_t N, int64_t K,
                             const void* A, int64_t lda, const void* scale_a, int64_t ldsa,
                             const void* B, int64_t ldb, const void* scale_b, int64_t ldsb,
                             void* C, int64_t ldc, int relu, void* stream);
TGEMM_API int mxfp4_gemm_f16_cfg(int idx, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                                 const void* B, int64_t ldb, const void* scale_b, int64_t ldsb,
                                 void* C, int64_t ldc, int relu, void* stream);
TGEMM_API int mxfp4_select_config(int f16_a, int64_t M, int64_t N, int64_t K,
                                        const void* A, int64_t lda, const void* scale_a, int64_t ldsa,
                                        const void* B, int64_t ldb, const void* scale_b, int64_t ldsb,
                                        const void* C, int64_t ldc);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_OPS_H_ */
