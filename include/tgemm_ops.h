/*
 * tgemm_ops.h -- C ABI of libtgemm, the operators beside the GEMMs of tgemm.h: MXFP4 (4-bit
 * microscaled) matrices with their quantiser and products, and the orthogonalisation of a
 * weight's update. The same library and conventions
 * (row-major storage, device pointers owned by the caller, nothing allocated, enqueue-only calls
 * on the given stream, the TGEMM_E* codes of tgemm.h, C not overlapping an input).
 */
#ifndef TGEMM_OPS_H_
#define TGEMM_OPS_H_

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

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
#define TGEMM_DTYPE_F16 0
#define TGEMM_DTYPE_F32 1
TGEMM_API int64_t orthogonalize_workspace_bytes(int64_t batch, int64_t R, int64_t C);
TGEMM_API int orthogonalize_f16(int64_t batch, int64_t R, int64_t C, int dtype,
                                const void* G, int64_t ldg, int64_t stride_g,
                                void* X, int64_t ldx, int64_t stride_x,
                                int steps, float a, float b, float c, float scale,
                                void* workspace, int64_t workspace_bytes, void* stream);

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
