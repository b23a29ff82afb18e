/*
 * mxfp4.h - MXFP4 quantisation and products in libnvfp4moe.so (sm_100a).
 *
 * MXFP4 (OCP Microscaling Formats v1.0) is the 4-bit sibling of the layer's
 * NVFP4: E2M1 elements in blocks of 32 under one E8M0 (power of two) scale,
 * without a global scale.  The calls here quantise, read back and multiply
 * such matrices outside the NVFP4 layer: dense, or grouped by expert on the
 * rows that moe_route orders.
 *
 * Format
 *   - A matrix of `rows` x `cols` has B = ceil(cols / 32) blocks a row.  Its
 *     codes are [rows][16 B] bytes, two E2M1 codes per byte, the element with
 *     the even index in the low nibble, the sign in bit 3 of a code; elements
 *     past `cols` in the last block are zero.
 *   - Scales, one E8M0 byte per block (value 2^(byte - 127), 255 is NaN):
 *       NVFP4_LAYOUT_CANONICAL: [rows][B].
 *       NVFP4_LAYOUT_TILED: the layout the tensor-core MMA reads.  Rows in
 *       tiles of 128 and blocks in groups of 4; each (row tile, group) is a
 *       512-byte atom, atoms ordered row tile major, and inside an atom row r
 *       (0..127), block b (0..3) sits at byte (r % 32) * 16 + (r / 32) * 4 + b.
 *       The bytes of a data row's padding blocks (past B in the last group)
 *       are 0.  Padding rows may hold anything.
 *     mxfp4_scale_bytes() gives the size of either.
 *   - A block with largest magnitude a gets the scale 2^(floor(log2 a) - 2),
 *     no less than 2^-127, and each element x the E2M1 value nearest to
 *     x / scale (ties to even, clamped at 6).  Every step is exact in fp32.  A
 *     zero block has scale byte 0.  A block that holds a NaN or an infinity
 *     gets scale byte 255 and codes 0: every value of it reads back as NaN,
 *     and so does every product it enters.
 *
 * Conventions are those of nvfp4_moe.h (device memory of the caller, nothing
 * allocated, work queued on `stream`, checks on the host before anything is
 * queued).  A workspace serves one call at a time: calls or captured graphs
 * that share one run one after the other.  Outputs share no memory with inputs
 * but where a call allows it.  Sizes of zero rows are legal and queue nothing.
 */
#ifndef NVFP4_MOE_MXFP4_H
#define NVFP4_MOE_MXFP4_H

#include "nvfp4_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of unquantised matrices. */
enum { MXFP4_DTYPE_BF16 = 0, MXFP4_DTYPE_F16 = 1, MXFP4_DTYPE_F32 = 2 };

/* Bytes of the scales of a rows x cols matrix in `layout` (0 for an unknown
 * layout or a negative size). */
NVFP4_API size_t mxfp4_scale_bytes(int rows, int cols, int layout);

/* Quantises x[rows][cols] (dtype, rows `row_stride` elements apart).  With
 * `perm` (device int32 [perm_rows], nullable) the quantised matrix has
 * perm_rows rows, row r being x[perm[r]], or zeros where perm[r] is negative
 * or not below `rows`.  codes and scales as above (codes 16-byte, scales
 * 4-byte aligned). */
NVFP4_API nvfp4_status mxfp4_quantize(const void* x, int dtype, int rows, int cols, long long row_stride,
                                      const int32_t* perm, int perm_rows, int layout, uint8_t* codes,
                                      uint8_t* scales, void* stream);

/* Quantises the transpose of x[rows][cols]: the result is a cols x rows
 * matrix with its blocks along x's columns, the operand of a product that
 * sums over x's rows (a gradient).  One read of x, no transposed copy. */
NVFP4_API nvfp4_status mxfp4_quantize_transposed(const void* x, int dtype, int rows, int cols, long long row_stride,
                                                 int layout, uint8_t* codes, uint8_t* scales, void* stream);

/* Reads a rows x cols matrix back: out[r * row_stride + c] = code * scale,
 * rounded once to dtype (exact for fp32; exact for bf16 too, whose subnormals
 * hold the smallest values). */
NVFP4_API nvfp4_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int layout, int rows, int cols,
                                        int dtype, void* out, long long row_stride, void* stream);

/* ------------------------------------------------------------------------
 * Products.
 *
 * y[m][n] = row_weight[m] * (sum_k a[m][k] * b[n][k] + bias[n])
 * with a (M x K) and b (N x K) in MXFP4, scales TILED, fp32 accumulation on
 * the tensor cores, one rounding to out_dtype.  y rows are y_stride elements
 * apart.  row_weight (fp32 [M]) and bias (fp32 [N]) are nullable.
 *
 * Grouped by expert: E >= 1 with expert_offsets (device int32 [E+1]) and b
 * holding E matrices of N rows each (N % 128 == 0), bias [E][N].  Rows
 * [expert_offsets[e], expert_offsets[e] + expert_counts[e]) of a meet expert
 * e's matrix; expert_counts NULL means the whole segment.  Offsets are
 * non-decreasing multiples of 128 as moe_route writes them; values outside
 * [0, M] are clamped (M may be any number: the last segment may end inside its
 * padding), and a segment that then starts elsewhere than at a multiple of 128
 * has no rows.  Rows of y that belong to no expert keep what they held.  Dense: E = 0 and expert_offsets = expert_counts = NULL; every row is
 * written.
 *
 * a codes, b codes and scales need 16-byte alignment.  E <= 1024, M, N and K
 * <= 2^30.  The result does not depend on scheduling.
 * ---------------------------------------------------------------------- */
NVFP4_API size_t mxfp4_matmul_workspace_size(void);
NVFP4_API nvfp4_status mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int M, const uint8_t* b_codes,
                                    const uint8_t* b_scales, int N, int K, int E, const int32_t* expert_offsets,
                                    const int32_t* expert_counts, const float* row_weight, const float* bias,
                                    int out_dtype, void* y, long long y_stride, void* ws, size_t ws_bytes,
                                    void* stream);

/* The product with a = x (or x[perm]) quantised in the call: mxfp4_quantize
 * into the workspace, then mxfp4_matmul on its M rows (M = perm_rows with
 * perm, else rows).  A dense product of few rows quantises them itself, with
 * the same result.  The workspace's status word is that of the product.  y may
 * take the place of x. */
NVFP4_API size_t mxfp4_linear_workspace_size(int M, int K);
NVFP4_API nvfp4_status mxfp4_linear(const void* x, int dtype, int rows, long long row_stride, const int32_t* perm,
                                    int perm_rows, const uint8_t* b_codes, const uint8_t* b_scales, int N, int K,
                                    int E, const int32_t* expert_offsets, const int32_t* expert_counts,
                                    const float* row_weight, const float* bias, int out_dtype, void* y,
                                    long long y_stride, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_MOE_MXFP4_H */
