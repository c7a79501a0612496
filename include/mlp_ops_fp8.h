/*
 * mlp_ops_fp8.h -- layers with 8-bit operands, beside the 16-bit ones of mlp_ops.h, same library: the norm that
 * feeds them, the rounding to 8 bits, one affine layer with its epilogue, and the experts' layers on routed rows.
 *
 * The format: E4M3 values (OCP, largest 448, one NaN) with FP32 scales.  A scale belongs to a block of
 * MLP_FP8_BLOCK columns, of one row (activations) or of MLP_FP8_BLOCK rows (weights); blocks begin at row and
 * column 0, the last of a row or column is as short as it has to be.  The element is value * scale.
 *   scale = max(amax / 448, 2^-126),  value = round(v * (1 / scale)),  to nearest, ties to even,
 * amax over the block's finite elements; a NaN or an infinity becomes NaN by itself and leaves the others as they are.  The
 * reciprocal and the product are rounded to FP32 first: v / scale within 2^-22 of itself of the middle between two E4M3
 * numbers may go to either.
 * Scales made elsewhere are taken as they are, of any sign; a layer multiplies those of its two operands' blocks in FP32, so a
 * block whose product is infinite gives infinities or NaN, whatever its values, and one below 2^-126 has fewer bits.
 *
 * Conventions as in mlp_ops.h: status codes and mlp_last_error, arguments checked on the host before any HIP call,
 * work enqueued on `stream` without allocating or waiting, scratch memory the caller's, no state, the same bits for
 * the same call.  Row strides (ld*) are in elements, scales' (ldxs, ...) in scales; 16-byte aligned rows are faster.
 */
#ifndef MLP_OPS_FP8_H
#define MLP_OPS_FP8_H

#include "mlp_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLP_FP8_BLOCK 128
#define MLP_DTYPE_FP8 3 /* an output in the format above: E4M3 values and their scales */
#define MLP_FP8_MAX_COUNT 65535 /* matrices of one mlp_quantize call */

/* The root-mean-square norm of the residual stream, and the next layer's input:
 *   total[r][i] = round(x[r][i] + residual[r][i]),  or x without a residual,
 *   y[r][i] = total[r][i] / sqrt(mean_j total[r][j]^2 + eps) * weight[i],
 * rounded once to y, or to values and scales, or to both.  The sum of squares is held in 64 bits. */
typedef struct mlp_rms_norm_args {
    int64_t rows;      /* 0 .. INT32_MAX                                                                */
    int32_t width;     /* 1 .. MLP_OPS_MAX_WIDTH                                                         */
    int32_t dtype;     /* of x, residual, total and weight: MLP_DTYPE_FP16, _BF16 or _FP32               */
    int32_t out_dtype; /* of y: dtype, or MLP_DTYPE_FP32                                                 */
    float eps;         /* 2^-126 or more, finite                                                        */
    const void *x;     /* [rows][width]                                                                 */
    int64_t ldx;
    const void *residual; /* [rows][width], or NULL                                                     */
    int64_t ldr;
    const void *weight; /* [width], or NULL for 1                                                       */
    void *total;        /* [rows][width], or NULL; with a residual only; may be x or residual itself      */
    int64_t ldt;
    void *y; /* [rows][width], or NULL                                                                  */
    int64_t ldy;
    uint8_t *values; /* [rows][width], or NULL where y is not                                           */
    int64_t ldv;
    float *scales; /* [rows][ceil(width / 128)], with values                                            */
    int64_t lds;
} mlp_rms_norm_args;

int mlp_rms_norm(const mlp_rms_norm_args *args, void *stream);

/* `count` matrices to the format above. */
typedef struct mlp_quantize_args {
    int64_t rows;       /* 0 .. INT32_MAX, of each matrix                                                */
    int32_t count;      /* 0 .. MLP_FP8_MAX_COUNT                                                        */
    int32_t width;      /* 1 .. MLP_OPS_MAX_WIDTH                                                        */
    int32_t dtype;      /* of x: MLP_DTYPE_FP16, _BF16 or _FP32                                          */
    int32_t block_rows; /* 1, or MLP_FP8_BLOCK                                                           */
    const void *x;      /* [count][rows][width]                                                         */
    int64_t ldx;
    int64_t x_stride; /* elements from one matrix to the next                                           */
    uint8_t *values;  /* [count][rows][width]                                                           */
    int64_t ldv;
    int64_t v_stride;
    float *scales; /* [count][ceil(rows / block_rows)][ceil(width / 128)]                               */
    int64_t lds;
    int64_t s_stride;
} mlp_quantize_args;

int mlp_quantize(const mlp_quantize_args *args, void *stream);

/* mlp_linear with operands in the format above:
 *   z[r][o] = sum_b x_scale[r][b] w_scale[o / 128][b] (sum_{i in block b} x[r][i] w[o][i]) + bias[o],
 *   y[r][o] = round(act(z[r][o]) + residual[r][o]),  or gated, round(act(z[r][o]) z[r][out_width + o] + residual[r][o]),
 * in FP32, rounded once.  16-bit outputs are sums of the matrix unit's 8-bit products: it adds 8 neighbouring columns'
 * products after cutting each to 2^-13 of the largest one's power of two.  A sum is off by less than 7 * 2^-13 of the groups'
 * largest |x| times largest |w|, summed over the groups of 8, whatever is left of it: an output whose products cancel can be
 * off by many of its own steps.  In the root mean square that is 2^-16 of the outputs' own where the columns are alike, and
 * 2^-14 where one of 8 outweighs the others; the rounding to FP16 is 2^-12, to BF16 2^-9.  FP32 and 8-bit outputs get sums
 * whose products are not cut, at half that unit's rate.  The halves of a gated
 * layer's w are matrices of their own: the blocks of the second begin at its row out_width, and its scales' rows follow
 * the ceil(out_width / 128) of the first. */
typedef struct mlp_fp8_linear_args {
    int64_t rows;      /* 0 .. INT32_MAX                                                                */
    int32_t in_width;  /* 1 .. MLP_OPS_MAX_WIDTH                                                         */
    int32_t out_width; /* 1 .. MLP_OPS_MAX_WIDTH                                                         */
    int32_t out_dtype; /* of y and residual: MLP_DTYPE_FP16, _BF16 or _FP32; or MLP_DTYPE_FP8, no residual */
    int32_t act;       /* MLP_EPI_*                                                                     */
    int32_t gated;     /* 0, or 1: w and bias have 2 * out_width rows, the gates first                  */
    const uint8_t *x;  /* [rows][in_width]                                                              */
    int64_t ldx;
    const float *x_scale; /* [rows][ceil(in_width / 128)]                                               */
    int64_t ldxs;
    const uint8_t *w; /* [out_width or 2 * out_width][in_width]                                         */
    int64_t ldw;
    const float *w_scale; /* [ceil(out_width / 128), twice if gated][ceil(in_width / 128)]              */
    int64_t ldws;
    const float *bias;    /* [out_width or 2 * out_width], or NULL                                      */
    const void *residual; /* [rows][out_width], or NULL; may be y itself (same pointer and stride)      */
    int64_t ldr;
    void *y; /* [rows][out_width]; overlaps no input but such a residual                                */
    int64_t ldy;
    float *y_scale; /* [rows][ceil(out_width / 128)] with MLP_DTYPE_FP8, else NULL                      */
    int64_t ldys;
    void *workspace; /* mlp_fp8_linear_workspace bytes, 16-byte aligned (NULL where that is 0)          */
    uint64_t workspace_bytes;
} mlp_fp8_linear_args;

/* Bytes of workspace mlp_fp8_linear needs for these sizes, strides and (by their alignment) pointers of x and w: FP32 rows
 * where 8-bit outputs are rounded by a kernel of its own, else 0. */
int mlp_fp8_linear_workspace(const mlp_fp8_linear_args *args, uint64_t *bytes);
int mlp_fp8_linear(const mlp_fp8_linear_args *args, void *stream);

/* mlp_expert_linear with operands in the format above, each expert's layer as in mlp_fp8_linear.  offsets, slots and
 * places are mlp_dispatch's, with the same clamping; x_scale has a row for each row of x, y_scale for each of y (rows
 * behind offsets[experts] are left as they were).  MLP_DTYPE_FP8 goes without combine.  Combined, a token's terms and their sum
 * are FP32, rounded once. */
typedef struct mlp_fp8_expert_linear_args {
    int64_t tokens; /* tokens * k: 0 .. INT32_MAX */
    int32_t k;
    int32_t experts;
    int32_t in_width, out_width;
    int32_t out_dtype, act, gated;
    int32_t x_slots, combine; /* as in mlp_expert_linear_args                                           */
    const uint8_t *x;         /* [tokens or tokens * k][in_width]                                       */
    int64_t ldx;
    const float *x_scale; /* [tokens or tokens * k][ceil(in_width / 128)]                               */
    int64_t ldxs;
    const uint8_t *w; /* [experts][out_width or 2 * out_width][in_width]                                */
    int64_t ldw;
    int64_t w_stride;
    const float *w_scale; /* [experts][ceil(out_width / 128), twice if gated][ceil(in_width / 128)]     */
    int64_t ldws;
    int64_t ws_stride;
    const float *bias; /* [experts][out_width or 2 * out_width], contiguous, or NULL                    */
    const int32_t *offsets;
    const int32_t *slots;
    const int32_t *places;
    const float *weight;  /* [tokens][k] with combine, or NULL for 1; NULL without combine              */
    const void *residual; /* [tokens][out_width] with combine, or NULL; may be y itself                 */
    int64_t ldr;
    void *y;
    int64_t ldy;
    float *y_scale;
    int64_t ldys;
    void *workspace; /* mlp_fp8_expert_linear_workspace bytes, 16-byte aligned (NULL where that is 0)   */
    uint64_t workspace_bytes;
} mlp_fp8_expert_linear_args;

/* Bytes of workspace mlp_fp8_expert_linear needs, as above; also the outputs by slot where it combines. */
int mlp_fp8_expert_linear_workspace(const mlp_fp8_expert_linear_args *args, uint64_t *bytes);
int mlp_fp8_expert_linear(const mlp_fp8_expert_linear_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MLP_OPS_FP8_H */
