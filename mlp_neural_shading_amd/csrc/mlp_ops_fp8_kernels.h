// mlp_ops_fp8_kernels.h -- launches of the operators of include/mlp_ops_fp8.h, arguments already checked.
#pragma once

#include "mlp_ops_kernels.h"

namespace mlpk {

constexpr int kFp8Block = 128;

struct NormArgs {
    const void *x;
    int64_t ldx;
    const void *residual;  // or NULL
    int64_t ldr;
    const void *weight;  // or NULL
    void *total;         // or NULL
    int64_t ldt;
    void *y;  // or NULL
    int64_t ldy;
    uint8_t *values;  // or NULL
    int64_t ldv;
    float *scales;
    int64_t lds;
    int64_t rows;
    int width;
    int y_fp32;
    float eps;
};
hipError_t launch_norm(const NormArgs &n, int dtype, hipStream_t stream);
// The kernel that launch_norm takes, for tests.
const char *norm_kernel(const NormArgs &n, int dtype);

struct QuantizeArgs {
    const void *x;
    int64_t ldx, x_stride;
    uint8_t *values;
    int64_t ldv, v_stride;
    float *scales;
    int64_t lds, s_stride;
    int64_t rows;
    int count, width;
    const int32_t *used;  // rows from *used on are left out (rows by slot); or NULL
};
hipError_t launch_quantize(const QuantizeArgs &q, int dtype, int block_rows, hipStream_t stream);

// A product of 8-bit operands: ProductArgs with bytes for x and w, FP32 bias, and the scales.
struct Fp8ProductArgs : ProductArgs {
    const float *xs;
    int64_t ldxs;
    const float *ws;
    int64_t ldws, ws_stride;
    bool eight;       // 8-bit outputs, here or by another kernel from FP32 rows
    uint8_t *values;  // 8-bit outputs, or NULL: then y
    int64_t ldv;
    float *ys;
    int64_t ldys;
};
// type: what becomes of the results, kFp16 or kBf16 (at once, or with y_fp32 from FP32 rows in a workspace), or kFp32 for FP32's
// accuracy.
hipError_t launch_fp8_product(const Fp8ProductArgs &p, int type, bool gated, bool grouped, hipStream_t stream);
bool fp8_product_fits(const Fp8ProductArgs &p, int type, bool gated, bool grouped);
// Whether the product's kernel (type kFp32) rounds to 8 bits itself: `values` and `ys` may be set, y is not used then.
bool fp8_product_rounds(const Fp8ProductArgs &p, bool gated, bool grouped);
const char *fp8_product_kernel(const Fp8ProductArgs &p, int type, bool gated, bool grouped);

}  // namespace mlpk
