// mlp_ops_kernels.h -- launches of the single operators (include/mlp_ops.h), arguments already checked.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace mlpk {

// One product with its epilogue: a dense layer, or the experts' layers over their slots.
struct ProductArgs {
    const void *x;
    int64_t ldx;
    const void *w;
    int64_t ldw;
    int64_t w_stride;  // grouped: elements between the experts' matrices
    const void *bias;
    const void *residual;  // dense only
    int64_t ldr;
    void *y;
    int64_t ldy;
    int64_t rows;  // dense: rows; grouped: slots, in use or not (tokens * k)
    int in, out;   // widths; a gated layer's w has 2 * out rows
    int act;       // MLP_EPI_*, or kSiluFull
    int y_fp32;    // 1: y and residual are FP32, 0: of the inputs' type
    // grouped only
    const int32_t *offsets;  // [experts + 1]
    const int32_t *slots;    // the assignment of each slot, or NULL: x is by slot
    int experts, k;
};

enum { kSiluFull = 5 };  // SiLU for FP32 outputs: the other form is exact to well below a 16-bit rounding only

enum { kFp16 = 0, kBf16 = 1, kFp32 = 2 };  // MLP_DTYPE_*

hipError_t launch_product(const ProductArgs &p, int dtype, bool gated, bool grouped, hipStream_t stream);
// Whether one launch holds the product's tiles.
bool product_fits(const ProductArgs &p, bool gated, bool grouped);

// The kernel that launch_product takes, for tests.
const char *product_kernel(const ProductArgs &p, bool gated, bool grouped);

// y[t] = round(sum_j weight[t][j] * part[places[t][j]] + residual[t]) over FP32 rows `part`.
struct CombineArgs {
    const float *part;  // [slots][ldp], 16-byte aligned rows
    int64_t ldp;
    const int32_t *places;
    const float *weight;  // NULL: 1
    const void *residual;
    int64_t ldr;
    void *y;
    int64_t ldy;
    int64_t tokens;
    int k, out;
};
hipError_t launch_combine(const CombineArgs &c, int out_dtype, hipStream_t stream);

struct RouteArgs {
    const void *logits;
    int64_t ld;
    const float *bias;
    int32_t *index;
    float *weight;
    int64_t tokens;
    int experts, k, groups, topk_groups, group_top;
    int lanes;  // of a group, set at the launch
    bool sigmoid, renormalise;
    float scale;
};
hipError_t launch_route(const RouteArgs &r, int dtype, hipStream_t stream);
// The kernel that launch_route takes, for tests.
const char *route_kernel(const RouteArgs &r);

struct DispatchArgs {
    const int32_t *index;
    int32_t *offsets, *slots, *places;
    int32_t *workspace;
    int64_t n;  // assignments
    int experts;
};
// Entries (int32) of the dispatch workspace.
int64_t dispatch_workspace_entries(int64_t n, int experts);
hipError_t launch_dispatch(const DispatchArgs &d, hipStream_t stream);

}  // namespace mlpk
