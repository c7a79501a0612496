// mlp_ops_fp8_api.cpp -- the entry points of include/mlp_ops_fp8.h: argument checks and launches.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mlp_error.h"
#include "mlp_ops_check.h"
#include "mlp_ops_fp8.h"
#include "mlp_ops_fp8_kernels.h"
#include "mlp_ops_kernels.h"
#include "mlp_testing.h"

using namespace mlpk;

namespace {

int64_t blocks_of(int64_t n) { return (n + MLP_FP8_BLOCK - 1) / MLP_FP8_BLOCK; }
int size_of(int dtype) { return dtype == MLP_DTYPE_FP32 ? 4 : dtype == MLP_DTYPE_FP8 ? 1 : 2; }
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Whether `out` shares a byte with one of `in`.
template <size_t N>
bool overlaps(const Span &out, const Span (&in)[N])
{
    for (const Span &s : in)
        if (overlap(out, s))
            return true;
    return false;
}

// `out` may be `in` itself, element by element.
bool itself(const Span &out, const Span &in) { return out.at == in.at && (out.ld == in.ld || out.rows == 1); }

int check_norm(const mlp_rms_norm_args *a)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    MLP_TRY(check_range("rows", a->rows, 0, INT32_MAX));
    MLP_TRY(check_range("width", a->width, 1, MLP_OPS_MAX_WIDTH));
    MLP_TRY(check_range("dtype", a->dtype, MLP_DTYPE_FP16, MLP_DTYPE_FP32));
    if (a->out_dtype != a->dtype && a->out_dtype != MLP_DTYPE_FP32)
        return fail(MLP_ERR_INVALID_ARGUMENT, "out_dtype must be dtype or MLP_DTYPE_FP32, got %d", a->out_dtype);
    if (!(a->eps >= 0x1p-126f) || !isfinite(a->eps))
        return fail(MLP_ERR_INVALID_ARGUMENT, "eps must be finite and at least 2^-126");
    return MLP_OK;
}

int prepare_norm(const mlp_rms_norm_args *a, NormArgs &n)
{
    MLP_TRY(check_norm(a));
    if (a->rows == 0)
        return MLP_OK;
    const int size = size_of(a->dtype), y_size = size_of(a->out_dtype);
    const int64_t rows = a->rows, width = a->width, blocks = blocks_of(width);
    MLP_TRY(check_matrix("x", a->x, rows, width, a->ldx, size));
    if (a->residual)
        MLP_TRY(check_matrix("residual", a->residual, rows, width, a->ldr, size));
    if (a->weight)
        MLP_TRY(check_vector("weight", a->weight, size));
    if (a->total) {
        if (!a->residual)
            return fail(MLP_ERR_INVALID_ARGUMENT, "total goes with a residual");
        MLP_TRY(check_matrix("total", a->total, rows, width, a->ldt, size));
    }
    if (!a->y && !a->values)
        return fail(MLP_ERR_INVALID_ARGUMENT, "y and values are NULL");
    if (a->y)
        MLP_TRY(check_matrix("y", a->y, rows, width, a->ldy, y_size));
    if (a->values) {
        MLP_TRY(check_matrix("values", a->values, rows, width, a->ldv, 1));
        MLP_TRY(check_matrix("scales", a->scales, rows, blocks, a->lds, 4));
    }
    const Span x = span(a->x, rows, width, a->ldx, size), r = span(a->residual, rows, width, a->ldr, size);
    const Span w = span(a->weight, 1, width, width, size), t = span(a->total, rows, width, a->ldt, size);
    const Span y = span(a->y, rows, width, a->ldy, y_size), v = span(a->values, rows, width, a->ldv, 1);
    const Span s = span(a->values ? a->scales : nullptr, rows, blocks, a->lds, 4);
    const Span before_y[] = {x, r, w, t}, before_v[] = {x, r, w, t, y}, before_s[] = {x, r, w, t, y, v};
    if (overlap(t, w) || (!itself(t, x) && overlap(t, x)) || (!itself(t, r) && overlap(t, r)))
        return fail(MLP_ERR_INVALID_ARGUMENT, "total overlaps an input without being x or residual");
    if (overlaps(y, before_y) || overlaps(v, before_v) || overlaps(s, before_s))
        return fail(MLP_ERR_INVALID_ARGUMENT, "y, values or scales overlaps another buffer");
    n.x = a->x;
    n.ldx = a->ldx;
    n.residual = a->residual;
    n.ldr = a->ldr;
    n.weight = a->weight;
    n.total = a->total;
    n.ldt = a->ldt;
    n.y = a->y;
    n.ldy = a->ldy;
    n.values = a->values;
    n.ldv = a->ldv;
    n.scales = a->scales;
    n.lds = a->lds;
    n.rows = rows;
    n.width = a->width;
    n.y_fp32 = a->out_dtype == MLP_DTYPE_FP32;
    n.eps = a->eps;
    return MLP_OK;
}

// Elements from the first to behind the last of `count` matrices `stride` apart.
int check_count(const char *name, int count, int64_t stride, int64_t rows, int64_t cols, int64_t ld)
{
    if (count > 1 && (stride < (rows - 1) * ld + cols || stride > (INT64_MAX >> 3) / count))
        return fail(MLP_ERR_INVALID_ARGUMENT, "%s %lld does not hold a matrix's %lld rows", name, (long long)stride, (long long)rows);
    return MLP_OK;
}

Span many(const void *p, int count, int64_t stride, int64_t rows, int64_t cols, int64_t ld, int size)
{
    const int64_t all = (count > 1 ? (count - 1) * stride : 0) + (rows - 1) * ld + cols;
    return count > 1 ? span(p, 1, all, all, size) : span(p, rows, cols, ld, size);
}

int check_fp8_layer(int in_width, int out_width, int out_dtype, int act, int gated)
{
    MLP_TRY(check_range("in_width", in_width, 1, MLP_OPS_MAX_WIDTH));
    MLP_TRY(check_range("out_width", out_width, 1, MLP_OPS_MAX_WIDTH));
    MLP_TRY(check_range("out_dtype", out_dtype, MLP_DTYPE_FP16, MLP_DTYPE_FP8));
    MLP_TRY(check_range("act", act, MLP_EPI_NONE, MLP_EPI_SILU));
    MLP_TRY(check_range("gated", gated, 0, 1));
    return MLP_OK;
}

int check_linear(const mlp_fp8_linear_args *a)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    MLP_TRY(check_range("rows", a->rows, 0, INT32_MAX));
    return check_fp8_layer(a->in_width, a->out_width, a->out_dtype, a->act, a->gated);
}

int check_expert_linear(const mlp_fp8_expert_linear_args *a)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    MLP_TRY(check_range("experts", a->experts, 1, MLP_OPS_MAX_EXPERTS));
    MLP_TRY(check_range("k", a->k, 1, MLP_OPS_MAX_TOPK));
    MLP_TRY(check_range("tokens", a->tokens, 0, INT32_MAX));
    MLP_TRY(check_range("tokens * k", a->tokens * a->k, 0, INT32_MAX));
    MLP_TRY(check_fp8_layer(a->in_width, a->out_width, a->out_dtype, a->act, a->gated));
    MLP_TRY(check_range("x_slots", a->x_slots, 0, 1));
    MLP_TRY(check_range("combine", a->combine, 0, 1));
    if (a->combine && a->out_dtype == MLP_DTYPE_FP8)
        return fail(MLP_ERR_INVALID_ARGUMENT, "MLP_DTYPE_FP8 goes without combine");
    return MLP_OK;
}

// Row stride (floats) of FP32 rows in a workspace.
int64_t part_stride(int out_width) { return round_up(out_width, 4); }

// What the choice of kernel depends on: sizes, strides and the operands' alignment.
Fp8ProductArgs sizes(const mlp_fp8_linear_args *a)
{
    Fp8ProductArgs p{};
    p.rows = a->rows;
    p.in = a->in_width;
    p.out = a->out_width;
    p.eight = a->out_dtype == MLP_DTYPE_FP8;
    p.x = a->x;
    p.ldx = a->ldx;
    p.w = a->w;
    p.ldw = a->ldw;
    return p;
}

Fp8ProductArgs sizes(const mlp_fp8_expert_linear_args *a)
{
    Fp8ProductArgs p{};
    p.rows = a->tokens * a->k;
    p.in = a->in_width;
    p.out = a->out_width;
    p.eight = a->out_dtype == MLP_DTYPE_FP8;
    p.x = a->x;
    p.ldx = a->ldx;
    p.w = a->w;
    p.ldw = a->ldw;
    p.experts = a->experts;
    p.k = a->k;
    p.w_stride = a->experts > 1 ? a->w_stride : 0;  // of one expert it may be anything
    return p;
}

// 8-bit outputs have FP32 scales.
int result_type(int out_dtype) { return out_dtype == MLP_DTYPE_FP8 ? kFp32 : out_dtype; }

// Whether the workspace holds FP32 rows, for another kernel to combine or to round to 8 bits.
bool needs_rows(const Fp8ProductArgs &p, int out_dtype, bool combine, bool gated, bool grouped)
{
    return combine || (out_dtype == MLP_DTYPE_FP8 && !fp8_product_rounds(p, gated, grouped));
}

template <class A>
uint64_t rows_need(const A *a, bool combine, bool grouped)
{
    const Fp8ProductArgs p = sizes(a);
    return p.rows && needs_rows(p, a->out_dtype, combine, a->gated, grouped) ? (uint64_t)p.rows * part_stride(p.out) * 4 : 0;
}

uint64_t linear_need(const mlp_fp8_linear_args *a) { return rows_need(a, false, false); }
uint64_t expert_linear_need(const mlp_fp8_expert_linear_args *a) { return rows_need(a, a->combine, true); }

int activation(int act, int out_dtype)
{
    return act == MLP_EPI_SILU && (out_dtype == MLP_DTYPE_FP32 || out_dtype == MLP_DTYPE_FP8) ? mlpk::kSiluFull : act;
}

// The operands and the scales of both calls: `experts` matrices, x_rows rows of x.
template <class A>
int check_operands(const A *a, int64_t x_rows, int experts, int64_t w_stride, int64_t ws_stride)
{
    const int64_t wide = (int64_t)a->out_width * (a->gated ? 2 : 1), blocks = blocks_of(a->in_width);
    const int64_t down = blocks_of(a->out_width) * (a->gated ? 2 : 1);
    MLP_TRY(check_matrix("x", a->x, x_rows, a->in_width, a->ldx, 1));
    MLP_TRY(check_matrix("x_scale", a->x_scale, x_rows, blocks, a->ldxs, 4));
    MLP_TRY(check_matrix("w", a->w, wide, a->in_width, a->ldw, 1));
    MLP_TRY(check_matrix("w_scale", a->w_scale, down, blocks, a->ldws, 4));
    MLP_TRY(check_count("w_stride", experts, w_stride, wide, a->in_width, a->ldw));
    MLP_TRY(check_count("ws_stride", experts, ws_stride, down, blocks, a->ldws));
    if (a->bias)
        MLP_TRY(check_vector("bias", a->bias, 4));
    return MLP_OK;
}

// y, its scales and the residual, and what they may not share; `in` holds the inputs.
template <class A, size_t N>
int check_outputs(const A *a, int64_t y_rows, uint64_t need, const Span (&in)[N])
{
    const int size = size_of(a->out_dtype);
    const bool eight = a->out_dtype == MLP_DTYPE_FP8;
    MLP_TRY(check_matrix("y", a->y, y_rows, a->out_width, a->ldy, size));
    MLP_TRY(check_stride("y", a->ldy));
    if (eight)
        MLP_TRY(check_matrix("y_scale", a->y_scale, y_rows, blocks_of(a->out_width), a->ldys, 4));
    else if (a->y_scale)
        return fail(MLP_ERR_INVALID_ARGUMENT, "y_scale goes with MLP_DTYPE_FP8");
    const Span y = span(a->y, y_rows, a->out_width, a->ldy, size);
    const Span ys = span(a->y_scale, y_rows, blocks_of(a->out_width), a->ldys, 4);
    const Span r = span(a->residual, y_rows, a->out_width, a->ldr, size);
    if (a->residual) {
        if (eight)
            return fail(MLP_ERR_INVALID_ARGUMENT, "a residual goes without MLP_DTYPE_FP8");
        MLP_TRY(check_matrix("residual", a->residual, y_rows, a->out_width, a->ldr, size));
        MLP_TRY(check_stride("residual", a->ldr));
        if (!itself(y, r) && overlap(y, r))
            return fail(MLP_ERR_INVALID_ARGUMENT, "y overlaps residual without being it");
    }
    if (overlaps(y, in) || overlaps(ys, in) || overlap(y, ys))
        return fail(MLP_ERR_INVALID_ARGUMENT, "y or y_scale overlaps another buffer");
    MLP_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    const Span ws = span(need ? a->workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1);
    if (overlaps(ws, in) || overlap(ws, y) || overlap(ws, ys) || overlap(ws, r))
        return fail(MLP_ERR_INVALID_ARGUMENT, "workspace overlaps another buffer");
    return MLP_OK;
}

// Where the product's results go.
template <class A>
void outputs(const A *a, bool combine, bool grouped, Fp8ProductArgs &p)
{
    p.xs = a->x_scale;
    p.ldxs = a->ldxs;
    p.ws = a->w_scale;
    p.ldws = a->ldws;
    p.bias = a->bias;
    p.act = activation(a->act, a->out_dtype);
    if (needs_rows(p, a->out_dtype, combine, a->gated, grouped)) {
        p.y = a->workspace;
        p.ldy = part_stride(p.out);
        p.y_fp32 = 1;
    } else if (a->out_dtype == MLP_DTYPE_FP8) {
        p.values = (uint8_t *)a->y;
        p.ldv = a->ldy;
        p.ys = a->y_scale;
        p.ldys = a->ldys;
    } else {
        p.y = a->y;
        p.ldy = a->ldy;
        p.y_fp32 = a->out_dtype == MLP_DTYPE_FP32;
        p.residual = a->residual;
        p.ldr = a->ldr;
    }
}

// The checked call as its product; rows are left 0 where there is nothing to do.
int prepare_linear(const mlp_fp8_linear_args *a, Fp8ProductArgs &p)
{
    MLP_TRY(check_linear(a));
    if (a->rows == 0)
        return MLP_OK;
    MLP_TRY(check_operands(a, a->rows, 1, 0, 0));
    const int64_t wide = (int64_t)a->out_width * (a->gated ? 2 : 1), blocks = blocks_of(a->in_width);
    const int64_t down = blocks_of(a->out_width) * (a->gated ? 2 : 1);
    const Span in[] = {span(a->x, a->rows, a->in_width, a->ldx, 1), span(a->x_scale, a->rows, blocks, a->ldxs, 4),
                       span(a->w, wide, a->in_width, a->ldw, 1), span(a->w_scale, down, blocks, a->ldws, 4),
                       span(a->bias, 1, wide, wide, 4)};
    MLP_TRY(check_outputs(a, a->rows, linear_need(a), in));
    p = sizes(a);
    outputs(a, false, false, p);
    if (!fp8_product_fits(p, result_type(a->out_dtype), a->gated, false))
        return fail(MLP_ERR_UNSUPPORTED, "%lld rows of %d outputs are more tiles than one launch holds", (long long)a->rows,
                    a->out_width);
    return MLP_OK;
}

// The checked call as its product; rows are left 0 where there is nothing to do.
int prepare_expert_linear(const mlp_fp8_expert_linear_args *a, Fp8ProductArgs &p)
{
    MLP_TRY(check_expert_linear(a));
    if (!a->combine && (a->weight || a->residual))
        return fail(MLP_ERR_INVALID_ARGUMENT, "weight and residual go with combine");
    const int64_t n = a->tokens * a->k;
    if (n == 0)
        return MLP_OK;
    const int64_t x_rows = a->x_slots ? n : a->tokens, y_rows = a->combine ? a->tokens : n;
    MLP_TRY(check_operands(a, x_rows, a->experts, a->w_stride, a->ws_stride));
    MLP_TRY(check_vector("offsets", a->offsets, 4));
    if (!a->x_slots)
        MLP_TRY(check_vector("slots", a->slots, 4));
    if (a->combine)
        MLP_TRY(check_vector("places", a->places, 4));
    if (a->weight)
        MLP_TRY(check_vector("weight", a->weight, 4));
    const int64_t wide = (int64_t)a->out_width * (a->gated ? 2 : 1), blocks = blocks_of(a->in_width);
    const int64_t down = blocks_of(a->out_width) * (a->gated ? 2 : 1), all = wide * a->experts;
    const Span in[] = {span(a->x, x_rows, a->in_width, a->ldx, 1), span(a->x_scale, x_rows, blocks, a->ldxs, 4),
                       many(a->w, a->experts, a->w_stride, wide, a->in_width, a->ldw, 1),
                       many(a->w_scale, a->experts, a->ws_stride, down, blocks, a->ldws, 4), span(a->bias, 1, all, all, 4),
                       span(a->offsets, 1, a->experts + 1, a->experts + 1, 4), span(a->slots, 1, n, n, 4),
                       span(a->places, 1, n, n, 4), span(a->weight, 1, n, n, 4)};
    MLP_TRY(check_outputs(a, y_rows, expert_linear_need(a), in));
    p = sizes(a);
    outputs(a, a->combine, true, p);
    p.ws_stride = a->experts > 1 ? a->ws_stride : 0;
    p.offsets = a->offsets;
    p.slots = a->x_slots ? nullptr : a->slots;
    if (!fp8_product_fits(p, result_type(a->out_dtype), a->gated, true))
        return fail(MLP_ERR_UNSUPPORTED, "%lld slots of %d outputs are more tiles than one launch holds", (long long)n,
                    a->out_width);
    return MLP_OK;
}

// The FP32 rows of the workspace into y and y_scale.
template <class A>
QuantizeArgs rounding(const A *a, int64_t rows, const int32_t *used)
{
    QuantizeArgs q{};
    q.x = a->workspace;
    q.ldx = part_stride(a->out_width);
    q.values = (uint8_t *)a->y;
    q.ldv = a->ldy;
    q.scales = a->y_scale;
    q.lds = a->ldys;
    q.rows = rows;
    q.count = 1;
    q.width = a->out_width;
    q.used = used;
    return q;
}

int put_name(const char *text, char *name, size_t cap)
{
    if (!name || cap == 0)
        return fail(MLP_ERR_INVALID_ARGUMENT, "name is NULL or empty");
    snprintf(name, cap, "%s", text);
    return ok();
}

}  // namespace

extern "C" {

int mlp_rms_norm(const mlp_rms_norm_args *a, void *stream)
{
    NormArgs n{};
    MLP_TRY(prepare_norm(a, n));
    if (n.rows == 0)
        return ok();
    const hipError_t err = launch_norm(n, a->dtype, (hipStream_t)stream);
    return err == hipSuccess ? ok() : hip_fail(err, "launching the norm");
}

int mlp_quantize(const mlp_quantize_args *a, void *stream)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    MLP_TRY(check_range("rows", a->rows, 0, INT32_MAX));
    MLP_TRY(check_range("count", a->count, 0, MLP_FP8_MAX_COUNT));
    MLP_TRY(check_range("width", a->width, 1, MLP_OPS_MAX_WIDTH));
    MLP_TRY(check_range("dtype", a->dtype, MLP_DTYPE_FP16, MLP_DTYPE_FP32));
    if (a->block_rows != 1 && a->block_rows != MLP_FP8_BLOCK)
        return fail(MLP_ERR_INVALID_ARGUMENT, "block_rows must be 1 or %d, got %d", MLP_FP8_BLOCK, a->block_rows);
    if (a->rows == 0 || a->count == 0)
        return ok();
    const int size = size_of(a->dtype);
    const int64_t across = blocks_of(a->width), down = a->block_rows == 1 ? a->rows : blocks_of(a->rows);
    MLP_TRY(check_matrix("x", a->x, a->rows, a->width, a->ldx, size));
    MLP_TRY(check_matrix("values", a->values, a->rows, a->width, a->ldv, 1));
    MLP_TRY(check_matrix("scales", a->scales, down, across, a->lds, 4));
    MLP_TRY(check_count("x_stride", a->count, a->x_stride, a->rows, a->width, a->ldx));
    MLP_TRY(check_count("v_stride", a->count, a->v_stride, a->rows, a->width, a->ldv));
    MLP_TRY(check_count("s_stride", a->count, a->s_stride, down, across, a->lds));
    const Span x = many(a->x, a->count, a->x_stride, a->rows, a->width, a->ldx, size);
    const Span v = many(a->values, a->count, a->v_stride, a->rows, a->width, a->ldv, 1);
    const Span s = many(a->scales, a->count, a->s_stride, down, across, a->lds, 4);
    if (overlap(x, v) || overlap(x, s) || overlap(v, s))
        return fail(MLP_ERR_INVALID_ARGUMENT, "values or scales overlaps another buffer");
    QuantizeArgs q{};
    q.x = a->x;
    q.ldx = a->ldx;
    q.values = a->values;
    q.ldv = a->ldv;
    q.scales = a->scales;
    q.lds = a->lds;
    if (a->count > 1) {
        q.x_stride = a->x_stride;
        q.v_stride = a->v_stride;
        q.s_stride = a->s_stride;
    }
    q.rows = a->rows;
    q.count = a->count;
    q.width = a->width;
    const hipError_t err = launch_quantize(q, a->dtype, a->block_rows, (hipStream_t)stream);
    return err == hipSuccess ? ok() : hip_fail(err, "launching the rounding to 8 bits");
}

int mlp_fp8_linear_workspace(const mlp_fp8_linear_args *a, uint64_t *bytes)
{
    if (!bytes)
        return fail(MLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
    MLP_TRY(check_linear(a));
    *bytes = linear_need(a);
    return ok();
}

int mlp_fp8_linear(const mlp_fp8_linear_args *a, void *stream)
{
    Fp8ProductArgs p{};
    MLP_TRY(prepare_linear(a, p));
    if (p.rows == 0)
        return ok();
    hipError_t err = launch_fp8_product(p, result_type(a->out_dtype), a->gated, false, (hipStream_t)stream);
    if (err != hipSuccess)
        return hip_fail(err, "launching the layer");
    if (a->out_dtype == MLP_DTYPE_FP8 && !p.values) {
        err = launch_quantize(rounding(a, a->rows, nullptr), kFp32, 1, (hipStream_t)stream);
        if (err != hipSuccess)
            return hip_fail(err, "launching the rounding to 8 bits");
    }
    return ok();
}

int mlp_fp8_expert_linear_workspace(const mlp_fp8_expert_linear_args *a, uint64_t *bytes)
{
    if (!bytes)
        return fail(MLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
    MLP_TRY(check_expert_linear(a));
    *bytes = expert_linear_need(a);
    return ok();
}

int mlp_fp8_expert_linear(const mlp_fp8_expert_linear_args *a, void *stream)
{
    Fp8ProductArgs p{};
    MLP_TRY(prepare_expert_linear(a, p));
    if (p.rows == 0)
        return ok();
    hipError_t err = launch_fp8_product(p, result_type(a->out_dtype), a->gated, true, (hipStream_t)stream);
    if (err != hipSuccess)
        return hip_fail(err, "launching the experts' layer");
    if (a->combine) {
        CombineArgs c{};
        c.part = (const float *)a->workspace;
        c.ldp = part_stride(a->out_width);
        c.places = a->places;
        c.weight = a->weight;
        c.residual = a->residual;
        c.ldr = a->ldr;
        c.y = a->y;
        c.ldy = a->ldy;
        c.tokens = a->tokens;
        c.k = a->k;
        c.out = a->out_width;
        err = launch_combine(c, a->out_dtype, (hipStream_t)stream);
        if (err != hipSuccess)
            return hip_fail(err, "launching the combination");
    } else if (a->out_dtype == MLP_DTYPE_FP8 && !p.values) {
        err = launch_quantize(rounding(a, p.rows, a->offsets + a->experts), kFp32, 1, (hipStream_t)stream);
        if (err != hipSuccess)
            return hip_fail(err, "launching the rounding to 8 bits");
    }
    return ok();
}

int mlp_testing_norm_kernel(const mlp_rms_norm_args *a, char *name, size_t cap)
{
    NormArgs n{};
    MLP_TRY(prepare_norm(a, n));
    return put_name(n.rows ? norm_kernel(n, a->dtype) : "none", name, cap);
}

int mlp_testing_fp8_linear_kernel(const mlp_fp8_linear_args *a, char *name, size_t cap)
{
    Fp8ProductArgs p{};
    MLP_TRY(prepare_linear(a, p));
    return put_name(p.rows ? fp8_product_kernel(p, result_type(a->out_dtype), a->gated, false) : "none", name, cap);
}

int mlp_testing_fp8_expert_linear_kernel(const mlp_fp8_expert_linear_args *a, char *name, size_t cap)
{
    Fp8ProductArgs p{};
    MLP_TRY(prepare_expert_linear(a, p));
    return put_name(p.rows ? fp8_product_kernel(p, result_type(a->out_dtype), a->gated, true) : "none", name, cap);
}

}  // extern "C"
