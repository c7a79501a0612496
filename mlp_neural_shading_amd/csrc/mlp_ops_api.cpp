// mlp_ops_api.cpp -- the entry points of include/mlp_ops.h: argument checks and launches.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mlp_error.h"
#include "mlp_ops.h"
#include "mlp_ops_check.h"
#include "mlp_ops_kernels.h"
#include "mlp_ops_tiles.h"
#include "mlp_testing.h"

using namespace mlpk;

namespace {

int elem_size(int dtype) { return dtype == MLP_DTYPE_FP32 ? 4 : 2; }

// The sizes and types that mlp_linear and mlp_expert_linear share.
int check_layer(int in_width, int out_width, int dtype, int out_dtype, int act, int gated)
{
    MLP_TRY(check_range("in_width", in_width, 1, MLP_OPS_MAX_WIDTH));
    MLP_TRY(check_range("out_width", out_width, 1, MLP_OPS_MAX_WIDTH));
    if (dtype != MLP_DTYPE_FP16 && dtype != MLP_DTYPE_BF16)
        return fail(MLP_ERR_INVALID_ARGUMENT, "dtype must be MLP_DTYPE_FP16 or MLP_DTYPE_BF16, got %d", dtype);
    if (out_dtype != dtype && out_dtype != MLP_DTYPE_FP32)
        return fail(MLP_ERR_INVALID_ARGUMENT, "out_dtype must be dtype or MLP_DTYPE_FP32, got %d", out_dtype);
    MLP_TRY(check_range("act", act, MLP_EPI_NONE, MLP_EPI_SILU));
    MLP_TRY(check_range("gated", gated, 0, 1));
    return MLP_OK;
}

int check_experts(int64_t tokens, int k, int experts)
{
    MLP_TRY(check_range("experts", experts, 1, MLP_OPS_MAX_EXPERTS));
    MLP_TRY(check_range("k", k, 1, MLP_OPS_MAX_TOPK));
    MLP_TRY(check_range("tokens", tokens, 0, INT32_MAX));
    MLP_TRY(check_range("tokens * k", tokens * k, 0, INT32_MAX));
    return MLP_OK;
}

int check_linear(const mlp_linear_args *a)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    MLP_TRY(check_range("rows", a->rows, 0, INT32_MAX));
    return check_layer(a->in_width, a->out_width, a->dtype, a->out_dtype, a->act, a->gated);
}

int check_expert_linear(const mlp_expert_linear_args *a)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    MLP_TRY(check_experts(a->tokens, a->k, a->experts));
    MLP_TRY(check_layer(a->in_width, a->out_width, a->dtype, a->out_dtype, a->act, a->gated));
    MLP_TRY(check_range("x_slots", a->x_slots, 0, 1));
    MLP_TRY(check_range("combine", a->combine, 0, 1));
    return MLP_OK;
}

// Row stride (floats) of the FP32 rows that a combined product leaves in its workspace.
int64_t part_stride(int out_width) { return ((int64_t)out_width + 3) / 4 * 4; }

uint64_t expert_linear_need(const mlp_expert_linear_args *a)
{
    return a->combine ? (uint64_t)a->tokens * a->k * part_stride(a->out_width) * 4 : 0;
}

int check_dispatch(const mlp_dispatch_args *a)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    return check_experts(a->tokens, a->k, a->experts);
}

uint64_t dispatch_need(const mlp_dispatch_args *a)
{
    return 4 * (uint64_t)mlpk::dispatch_workspace_entries(a->tokens * a->k, a->experts);
}

// The kernels' activation.
int activation(int act, int out_dtype)
{
    return act == MLP_EPI_SILU && out_dtype == MLP_DTYPE_FP32 ? mlpk::kSiluFull : act;
}

// The checked call as its product; rows are left 0 where there is nothing to do.
int prepare_linear(const mlp_linear_args *a, mlpk::ProductArgs &p)
{
    MLP_TRY(check_linear(a));
    if (a->rows == 0)
        return MLP_OK;
    const int64_t wide = (int64_t)a->out_width * (a->gated ? 2 : 1);
    const int out_size = elem_size(a->out_dtype);
    MLP_TRY(check_matrix("x", a->x, a->rows, a->in_width, a->ldx, 2));
    MLP_TRY(check_matrix("w", a->w, wide, a->in_width, a->ldw, 2));
    MLP_TRY(check_matrix("y", a->y, a->rows, a->out_width, a->ldy, out_size));
    MLP_TRY(check_stride("y", a->ldy));
    if (a->bias)
        MLP_TRY(check_vector("bias", a->bias, 2));
    const Span y = span(a->y, a->rows, a->out_width, a->ldy, out_size);
    if (overlap(y, span(a->x, a->rows, a->in_width, a->ldx, 2)) || overlap(y, span(a->w, wide, a->in_width, a->ldw, 2)) ||
        overlap(y, span(a->bias, 1, wide, wide, 2)))
        return fail(MLP_ERR_INVALID_ARGUMENT, "y overlaps x, w or bias");
    if (a->residual) {
        MLP_TRY(check_matrix("residual", a->residual, a->rows, a->out_width, a->ldr, out_size));
        MLP_TRY(check_stride("residual", a->ldr));
        if (!(a->residual == a->y && (a->ldr == a->ldy || a->rows == 1)) &&
            overlap(y, span(a->residual, a->rows, a->out_width, a->ldr, out_size)))
            return fail(MLP_ERR_INVALID_ARGUMENT, "y overlaps residual without being it");
    }
    p.x = a->x;
    p.ldx = a->ldx;
    p.w = a->w;
    p.ldw = a->ldw;
    p.bias = a->bias;
    p.residual = a->residual;
    p.ldr = a->ldr;
    p.y = a->y;
    p.ldy = a->ldy;
    p.rows = a->rows;
    p.in = a->in_width;
    p.out = a->out_width;
    p.act = activation(a->act, a->out_dtype);
    p.y_fp32 = a->out_dtype == MLP_DTYPE_FP32;
    if (!mlpk::product_fits(p, a->gated, false))
        return fail(MLP_ERR_UNSUPPORTED, "%lld rows of %d outputs are more tiles than one launch holds", (long long)a->rows,
                    a->out_width);
    return MLP_OK;
}

// The checked call as its product; rows are left 0 where there is nothing to do.
int prepare_expert_linear(const mlp_expert_linear_args *a, mlpk::ProductArgs &p)
{
    MLP_TRY(check_expert_linear(a));
    if (!a->combine && (a->weight || a->residual))
        return fail(MLP_ERR_INVALID_ARGUMENT, "weight and residual go with combine");
    const int64_t n = a->tokens * a->k;
    if (n == 0)
        return MLP_OK;
    const int64_t wide = (int64_t)a->out_width * (a->gated ? 2 : 1), x_rows = a->x_slots ? n : a->tokens;
    const int64_t y_rows = a->combine ? a->tokens : n;
    const int out_size = elem_size(a->out_dtype);
    MLP_TRY(check_matrix("x", a->x, x_rows, a->in_width, a->ldx, 2));
    MLP_TRY(check_matrix("w", a->w, wide, a->in_width, a->ldw, 2));
    if (a->experts > 1 && (a->w_stride < wide * a->ldw - (a->ldw - a->in_width) ||
                           a->w_stride > (INT64_MAX >> 3) / a->experts))
        return fail(MLP_ERR_INVALID_ARGUMENT, "w_stride %lld does not hold an expert's %lld rows", (long long)a->w_stride,
                    (long long)wide);
    MLP_TRY(check_matrix("y", a->y, y_rows, a->out_width, a->ldy, out_size));
    MLP_TRY(check_stride("y", a->ldy));
    if (a->bias)
        MLP_TRY(check_vector("bias", a->bias, 2));
    MLP_TRY(check_vector("offsets", a->offsets, 4));
    if (!a->x_slots)
        MLP_TRY(check_vector("slots", a->slots, 4));
    if (a->combine)
        MLP_TRY(check_vector("places", a->places, 4));
    if (a->weight)
        MLP_TRY(check_vector("weight", a->weight, 4));
    const Span y = span(a->y, y_rows, a->out_width, a->ldy, out_size);
    const int64_t w_cols = (a->experts - 1) * (a->experts > 1 ? a->w_stride : 0) + (wide - 1) * a->ldw + a->in_width;
    if (overlap(y, span(a->x, x_rows, a->in_width, a->ldx, 2)) || overlap(y, span(a->w, 1, w_cols, w_cols, 2)) ||
        overlap(y, span(a->bias, 1, wide * a->experts, wide * a->experts, 2)) ||
        overlap(y, span(a->offsets, 1, a->experts + 1, a->experts + 1, 4)) || overlap(y, span(a->slots, 1, n, n, 4)) ||
        overlap(y, span(a->places, 1, n, n, 4)) || overlap(y, span(a->weight, 1, n, n, 4)))
        return fail(MLP_ERR_INVALID_ARGUMENT, "y overlaps an input");
    if (a->residual) {
        MLP_TRY(check_matrix("residual", a->residual, y_rows, a->out_width, a->ldr, out_size));
        MLP_TRY(check_stride("residual", a->ldr));
        if (!(a->residual == a->y && (a->ldr == a->ldy || y_rows == 1)) &&
            overlap(y, span(a->residual, y_rows, a->out_width, a->ldr, out_size)))
            return fail(MLP_ERR_INVALID_ARGUMENT, "y overlaps residual without being it");
    }
    const uint64_t need = expert_linear_need(a);
    MLP_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    const Span ws = span(need ? a->workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1);
    if (overlap(ws, y) || overlap(ws, span(a->x, x_rows, a->in_width, a->ldx, 2)) || overlap(ws, span(a->w, 1, w_cols, w_cols, 2)) ||
        overlap(ws, span(a->bias, 1, wide * a->experts, wide * a->experts, 2)) || overlap(ws, span(a->slots, 1, n, n, 4)) ||
        overlap(ws, span(a->offsets, 1, a->experts + 1, a->experts + 1, 4)) || overlap(ws, span(a->places, 1, n, n, 4)) ||
        overlap(ws, span(a->weight, 1, n, n, 4)) ||
        (a->residual && overlap(ws, span(a->residual, y_rows, a->out_width, a->ldr, out_size))))
        return fail(MLP_ERR_INVALID_ARGUMENT, "workspace overlaps another buffer");
    p.x = a->x;
    p.ldx = a->ldx;
    p.w = a->w;
    p.ldw = a->ldw;
    p.w_stride = a->experts > 1 ? a->w_stride : 0;  // of one expert it may be anything
    p.bias = a->bias;
    p.y = a->combine ? a->workspace : a->y;
    p.ldy = a->combine ? part_stride(a->out_width) : a->ldy;
    p.rows = n;
    p.in = a->in_width;
    p.out = a->out_width;
    p.act = activation(a->act, a->out_dtype);
    p.y_fp32 = a->combine || a->out_dtype == MLP_DTYPE_FP32;
    p.offsets = a->offsets;
    p.slots = a->x_slots ? nullptr : a->slots;
    p.experts = a->experts;
    p.k = a->k;
    if (!mlpk::product_fits(p, a->gated, true))
        return fail(MLP_ERR_UNSUPPORTED, "%lld slots of %d outputs are more tiles than one launch holds", (long long)n,
                    a->out_width);
    return MLP_OK;
}

// The route call's sizes, without its buffers.
int check_route(const mlp_route_args *a)
{
    if (!a)
        return fail(MLP_ERR_INVALID_ARGUMENT, "args is NULL");
    MLP_TRY(check_range("tokens", a->tokens, 0, INT32_MAX));
    MLP_TRY(check_range("experts", a->experts, 1, MLP_OPS_MAX_EXPERTS));
    MLP_TRY(check_range("k", a->k, 1, a->experts < MLP_OPS_MAX_TOPK ? a->experts : MLP_OPS_MAX_TOPK));
    MLP_TRY(check_range("dtype", a->dtype, MLP_DTYPE_FP16, MLP_DTYPE_FP32));
    MLP_TRY(check_range("score", a->score, MLP_SCORE_SOFTMAX, MLP_SCORE_SIGMOID));
    MLP_TRY(check_range("groups", a->groups, 1, a->experts));
    if (a->experts % a->groups)
        return fail(MLP_ERR_INVALID_ARGUMENT, "%d experts do not divide into %d groups", a->experts, a->groups);
    MLP_TRY(check_range("topk_groups", a->topk_groups, 1, a->groups));
    MLP_TRY(check_range("group_top", a->group_top, 1, 2));
    MLP_TRY(check_range("renormalise", a->renormalise, 0, 1));
    if (!isfinite(a->scale))
        return fail(MLP_ERR_INVALID_ARGUMENT, "scale is not finite");
    return MLP_OK;
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

int mlp_linear(const mlp_linear_args *a, void *stream)
{
    mlpk::ProductArgs p{};
    MLP_TRY(prepare_linear(a, p));
    if (p.rows == 0)
        return ok();
    const hipError_t err = mlpk::launch_product(p, a->dtype, a->gated, false, (hipStream_t)stream);
    return err == hipSuccess ? ok() : hip_fail(err, "launching the layer");
}

int mlp_route(const mlp_route_args *a, void *stream)
{
    MLP_TRY(check_route(a));
    if (a->tokens == 0)
        return ok();
    MLP_TRY(check_matrix("logits", a->logits, a->tokens, a->experts, a->ld, elem_size(a->dtype)));
    if (a->bias)
        MLP_TRY(check_vector("bias", a->bias, 4));
    MLP_TRY(check_vector("index", a->index, 4));
    MLP_TRY(check_vector("weight", a->weight, 4));
    const Span in[2] = {span(a->logits, a->tokens, a->experts, a->ld, elem_size(a->dtype)),
                        span(a->bias, 1, a->experts, a->experts, 4)};
    const Span out[2] = {span(a->index, 1, a->tokens * a->k, a->tokens * a->k, 4),
                         span(a->weight, 1, a->tokens * a->k, a->tokens * a->k, 4)};
    if (overlap(out[0], in[0]) || overlap(out[1], in[0]) || overlap(out[0], in[1]) || overlap(out[1], in[1]) ||
        overlap(out[0], out[1]))
        return fail(MLP_ERR_INVALID_ARGUMENT, "index or weight overlaps another buffer");
    mlpk::RouteArgs r{};
    r.logits = a->logits;
    r.ld = a->ld;
    r.bias = a->bias;
    r.index = a->index;
    r.weight = a->weight;
    r.tokens = a->tokens;
    r.experts = a->experts;
    r.k = a->k;
    r.groups = a->groups;
    r.topk_groups = a->topk_groups;
    r.group_top = a->group_top;
    r.sigmoid = a->score == MLP_SCORE_SIGMOID;
    r.renormalise = a->renormalise != 0;
    r.scale = a->scale;
    const hipError_t err = mlpk::launch_route(r, a->dtype, (hipStream_t)stream);
    return err == hipSuccess ? ok() : hip_fail(err, "launching the router");
}

int mlp_dispatch_workspace(const mlp_dispatch_args *a, uint64_t *bytes)
{
    if (!bytes)
        return fail(MLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
    MLP_TRY(check_dispatch(a));
    *bytes = dispatch_need(a);
    return ok();
}

int mlp_dispatch(const mlp_dispatch_args *a, void *stream)
{
    MLP_TRY(check_dispatch(a));
    MLP_TRY(check_vector("offsets", a->offsets, 4));
    const int64_t n = a->tokens * a->k;
    if (n > 0) {
        MLP_TRY(check_vector("index", a->index, 4));
        MLP_TRY(check_vector("slots", a->slots, 4));
        MLP_TRY(check_vector("places", a->places, 4));
        const Span s[4] = {span(a->index, 1, n, n, 4), span(a->slots, 1, n, n, 4), span(a->places, 1, n, n, 4),
                           span(a->offsets, 1, a->experts + 1, a->experts + 1, 4)};
        for (int i = 0; i < 4; ++i)
            for (int j = i + 1; j < 4; ++j)
                if (overlap(s[i], s[j]))
                    return fail(MLP_ERR_INVALID_ARGUMENT, "index, slots, places and offsets overlap");
    }
    const uint64_t need = dispatch_need(a);
    MLP_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    const Span ws = span(need ? a->workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1);
    if (overlap(ws, span(a->index, 1, n, n, 4)) || overlap(ws, span(a->slots, 1, n, n, 4)) ||
        overlap(ws, span(a->places, 1, n, n, 4)) || overlap(ws, span(a->offsets, 1, a->experts + 1, a->experts + 1, 4)))
        return fail(MLP_ERR_INVALID_ARGUMENT, "workspace overlaps another buffer");
    mlpk::DispatchArgs d{};
    d.index = a->index;
    d.offsets = a->offsets;
    d.slots = a->slots;
    d.places = a->places;
    d.workspace = (int32_t *)a->workspace;
    d.n = n;
    d.experts = a->experts;
    const hipError_t err = mlpk::launch_dispatch(d, (hipStream_t)stream);
    return err == hipSuccess ? ok() : hip_fail(err, "launching the dispatch");
}

int mlp_expert_linear_workspace(const mlp_expert_linear_args *a, uint64_t *bytes)
{
    if (!bytes)
        return fail(MLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
    MLP_TRY(check_expert_linear(a));
    *bytes = expert_linear_need(a);
    return ok();
}

int mlp_expert_linear(const mlp_expert_linear_args *a, void *stream)
{
    mlpk::ProductArgs p{};
    MLP_TRY(prepare_expert_linear(a, p));
    if (p.rows == 0)
        return ok();
    hipError_t err = mlpk::launch_product(p, a->dtype, a->gated, true, (hipStream_t)stream);
    if (err != hipSuccess)
        return hip_fail(err, "launching the experts' layer");
    if (a->combine) {
        mlpk::CombineArgs c{};
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
        err = mlpk::launch_combine(c, a->out_dtype, (hipStream_t)stream);
        if (err != hipSuccess)
            return hip_fail(err, "launching the combination");
    }
    return ok();
}

int mlp_testing_expert_tile(int32_t begin, int32_t end, int32_t rows_per_tile, int32_t tile, int32_t *row0, int32_t *row1)
{
    if (!row0 || !row1)
        return fail(MLP_ERR_INVALID_ARGUMENT, "row0 or row1 is NULL");
    MLP_TRY(check_range("begin", begin, 0, INT32_MAX));
    MLP_TRY(check_range("rows_per_tile", rows_per_tile, 1, INT32_MAX));
    MLP_TRY(check_range("tile", tile, 0, (int64_t)mlpk::tiles_in(begin, end, rows_per_tile) - 1));
    *row0 = mlpk::tile_begin(begin, rows_per_tile, tile);
    *row1 = mlpk::tile_end(*row0, end, rows_per_tile);
    return ok();
}

int mlp_testing_linear_kernel(const mlp_linear_args *a, char *name, size_t cap)
{
    mlpk::ProductArgs p{};
    MLP_TRY(prepare_linear(a, p));
    return put_name(p.rows ? mlpk::product_kernel(p, a->gated, false) : "none", name, cap);
}

int mlp_testing_expert_linear_kernel(const mlp_expert_linear_args *a, char *name, size_t cap)
{
    mlpk::ProductArgs p{};
    MLP_TRY(prepare_expert_linear(a, p));
    return put_name(p.rows ? mlpk::product_kernel(p, a->gated, true) : "none", name, cap);
}

int mlp_testing_route_kernel(const mlp_route_args *a, char *name, size_t cap)
{
    MLP_TRY(check_route(a));
    mlpk::RouteArgs r{};
    r.experts = a->experts;
    r.k = a->k;
    r.groups = a->groups;
    r.topk_groups = a->topk_groups;
    return put_name(mlpk::route_kernel(r), name, cap);
}

}  // extern "C"
