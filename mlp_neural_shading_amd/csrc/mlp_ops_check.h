// mlp_ops_check.h -- the checks of arguments that the entry points of mlp_ops.h and mlp_ops_fp8.h share.
#pragma once

#include <stdint.h>

#include "mlp_error.h"
#include "mlp_ops.h"

namespace mlpk {

namespace {

// A matrix as the checks see it: `rows` rows of `cols` bytes, `ld` bytes apart.
struct Span {
    uintptr_t at;
    int64_t rows, cols, ld;
};

Span span(const void *p, int64_t rows, int64_t cols, int64_t ld, int size)
{
    return Span{(uintptr_t)p, rows, cols * size, ld * size};
}

// Whether two matrices share a byte.  Column blocks of one matrix (equal strides, disjoint columns) do not;
// other strides over the same memory are taken to.
bool overlap(const Span &a, const Span &b)
{
    if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0)
        return false;
    const uintptr_t a1 = a.at + (uintptr_t)((a.rows - 1) * a.ld + a.cols), b1 = b.at + (uintptr_t)((b.rows - 1) * b.ld + b.cols);
    if (a.at >= b1 || b.at >= a1)
        return false;
    if (a.ld == b.ld && a.ld > 0) {
        const int64_t ld = a.ld, d = (int64_t)b.at - (int64_t)a.at;
        const int64_t shift = (d % ld + ld) % ld;  // the column of a at which b's rows begin
        if (shift >= a.cols && shift + b.cols <= a.ld)
            return false;
    }
    return true;
}

int check_matrix(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int size)
{
    if (!p)
        return fail(MLP_ERR_INVALID_ARGUMENT, "%s is NULL", name);
    if ((uintptr_t)p % size)
        return fail(MLP_ERR_INVALID_ARGUMENT, "%s is not %d-byte aligned", name, size);
    if (ld < cols)
        return fail(MLP_ERR_INVALID_ARGUMENT, "the row stride of %s, %lld, is less than its %lld columns", name,
                    (long long)ld, (long long)cols);
    if (ld > (INT64_MAX >> 3) / (rows > 0 ? rows : 1))
        return fail(MLP_ERR_INVALID_ARGUMENT, "the row stride of %s, %lld, is too large", name, (long long)ld);
    return MLP_OK;
}

// The kernels step through y and residual in 32 bits.
int check_stride(const char *name, int64_t ld)
{
    if (ld > MLP_OPS_MAX_STRIDE)
        return fail(MLP_ERR_INVALID_ARGUMENT, "the row stride of %s, %lld, is larger than %d", name, (long long)ld,
                    MLP_OPS_MAX_STRIDE);
    return MLP_OK;
}

int check_vector(const char *name, const void *p, int size)
{
    if (!p)
        return fail(MLP_ERR_INVALID_ARGUMENT, "%s is NULL", name);
    if ((uintptr_t)p % size)
        return fail(MLP_ERR_INVALID_ARGUMENT, "%s is not %d-byte aligned", name, size);
    return MLP_OK;
}

int check_range(const char *name, int64_t v, int64_t lo, int64_t hi)
{
    if (v < lo || v > hi)
        return fail(MLP_ERR_INVALID_ARGUMENT, "%s must be in [%lld, %lld], got %lld", name, (long long)lo, (long long)hi,
                    (long long)v);
    return MLP_OK;
}

int check_workspace(const void *p, uint64_t have, uint64_t need)
{
    if (need == 0)
        return MLP_OK;
    if (!p)
        return fail(MLP_ERR_INVALID_ARGUMENT, "workspace is NULL, %llu bytes are needed", (unsigned long long)need);
    if ((uintptr_t)p % 16)
        return fail(MLP_ERR_INVALID_ARGUMENT, "workspace is not 16-byte aligned");
    if (have < need)
        return fail(MLP_ERR_INVALID_ARGUMENT, "workspace holds %llu bytes, %llu are needed", (unsigned long long)have,
                    (unsigned long long)need);
    return MLP_OK;
}

#define MLP_TRY(call)                                                                                          \
    do {                                                                                                       \
        const int rc_ = (call);                                                                                \
        if (rc_ != MLP_OK)                                                                                     \
            return rc_;                                                                                        \
    } while (0)

}  // namespace

}  // namespace mlpk
