/*
 * mlp_ops.h -- single operators beside the whole-network inference of mlp.h, same library: one affine
 * layer with its epilogue, and the parts of a layer of experts (several networks' layers, each row
 * routed to its own): the router's choice, the order of the rows by expert, the experts' products.
 *
 * Conventions, for every function (as in mlp.h):
 *   - returns MLP_OK (0) or a negative mlp_status; never aborts, throws or exits; after an error,
 *     mlp_last_error() returns a message for the calling thread;
 *   - arguments are validated on the host before any HIP call;
 *   - work is enqueued on `stream` (hipStream_t, NULL = the default stream) and the call returns; it
 *     allocates, frees and waits for nothing, so it can be recorded into a HIP graph.  Stream and
 *     pointers belong to the current device, and the buffers stay valid until the stream's work is done;
 *   - no state is kept between calls: weights are read row-major as they are, scratch memory is the
 *     caller's `workspace` (its size from the *_workspace function, which makes no HIP call).  Two calls
 *     whose work may overlap on the GPU (other streams, or graphs replayed side by side) need workspaces
 *     of their own; its contents need no clearing and mean nothing afterwards;
 *   - results do not depend on timing: the same call gives the same bits;
 *   - matrices are row-major with a row stride in elements (ld*), at least the row's length; pointers
 *     are aligned to their element, and 16-byte aligned rows are faster;
 *   - the struct is read before the call returns and can be reused.
 */
#ifndef MLP_OPS_H
#define MLP_OPS_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum {
    MLP_DTYPE_FP16 = 0,
    MLP_DTYPE_BF16 = 1,
    MLP_DTYPE_FP32 = 2
};

/* Activations of the epilogue, computed in FP32 on the FP32 sum v: GELU is off by at most 3 * 2^-24 of |v|, SiLU by
 * 10 * 2^-24 of its value, but by (2 |v| + 40) * 2^-24 of it before the rounding to a 16-bit output. */
enum {
    MLP_EPI_NONE = 0,
    MLP_EPI_LEAKY_RELU = 1, /* v < 0 ? v * half(0.01) : v, the slope of mlp.h's networks */
    MLP_EPI_RELU = 2,
    MLP_EPI_GELU = 3, /* v * (1 + erf(v / sqrt 2)) / 2 */
    MLP_EPI_SILU = 4  /* v / (1 + exp(-v)) */
};

#define MLP_OPS_MAX_WIDTH (1 << 20) /* widths of mlp_linear and mlp_expert_linear */
#define MLP_OPS_MAX_STRIDE (1 << 24) /* row strides of y and residual there, in elements */
#define MLP_OPS_MAX_EXPERTS 1024
#define MLP_OPS_MAX_TOPK 32 /* experts per token */

/* One affine layer:  y[r][o] = round(act(sum_i x[r][i] w[o][i] + bias[o]) + residual[r][o]),
 * or gated, with twice the weight rows:  y[r][o] = round(act(z[r][o]) * z[r][out_width + o] +
 * residual[r][o]),  z = x w^T + bias.  Sums, activation, gate and residual in FP32, rounded once. */
typedef struct mlp_linear_args {
    int64_t rows;      /* 0 .. INT32_MAX; 0: nothing is launched                                     */
    int32_t in_width;  /* 1 .. MLP_OPS_MAX_WIDTH                                                      */
    int32_t out_width; /* 1 .. MLP_OPS_MAX_WIDTH, columns of y                                        */
    int32_t dtype;     /* of x, w and bias: MLP_DTYPE_FP16 or MLP_DTYPE_BF16                          */
    int32_t out_dtype; /* of y and residual: dtype, or MLP_DTYPE_FP32                                 */
    int32_t act;       /* MLP_EPI_*                                                                   */
    int32_t gated;     /* 0, or 1: w and bias have 2 * out_width rows, the gates first                */
    const void *x;     /* [rows][in_width]                                                            */
    int64_t ldx;
    const void *w; /* [out_width or 2 * out_width][in_width]                                      */
    int64_t ldw;
    const void *bias;     /* [out_width or 2 * out_width], or NULL                                   */
    const void *residual; /* [rows][out_width], or NULL; may be y itself (same pointer and stride)   */
    int64_t ldr;
    void *y; /* [rows][out_width]; overlaps no input but such a residual                        */
    int64_t ldy;
} mlp_linear_args;

/* Errors: INVALID_ARGUMENT, UNSUPPORTED (more tiles than one launch holds), HIP. */
int mlp_linear(const mlp_linear_args *args, void *stream);

/* Scores of the router. */
enum {
    MLP_SCORE_SOFTMAX = 0, /* over all experts of the token */
    MLP_SCORE_SIGMOID = 1
};

/* The router: for each token the k experts of largest choice = score + bias, largest first, and their
 * weights.  With groups > 1 (consecutive experts, equally many in each) only the topk_groups groups of
 * largest value are chosen from; a group's value is the sum of its group_top largest choices (of as many
 * as it has).  Equal choices, and equal groups, go to the lower index.  Choices are compared as if computed
 * exactly: without a bias and without group_top 2 by the logits themselves, whose order is the scores' (with a
 * +infinite logit the softmax's other scores are 0, and equal), else to about 50 bits.  A token's choice and
 * weights do not depend on the other tokens of the call.  The weight is the score (not the choice), divided by the sum of the token's
 * chosen scores if `renormalise` (0 where that sum is 0), times `scale`.
 * An expert whose logit is NaN or -infinity (a masked expert) or whose bias is NaN or -infinity is never
 * chosen, and a group without other experts neither; the softmax leaves NaN and -infinity out, and logits of
 * +infinity share all of it.  Where fewer than k experts are left, the rest of the row is index -1, weight 0. */
typedef struct mlp_route_args {
    int64_t tokens;      /* 0 .. INT32_MAX                                                           */
    int32_t experts;     /* 1 .. MLP_OPS_MAX_EXPERTS                                                  */
    int32_t k;           /* 1 .. min(MLP_OPS_MAX_TOPK, experts)                                       */
    int32_t dtype;       /* of the logits: MLP_DTYPE_FP32, _FP16 or _BF16                             */
    int32_t score;       /* MLP_SCORE_*                                                               */
    int32_t groups;      /* 1 .. experts, a divisor of experts                                        */
    int32_t topk_groups; /* 1 .. groups                                                               */
    int32_t group_top;   /* 1 or 2                                                                    */
    int32_t renormalise; /* 0 or 1                                                                    */
    float scale;         /* finite                                                                    */
    const void *logits;  /* [tokens][experts]                                                         */
    int64_t ld;
    const float *bias; /* [experts], or NULL                                                        */
    int32_t *index;    /* [tokens][k], contiguous                                                    */
    float *weight;     /* [tokens][k], contiguous                                                    */
} mlp_route_args;

int mlp_route(const mlp_route_args *args, void *stream);

/* The order of rows by expert.  Assignment a = token * k + j is row `token` going to expert index[a]; the
 * assignments of expert e take the slots offsets[e] .. offsets[e + 1] - 1, in rising order of a.  An index
 * outside 0 .. experts - 1 (the router's -1, a padded row) is dropped: it takes no slot.  The index may be
 * the router's, or any tag of the caller's (which of several networks evaluates a row, with k = 1); the
 * same expert may appear twice in a row. */
typedef struct mlp_dispatch_args {
    int64_t tokens;       /* tokens * k: 0 .. INT32_MAX                                              */
    int32_t k;            /* 1 .. MLP_OPS_MAX_TOPK                                                    */
    int32_t experts;      /* 1 .. MLP_OPS_MAX_EXPERTS                                                 */
    const int32_t *index; /* [tokens][k], contiguous                                                  */
    int32_t *offsets;     /* [experts + 1]                                                            */
    int32_t *slots;       /* [tokens * k]: the assignment in each slot; -1 from offsets[experts] on   */
    int32_t *places;      /* [tokens * k]: the slot of each assignment, -1 if dropped                 */
    void *workspace; /* mlp_dispatch_workspace bytes, 16-byte aligned (NULL where that is 0)         */
    uint64_t workspace_bytes;
} mlp_dispatch_args;

/* Bytes of workspace mlp_dispatch needs for these sizes (pointers are not looked at). */
int mlp_dispatch_workspace(const mlp_dispatch_args *args, uint64_t *bytes);
int mlp_dispatch(const mlp_dispatch_args *args, void *stream);

/* The experts' layer on routed rows: f_e(x) = act(x w[e]^T + bias[e]) or gated, as in mlp_linear, for the
 * rows of each expert e.
 *   x by tokens (x_slots 0): slot s reads row slots[s] / k of x;  by slots (1): row s.
 *   y by slots (combine 0):  y[s] = round(f_e(x of s)) for every slot in use; rows of y from
 *     offsets[experts] on are left as they were.
 *   combined (1):  y[t] = round(sum_j weight[t][j] f(x of the slot of (t, j)) + residual[t]), in the order of
 *     j and in FP32; a dropped assignment adds nothing, so a token without any gets its residual, or 0.
 * offsets, slots and places are mlp_dispatch's; entries outside their ranges are clamped to them (a place
 * to "dropped"), so no call reads or writes out of bounds whatever they hold. */
typedef struct mlp_expert_linear_args {
    int64_t tokens; /* tokens * k: 0 .. INT32_MAX */
    int32_t k;
    int32_t experts;
    int32_t in_width, out_width;
    int32_t dtype, out_dtype, act, gated; /* as in mlp_linear_args                                   */
    int32_t x_slots, combine;
    const void *x; /* [tokens or tokens * k][in_width]                                               */
    int64_t ldx;
    const void *w; /* [experts][out_width or 2 * out_width][in_width]                                */
    int64_t ldw;
    int64_t w_stride;       /* elements from one expert's matrix to the next                          */
    const void *bias;       /* [experts][out_width or 2 * out_width], contiguous, or NULL             */
    const int32_t *offsets; /* [experts + 1]                                                          */
    const int32_t *slots;   /* [tokens * k]; NULL allowed with x_slots                                */
    const int32_t *places;  /* [tokens * k]; NULL allowed without combine                             */
    const float *weight;    /* [tokens][k] with combine, or NULL for 1; NULL without combine          */
    const void *residual;   /* [tokens][out_width] with combine, or NULL; may be y itself             */
    int64_t ldr;
    void *y; /* [tokens * k or tokens][out_width]                                               */
    int64_t ldy;
    void *workspace; /* mlp_expert_linear_workspace bytes, 16-byte aligned (NULL where that is 0)    */
    uint64_t workspace_bytes;
} mlp_expert_linear_args;

/* Bytes of workspace mlp_expert_linear needs for these sizes: the FP32 outputs by slot where it combines. */
int mlp_expert_linear_workspace(const mlp_expert_linear_args *args, uint64_t *bytes);
int mlp_expert_linear(const mlp_expert_linear_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MLP_OPS_H */
