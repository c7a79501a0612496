// mlp_torch_fp8.cpp -- the usual call of ops_fp8's operators, from torch's tensors to the C entry points of
// include/mlp_ops_fp8.h, as a Python extension: a small layer's kernel takes 3 to 6 us, its checks, allocations and
// arguments in Python 5 to 6 more, here about 2.  Each function takes its operator's arguments in order and answers None
// for anything out of the ordinary (other tensors, devices, types, shapes, modes; an error), which ops_fp8.py then takes
// through all of its checks, with its own messages.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mlp_ops_fp8.h"

namespace {

typedef at::ScalarType Type;

int64_t blocks(int64_t n) { return (n + MLP_FP8_BLOCK - 1) / MLP_FP8_BLOCK; }

// Something the call does not take: the answer is None.
struct Unusual {};

void need(bool ok)
{
    if (!ok)
        throw Unusual();
}

bool is_none(PyObject *o) { return o == Py_None; }

const at::Tensor &tensor(PyObject *o)
{
    need(THPVariable_CheckExact(o));
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.is_cuda() && t.layout() == at::kStrided && !(t.requires_grad() && c10::GradMode::is_enabled()));
    return t;
}

// What a call's tensors share.
struct Call {
    c10::Device device;

    explicit Call(const at::Tensor &t) : device(t.device())
    {
        need(device.index() == c10::hip::current_device() && !c10::impl::TorchDispatchModeTLS::any_modes_set());
    }
    const at::Tensor &take(PyObject *o, Type type) const
    {
        const at::Tensor &t = tensor(o);
        need(t.scalar_type() == type && t.device() == device);
        return t;
    }
    // The row stride of a matrix with contiguous rows.
    int64_t matrix(const at::Tensor &t, int64_t rows, int64_t cols) const
    {
        need(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && (t.stride(1) == 1 || cols <= 1));
        return rows > 1 ? t.stride(0) : cols;
    }
    const void *vector(PyObject *o, Type type, int64_t numel) const
    {
        if (is_none(o))
            return nullptr;
        const at::Tensor &t = take(o, type);
        need(t.numel() == numel && t.is_contiguous());
        return t.data_ptr();
    }
    at::Tensor empty(int64_t rows, int64_t cols, Type type) const
    {
        return at::detail::empty_cuda({rows, cols}, type, device, std::nullopt);
    }
    // 8-bit values in rows of whole 16 bytes.
    at::Tensor values(int64_t rows, int64_t width) const
    {
        const int64_t pad = (width + 15) / 16 * 16;
        at::Tensor t = empty(rows, pad, Type::Float8_e4m3fn);
        return pad == width ? t : t.narrow(1, 0, width);
    }
    at::Tensor workspace(uint64_t bytes) const
    {
        return bytes ? at::detail::empty_cuda({(int64_t)bytes}, Type::Byte, device, std::nullopt) : at::Tensor();
    }
    void *stream() const { return (void *)c10::hip::getCurrentHIPStream(device.index()).stream(); }
};

int64_t number(PyObject *o)
{
    need(PyLong_CheckExact(o));
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unusual();
    }
    return v;
}

bool truth(PyObject *o)
{
    need(PyBool_Check(o));
    return o == Py_True;
}

// MLP_DTYPE_* of a float type and back.
int code(Type t)
{
    need(t == Type::Half || t == Type::BFloat16 || t == Type::Float);
    return t == Type::Half ? MLP_DTYPE_FP16 : t == Type::BFloat16 ? MLP_DTYPE_BF16 : MLP_DTYPE_FP32;
}

Type type_of(int64_t code)
{
    need(code >= MLP_DTYPE_FP16 && code <= MLP_DTYPE_FP8);
    return code == MLP_DTYPE_FP16 ? Type::Half : code == MLP_DTYPE_BF16 ? Type::BFloat16 : code == MLP_DTYPE_FP32 ? Type::Float : Type::Float8_e4m3fn;
}

PyObject *wrap(at::Tensor t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(t));
}

PyObject *tuple(std::initializer_list<at::Tensor> all)
{
    PyObject *r = PyTuple_New((Py_ssize_t)all.size());
    Py_ssize_t i = 0;
    for (const at::Tensor &t : all)
        PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

// Runs f; None where it throws.
template <class F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F f)
{
    try {
        need(given == wanted);
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// x, weight, residual, eps, y wanted, 8 bits wanted, y in FP32 -> (y, values, scales, total)
PyObject *rms_norm(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    return guarded(n, 7, [&]() {
        const at::Tensor &x = tensor(o[0]);
        need(x.dim() == 2);
        const Call c(x);
        const Type type = x.scalar_type();
        const int64_t rows = x.size(0), width = x.size(1);
        mlp_rms_norm_args a{};
        a.rows = rows;
        need(width <= MLP_OPS_MAX_WIDTH && PyFloat_CheckExact(o[3]));
        a.width = (int32_t)width;
        a.dtype = code(type);
        a.eps = (float)PyFloat_AS_DOUBLE(o[3]);
        a.x = x.data_ptr();
        a.ldx = c.matrix(x, rows, width);
        a.weight = c.vector(o[1], type, width);
        at::Tensor total, y, values, scales;
        if (!is_none(o[2])) {
            const at::Tensor &r = c.take(o[2], type);
            a.residual = r.data_ptr();
            a.ldr = c.matrix(r, rows, width);
            total = c.empty(rows, width, type);
            a.total = total.data_ptr();
            a.ldt = width;
        }
        a.out_dtype = truth(o[6]) ? MLP_DTYPE_FP32 : a.dtype;
        if (truth(o[4])) {
            y = c.empty(rows, width, type_of(a.out_dtype));
            a.y = y.data_ptr();
            a.ldy = width;
        }
        if (truth(o[5])) {
            values = c.values(rows, width);
            scales = c.empty(rows, blocks(width), Type::Float);
            a.values = (uint8_t *)values.data_ptr();
            a.ldv = values.stride(0);
            a.scales = (float *)scales.data_ptr();
            a.lds = blocks(width);
        }
        need(mlp_rms_norm(&a, c.stream()) == MLP_OK);
        return tuple({y, values, scales, total});
    });
}

// x, block_rows -> (values, scales); one matrix, or several
PyObject *quantize(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    return guarded(n, 2, [&]() {
        const at::Tensor &x = tensor(o[0]);
        const Call c(x);
        const bool many = x.dim() == 3;
        need(many || x.dim() == 2);
        const int64_t count = many ? x.size(0) : 1, rows = x.size(many), width = x.size(many + 1), block_rows = number(o[1]);
        need((block_rows == 1 || block_rows == MLP_FP8_BLOCK) && width <= MLP_OPS_MAX_WIDTH && count <= MLP_FP8_MAX_COUNT);
        const int64_t down = block_rows == 1 ? rows : blocks(rows);
        at::Tensor values = c.values(count * rows, width), scales = c.empty(count * down, blocks(width), Type::Float);
        mlp_quantize_args a{};
        a.rows = rows;
        a.count = (int32_t)count;
        a.width = (int32_t)width;
        a.dtype = code(x.scalar_type());
        a.block_rows = (int32_t)block_rows;
        a.x = x.data_ptr();
        if (many) {
            need(x.stride(2) == 1 || width <= 1);
            a.ldx = rows > 1 ? x.stride(1) : width;
            a.x_stride = x.stride(0);
        } else {
            a.ldx = c.matrix(x, rows, width);
        }
        a.values = (uint8_t *)values.data_ptr();
        a.ldv = values.stride(0);
        a.v_stride = rows * a.ldv;
        a.scales = (float *)scales.data_ptr();
        a.lds = blocks(width);
        a.s_stride = down * a.lds;
        need(mlp_quantize(&a, c.stream()) == MLP_OK);
        if (many) {
            values = values.unflatten(0, {count, rows});
            scales = scales.unflatten(0, {count, down});
        }
        return tuple({values, scales});
    });
}

PyObject *part(PyObject *pair, int i)
{
    need(PyTuple_Check(pair) && PyTuple_GET_SIZE(pair) == 2);
    return PyTuple_GET_ITEM(pair, i);
}

// The fields that both layers have, from x, w, bias, residual, act, gated, out_dtype; w is 3-D where experts > 0.
template <class A>
void layer(A &a, const Call &c, const at::Tensor &x, PyObject *xs_, const at::Tensor &w, PyObject *ws_, int64_t experts, PyObject *bias, PyObject *act,
           PyObject *gated, PyObject *dtype)
{
    const int64_t rows = x.size(0), k = x.size(1), nb = blocks(k);
    const bool two = truth(gated);
    const int64_t wide = w.size(experts ? 1 : 0), out = two ? wide / 2 : wide, down = blocks(out) * (two ? 2 : 1);
    need((!two || wide % 2 == 0) && k <= MLP_OPS_MAX_WIDTH && out <= MLP_OPS_MAX_WIDTH);
    a.in_width = (int32_t)k;
    a.out_width = (int32_t)out;
    a.act = (int32_t)number(act);
    a.gated = two;
    a.out_dtype = (int32_t)number(dtype);
    const at::Tensor &xs = c.take(xs_, Type::Float), &ws = c.take(ws_, Type::Float);
    a.x = (const uint8_t *)x.data_ptr();
    a.ldx = c.matrix(x, rows, k);
    a.x_scale = (const float *)xs.data_ptr();
    a.ldxs = c.matrix(xs, rows, nb);
    a.w = (const uint8_t *)w.data_ptr();
    a.w_scale = (const float *)ws.data_ptr();
    if (experts) {
        need(w.dim() == 3 && w.size(2) == k && (w.stride(2) == 1 || k <= 1));
        need(ws.dim() == 3 && ws.size(0) == experts && ws.size(1) == down && ws.size(2) == nb && (ws.stride(2) == 1 || nb <= 1));
        a.ldw = wide > 1 ? w.stride(1) : k;
        a.ldws = down > 1 ? ws.stride(1) : nb;
    } else {
        a.ldw = c.matrix(w, wide, k);
        a.ldws = c.matrix(ws, down, nb);
    }
    a.bias = (const float *)c.vector(bias, Type::Float, wide * (experts ? experts : 1));
}

// New outputs of the layers, and the residual.
template <class A>
PyObject *outputs(A &a, const Call &c, int64_t rows, PyObject *residual, bool scratch, int (*query)(const A *, uint64_t *), int (*run)(const A *, void *))
{
    const Type type = type_of(a.out_dtype);
    const bool eight = a.out_dtype == MLP_DTYPE_FP8;
    const at::Tensor y = eight ? c.values(rows, a.out_width) : c.empty(rows, a.out_width, type);
    at::Tensor ys;
    a.y = y.data_ptr();
    a.ldy = rows > 1 ? y.stride(0) : a.out_width;
    if (eight) {
        ys = c.empty(rows, blocks(a.out_width), Type::Float);
        a.y_scale = (float *)ys.data_ptr();
        a.ldys = blocks(a.out_width);
    }
    if (!is_none(residual)) {
        const at::Tensor &r = c.take(residual, type);
        a.residual = r.data_ptr();
        a.ldr = c.matrix(r, rows, a.out_width);
    }
    at::Tensor ws;
    if (eight || scratch) {
        uint64_t bytes = 0;
        need(query(&a, &bytes) == MLP_OK);
        ws = c.workspace(bytes);
        a.workspace = bytes ? ws.data_ptr() : nullptr;
        a.workspace_bytes = bytes;
    }
    need(run(&a, c.stream()) == MLP_OK);
    return eight ? tuple({y, ys}) : wrap(y);
}

// x, w, bias, residual, act, gated, out_dtype -> y, or (values, scales)
PyObject *linear(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    return guarded(n, 7, [&]() {
        const at::Tensor &x = tensor(part(o[0], 0));
        const Call c(x);
        need(x.dim() == 2 && x.scalar_type() == Type::Float8_e4m3fn);
        const at::Tensor &w = c.take(part(o[1], 0), Type::Float8_e4m3fn);
        need(w.dim() == 2);
        mlp_fp8_linear_args a{};
        a.rows = x.size(0);
        layer(a, c, x, part(o[0], 1), w, part(o[1], 1), 0, o[2], o[4], o[5], o[6]);
        return outputs(a, c, a.rows, o[3], false, mlp_fp8_linear_workspace, mlp_fp8_linear);
    });
}

// x, w, offsets, slots, places, bias, k, act, gated, x by slots, combine, weight, residual, out_dtype -> y, or (values, scales)
PyObject *expert_linear(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    return guarded(n, 14, [&]() {
        const at::Tensor &x = tensor(part(o[0], 0));
        const Call c(x);
        need(x.dim() == 2 && x.scalar_type() == Type::Float8_e4m3fn);
        const at::Tensor &w = c.take(part(o[1], 0), Type::Float8_e4m3fn);
        need(w.dim() == 3 && w.size(0) >= 1 && w.size(0) <= MLP_OPS_MAX_EXPERTS);
        const int64_t experts = w.size(0), k = number(o[6]), total = c.take(o[4], Type::Int).numel();
        need(k >= 1 && k <= MLP_OPS_MAX_TOPK && total % k == 0);
        mlp_fp8_expert_linear_args a{};
        a.tokens = total / k;
        a.k = (int32_t)k;
        a.experts = (int32_t)experts;
        a.x_slots = truth(o[9]);
        a.combine = truth(o[10]);
        need(x.size(0) == (a.x_slots ? total : a.tokens));
        layer(a, c, x, part(o[0], 1), w, part(o[1], 1), experts, o[5], o[7], o[8], o[13]);
        a.w_stride = experts > 1 ? w.stride(0) : 0;
        a.ws_stride = experts > 1 ? THPVariable_Unpack(part(o[1], 1)).stride(0) : 0;
        need(!is_none(o[2]) && !is_none(o[3]));
        a.offsets = (const int32_t *)c.vector(o[2], Type::Int, experts + 1);
        a.slots = (const int32_t *)c.vector(o[3], Type::Int, total);
        a.places = (const int32_t *)c.vector(o[4], Type::Int, total);
        a.weight = (const float *)c.vector(o[11], Type::Float, total);
        return outputs(a, c, a.combine ? a.tokens : total, o[12], a.combine, mlp_fp8_expert_linear_workspace, mlp_fp8_expert_linear);
    });
}

PyMethodDef methods[] = {{"rms_norm", (PyCFunction)(void *)rms_norm, METH_FASTCALL, nullptr},
                         {"quantize", (PyCFunction)(void *)quantize, METH_FASTCALL, nullptr},
                         {"linear", (PyCFunction)(void *)linear, METH_FASTCALL, nullptr},
                         {"expert_linear", (PyCFunction)(void *)expert_linear, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_fp8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_fp8() { return PyModule_Create(&module); }
