// binding.h -- what the compiled Python module's calls share: checks of the tensors,
// allocation of outputs and scratch, results.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace moe_py {

using at::ScalarType;
using at::Tensor;

constexpr int64_t kBlock = 128;
inline int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

inline const Tensor &tensor_of(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
inline bool given(PyObject *o) { return o != Py_None; }

inline int int_of(int64_t v, const char *name)
{
    TORCH_CHECK_VALUE(v >= 0 && v <= INT32_MAX, name, ": ", v, " is out of range");
    return (int)v;
}

// Sets of element types an operand may have.
enum Kind { CODES, REAL, FLOAT32, BFLOAT16, INT8, INT32 };
inline bool is_kind(ScalarType t, Kind k)
{
    switch (k) {
    case CODES: return t == ScalarType::Float8_e4m3fn || t == ScalarType::Byte;
    case REAL: return t == ScalarType::Float || t == ScalarType::BFloat16;
    case FLOAT32: return t == ScalarType::Float;
    case BFLOAT16: return t == ScalarType::BFloat16;
    case INT8: return t == ScalarType::Char;
    default: return t == ScalarType::Int;
    }
}
inline const char *kind_name(Kind k)
{
    static const char *const names[] = {"float8_e4m3fn or uint8", "float32 or bfloat16", "float32", "bfloat16", "int8", "int32"};
    return names[k];
}

// The operand's pointer, after checks of device, type, shape and strides
// (`strided`: its rows may be further apart than their length).
inline void *need(const Tensor &t, const char *name, at::IntArrayRef shape, Kind kind, c10::Device dev, bool strided = false)
{
    TORCH_CHECK_VALUE(t.device() == dev, name, ": on ", t.device(), ", expected ", dev);
    TORCH_CHECK_TYPE(is_kind(t.scalar_type(), kind), name, ": ", t.scalar_type(), ", expected ", kind_name(kind));
    TORCH_CHECK_VALUE(t.sizes() == shape, name, ": shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(t.is_contiguous() || (strided && t.stride(-1) == 1), name, ": strides ", t.strides(),
                      " are not supported, make it contiguous");
    return t.data_ptr();
}
inline int64_t row_stride(const Tensor &t) { return t.size(-2) > 1 ? t.stride(-2) : t.size(-1); }
inline moe_dtype real_dtype(const Tensor &t) { return t.scalar_type() == ScalarType::Float ? MOE_F32 : MOE_BF16; }

inline Tensor empty(at::IntArrayRef shape, ScalarType t, c10::Device dev)
{
    return at::detail::empty_cuda(shape, t, dev, c10::nullopt);
}
// `o` if it is a tensor, else a new one (`holder` keeps it)
inline const Tensor &given_or_empty(PyObject *o, const char *name, Tensor &holder, at::IntArrayRef shape, ScalarType t,
                             c10::Device dev)
{
    if (given(o)) return tensor_of(o, name);
    holder = empty(shape, t, dev);
    return holder;
}
inline void need_cuda(const Tensor &t, const char *name)
{
    TORCH_CHECK_VALUE(t.is_cuda(), name, ": on ", t.device(), ", expected a CUDA device");
}
inline moe_stream stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// What a call returns: its outputs, or the status it failed with as an int
// (the Python side raises MoeError).
inline PyObject *wrap(PyObject *o, const Tensor &t)
{
    if (o && given(o) && THPVariable_Check(o)) {
        Py_INCREF(o);
        return o;
    }
    return THPVariable_Wrap(t);
}
inline PyObject *failed(moe_status st) { return PyLong_FromLong(st); }

inline void need_args(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }


// What the products share: x, its groups, the scratch of gathered rows, status.
struct Rows {
    const void *x_q;
    const float *x_s;
    int x_rows, K, rows;
    int64_t ldx;
    const int32_t *offsets = nullptr, *perm_tok = nullptr;
    uint32_t *status = nullptr;
    c10::Device dev;
};
inline Rows rows_of(PyObject *x_q, PyObject *x_s, PyObject *offsets, PyObject *perm_tok, PyObject *status, int64_t E,
                    Kind codes = CODES)
{
    const Tensor &x = tensor_of(x_q, "x_q");
    TORCH_CHECK_VALUE(x.dim() == 2, "x_q: ", x.dim(), " dimensions, expected 2");
    Rows r{nullptr, nullptr, int_of(x.size(0), "x_q"), int_of(x.size(1), "x_q"), 0, row_stride(x),
           nullptr, nullptr, nullptr, x.device()};
    r.x_q = need(x, "x_q", x.sizes(), codes, r.dev, true);
    // (block-scaled fp8: a scale for each row and 128 columns; int8: one for each row)
    const int64_t s_shape[2] = {r.x_rows, blocks(r.K)};
    r.x_s = static_cast<const float *>(need(tensor_of(x_s, "x_s"), "x_s", at::IntArrayRef(s_shape, codes == CODES ? 2 : 1),
                                            FLOAT32, r.dev));
    r.rows = r.x_rows;
    if (given(perm_tok)) {
        const Tensor &p = tensor_of(perm_tok, "perm_tok");
        const int64_t shape[1] = {p.numel()};
        r.rows = int_of(p.numel(), "perm_tok");
        r.perm_tok = static_cast<const int32_t *>(need(p, "perm_tok", shape, INT32, r.dev));
    }
    if (given(offsets)) {
        const int64_t shape[1] = {E + 1};
        r.offsets = static_cast<const int32_t *>(need(tensor_of(offsets, "offsets"), "offsets", shape, INT32, r.dev));
    } else {
        TORCH_CHECK_VALUE(E == 1, "offsets are required for ", E, " experts");
    }
    if (given(status)) {
        const Tensor &t = tensor_of(status, "status");
        TORCH_CHECK_VALUE(t.numel() > 0, "status: empty");
        r.status = static_cast<uint32_t *>(need(t, "status", t.sizes(), INT32, r.dev));
    }
    return r;
}
// scratch of `need_bytes`: the caller's, or a new one (the allocator hands it on in
// stream order)
inline void *scratch_of(PyObject *o, c10::Device dev, size_t need_bytes, Tensor &holder, size_t *bytes)
{
    if (given(o)) {
        const Tensor &t = tensor_of(o, "workspace");
        TORCH_CHECK_VALUE(t.device() == dev, "workspace: on ", t.device(), ", expected ", dev);
        TORCH_CHECK_VALUE(t.is_contiguous(), "workspace: make it contiguous");
        *bytes = t.nbytes();
        return t.data_ptr();
    }
    *bytes = need_bytes;
    const int64_t shape[1] = {(int64_t)need_bytes};
    holder = empty(shape, ScalarType::Byte, dev);
    return holder.data_ptr();
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(F)), METH_FASTCALL, nullptr};
}

extern PyMethodDef i8_methods[];   // i8_binding.cpp

}  // namespace moe_py
