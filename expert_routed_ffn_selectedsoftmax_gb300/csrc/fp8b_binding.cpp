// fp8b_binding.cpp -- the Python side of the block-scaled fp8 operators: checks
// of the tensors, allocation of the outputs and the call into the C ABI.
//
// The other calls of the binding go through ctypes.  These take up to ten
// tensors that have to fit one another (a wrong pairing would read out of
// bounds), and in Python the checks, the allocations and the marshalling took
// 15-23 us a call on the host where the kernels of a decode step take 2-7 us;
// here they take 3-6 us.  Nothing of the operators is computed here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int64_t kBlock = 128;
int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

const Tensor &tensor_of(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
bool given(PyObject *o) { return o != Py_None; }

int int_of(int64_t v, const char *name)
{
    TORCH_CHECK_VALUE(v >= 0 && v <= INT32_MAX, name, ": ", v, " is out of range");
    return (int)v;
}

// Sets of element types an operand may have.
enum Kind { CODES, REAL, FLOAT32, BFLOAT16, INT32 };
bool is_kind(ScalarType t, Kind k)
{
    switch (k) {
    case CODES: return t == ScalarType::Float8_e4m3fn || t == ScalarType::Byte;
    case REAL: return t == ScalarType::Float || t == ScalarType::BFloat16;
    case FLOAT32: return t == ScalarType::Float;
    case BFLOAT16: return t == ScalarType::BFloat16;
    default: return t == ScalarType::Int;
    }
}
const char *kind_name(Kind k)
{
    static const char *const names[] = {"float8_e4m3fn or uint8", "float32 or bfloat16", "float32", "bfloat16", "int32"};
    return names[k];
}

// The operand's pointer, after checks of device, type, shape and strides
// (`strided`: its rows may be further apart than their length).
void *need(const Tensor &t, const char *name, at::IntArrayRef shape, Kind kind, c10::Device dev, bool strided = false)
{
    TORCH_CHECK_VALUE(t.device() == dev, name, ": on ", t.device(), ", expected ", dev);
    TORCH_CHECK_TYPE(is_kind(t.scalar_type(), kind), name, ": ", t.scalar_type(), ", expected ", kind_name(kind));
    TORCH_CHECK_VALUE(t.sizes() == shape, name, ": shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(t.is_contiguous() || (strided && t.stride(-1) == 1), name, ": strides ", t.strides(),
                      " are not supported, make it contiguous");
    return t.data_ptr();
}
int64_t row_stride(const Tensor &t) { return t.size(-2) > 1 ? t.stride(-2) : t.size(-1); }
moe_dtype real_dtype(const Tensor &t) { return t.scalar_type() == ScalarType::Float ? MOE_F32 : MOE_BF16; }

Tensor empty(at::IntArrayRef shape, ScalarType t, c10::Device dev)
{
    return at::detail::empty_cuda(shape, t, dev, c10::nullopt);
}
// `o` if it is a tensor, else a new one (`holder` keeps it)
const Tensor &given_or_empty(PyObject *o, const char *name, Tensor &holder, at::IntArrayRef shape, ScalarType t,
                             c10::Device dev)
{
    if (given(o)) return tensor_of(o, name);
    holder = empty(shape, t, dev);
    return holder;
}
void need_cuda(const Tensor &t, const char *name)
{
    TORCH_CHECK_VALUE(t.is_cuda(), name, ": on ", t.device(), ", expected a CUDA device");
}
moe_stream stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// What a call returns: its outputs, or the status it failed with as an int
// (the Python side raises MoeError).
PyObject *wrap(PyObject *o, const Tensor &t)
{
    if (o && given(o) && THPVariable_Check(o)) {
        Py_INCREF(o);
        return o;
    }
    return THPVariable_Wrap(t);
}
PyObject *failed(moe_status st) { return PyLong_FromLong(st); }

void need_args(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// quant(x, block_rows, codes, scales)
PyObject *quant(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 4);
    const Tensor &x = tensor_of(a[0], "x");
    const long block_rows = PyLong_AsLong(a[1]);
    if (block_rows == -1 && PyErr_Occurred()) return nullptr;
    TORCH_CHECK_VALUE(x.dim() == 2 || x.dim() == 3, "x: ", x.dim(), " dimensions, expected 2 or 3");
    TORCH_CHECK_VALUE(block_rows == 1 || block_rows == kBlock, "block_rows: ", block_rows, ", expected 1 or 128");
    const c10::Device dev = x.device();
    const int64_t rows = x.size(-2), cols = x.size(-1), batch = x.dim() == 3 ? x.size(0) : 1;
    const void *px = need(x, "x", x.sizes(), REAL, dev, true);
    const int64_t ldx = row_stride(x);
    TORCH_CHECK_VALUE(x.dim() == 2 || batch <= 1 || rows == 0 || x.stride(0) == rows * ldx, "x: strides ", x.strides(),
                      " are not supported, make it contiguous");
    const int64_t sr = (rows + block_rows - 1) / block_rows, sc = blocks(cols);
    const int64_t s2[2] = {sr, sc}, s3[3] = {batch, sr, sc};
    const at::IntArrayRef s_shape = x.dim() == 3 ? at::IntArrayRef(s3) : at::IntArrayRef(s2);
    if (given(a[2])) need(tensor_of(a[2], "codes"), "codes", x.sizes(), CODES, dev);
    if (given(a[3])) need(tensor_of(a[3], "scales"), "scales", s_shape, FLOAT32, dev);
    need_cuda(x, "x");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor h0, h1;
    const Tensor &codes = given_or_empty(a[2], "codes", h0, x.sizes(), ScalarType::Float8_e4m3fn, dev);
    const Tensor &scales = given_or_empty(a[3], "scales", h1, s_shape, ScalarType::Float, dev);
    const moe_status st = moe_quant_fp8b(px, real_dtype(x), int_of(batch, "x"), int_of(rows, "x"), int_of(cols, "x"),
                                         ldx, (int)block_rows, codes.data_ptr(), scales.data_ptr<float>(), stream_of(dev));
    if (st != MOE_OK) return failed(st);
    return Py_BuildValue("(NN)", wrap(a[2], codes), wrap(a[3], scales));
    END_HANDLE_TH_ERRORS
}

// norm(x, weight, eps, delta, topk_w, inv, want_normed, resid, normed, codes, scales)
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 11);
    const Tensor &x = tensor_of(a[0], "x"), &weight = tensor_of(a[1], "weight");
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const int wants = PyObject_IsTrue(a[6]);
    if (wants < 0) return nullptr;
    const bool adds = given(a[3]), combines = given(a[5]), want_normed = wants != 0;
    TORCH_CHECK_VALUE(x.dim() == 2, "x: ", x.dim(), " dimensions, expected 2");
    TORCH_CHECK_VALUE(given(a[4]) == combines, "topk_w and inv go together");
    TORCH_CHECK_VALUE(adds || !combines, "topk_w and inv need delta");
    TORCH_CHECK_VALUE(adds || !given(a[7]), "resid is written only with delta");
    TORCH_CHECK_VALUE(want_normed || !given(a[8]), "normed is given but not wanted");
    const c10::Device dev = x.device();
    const int64_t T = x.size(0), d = x.size(1);
    const int64_t td[2] = {T, d}, tb[2] = {T, blocks(d)};
    const void *px = need(x, "x", td, REAL, dev, true);
    const void *pg = need(weight, "weight", at::IntArrayRef(td + 1, 1), REAL, dev);
    const void *pd = nullptr;
    const float *pw = nullptr;
    const int32_t *pi = nullptr;
    moe_dtype dd = MOE_F32;
    int64_t delta_rows = 0, ldd = 0, k = 0;
    if (adds) {
        const Tensor &delta = tensor_of(a[3], "delta");
        TORCH_CHECK_VALUE(delta.dim() == 2, "delta: ", delta.dim(), " dimensions, expected 2");
        delta_rows = delta.size(0);
        if (combines) {
            const Tensor &topk_w = tensor_of(a[4], "topk_w"), &inv = tensor_of(a[5], "inv");
            TORCH_CHECK_VALUE(topk_w.dim() == 2 && topk_w.size(1) > 0, "topk_w: shape ", topk_w.sizes(), ", expected [", T, ", k]");
            k = topk_w.size(1);
            const int64_t tk[2] = {T, k};
            pw = static_cast<const float *>(need(topk_w, "topk_w", tk, FLOAT32, dev));
            pi = static_cast<const int32_t *>(need(inv, "inv", inv.sizes(), INT32, dev));
            TORCH_CHECK_VALUE(inv.numel() == T * k, "inv: ", inv.numel(), " values, expected ", T * k);
        }
        const int64_t shape[2] = {combines ? delta_rows : T, d};
        pd = need(delta, "delta", shape, REAL, dev, true);
        dd = real_dtype(delta);
        ldd = row_stride(delta);
        if (given(a[7]))
            need(tensor_of(a[7], "resid"), "resid", td, x.scalar_type() == ScalarType::Float ? FLOAT32 : BFLOAT16, dev);
    }
    if (given(a[8])) need(tensor_of(a[8], "normed"), "normed", td, BFLOAT16, dev);
    if (given(a[9])) need(tensor_of(a[9], "codes"), "codes", td, CODES, dev);
    if (given(a[10])) need(tensor_of(a[10], "scales"), "scales", tb, FLOAT32, dev);
    need_cuda(x, "x");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor h0, h1, h2, h3;
    void *pr = nullptr, *pn = nullptr;
    if (adds) pr = given_or_empty(a[7], "resid", h0, td, x.scalar_type(), dev).data_ptr();
    if (want_normed) pn = given_or_empty(a[8], "normed", h1, td, ScalarType::BFloat16, dev).data_ptr();
    const Tensor &codes = given_or_empty(a[9], "codes", h2, td, ScalarType::Float8_e4m3fn, dev);
    const Tensor &scales = given_or_empty(a[10], "scales", h3, tb, ScalarType::Float, dev);
    const moe_status st = moe_norm_fp8b(px, real_dtype(x), int_of(T, "x"), int_of(d, "x"), row_stride(x), pd, dd,
                                        int_of(delta_rows, "delta"), ldd, pw, pi, int_of(k, "topk_w"), pg,
                                        real_dtype(weight), (float)eps, pr, pn, codes.data_ptr(),
                                        scales.data_ptr<float>(), stream_of(dev));
    if (st != MOE_OK) return failed(st);
    PyObject *resid = adds ? wrap(a[7], h0) : wrap(a[0], x);
    PyObject *normed = Py_None;
    if (want_normed) normed = wrap(a[8], h1);
    else Py_INCREF(normed);
    return Py_BuildValue("(NNNN)", resid, normed, wrap(a[9], codes), wrap(a[10], scales));
    END_HANDLE_TH_ERRORS
}

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
Rows rows_of(PyObject *x_q, PyObject *x_s, PyObject *offsets, PyObject *perm_tok, PyObject *status, int64_t E)
{
    const Tensor &x = tensor_of(x_q, "x_q");
    TORCH_CHECK_VALUE(x.dim() == 2, "x_q: ", x.dim(), " dimensions, expected 2");
    Rows r{nullptr, nullptr, int_of(x.size(0), "x_q"), int_of(x.size(1), "x_q"), 0, row_stride(x),
           nullptr, nullptr, nullptr, x.device()};
    r.x_q = need(x, "x_q", x.sizes(), CODES, r.dev, true);
    const int64_t s_shape[2] = {r.x_rows, blocks(r.K)};
    r.x_s = static_cast<const float *>(need(tensor_of(x_s, "x_s"), "x_s", s_shape, FLOAT32, r.dev));
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
// scratch of gathered rows: the caller's, or a new one (the allocator hands it
// on in stream order)
void *workspace_of(PyObject *o, const Rows &r, Tensor &holder, size_t *bytes)
{
    *bytes = 0;
    if (!r.perm_tok) return nullptr;
    if (given(o)) {
        const Tensor &t = tensor_of(o, "workspace");
        TORCH_CHECK_VALUE(t.device() == r.dev, "workspace: on ", t.device(), ", expected ", r.dev);
        TORCH_CHECK_VALUE(t.is_contiguous(), "workspace: make it contiguous");
        *bytes = t.nbytes();
        return t.data_ptr();
    }
    *bytes = moe_fp8b_workspace_size(r.rows, r.K);
    const int64_t shape[1] = {(int64_t)*bytes};
    holder = empty(shape, ScalarType::Byte, r.dev);
    return holder.data_ptr();
}

// product(x_q, x_s, w_q, w_s, offsets, perm_tok, out, out_dtype, workspace, status): w_q [N, K] or [E, N, K]
PyObject *product(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 10);
    const Tensor &w = tensor_of(a[2], "w_q");
    TORCH_CHECK_VALUE(w.dim() == 2 || w.dim() == 3, "w_q: ", w.dim(), " dimensions, expected 2 or 3");
    TORCH_CHECK_TYPE(THPDtype_Check(a[7]), "out_dtype: expected a torch.dtype, got ", Py_TYPE(a[7])->tp_name);
    const ScalarType out_dtype = reinterpret_cast<THPDtype *>(a[7])->scalar_type;
    TORCH_CHECK_TYPE(is_kind(out_dtype, REAL), "out_dtype: ", out_dtype, ", expected float32 or bfloat16");
    const bool grouped = w.dim() == 3;
    const int64_t E = grouped ? w.size(0) : 1, N = w.size(-2);
    const Rows r = rows_of(a[0], a[1], a[4], a[5], a[9], E);
    const int64_t w3[3] = {E, N, r.K}, s3[3] = {E, blocks(N), blocks(r.K)};
    const void *pw = need(w, "w_q", grouped ? at::IntArrayRef(w3) : at::IntArrayRef(w3 + 1, 2), CODES, r.dev);
    const void *ps = need(tensor_of(a[3], "w_s"), "w_s", grouped ? at::IntArrayRef(s3) : at::IntArrayRef(s3 + 1, 2), FLOAT32, r.dev);
    const int64_t o_shape[2] = {r.rows, N};
    if (given(a[6])) need(tensor_of(a[6], "out"), "out", o_shape, REAL, r.dev, true);
    need_cuda(w, "w_q");
    const c10::cuda::CUDAGuard guard(r.dev);
    Tensor h0, h1;
    const Tensor &out = given_or_empty(a[6], "out", h0, o_shape, out_dtype, r.dev);
    size_t ws_bytes;
    void *ws = workspace_of(a[8], r, h1, &ws_bytes);
    const moe_status st =
        moe_grouped_gemm_fp8b(r.x_q, r.x_s, r.x_rows, r.K, r.ldx, pw, static_cast<const float *>(ps), int_of(E, "w_q"),
                              int_of(N, "w_q"), r.offsets, r.perm_tok, r.rows, out.data_ptr(), real_dtype(out),
                              row_stride(out), ws, ws_bytes, r.status, stream_of(r.dev));
    if (st != MOE_OK) return failed(st);
    return wrap(a[6], out);
    END_HANDLE_TH_ERRORS
}

// gate_up(x_q, x_s, wg_q, wg_s, wu_q, wu_s, offsets, perm_tok, h_q, h_s, workspace, status)
PyObject *gate_up(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 12);
    const Tensor &wg = tensor_of(a[2], "wg_q");
    TORCH_CHECK_VALUE(wg.dim() == 2 || wg.dim() == 3, "wg_q: ", wg.dim(), " dimensions, expected 2 or 3");
    const bool grouped = wg.dim() == 3;
    const int64_t E = grouped ? wg.size(0) : 1, F = wg.size(-2);
    const Rows r = rows_of(a[0], a[1], a[6], a[7], a[11], E);
    const int64_t w3[3] = {E, F, r.K}, s3[3] = {E, blocks(F), blocks(r.K)};
    const at::IntArrayRef w_shape = grouped ? at::IntArrayRef(w3) : at::IntArrayRef(w3 + 1, 2);
    const at::IntArrayRef s_shape = grouped ? at::IntArrayRef(s3) : at::IntArrayRef(s3 + 1, 2);
    const void *pg = need(wg, "wg_q", w_shape, CODES, r.dev);
    const void *pgs = need(tensor_of(a[3], "wg_s"), "wg_s", s_shape, FLOAT32, r.dev);
    const void *pu = need(tensor_of(a[4], "wu_q"), "wu_q", w_shape, CODES, r.dev);
    const void *pus = need(tensor_of(a[5], "wu_s"), "wu_s", s_shape, FLOAT32, r.dev);
    const int64_t h_shape[2] = {r.rows, F}, hs_shape[2] = {r.rows, blocks(F)};
    if (given(a[8])) need(tensor_of(a[8], "h_q"), "h_q", h_shape, CODES, r.dev);
    if (given(a[9])) need(tensor_of(a[9], "h_s"), "h_s", hs_shape, FLOAT32, r.dev);
    need_cuda(wg, "wg_q");
    const c10::cuda::CUDAGuard guard(r.dev);
    Tensor h0, h1, h2;
    const Tensor &h_q = given_or_empty(a[8], "h_q", h0, h_shape, ScalarType::Float8_e4m3fn, r.dev);
    const Tensor &h_s = given_or_empty(a[9], "h_s", h1, hs_shape, ScalarType::Float, r.dev);
    size_t ws_bytes;
    void *ws = workspace_of(a[10], r, h2, &ws_bytes);
    const moe_status st =
        moe_gate_up_fp8b(r.x_q, r.x_s, r.x_rows, r.K, r.ldx, pg, static_cast<const float *>(pgs), pu,
                         static_cast<const float *>(pus), int_of(E, "wg_q"), int_of(F, "wg_q"), r.offsets, r.perm_tok,
                         r.rows, h_q.data_ptr(), h_s.data_ptr<float>(), ws, ws_bytes, r.status, stream_of(r.dev));
    if (st != MOE_OK) return failed(st);
    return Py_BuildValue("(NN)", wrap(a[8], h_q), wrap(a[9], h_s));
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<quant>("quant"), method<norm>("norm"), method<product>("product"),
                         method<gate_up>("gate_up"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8b", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8b(void) { return PyModule_Create(&module); }
