// i8_binding.cpp -- the Python side of the 8-bit integer operators and of dispatch and
// combine (checks, outputs, the call into the C ABI), part of the module of
// fp8b_binding.cpp.  Nothing of the operators is computed here.
#include <c10/core/GradMode.h>

#include "binding.h"

namespace {

using namespace moe_py;

ScalarType real_type_of(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPDtype_Check(o), name, ": expected a torch.dtype, got ", Py_TYPE(o)->tp_name);
    const ScalarType t = reinterpret_cast<THPDtype *>(o)->scalar_type;
    TORCH_CHECK_TYPE(is_kind(t, REAL), name, ": ", t, ", expected float32 or bfloat16");
    return t;
}
Kind kind_of(const Tensor &t) { return t.scalar_type() == ScalarType::Float ? FLOAT32 : BFLOAT16; }

// quant_i8(x, codes, scales)
PyObject *quant_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 3);
    const Tensor &x = tensor_of(a[0], "x");
    TORCH_CHECK_VALUE(x.dim() == 2 || x.dim() == 3, "x: ", x.dim(), " dimensions, expected 2 or 3");
    const c10::Device dev = x.device();
    const int64_t per = x.size(-2), cols = x.size(-1), batch = x.dim() == 3 ? x.size(0) : 1;
    const void *px = need(x, "x", x.sizes(), REAL, dev, true);
    // (rows of a batch of one row each lie a batch apart)
    const int64_t ldx = x.dim() == 3 && per == 1 && batch > 1 ? x.stride(0) : row_stride(x);
    TORCH_CHECK_VALUE(x.dim() == 2 || batch <= 1 || per == 0 || x.stride(0) == per * ldx, "x: strides ", x.strides(),
                      " are not supported, make it contiguous");
    const at::IntArrayRef s_shape = x.sizes().slice(0, x.dim() - 1);
    if (given(a[1])) need(tensor_of(a[1], "codes"), "codes", x.sizes(), INT8, dev);
    if (given(a[2])) need(tensor_of(a[2], "scales"), "scales", s_shape, FLOAT32, dev);
    need_cuda(x, "x");
    const int rows = int_of(batch * per, "x");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor h0, h1;
    const Tensor &codes = given_or_empty(a[1], "codes", h0, x.sizes(), ScalarType::Char, dev);
    const Tensor &scales = given_or_empty(a[2], "scales", h1, s_shape, ScalarType::Float, dev);
    const moe_status st = moe_quant_i8(px, real_dtype(x), rows, int_of(cols, "x"), ldx, static_cast<int8_t *>(codes.data_ptr()),
                                       scales.data_ptr<float>(), stream_of(dev));
    if (st != MOE_OK) return failed(st);
    return Py_BuildValue("(NN)", wrap(a[1], codes), wrap(a[2], scales));
    END_HANDLE_TH_ERRORS
}

// product_i8(x_q, x_s, w_q, w_s, offsets, perm_tok, out, out_dtype, workspace, status): w_q [N, K] or [E, N, K]
PyObject *product_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 10);
    const Tensor &w = tensor_of(a[2], "w_q");
    TORCH_CHECK_VALUE(w.dim() == 2 || w.dim() == 3, "w_q: ", w.dim(), " dimensions, expected 2 or 3");
    const ScalarType out_dtype = real_type_of(a[7], "out_dtype");
    const bool grouped = w.dim() == 3;
    const int64_t E = grouped ? w.size(0) : 1, N = w.size(-2);
    const Rows r = rows_of(a[0], a[1], a[4], a[5], a[9], E, INT8);
    const int64_t w3[3] = {E, N, r.K};
    const void *pw = need(w, "w_q", grouped ? at::IntArrayRef(w3) : at::IntArrayRef(w3 + 1, 2), INT8, r.dev);
    const void *ps = need(tensor_of(a[3], "w_s"), "w_s", grouped ? at::IntArrayRef(w3, 2) : at::IntArrayRef(w3 + 1, 1), FLOAT32, r.dev);
    const int64_t o_shape[2] = {r.rows, N};
    if (given(a[6])) need(tensor_of(a[6], "out"), "out", o_shape, REAL, r.dev, true);
    need_cuda(w, "w_q");
    const c10::cuda::CUDAGuard guard(r.dev);
    Tensor h0, h1;
    const Tensor &out = given_or_empty(a[6], "out", h0, o_shape, out_dtype, r.dev);
    size_t ws_bytes;
    void *ws = scratch_of(a[8], r.dev, moe_i8_workspace_size(r.rows, r.K), h1, &ws_bytes);
    const moe_status st =
        moe_grouped_gemm_i8(r.x_q, r.x_s, r.x_rows, r.K, r.ldx, pw, static_cast<const float *>(ps), int_of(E, "w_q"),
                            int_of(N, "w_q"), r.offsets, r.perm_tok, r.rows, out.data_ptr(), real_dtype(out), row_stride(out),
                            ws, ws_bytes, r.status, stream_of(r.dev));
    if (st != MOE_OK) return failed(st);
    return wrap(a[6], out);
    END_HANDLE_TH_ERRORS
}

// gate_up_i8(x_q, x_s, wg_q, wg_s, wu_q, wu_s, offsets, perm_tok, h, h_dtype, workspace, status)
PyObject *gate_up_i8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 12);
    const Tensor &wg = tensor_of(a[2], "wg_q");
    TORCH_CHECK_VALUE(wg.dim() == 2 || wg.dim() == 3, "wg_q: ", wg.dim(), " dimensions, expected 2 or 3");
    const ScalarType h_dtype = real_type_of(a[9], "h_dtype");
    const bool grouped = wg.dim() == 3;
    const int64_t E = grouped ? wg.size(0) : 1, F = wg.size(-2);
    const Rows r = rows_of(a[0], a[1], a[6], a[7], a[11], E, INT8);
    const int64_t w3[3] = {E, F, r.K};
    const at::IntArrayRef w_shape = grouped ? at::IntArrayRef(w3) : at::IntArrayRef(w3 + 1, 2);
    const at::IntArrayRef s_shape = grouped ? at::IntArrayRef(w3, 2) : at::IntArrayRef(w3 + 1, 1);
    const void *pg = need(wg, "wg_q", w_shape, INT8, r.dev);
    const void *pgs = need(tensor_of(a[3], "wg_s"), "wg_s", s_shape, FLOAT32, r.dev);
    const void *pu = need(tensor_of(a[4], "wu_q"), "wu_q", w_shape, INT8, r.dev);
    const void *pus = need(tensor_of(a[5], "wu_s"), "wu_s", s_shape, FLOAT32, r.dev);
    const int64_t h_shape[2] = {r.rows, F};
    if (given(a[8])) need(tensor_of(a[8], "h"), "h", h_shape, REAL, r.dev, true);
    need_cuda(wg, "wg_q");
    const c10::cuda::CUDAGuard guard(r.dev);
    Tensor h0, h1;
    const Tensor &h = given_or_empty(a[8], "h", h0, h_shape, h_dtype, r.dev);
    size_t ws_bytes;
    void *ws = scratch_of(a[10], r.dev, moe_i8_workspace_size(r.rows, r.K), h1, &ws_bytes);
    const moe_status st =
        moe_gate_up_i8(r.x_q, r.x_s, r.x_rows, r.K, r.ldx, pg, static_cast<const float *>(pgs), pu,
                       static_cast<const float *>(pus), int_of(E, "wg_q"), int_of(F, "wg_q"), r.offsets, r.perm_tok, r.rows,
                       h.data_ptr(), real_dtype(h), row_stride(h), ws, ws_bytes, r.status, stream_of(r.dev));
    if (st != MOE_OK) return failed(st);
    return wrap(a[8], h);
    END_HANDLE_TH_ERRORS
}

// inv of k slots a token (as moe_permute gives it, or [T, k])
struct Slots { const int32_t *inv; int64_t T; int k; };
Slots slots_of(PyObject *o, int64_t k, c10::Device dev)
{
    const Tensor &inv = tensor_of(o, "inv");
    TORCH_CHECK_VALUE(k > 0, "k: ", k, ", expected a positive number");
    const void *p = need(inv, "inv", inv.sizes(), INT32, dev);
    TORCH_CHECK_VALUE(inv.numel() % k == 0, "inv: ", inv.numel(), " values, expected ", k, " a token");
    return {static_cast<const int32_t *>(p), inv.numel() / k, int_of(k, "k")};
}
// Whether an input requires grad where gradients are recorded: the call is then left to the
// Python side (the answer is NotImplemented), which comes again without recording.  An output that is
// given keeps no graph: such a call runs as it is, with a warning.
bool recorded(const char *call, bool has_output, std::initializer_list<const Tensor *> inputs)
{
    if (!c10::GradMode::is_enabled()) return false;
    for (const Tensor *t : inputs)
        if (t->requires_grad()) {
            if (has_output)
                TORCH_WARN(call, ": an output that is given keeps no graph, and an input requires grad: detach it, or let the "
                           "call allocate its outputs");
            return !has_output;
        }
    return false;
}
void need_matrix(const Tensor &t, const char *name)
{
    TORCH_CHECK_VALUE(t.dim() == 2, name, ": ", t.dim(), " dimensions, expected 2");
}

// dispatch(x, inv, k, out)
PyObject *dispatch(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 4);
    const Tensor &x = tensor_of(a[0], "x");
    const long k = PyLong_AsLong(a[2]);
    if (k == -1 && PyErr_Occurred()) return nullptr;
    need_matrix(x, "x");
    const c10::Device dev = x.device();
    const void *px = need(x, "x", x.sizes(), REAL, dev, true);
    const Slots s = slots_of(a[1], k, dev);
    TORCH_CHECK_VALUE(s.T == x.size(0), "inv: ", s.T * k, " values, expected ", x.size(0) * k);
    int64_t shape[2] = {s.T * k, x.size(1)};
    if (given(a[3])) {
        const Tensor &out = tensor_of(a[3], "out");
        need_matrix(out, "out");
        shape[0] = out.size(0);
        need(out, "out", shape, kind_of(x), dev, true);
    }
    need_cuda(x, "x");
    if (recorded("moe_dispatch", given(a[3]), {&x})) Py_RETURN_NOTIMPLEMENTED;
    const c10::cuda::CUDAGuard guard(dev);
    Tensor h0;
    const Tensor &out = given_or_empty(a[3], "out", h0, shape, x.scalar_type(), dev);
    // (a new output is written as a whole)
    const moe_status st = (given(a[3]) ? moe_dispatch : moe_dispatch_filled)(
        px, real_dtype(x), int_of(s.T, "x"), int_of(x.size(1), "x"), row_stride(x), s.inv, s.k, out.data_ptr(),
        int_of(shape[0], "out"), row_stride(out), stream_of(dev));
    if (st != MOE_OK) return failed(st);
    return wrap(a[3], out);
    END_HANDLE_TH_ERRORS
}

// dispatch_backward(grad, inv, k, out)
PyObject *dispatch_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 4);
    const Tensor &g = tensor_of(a[0], "grad");
    const long k = PyLong_AsLong(a[2]);
    if (k == -1 && PyErr_Occurred()) return nullptr;
    need_matrix(g, "grad");
    const c10::Device dev = g.device();
    const void *pg = need(g, "grad", g.sizes(), REAL, dev, true);
    const Slots s = slots_of(a[1], k, dev);
    const int64_t shape[2] = {s.T, g.size(1)};
    if (given(a[3])) need(tensor_of(a[3], "out"), "out", shape, kind_of(g), dev, true);
    need_cuda(g, "grad");
    if (recorded("moe_dispatch_backward", given(a[3]), {&g})) Py_RETURN_NOTIMPLEMENTED;
    const c10::cuda::CUDAGuard guard(dev);
    Tensor h0;
    const Tensor &out = given_or_empty(a[3], "out", h0, shape, g.scalar_type(), dev);
    const moe_status st = moe_dispatch_backward(pg, real_dtype(g), int_of(g.size(0), "grad"), int_of(g.size(1), "grad"),
                                                row_stride(g), s.inv, int_of(s.T, "inv"), s.k, out.data_ptr(), row_stride(out),
                                                stream_of(dev));
    if (st != MOE_OK) return failed(st);
    return wrap(a[3], out);
    END_HANDLE_TH_ERRORS
}

// topk_w [T, k] and its inv
Slots weighted_slots(PyObject *topk_w, PyObject *inv, c10::Device dev, const float **pw)
{
    const Tensor &w = tensor_of(topk_w, "topk_w");
    TORCH_CHECK_VALUE(w.dim() == 2 && w.size(1) > 0, "topk_w: shape ", w.sizes(), ", expected [T, k]");
    *pw = static_cast<const float *>(need(w, "topk_w", w.sizes(), FLOAT32, dev));
    const Slots s = slots_of(inv, w.size(1), dev);
    TORCH_CHECK_VALUE(s.T == w.size(0), "inv: ", s.T * s.k, " values, expected ", w.numel());
    return s;
}

// combine(y, topk_w, inv, out, out_dtype)
PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 5);
    const Tensor &y = tensor_of(a[0], "y");
    const ScalarType out_dtype = real_type_of(a[4], "out_dtype");
    need_matrix(y, "y");
    const c10::Device dev = y.device();
    const void *py = need(y, "y", y.sizes(), REAL, dev, true);
    const float *pw;
    const Slots s = weighted_slots(a[1], a[2], dev, &pw);
    const int64_t shape[2] = {s.T, y.size(1)};
    if (given(a[3])) need(tensor_of(a[3], "out"), "out", shape, REAL, dev, true);
    need_cuda(y, "y");
    if (recorded("moe_combine", given(a[3]), {&y, &tensor_of(a[1], "topk_w")})) Py_RETURN_NOTIMPLEMENTED;
    const c10::cuda::CUDAGuard guard(dev);
    Tensor h0;
    const Tensor &out = given_or_empty(a[3], "out", h0, shape, out_dtype, dev);
    const moe_status st = moe_combine(py, real_dtype(y), int_of(y.size(0), "y"), int_of(y.size(1), "y"), row_stride(y), pw,
                                      s.inv, int_of(s.T, "topk_w"), s.k, out.data_ptr(), real_dtype(out), row_stride(out),
                                      stream_of(dev));
    if (st != MOE_OK) return failed(st);
    return wrap(a[3], out);
    END_HANDLE_TH_ERRORS
}

// combine_backward(grad, y, topk_w, inv, want_dy, want_dw, dy, dw)
PyObject *combine_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_args(n, 8);
    const Tensor &g = tensor_of(a[0], "grad"), &y = tensor_of(a[1], "y");
    const int want_dy = PyObject_IsTrue(a[4]);
    if (want_dy < 0) return nullptr;
    const int want_dw = PyObject_IsTrue(a[5]);
    if (want_dw < 0) return nullptr;
    need_matrix(g, "grad");
    need_matrix(y, "y");
    TORCH_CHECK_VALUE(want_dy || !given(a[6]), "dy is given but not wanted");
    TORCH_CHECK_VALUE(want_dw || !given(a[7]), "dw is given but not wanted");
    const c10::Device dev = g.device();
    const float *pw;
    const Slots s = weighted_slots(a[2], a[3], dev, &pw);
    const int64_t g_shape[2] = {s.T, y.size(1)}, w_shape[2] = {s.T, s.k};
    const void *pg = need(g, "grad", g_shape, REAL, dev, true);
    const void *py = need(y, "y", y.sizes(), REAL, dev, true);
    if (given(a[6])) need(tensor_of(a[6], "dy"), "dy", y.sizes(), kind_of(y), dev, true);
    if (given(a[7])) need(tensor_of(a[7], "dw"), "dw", w_shape, FLOAT32, dev);
    need_cuda(g, "grad");
    if (recorded("moe_combine_backward", given(a[6]) || given(a[7]), {&g, &y, &tensor_of(a[2], "topk_w")}))
        Py_RETURN_NOTIMPLEMENTED;
    const c10::cuda::CUDAGuard guard(dev);
    Tensor h0, h1;
    void *pdy = nullptr;
    float *pdw = nullptr;
    int64_t lddy = y.size(1);
    if (want_dy) {
        const Tensor &dy = given_or_empty(a[6], "dy", h0, y.sizes(), y.scalar_type(), dev);
        pdy = dy.data_ptr();
        lddy = row_stride(dy);
    }
    if (want_dw) pdw = given_or_empty(a[7], "dw", h1, w_shape, ScalarType::Float, dev).data_ptr<float>();
    const moe_status st = (given(a[6]) ? moe_combine_backward : moe_combine_backward_filled)(
        pg, real_dtype(g), int_of(s.T, "topk_w"), int_of(y.size(1), "y"), row_stride(g), py, real_dtype(y), int_of(y.size(0), "y"),
        row_stride(y), pw, s.inv, s.k, pdy, lddy, pdw, stream_of(dev));
    if (st != MOE_OK) return failed(st);
    auto result = [](bool wanted, PyObject *o, const Tensor &t) {
        if (wanted) return wrap(o, t);
        Py_INCREF(Py_None);
        return Py_None;
    };
    return Py_BuildValue("(NN)", result(want_dy, a[6], h0), result(want_dw, a[7], h1));
    END_HANDLE_TH_ERRORS
}

}  // namespace

namespace moe_py {

PyMethodDef i8_methods[] = {method<quant_i8>("quant_i8"), method<product_i8>("product_i8"), method<gate_up_i8>("gate_up_i8"),
                            method<dispatch>("dispatch"), method<dispatch_backward>("dispatch_backward"),
                            method<combine>("combine"), method<combine_backward>("combine_backward"),
                            {nullptr, nullptr, 0, nullptr}};

}  // namespace moe_py
