// fp8b_binding.cpp -- the Python side of the block-scaled fp8 operators: checks
// of the tensors, allocation of the outputs and the call into the C ABI.
//
// The other calls of the binding go through ctypes.  These take up to ten
// tensors that have to fit one another (a wrong pairing would read out of
// bounds), and in Python the checks, the allocations and the marshalling took
// 15-23 us a call on the host where the kernels of a decode step take 2-7 us;
// here they take 3-6 us.  Nothing of the operators is computed here.
#include "binding.h"

namespace {

using namespace moe_py;

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

// scratch of gathered rows
void *workspace_of(PyObject *o, const Rows &r, Tensor &holder, size_t *bytes)
{
    *bytes = 0;
    return r.perm_tok ? scratch_of(o, r.dev, moe_fp8b_workspace_size(r.rows, r.K), holder, bytes) : nullptr;
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

PyMethodDef methods[] = {method<quant>("quant"), method<norm>("norm"), method<product>("product"),
                         method<gate_up>("gate_up"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8b", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8b(void)
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddFunctions(m, moe_py::i8_methods) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
