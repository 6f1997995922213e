// The expert block's part of the Python binding, as an extension module like the
// attention block's (attention_binding.cpp): checks of arguments (ValueError),
// results and workspaces in the memory of the call's stream; a status other
// than FP8_OK is returned as an int.
#include "binding_args.h"

namespace {

// A matrix with unit stride along a row; its leading dimension.
int64_t rows(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
    expect(t, name, dtype, shape, false);
    TORCH_CHECK_VALUE(t.numel() == 0 || t.size(1) == 1 || t.stride(1) == 1, name,
                      " must have unit stride along a row");
    TORCH_CHECK_VALUE(t.size(0) <= 1 || t.numel() == 0 || t.stride(0) >= t.size(1), name,
                      " must have rows that do not overlap");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// The given tensor, or a new one.
void result(Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape, const Tensor& like) {
    if (t.defined()) expect(t, name, dtype, shape);
    else t = make(shape, dtype, like);
}

void scratch(Tensor& ws, size_t need, const Tensor& like) {
    if (ws.defined()) expect(ws, "workspace", at::kByte, {-1});
    else ws = make({static_cast<int64_t>(need ? need : 1)}, at::kByte, like);
}

PyObject* tuple(std::initializer_list<const Tensor*> all) {
    PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(all.size()));
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor* t : all) {
        PyObject* o = Py_None;
        if (t->defined()) o = THPVariable_Wrap(*t);
        else Py_INCREF(o);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

template <typename T>
T* data(const Tensor& t) {
    return static_cast<T*>(ptr(t));
}

PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(11);
    const Tensor logits = tensor_of(a[0], "logits");
    const int64_t k = int_of(a[1], "top_k");
    const bool renorm = bool_of(a[2], "renormalize");
    const float scale = float_of(a[3], "scale");
    Tensor ids = tensor_of(a[4], "expert_ids"), weights = tensor_of(a[5], "weights"),
           offsets = tensor_of(a[6], "offsets"), row_token = tensor_of(a[7], "row_token"),
           token_row = tensor_of(a[8], "token_row"), ws = tensor_of(a[9], "workspace");
    const bool fp32 = logits.defined() && logits.scalar_type() == at::kFloat;
    const int64_t ld = rows(logits, "logits", fp32 ? at::kFloat : at::kBFloat16, {-1, -1});
    const int64_t T = logits.size(0), E = logits.size(1);
    TORCH_CHECK_VALUE(k >= 1 && k <= E && k <= 32 && E <= 1024, "top_k must be 1 .. min(experts, 32) and experts "
                      "at most 1024; got ", k, " of ", E);
    TORCH_CHECK_VALUE(T <= int64_t(1) << 23, "at most 2^23 tokens; got ", T);
    const Place place(logits, a[10]);
    if (!ids.defined() && !weights.defined() && !offsets.defined() && !row_token.defined() && !token_row.defined() &&
        !ws.defined()) {
        // one allocation for all of them
        auto bytes = [](int64_t n) { return (n + 255) / 256 * 256; };
        const int64_t pairs = bytes(4 * T * k), bounds = bytes(4 * (E + 1));
        const int64_t need = static_cast<int64_t>(fp8_moe_route_workspace_size(T, E, k));
        const Tensor block = make({4 * pairs + bounds + need + 1}, at::kByte, logits);
        ids = carve(block, 0, {T, k}, at::kInt);
        weights = carve(block, pairs, {T, k}, at::kFloat);
        row_token = carve(block, 2 * pairs, {T * k}, at::kInt);
        token_row = carve(block, 3 * pairs, {T, k}, at::kInt);
        offsets = carve(block, 4 * pairs, {E + 1}, at::kInt);
        ws = carve(block, 4 * pairs + bounds, {need}, at::kByte);
    }
    result(ids, "expert_ids", at::kInt, {T, k}, logits);
    result(weights, "weights", at::kFloat, {T, k}, logits);
    result(offsets, "offsets", at::kInt, {E + 1}, logits);
    result(row_token, "row_token", at::kInt, {T * k}, logits);
    result(token_row, "token_row", at::kInt, {T, k}, logits);
    scratch(ws, fp8_moe_route_workspace_size(T, E, k), logits);
    same_device(logits, {&ids, &weights, &offsets, &row_token, &token_row, &ws});
    const fp8_status_t st = fp8_moe_route(
        ptr(logits), fp32, ld, T, E, k, renorm, scale, data<int32_t>(ids), data<float>(weights), data<int32_t>(offsets),
        data<int32_t>(row_token), data<int32_t>(token_row), ptr(ws), static_cast<size_t>(ws.numel()), place.stream);
    return st != FP8_OK ? status(st) : tuple({&ids, &weights, &offsets, &row_token, &token_row});
    END_HANDLE_TH_ERRORS
}

// The experts' weights and bounds, and the output [R, N] or [R, N / 2].
struct Experts {
    int64_t E, N, K;
    Experts(const Tensor& wq, const Tensor& s_w, const Tensor& offsets, int64_t width, bool swiglu) {
        expect(wq, "wq", at::kByte, {-1, -1, width});
        E = wq.size(0), N = wq.size(1), K = width;
        expect(s_w, "s_w", at::kFloat, {E, N});
        expect(offsets, "offsets", at::kInt, {E + 1});
        TORCH_CHECK_VALUE(!swiglu || N % 2 == 0, "swiglu needs an even number of weight rows; got ", N);
    }
};

PyObject* grouped_gemm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(9);
    const Tensor xq = tensor_of(a[0], "xq"), s_tok = tensor_of(a[1], "s_tok"), wq = tensor_of(a[2], "wq"),
                 s_w = tensor_of(a[3], "s_w"), offsets = tensor_of(a[4], "offsets");
    const bool swiglu = bool_of(a[5], "swiglu");
    Tensor y = tensor_of(a[6], "y"), ws = tensor_of(a[7], "workspace");
    expect(xq, "xq", at::kByte, {-1, -1});
    const int64_t R = xq.size(0);
    expect(s_tok, "s_tok", at::kFloat, {R});
    const Experts x(wq, s_w, offsets, xq.size(1), swiglu);
    const Place place(xq, a[8]);
    result(y, "y", at::kBFloat16, {R, swiglu ? x.N / 2 : x.N}, xq);
    scratch(ws, ws.defined() ? 0 : fp8_grouped_gemm_workspace_size(x.E, R, x.N, x.K), xq);
    same_device(xq, {&s_tok, &wq, &s_w, &offsets, &y, &ws});
    const fp8_status_t st = fp8_grouped_gemm(
        data<uint8_t>(xq), data<float>(s_tok), data<uint8_t>(wq), data<float>(s_w), data<int32_t>(offsets), x.E, R, x.N,
        x.K, swiglu, ptr(y), ptr(ws), static_cast<size_t>(ws.numel()), place.stream);
    return st != FP8_OK ? status(st) : THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject* grouped_linear(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(9);
    const Tensor x = tensor_of(a[0], "x"), wq = tensor_of(a[1], "wq"), s_w = tensor_of(a[2], "s_w"),
                 offsets = tensor_of(a[3], "offsets"), row_token = tensor_of(a[4], "row_token");
    const bool swiglu = bool_of(a[5], "swiglu");
    Tensor y = tensor_of(a[6], "y"), ws = tensor_of(a[7], "workspace");
    const int64_t ldx = rows(x, "x", at::kBFloat16, {-1, -1});
    if (row_token.defined()) expect(row_token, "row_token", at::kInt, {-1});
    const int64_t T = x.size(0), R = row_token.defined() ? row_token.size(0) : T;
    const Experts w(wq, s_w, offsets, x.size(1), swiglu);
    const Place place(x, a[8]);
    result(y, "y", at::kBFloat16, {R, swiglu ? w.N / 2 : w.N}, x);
    scratch(ws, ws.defined() ? 0 : fp8_grouped_linear_workspace_size(w.E, R, w.N, w.K), x);
    same_device(x, {&wq, &s_w, &offsets, &row_token, &y, &ws});
    const fp8_status_t st = fp8_grouped_linear(
        ptr(x), T, ldx, data<int32_t>(row_token), data<uint8_t>(wq), data<float>(s_w), data<int32_t>(offsets), w.E, R,
        w.N, w.K, swiglu, ptr(y), ptr(ws), static_cast<size_t>(ws.numel()), place.stream);
    return st != FP8_OK ? status(st) : THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject* residual_norm_quant(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(17);
    const Tensor h = tensor_of(a[0], "h"), y = tensor_of(a[1], "y"), gamma = tensor_of(a[2], "gamma"),
                 gamma_post = tensor_of(a[4], "gamma_post"), gate = tensor_of(a[5], "gate"),
                 token_row = tensor_of(a[8], "token_row"), weights = tensor_of(a[9], "weights");
    const float eps = float_of(a[3], "eps"), residual_scale = float_of(a[6], "residual_scale"),
                branch_scale = float_of(a[7], "branch_scale");
    const bool want_z = bool_of(a[10], "rows"), want_codes = bool_of(a[11], "codes");
    Tensor h_out = tensor_of(a[12], "h_out"), z = tensor_of(a[13], "z"), xq = tensor_of(a[14], "xq"),
           s_tok = tensor_of(a[15], "s_tok");
    const int64_t ldh = rows(h, "h", at::kBFloat16, {-1, -1});
    const int64_t T = h.size(0), K = h.size(1);
    const int64_t ldy = rows(y, "y", at::kBFloat16, {token_row.defined() ? -1 : T, K});
    int64_t k = 0, ldg = 0;
    if (token_row.defined()) {
        expect(token_row, "token_row", at::kInt, {T, -1});
        k = token_row.size(1);
        TORCH_CHECK_VALUE(k >= 1 && k <= 32, "token_row must have 1 .. 32 rows a token; got ", k);
        if (weights.defined()) expect(weights, "weights", at::kFloat, {T, k});
    } else {
        TORCH_CHECK_VALUE(!weights.defined(), "weights need token_row");
    }
    if (gamma_post.defined()) expect(gamma_post, "gamma_post", at::kBFloat16, {K});
    if (gamma.defined() || want_z || want_codes) expect(gamma, "gamma", at::kBFloat16, {K});
    if (gate.defined()) {
        if (gate.dim() == 1) expect(gate, "gate", at::kBFloat16, {K});
        else ldg = rows(gate, "gate", at::kBFloat16, {T, K});
    }
    TORCH_CHECK_VALUE(want_z || !z.defined(), "z needs rows=True");
    TORCH_CHECK_VALUE(want_codes || (!xq.defined() && !s_tok.defined()), "xq and s_tok need codes=True");
    const Place place(h, a[16]);
    int64_t ldho = K, ldq = K;
    if (!h_out.defined() && !z.defined() && !xq.defined() && !s_tok.defined()) {
        // one allocation for all of them
        auto bytes = [](int64_t n) { return (n + 255) / 256 * 256; };
        const int64_t wide = bytes(2 * T * K), at_q = wide + (want_z ? wide : 0), at_s = at_q + bytes(T * K);
        const Tensor block = make({want_codes ? at_s + 4 * T : at_q}, at::kByte, h);
        h_out = carve(block, 0, {T, K}, at::kBFloat16);
        if (want_z) z = carve(block, wide, {T, K}, at::kBFloat16);
        if (want_codes) {
            xq = carve(block, at_q, {T, K}, at::kByte);
            s_tok = carve(block, at_s, {T}, at::kFloat);
        }
    }
    if (h_out.defined()) ldho = rows(h_out, "h_out", at::kBFloat16, {T, K});
    else h_out = make({T, K}, at::kBFloat16, h);
    if (want_z) result(z, "z", at::kBFloat16, {T, K}, h);
    if (want_codes) {
        if (xq.defined()) ldq = rows(xq, "xq", at::kByte, {T, K});
        else xq = make({T, K}, at::kByte, h);
        result(s_tok, "s_tok", at::kFloat, {T}, h);
    }
    same_device(h, {&y, &gamma, &gamma_post, &gate, &token_row, &weights, &h_out, &z, &xq, &s_tok});
    const fp8_status_t st = fp8_residual_norm_quant(
        ptr(h), ldh, ptr(y), ldy, y.size(0), data<int32_t>(token_row), data<float>(weights), k, ptr(gamma_post), ptr(gate),
        ldg, ptr(gamma), eps, residual_scale, branch_scale, T, K, ptr(h_out), ldho, ptr(z), data<uint8_t>(xq), ldq,
        data<float>(s_tok), place.stream);
    return st != FP8_OK ? status(st) : tuple({&h_out, &z, &xq, &s_tok});
    END_HANDLE_TH_ERRORS
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(moe_route), METHOD(grouped_gemm), METHOD(grouped_linear), METHOD(residual_norm_quant),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fp8_experts_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fp8_experts_binding() { return PyModule_Create(&module); }
