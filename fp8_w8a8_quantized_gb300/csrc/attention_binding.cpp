// The attention block's part of the Python binding, as an extension module: a
// decode step calls these operators for every layer, and the same checks and
// allocations written in Python took 20 to 30 us a call, several times what
// the kernels need.  Argument marshalling only: device, dtype, shape and
// layout of every tensor are checked here (ValueError), results and workspaces
// allocated in the memory of the stream that the call runs on, and the C ABI
// (fp8w8a8.h) does the rest; a status other than FP8_OK is returned as an int.
#include "binding_args.h"

#include <cmath>

namespace {

// The token stride of a bf16 [tokens, heads, D] tensor whose heads are
// contiguous within a token (a view into a wider projection will do).
int64_t tokens(const Tensor& t, const char* name, at::IntArrayRef shape = {-1, -1, -1}) {
    expect(t, name, at::kBFloat16, shape, false);
    const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
    TORCH_CHECK_VALUE(t.numel() == 0 || ((d == 1 || t.stride(2) == 1) && (h == 1 || t.stride(1) == d)),
                      name, " must have the heads of a token contiguous; got strides ",
                      shape_text(t.strides()));
    return n > 1 ? t.stride(0) : h * d;
}

int64_t scale_stride(const Tensor& t, const char* name, int64_t heads) {
    if (t.defined() && t.numel() == 1) {
        expect(t, name, at::kFloat, t.sizes());
        return 0;
    }
    expect(t, name, at::kFloat, {heads});
    return 1;
}

int64_t cache_slots(const Tensor& k, const Tensor& v, int64_t heads, int64_t dim) {
    expect(k, "k_cache", at::kByte, {-1, heads, dim});
    expect(v, "v_cache", at::kByte, {k.size(0), heads, dim});
    return k.size(0);
}

int64_t table_stride(const Tensor& t, int64_t rows) {
    expect(t, "block_table", at::kInt, {rows, -1}, false);
    TORCH_CHECK_VALUE(t.numel() == 0 || t.size(1) == 1 || t.stride(1) == 1,
                      "block_table must have unit stride along a row");
    return rows > 1 ? t.stride(0) : t.size(1);
}

PyObject* kv_slots(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(12);
    const Tensor ctx = tensor_of(a[0], "ctx_lens"), fresh = tensor_of(a[1], "new_lens"),
                 pages = tensor_of(a[2], "free_pages"), table = tensor_of(a[4], "block_table");
    const int64_t page = int_of(a[3], "page_size"), room = int_of(a[5], "max_tokens");
    Tensor slot = tensor_of(a[6], "slot_mapping"), pos = tensor_of(a[7], "positions"),
           cu = tensor_of(a[8], "cu_seqlens"), lens = tensor_of(a[9], "seq_lens"),
           used = tensor_of(a[10], "pages_used");
    TORCH_CHECK_VALUE(room >= 0 && room < int64_t(1) << 31, "max_tokens must be 0 .. 2^31 - 1");
    expect(ctx, "ctx_lens", at::kInt, {-1});
    const int64_t B = ctx.size(0);
    expect(fresh, "new_lens", at::kInt, {B});
    expect(pages, "free_pages", at::kInt, {-1});
    const int64_t ld = table_stride(table, B);
    const Place place(ctx, a[11]);
    if (!slot.defined() && !pos.defined() && !cu.defined() && !lens.defined() && !used.defined()) {
        // one allocation for all five (with five the call takes the host 7.7 us instead of 5.2)
        auto bytes = [](int64_t n) { return (n + 255) / 256 * 256; };
        const int64_t at_pos = bytes(room * 8), at_cu = at_pos + bytes(room * 4),
                      at_lens = at_cu + bytes((B + 1) * 4), at_used = at_lens + bytes(B * 4);
        const Tensor block = make({at_used + 4}, at::kByte, ctx);
        slot = carve(block, 0, {room}, at::kLong);
        pos = carve(block, at_pos, {room}, at::kInt);
        cu = carve(block, at_cu, {B + 1}, at::kInt);
        lens = carve(block, at_lens, {B}, at::kInt);
        used = carve(block, at_used, {1}, at::kInt);
    }
    if (!slot.defined()) slot = make({room}, at::kLong, ctx);
    else expect(slot, "slot_mapping", at::kLong, {room});
    if (!pos.defined()) pos = make({room}, at::kInt, ctx);
    else expect(pos, "positions", at::kInt, {room});
    if (!cu.defined()) cu = make({B + 1}, at::kInt, ctx);
    else expect(cu, "cu_seqlens", at::kInt, {B + 1});
    if (!lens.defined()) lens = make({B}, at::kInt, ctx);
    else expect(lens, "seq_lens", at::kInt, {B});
    if (!used.defined()) used = make({1}, at::kInt, ctx);
    else expect(used, "pages_used", at::kInt, {1});
    same_device(ctx, {&fresh, &pages, &table, &slot, &pos, &cu, &lens, &used});
    const fp8_status_t st = fp8_kv_slots(
        static_cast<const int32_t*>(ptr(ctx)), static_cast<const int32_t*>(ptr(fresh)), B,
        static_cast<const int32_t*>(ptr(pages)), pages.size(0), page, static_cast<int32_t*>(ptr(table)),
        table.size(1), ld, room, static_cast<int64_t*>(ptr(slot)), static_cast<int32_t*>(ptr(pos)),
        static_cast<int32_t*>(ptr(cu)), static_cast<int32_t*>(ptr(lens)), static_cast<int32_t*>(ptr(used)),
        place.stream);
    if (st != FP8_OK) return status(st);
    PyObject* out = PyTuple_New(5);
    if (!out) return nullptr;
    const Tensor* all[5] = {&slot, &pos, &cu, &lens, &used};
    for (int i = 0; i < 5; ++i) {
        PyObject* o = THPVariable_Wrap(*all[i]);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, o);
    }
    return out;
    END_HANDLE_TH_ERRORS
}

PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(18);
    const Tensor q = tensor_of(a[0], "q"), k = tensor_of(a[1], "k"), pos = tensor_of(a[2], "positions"),
                 turns = tensor_of(a[3], "turns"), gq = tensor_of(a[4], "gamma_q"),
                 gk = tensor_of(a[5], "gamma_k"), v = tensor_of(a[10], "v"),
                 ks = tensor_of(a[11], "k_scale"), vs = tensor_of(a[12], "v_scale"),
                 slot = tensor_of(a[13], "slot_mapping"), kc = tensor_of(a[14], "k_cache"),
                 vc = tensor_of(a[15], "v_cache");
    Tensor qo = tensor_of(a[8], "q_out"), ko = tensor_of(a[9], "k_out");
    const float eps = float_of(a[6], "eps");
    const bool pairs = bool_of(a[7], "interleaved"), cache_only = bool_of(a[16], "cache_only");
    const int64_t ldq = tokens(q, "q");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    const int64_t ldk = tokens(k, "k", {T, -1, D}), Hkv = k.size(1);
    expect(pos, "positions", at::kInt, {T});
    expect(turns, "turns", at::kLong, {-1});
    if (gq.defined()) expect(gq, "gamma_q", at::kBFloat16, {D});
    if (gk.defined()) expect(gk, "gamma_k", at::kBFloat16, {D});
    const bool cached = kc.defined() || vc.defined();
    int64_t ldv = 0, stride = 0, slots = 0;
    if (cached) {
        ldv = tokens(v, "v", {T, Hkv, D});
        slots = cache_slots(kc, vc, Hkv, D);
        stride = scale_stride(ks, "k_scale", Hkv);
        TORCH_CHECK_VALUE(scale_stride(vs, "v_scale", Hkv) == stride,
                          "k_scale and v_scale must both be per head or both single");
        if (slot.defined()) expect(slot, "slot_mapping", at::kLong, {T});
    }
    const Place place(q, a[17]);
    int64_t ldqo = Hq * D, ldko = Hkv * D;
    if (!qo.defined()) qo = make({T, Hq, D}, at::kBFloat16, q);
    else ldqo = tokens(qo, "q_out", {T, Hq, D});
    if (cached && cache_only) ko = Tensor();
    else if (!ko.defined()) ko = make({T, Hkv, D}, at::kBFloat16, q);
    else ldko = tokens(ko, "k_out", {T, Hkv, D});
    same_device(q, {&k, &pos, &turns, &gq, &gk, &qo, &ko, &v, &ks, &vs, &slot, &kc, &vc});
    const fp8_status_t st = fp8_qk_norm_rope(
        ptr(q), ldq, ptr(k), ldk, cached ? ptr(v) : nullptr, ldv, T, Hq, Hkv, D, ptr(gq), ptr(gk), eps,
        static_cast<const int32_t*>(ptr(pos)), static_cast<const uint64_t*>(ptr(turns)), 2 * turns.size(0),
        pairs, ptr(qo), ldqo, ptr(ko), ldko, static_cast<const float*>(ptr(ks)),
        static_cast<const float*>(ptr(vs)), stride, cached ? static_cast<const int64_t*>(ptr(slot)) : nullptr,
        static_cast<uint8_t*>(ptr(kc)), static_cast<uint8_t*>(ptr(vc)), slots, place.stream);
    if (st != FP8_OK) return status(st);
    PyObject* out = PyTuple_New(2);
    if (!out) return nullptr;
    PyObject* o = THPVariable_Wrap(qo);
    PyObject* p = nullptr;
    if (ko.defined()) {
        p = THPVariable_Wrap(ko);
    } else {
        p = Py_None;
        Py_INCREF(p);
    }
    if (!o || !p) {
        Py_XDECREF(o);
        Py_XDECREF(p);
        Py_DECREF(out);
        return nullptr;
    }
    PyTuple_SET_ITEM(out, 0, o);
    PyTuple_SET_ITEM(out, 1, p);
    return out;
    END_HANDLE_TH_ERRORS
}

// 1 / sqrt(D) unless a scale is given.
float softmax_scale(PyObject* o, int64_t D) {
    if (o == Py_None) return D > 0 ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : 1.0f;
    return float_of(o, "scale");
}

PyObject* attention_prompt(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(7);
    const Tensor q = tensor_of(a[0], "q"), k = tensor_of(a[1], "k"), v = tensor_of(a[2], "v"),
                 cu = tensor_of(a[3], "cu_seqlens");
    Tensor out = tensor_of(a[5], "out");
    const int64_t ldq = tokens(q, "q");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    const int64_t ldk = tokens(k, "k", {T, -1, D}), Hkv = k.size(1);
    const int64_t ldv = tokens(v, "v", {T, Hkv, D});
    expect(cu, "cu_seqlens", at::kInt, {-1});
    TORCH_CHECK_VALUE(cu.size(0) >= 1, "cu_seqlens must hold the sequences' bounds");
    const float scale = softmax_scale(a[4], D);
    const Place place(q, a[6]);
    int64_t ldo = Hq * D;
    if (!out.defined()) out = make({T, Hq, D}, at::kBFloat16, q);
    else ldo = tokens(out, "out", {T, Hq, D});
    same_device(q, {&k, &v, &cu, &out});
    const fp8_status_t st =
        fp8_attention_prompt(ptr(q), ldq, ptr(k), ldk, ptr(v), ldv, T, Hq, Hkv, D,
                             static_cast<const int32_t*>(ptr(cu)), cu.size(0) - 1, scale, ptr(out), ldo,
                             place.stream);
    return st != FP8_OK ? status(st) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

PyObject* attention_decode(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    NARGS(13);
    const Tensor q = tensor_of(a[0], "q"), kc = tensor_of(a[1], "k_cache"), vc = tensor_of(a[2], "v_cache"),
                 ks = tensor_of(a[3], "k_scale"), vs = tensor_of(a[4], "v_scale"),
                 table = tensor_of(a[5], "block_table"), lens = tensor_of(a[6], "seq_lens");
    const int64_t page = int_of(a[7], "page_size"), prefix = int_of(a[8], "prefix_len");
    Tensor out = tensor_of(a[10], "out"), ws = tensor_of(a[11], "workspace");
    const int64_t ldq = tokens(q, "q");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    expect(kc, "k_cache", at::kByte, {-1, -1, D});
    const int64_t Hkv = kc.size(1), slots = cache_slots(kc, vc, Hkv, D);
    const int64_t stride = scale_stride(ks, "k_scale", Hkv);
    TORCH_CHECK_VALUE(scale_stride(vs, "v_scale", Hkv) == stride,
                      "k_scale and v_scale must both be per head or both single");
    const int64_t ld = table_stride(table, B), width = table.size(1);
    expect(lens, "seq_lens", at::kInt, {B});
    const float scale = softmax_scale(a[9], D);
    const Place place(q, a[12]);
    int64_t ldo = Hq * D;
    if (!out.defined()) out = make({B, Hq, D}, at::kBFloat16, q);
    else ldo = tokens(out, "out", {B, Hq, D});
    if (!ws.defined()) {
        const size_t need = fp8_attention_decode_workspace_size(B, Hq, Hkv, D, width, page, prefix);
        ws = make({static_cast<int64_t>(need ? need : 1)}, at::kByte, q);
    } else {
        expect(ws, "workspace", at::kByte, {-1});
    }
    same_device(q, {&kc, &vc, &ks, &vs, &table, &lens, &out, &ws});
    const fp8_status_t st = fp8_attention_decode(
        ptr(q), ldq, B, Hq, Hkv, D, static_cast<const uint8_t*>(ptr(kc)),
        static_cast<const uint8_t*>(ptr(vc)), slots, static_cast<const float*>(ptr(ks)),
        static_cast<const float*>(ptr(vs)), stride, static_cast<const int32_t*>(ptr(table)), width, ld, page,
        static_cast<const int32_t*>(ptr(lens)), prefix, scale, ptr(out), ldo, ptr(ws),
        static_cast<size_t>(ws.numel()), place.stream);
    return st != FP8_OK ? status(st) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(kv_slots), METHOD(qk_norm_rope), METHOD(attention_prompt),
                         METHOD(attention_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fp8_attention_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fp8_attention_binding() { return PyModule_Create(&module); }
