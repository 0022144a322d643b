// py_calls.cpp -- the calls of the training operators, of windowed attention and of
// the paged cache from Python, as a CPython extension module: argument checks, output and workspace allocation through
// PyTorch, and one call of the C ABI (include/dit_attn.h).
//
// Marshalling only.  A small call's time is its host time: through ctypes a
// single-token rotation cost 15 us and the backward pass of a small attention
// 41 us on the GB300's host cores, most of it Python statements and argument
// conversions.  Every function returns the C status with its results; binding.py
// turns a status other than DIT_OK into DitError.  The library's functions are
// handed over by bind(), so that the debug library can take the product
// library's place.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/types.h>

#include <cmath>
#include <cstdint>
#include <exception>
#include <optional>
#include <vector>

#include "dit_attn.h"

namespace {

decltype(&dit_attn_bwd) g_attn_bwd;
decltype(&dit_attn_bwd_masked) g_attn_bwd_masked;
decltype(&dit_attn_bwd_workspace_bytes) g_attn_bwd_ws;
decltype(&dit_layer_norm_fwd) g_norm_fwd;
decltype(&dit_layer_norm_bwd) g_norm_bwd;
decltype(&dit_layer_norm_bwd_workspace_bytes) g_norm_bwd_ws;
decltype(&dit_rope) g_rope;
decltype(&dit_attn_fwd_window) g_window_fwd;
decltype(&dit_attn_fwd_window_workspace_bytes) g_window_fwd_ws;
decltype(&dit_attn_bwd_window) g_window_bwd;
decltype(&dit_attn_bwd_window_workspace_bytes) g_window_bwd_ws;
decltype(&dit_paged_append) g_append;
decltype(&dit_attn_fwd_paged) g_paged;
decltype(&dit_attn_fwd_paged_workspace_bytes) g_paged_ws;

// A failed check, carried to the function's end.
struct Refused {
    PyObject* type;
    const char* what;
};
[[noreturn]] void type_error(const char* what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const char* what) { throw Refused{PyExc_ValueError, what}; }
[[noreturn]] void python_error() { throw Refused{nullptr, nullptr}; }

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) type_error(what);
    return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }
long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) python_error();
    return v;
}
int small_int(PyObject* o) {
    const long long v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) value_error("an integer argument is out of range");
    return static_cast<int>(v);
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) python_error();
    return v;
}
dit_stream_t stream_of(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) python_error();
    return reinterpret_cast<dit_stream_t>(p);
}

bool is(const at::Tensor& t, at::ScalarType s) { return t.scalar_type() == s; }
bool bf16_or_f32(const at::Tensor& t) { return is(t, at::kBFloat16) || is(t, at::kFloat); }
dit_dtype_t code(const at::Tensor& t) { return is(t, at::kFloat) ? DIT_F32 : DIT_BF16; }
int extent(int64_t n) {
    if (n > INT32_MAX) value_error("a dimension is out of range");
    return static_cast<int>(n);
}
template <typename T>
T* data(const at::Tensor* t) {
    return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}
dit_strides4_t strides4(const at::Tensor& t) {
    const auto s = t.strides();
    return s.size() == 4 ? dit_strides4_t{s[0], s[1], s[2], s[3]} : dit_strides4_t{s[0], s[1], s[1], s[2]};
}
bool contiguous_f32(const at::Tensor& t, at::IntArrayRef shape) {
    return is(t, at::kFloat) && t.sizes() == shape && t.is_contiguous();
}
// (PyTorch's allocation without its dispatcher: 0.3 to 0.5 us less a tensor)
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
// f() with the interpreter's lock let go: allocations and launches can wait for
// the device, and other Python threads run meanwhile.  f touches no Python object
// and takes no reference of a tensor that has one.
template <typename F>
int unlocked(F&& f) {
    struct Lock {
        PyThreadState* const state = PyEval_SaveThread();
        ~Lock() { PyEval_RestoreThread(state); }
    } lock;
    return f();
}
// (status, tensors...), None for those not there
PyObject* result(int status, std::initializer_list<const at::Tensor*> ts) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(1 + ts.size()));
    if (r == nullptr) python_error();
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
    Py_ssize_t i = 1;
    for (const at::Tensor* t : ts)
        PyTuple_SET_ITEM(r, i++, t == nullptr ? Py_NewRef(Py_None) : THPVariable_Wrap(*t));
    return r;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused& r) {
        if (r.type != nullptr) PyErr_SetString(r.type, r.what);
    } catch (...) {      // PyTorch's own, as the Python errors its functions raise (torch.OutOfMemoryError)
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// left, right, sinks, frame at a[0..3]; None: no bound on that side.
dit_window_t window_of(PyObject* const* a) {
    dit_window_t w;
    w.left = a[0] == Py_None ? -1 : small_int(a[0]);
    w.right = a[1] == Py_None ? -1 : small_int(a[1]);
    w.sinks = small_int(a[2]);
    w.frame = small_int(a[3]);
    if ((a[0] != Py_None && w.left < 0) || (a[1] != Py_None && w.right < 0)) value_error("left and right are None or at least 0");
    if (w.sinks < 0 || w.frame < 1) value_error("sinks must be at least 0 and frame at least 1");
    return w;
}
float scale_of(PyObject* o, int D) {
    return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D > 0 ? D : 1))) : static_cast<float>(real(o));
}

// attn_bwd(q, k, v, out, lse, dout, dlse, mask_bits, mask_rows, key_valid_len, scale,
//          dq, dk, dv, grads_fp32, workspace, stream); None where there is none.
// With a window: its heads may share K and V, q begins at `offset`.
PyObject* attn_bwd_of(PyObject* const* a, const dit_window_t* window, int offset) {
    const char* kIn = "q, k, v and dout must be bf16 CUDA tensors";
    const at::Tensor &q = tensor(a[0], kIn), &k = tensor(a[1], kIn), &v = tensor(a[2], kIn), &dout = tensor(a[5], kIn);
    const at::Tensor& out = tensor(a[3], "out must be a tensor");
    const at::Tensor& lse = tensor(a[4], "lse must be a tensor");
    const at::Tensor* dlse = maybe(a[6], "dlse must be a tensor");
    const at::Tensor* mask = maybe(a[7], "mask_bits must be a tensor");
    for (const at::Tensor* t : {&q, &k, &v, &dout})
        if (!is(*t, at::kBFloat16) || !t->is_cuda()) type_error(kIn);
    if (q.dim() != 4 || k.dim() != 4) value_error("q, k and v must be [B, N, H, D]");
    const int B = extent(q.size(0)), Nq = extent(q.size(1)), H = extent(q.size(2)), D = extent(q.size(3));
    const int Nkv = extent(k.size(1));
    const int Hkv = extent(k.size(2));
    if (k.size(0) != B || (window == nullptr && Hkv != H) || k.size(3) != D || v.sizes() != k.sizes() || dout.sizes() != q.sizes())
        value_error("k and v must be [B, Nkv, H, D] matching q, dout [B, Nq, H, D]");
    if (!bf16_or_f32(out) || out.sizes() != q.sizes()) value_error("out must be a [B, Nq, H, D] fp32 or bf16 tensor");
    const int64_t rows[3] = {B, H, Nq};
    if (!contiguous_f32(lse, rows) || (dlse != nullptr && !contiguous_f32(*dlse, rows)))
        value_error("lse and dlse must be contiguous fp32 [B, H, Nq] tensors");
    const int kvl = a[9] == Py_None ? Nkv : small_int(a[9]);
    int mask_rows = 0;
    if (mask != nullptr) {
        if (!is(*mask, at::kInt) || mask->dim() != 3 || !mask->is_cuda() || (mask->size(2) > 1 && mask->stride(2) != 1))
            value_error("mask_bits must be an int32 CUDA tensor [B or 1, rows, words], words contiguous");
        if (mask->size(0) != 1 && mask->size(0) != B) value_error("mask_bits must have B or 1 batch entries");
        mask_rows = a[8] == Py_None ? extent(mask->size(1)) : small_int(a[8]);
        if (mask_rows > mask->size(1)) value_error("mask_rows exceeds the mask's rows");
        if (kvl >= 0 && 4 * ((static_cast<int64_t>(kvl) + 127) / 128) > mask->size(2))
            value_error("mask_bits must have 4 * ceil(key_valid_len / 128) words a row");
    }
    const float scale = scale_of(a[10], D);
    const at::Tensor* given[3] = {maybe(a[11], "dq must be a tensor"), maybe(a[12], "dk must be a tensor"),
                                  maybe(a[13], "dv must be a tensor")};
    at::ScalarType type = integer(a[14]) ? at::kFloat : at::kBFloat16;
    for (const at::Tensor* g : given)
        if (g != nullptr) {
            type = g->scalar_type();
            break;
        }
    at::Tensor grads[3];
    for (int i = 0; i < 3; ++i)
        if (given[i] != nullptr) {
            if (!bf16_or_f32(*given[i]) || !is(*given[i], type) || given[i]->sizes() != (i == 0 ? q : k).sizes())
                value_error("dq must be [B, Nq, H, D], dk and dv [B, Nkv, H, D] tensors of one type, fp32 or bf16");
            grads[i] = *given[i];
        }
    const at::Tensor* workspace = maybe(a[15], "workspace must be a tensor");
    const dit_stream_t stream = stream_of(a[16]);
    at::Tensor own;
    const int rc = unlocked([&] {
        for (int i = 0; i < 3; ++i)
            if (given[i] == nullptr) grads[i] = fresh((i == 0 ? q : k).sizes(), type, q);
        size_t ws_bytes = 0;
        if (workspace != nullptr) {
            ws_bytes = workspace->nbytes();
        } else if ((ws_bytes = window != nullptr ? g_window_bwd_ws(B, Nq, Nkv, H, Hkv, D, kvl, window, offset)
                                                 : g_attn_bwd_ws(B, Nq, Nkv, H, D, kvl, mask != nullptr)) > 0) {
            own = fresh({static_cast<int64_t>(ws_bytes)}, at::kByte, q);
            workspace = &own;
        }
        const dit_attn_bwd_strides_t st{strides4(q),        strides4(k),        strides4(v),        strides4(out), strides4(dout),
                                        strides4(grads[0]), strides4(grads[1]), strides4(grads[2])};
        const dit_dtype_t gt = type == at::kFloat ? DIT_F32 : DIT_BF16;
        if (window != nullptr)
            return g_window_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), code(out), data<float>(&lse),
                                dout.data_ptr(), data<float>(dlse), &st, B, Nq, Nkv, H, Hkv, D, kvl, window, offset, scale,
                                grads[0].data_ptr(), grads[1].data_ptr(), grads[2].data_ptr(), gt, data<void>(workspace), ws_bytes,
                                stream);
        if (mask != nullptr)
            return g_attn_bwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), code(out), data<float>(&lse),
                                     dout.data_ptr(), data<float>(dlse), &st, B, Nq, Nkv, H, D, kvl, data<uint32_t>(mask),
                                     mask->size(0) == 1 ? 0 : mask->stride(0), mask->stride(1), mask_rows, scale,
                                     grads[0].data_ptr(), grads[1].data_ptr(), grads[2].data_ptr(), gt,
                                     data<void>(workspace), ws_bytes, stream);
        return g_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), code(out), data<float>(&lse),
                          dout.data_ptr(), data<float>(dlse), &st, B, Nq, Nkv, H, D, kvl, scale, grads[0].data_ptr(),
                          grads[1].data_ptr(), grads[2].data_ptr(), gt, data<void>(workspace), ws_bytes, stream);
    });
    return result(rc, {&grads[0], &grads[1], &grads[2]});
}
PyObject* attn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&] { return attn_bwd_of(a, nullptr, 0); });
}
// window_bwd(left, right, sinks, frame, offset, then attn_bwd's arguments without a mask)
PyObject* window_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 22, [&] {
        const dit_window_t w = window_of(a);
        return attn_bwd_of(a + 5, &w, small_int(a[4]));
    });
}

// A forward call's results, given ones checked.
struct Results {
    at::Tensor out, lse;
    const at::Tensor *given_out, *given_lse;
    at::ScalarType type;
    Results(PyObject* o, PyObject* l, PyObject* fp32, const at::Tensor& q) {
        given_out = maybe(o, "out must be a tensor");
        given_lse = maybe(l, "lse must be a tensor");
        type = integer(fp32) ? at::kFloat : at::kBFloat16;
        const int64_t rows[3] = {q.size(0), q.size(2), q.size(1)};
        if (given_out != nullptr) {
            if (!bf16_or_f32(*given_out) || given_out->sizes() != q.sizes()) value_error("out must be a [B, N, H, D] fp32 or bf16 tensor");
            out = *given_out;
        }
        if (given_lse != nullptr) {
            if (!contiguous_f32(*given_lse, rows)) value_error("lse must be a contiguous fp32 [B, H, N] tensor");
            lse = *given_lse;
        }
    }
    void allocate(const at::Tensor& q) {
        if (given_out == nullptr) out = fresh(q.sizes(), type, q);
        if (given_lse == nullptr) lse = fresh({q.size(0), q.size(2), q.size(1)}, at::kFloat, q);
    }
};

// window_fwd(q, k, v, left, right, sinks, frame, offset, key_valid_len, scale, out, lse, out_fp32, workspace, stream)
PyObject* window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const char* kIn = "q, k and v must be bf16 CUDA tensors";
        const at::Tensor &q = tensor(a[0], kIn), &k = tensor(a[1], kIn), &v = tensor(a[2], kIn);
        for (const at::Tensor* t : {&q, &k, &v})
            if (!is(*t, at::kBFloat16) || !t->is_cuda()) type_error(kIn);
        if (q.dim() != 4 || k.dim() != 4) value_error("q, k and v must be [B, N, H, D]");
        const int B = extent(q.size(0)), Nq = extent(q.size(1)), H = extent(q.size(2)), D = extent(q.size(3));
        const int Nkv = extent(k.size(1)), Hkv = extent(k.size(2));
        if (k.size(0) != B || k.size(3) != D || v.sizes() != k.sizes()) value_error("k and v must be [B, Nkv, Hkv, D] matching q");
        const dit_window_t w = window_of(a + 3);
        const int offset = small_int(a[7]), kvl = a[8] == Py_None ? Nkv : small_int(a[8]);
        const float scale = scale_of(a[9], D);
        Results r(a[10], a[11], a[12], q);
        const at::Tensor* workspace = maybe(a[13], "workspace must be a tensor");
        const dit_stream_t stream = stream_of(a[14]);
        at::Tensor own;
        const int rc = unlocked([&] {
            r.allocate(q);
            size_t ws_bytes = 0;
            if (workspace != nullptr) {
                ws_bytes = workspace->nbytes();
            } else if ((ws_bytes = g_window_fwd_ws(B, Nq, H, Hkv, D, kvl, &w, offset)) > 0) {
                own = fresh({static_cast<int64_t>(ws_bytes)}, at::kByte, q);
                workspace = &own;
            }
            const dit_attn_strides_t st{strides4(q), strides4(k), strides4(v), strides4(r.out)};
            return g_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), &st, B, Nq, Nkv, H, Hkv, D, kvl, &w, offset, scale,
                                r.out.data_ptr(), code(r.out), data<float>(&r.lse), data<void>(workspace), ws_bytes, stream);
        });
        return result(rc, {&r.out, &r.lse});
    });
}

// The cache of k_cache, v_cache [pages, page, Hkv, D], page_table [B, width], kv_lens [B] at a[0..3].
dit_paged_cache_t cache_of(PyObject* const* a, int64_t B, int64_t D) {
    const char* kCache = "k_cache and v_cache must be bf16 CUDA tensors";
    const at::Tensor &k = tensor(a[0], kCache), &v = tensor(a[1], kCache);
    for (const at::Tensor* t : {&k, &v})
        if (!is(*t, at::kBFloat16) || !t->is_cuda()) type_error(kCache);
    if (k.dim() != 4 || v.sizes() != k.sizes() || k.size(3) != D) value_error("k_cache and v_cache must be [pages, page_size, Hkv, D]");
    const char* kTable = "page_table must be an int32 CUDA tensor [B, width], each row contiguous";
    const at::Tensor& table = tensor(a[2], kTable);
    if (!is(table, at::kInt) || !table.is_cuda()) type_error(kTable);
    if (table.dim() != 2 || table.size(0) != B || (table.size(1) > 1 && table.stride(1) != 1)) value_error(kTable);
    const char* kLens = "kv_lens must be a contiguous int32 CUDA tensor [B]";
    const at::Tensor& lens = tensor(a[3], kLens);
    if (!is(lens, at::kInt) || !lens.is_cuda()) type_error(kLens);
    if (lens.dim() != 1 || lens.size(0) != B || !lens.is_contiguous()) value_error(kLens);
    dit_paged_cache_t c;
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.k_strides = strides4(k);
    c.v_strides = strides4(v);
    c.pages = extent(k.size(0));
    c.page_size = extent(k.size(1));
    c.table = data<const int32_t>(&table);
    c.table_stride = table.stride(0);
    c.table_width = extent(table.size(1));
    c.kv_lens = data<const int32_t>(&lens);
    return c;
}
// An int32 [B] tensor of new tokens, or none.
const int32_t* counts_of(PyObject* o, int64_t B, const char* what) {
    const at::Tensor* t = maybe(o, what);
    if (t == nullptr) return nullptr;
    if (!is(*t, at::kInt) || !t->is_cuda()) type_error(what);
    if (t->dim() != 1 || t->size(0) != B || !t->is_contiguous()) value_error(what);
    return data<const int32_t>(t);
}

// append(k, v, k_cache, v_cache, page_table, kv_lens, new_lens, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        const char* kIn = "k and v must be bf16 CUDA tensors";
        const at::Tensor &k = tensor(a[0], kIn), &v = tensor(a[1], kIn);
        for (const at::Tensor* t : {&k, &v})
            if (!is(*t, at::kBFloat16) || !t->is_cuda()) type_error(kIn);
        if (k.dim() != 4 || v.sizes() != k.sizes()) value_error("k and v must be [B, T, Hkv, D] tensors of one shape");
        const int B = extent(k.size(0)), T = extent(k.size(1)), Hkv = extent(k.size(2)), D = extent(k.size(3));
        const dit_paged_cache_t c = cache_of(a + 2, B, D);
        if (tensor(a[2], kIn).size(2) != Hkv) value_error("k_cache and v_cache must have the heads of k and v");
        const int32_t* lens = counts_of(a[6], B, "new_lens must be a contiguous int32 CUDA tensor [B]");
        const dit_stream_t stream = stream_of(a[7]);
        const int rc = unlocked([&] {
            const dit_strides4_t sk = strides4(k), sv = strides4(v);
            return g_append(k.data_ptr(), &sk, v.data_ptr(), &sv, &c, lens, B, T, Hkv, D, stream);
        });
        return result(rc, {});
    });
}

// paged(q, k_cache, v_cache, page_table, kv_lens, q_lens, left, right, sinks, frame, scale, out, lse, out_fp32, workspace, stream)
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const char* kIn = "q must be a bf16 CUDA tensor";
        const at::Tensor& q = tensor(a[0], kIn);
        if (!is(q, at::kBFloat16) || !q.is_cuda()) type_error(kIn);
        if (q.dim() != 4) value_error("q must be [B, T, H, D]");
        const int B = extent(q.size(0)), T = extent(q.size(1)), H = extent(q.size(2)), D = extent(q.size(3));
        const dit_paged_cache_t c = cache_of(a + 1, B, D);
        const int Hkv = extent(tensor(a[1], kIn).size(2));
        const int32_t* lens = counts_of(a[5], B, "q_lens must be a contiguous int32 CUDA tensor [B]");
        const dit_window_t w = window_of(a + 6);
        const float scale = scale_of(a[10], D);
        Results r(a[11], a[12], a[13], q);
        const at::Tensor* workspace = maybe(a[14], "workspace must be a tensor");
        const dit_stream_t stream = stream_of(a[15]);
        at::Tensor own;
        const int rc = unlocked([&] {
            r.allocate(q);
            size_t ws_bytes = 0;
            if (workspace != nullptr) {
                ws_bytes = workspace->nbytes();
            } else if ((ws_bytes = g_paged_ws(B, T, H, Hkv, D, c.page_size, c.table_width, &w)) > 0) {
                own = fresh({static_cast<int64_t>(ws_bytes)}, at::kByte, q);
                workspace = &own;
            }
            const dit_strides4_t sq = strides4(q), so = strides4(r.out);
            return g_paged(q.data_ptr(), &sq, &c, lens, B, T, H, Hkv, D, &w, scale, r.out.data_ptr(), code(r.out), &so,
                           data<float>(&r.lse), data<void>(workspace), ws_bytes, stream);
        });
        return result(rc, {&r.out, &r.lse});
    });
}

// B, N, H, C of a [B, N, C] or [B, N, H, C] tensor.
struct Rows {
    int B, N, H, C;
    explicit Rows(const at::Tensor& t) {
        if (t.dim() != 3 && t.dim() != 4) value_error("expected a [B, N, C] or [B, N, H, C] tensor");
        B = extent(t.size(0));
        N = extent(t.size(1));
        H = t.dim() == 4 ? extent(t.size(2)) : 1;
        C = extent(t.size(-1));
    }
};
// The parameter sets of weight-like tensors, [C] or [B, C], all of one shape.
int param_batches(const Rows& r, std::initializer_list<const at::Tensor*> ps) {
    const at::Tensor* one = nullptr;
    for (const at::Tensor* p : ps) {
        if (p == nullptr) continue;
        const bool whole = p->dim() == 1 && p->size(0) == r.C;
        const bool each = p->dim() == 2 && p->size(0) == r.B && p->size(1) == r.C;
        if (!is(*p, at::kFloat) || !p->is_contiguous() || (!whole && !each))
            value_error("weight, bias and their gradients must be contiguous fp32 [C] or [B, C] tensors");
        if (one != nullptr && one->sizes() != p->sizes()) value_error("weight, bias and their gradients must have one shape");
        one = p;
    }
    return one != nullptr && one->dim() == 2 ? r.B : 1;
}

// norm_fwd(x, weight, bias, eps, center, out, out_fp32, stream); out_fp32 None: x's type
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        const char* kX = "x must be a bf16 or fp32 CUDA tensor";
        const at::Tensor& x = tensor(a[0], kX);
        if (!bf16_or_f32(x) || !x.is_cuda()) type_error(kX);
        const Rows r(x);
        const at::Tensor *weight = maybe(a[1], "weight must be a tensor"), *bias = maybe(a[2], "bias must be a tensor");
        const int groups = param_batches(r, {weight, bias});
        const float eps = static_cast<float>(real(a[3]));
        const bool center = integer(a[4]) != 0;
        const at::Tensor* given = maybe(a[5], "out must be a tensor");
        if (given != nullptr && (!bf16_or_f32(*given) || given->sizes() != x.sizes()))
            value_error("out must have x's shape, bf16 or fp32");
        const at::ScalarType type = a[6] == Py_None ? x.scalar_type() : (integer(a[6]) ? at::kFloat : at::kBFloat16);
        const dit_stream_t stream = stream_of(a[7]);
        at::Tensor y, mean, rstd;
        if (given != nullptr) y = *given;
        const int rc = unlocked([&] {
            if (given == nullptr) y = fresh(x.sizes(), type, x);
            const at::IntArrayRef rows = x.sizes().slice(0, x.dim() - 1);
            rstd = fresh(rows, at::kFloat, x);
            if (center) mean = fresh(rows, at::kFloat, x);
            const dit_strides4_t sx = strides4(x), sy = strides4(y);
            return g_norm_fwd(x.data_ptr(), code(x), &sx, r.B, r.N, r.H, r.C, data<float>(weight), data<float>(bias), groups, eps,
                              center, y.data_ptr(), code(y), &sy, center ? data<float>(&mean) : nullptr, data<float>(&rstd), stream);
        });
        return result(rc, {&y, center ? &mean : nullptr, &rstd});
    });
}

// norm_bwd(dy, x, mean, rstd, weight, has_bias, dx, dweight, dbias, workspace, stream)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const char* kX = "x and dy must be bf16 or fp32 CUDA tensors";
        const at::Tensor &dy = tensor(a[0], kX), &x = tensor(a[1], kX);
        if (!bf16_or_f32(x) || !x.is_cuda() || !bf16_or_f32(dy) || !dy.is_cuda()) type_error(kX);
        const Rows r(x);
        if (dy.sizes() != x.sizes()) value_error("dy must have x's shape");
        const at::Tensor* mean = maybe(a[2], "mean must be a tensor");
        const at::Tensor& rstd = tensor(a[3], "rstd must be a tensor");
        const at::IntArrayRef rows = x.sizes().slice(0, x.dim() - 1);
        if (!contiguous_f32(rstd, rows) || (mean != nullptr && !contiguous_f32(*mean, rows)))
            value_error("mean and rstd must be contiguous fp32 tensors of x's shape without the channels");
        const at::Tensor* weight = maybe(a[4], "weight must be a tensor");
        const at::Tensor *given = maybe(a[6], "dx must be a tensor"), *dweight = maybe(a[7], "dweight must be a tensor"),
                         *dbias = maybe(a[8], "dbias must be a tensor");
        if (given != nullptr && (!is(*given, x.scalar_type()) || given->sizes() != x.sizes()))
            value_error("dx must have x's shape and type");
        const int groups = param_batches(r, {weight, dweight, dbias});
        const bool own_dw = weight != nullptr && dweight == nullptr;
        const bool own_db = weight != nullptr && dbias == nullptr && integer(a[5]) != 0;
        const at::Tensor* workspace = maybe(a[9], "workspace must be a tensor");
        const dit_stream_t stream = stream_of(a[10]);
        at::Tensor dx, dw, db, own;
        if (given != nullptr) dx = *given;
        const int rc = unlocked([&] {
            if (given == nullptr) dx = fresh(x.sizes(), x.scalar_type(), x);
            if (own_dw) {
                dw = fresh(weight->sizes(), at::kFloat, x);
                dweight = &dw;
            }
            if (own_db) {
                db = fresh(weight->sizes(), at::kFloat, x);
                dbias = &db;
            }
            size_t ws_bytes = workspace != nullptr ? workspace->nbytes() : 0;
            if (workspace == nullptr && (dweight != nullptr || dbias != nullptr) &&
                (ws_bytes = g_norm_bwd_ws(r.B, r.N, r.H, r.C, groups)) > 0) {
                own = fresh({static_cast<int64_t>(ws_bytes)}, at::kByte, x);
                workspace = &own;
            }
            const dit_strides4_t sdy = strides4(dy), sx = strides4(x), sdx = strides4(dx);
            return g_norm_bwd(dy.data_ptr(), code(dy), &sdy, x.data_ptr(), code(x), &sx, data<float>(mean), data<float>(&rstd),
                              data<float>(weight), r.B, r.N, r.H, r.C, groups, mean != nullptr, dx.data_ptr(), &sdx,
                              data<float>(dweight), data<float>(dbias), data<void>(workspace), ws_bytes, stream);
        });
        return result(rc, {&dx, dweight, dbias});
    });
}

// rope(x, inv_freq, positions, half, axis_pairs, offset, mscale, inverse, out, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const char* kX = "x must be a bf16 or fp32 CUDA tensor";
        const at::Tensor& x = tensor(a[0], kX);
        if (!bf16_or_f32(x) || !x.is_cuda()) type_error(kX);
        if (x.dim() != 4) value_error("x must be [B, N, H, D]");
        const Rows r(x);
        const char* kFreq = "inv_freq must be a contiguous one-dimensional fp64 CPU tensor";
        const at::Tensor& freq = tensor(a[1], kFreq);
        if (!is(freq, at::kDouble) || !freq.is_cpu() || freq.dim() != 1 || !freq.is_contiguous()) value_error(kFreq);
        const int pairs = extent(freq.size(0));
        if (pairs > INT32_MAX / 2) value_error("inv_freq is out of range");
        std::vector<int> axes;
        if (a[4] == Py_None) {
            axes.push_back(pairs);
        } else {
            PyObject* seq = PySequence_Fast(a[4], "axis_pairs must be a sequence of integers");
            if (seq == nullptr) python_error();
            const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
            long long sum = 0;
            bool fine = true;
            for (Py_ssize_t i = 0; fine && i < len; ++i) {
                const long long p = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
                if (p == -1 && PyErr_Occurred()) {
                    Py_DECREF(seq);
                    python_error();
                }
                fine = p >= 0 && p <= pairs;
                sum += p;
                axes.push_back(static_cast<int>(p));
            }
            Py_DECREF(seq);
            if (!fine || sum != pairs) value_error("axis_pairs must sum to the number of pairs");
        }
        const int64_t n_axes = static_cast<int64_t>(axes.size());
        const at::Tensor* pos = maybe(a[2], "positions must be an int32 CUDA tensor");
        int64_t pos_sb = 0;
        if (pos != nullptr) {
            if (!is(*pos, at::kInt) || !pos->is_cuda()) type_error("positions must be an int32 CUDA tensor");
            const bool flat = pos->dim() == 1 && n_axes == 1 && pos->size(0) == r.N;
            const bool full = pos->dim() == 3 && (pos->size(0) == 1 || pos->size(0) == r.B) && pos->size(1) == r.N && pos->size(2) == n_axes;
            if (!flat && !full) value_error("positions must be [N] (one axis) or [B or 1, N, axes]");
            const int64_t step_n = pos->stride(flat ? 0 : 1), step_a = flat ? 1 : pos->stride(2);
            if ((r.N > 1 && step_n != n_axes) || (n_axes > 1 && step_a != 1))
                value_error("each batch entry's positions must be contiguous");
            if (full && pos->size(0) > 1) pos_sb = pos->stride(0);
        }
        const at::Tensor* given = maybe(a[8], "out must be a tensor");
        if (given != nullptr && (!is(*given, x.scalar_type()) || given->sizes() != x.sizes()))
            value_error("out must have x's shape and type");
        const int64_t offset = integer(a[5]);
        const float mscale = static_cast<float>(real(a[6]));
        const dit_rope_layout_t layout = integer(a[3]) ? DIT_ROPE_HALF : DIT_ROPE_INTERLEAVED;
        const bool inverse = integer(a[7]) != 0;
        const dit_stream_t stream = stream_of(a[9]);
        const int axis_count = extent(n_axes);
        at::Tensor y;
        if (given != nullptr) y = *given;
        const int rc = unlocked([&] {
            if (given == nullptr) y = fresh(x.sizes(), x.scalar_type(), x);
            const dit_strides4_t sx = strides4(x), sy = strides4(y);
            return g_rope(x.data_ptr(), code(x), &sx, r.B, r.N, r.H, r.C, 2 * pairs, layout, data<const double>(&freq), axes.data(),
                          axis_count, data<const int32_t>(pos), pos_sb, offset, mscale, inverse, y.data_ptr(), &sy, stream);
        });
        return result(rc, {&y});
    });
}

// The seven addresses of a bind call.
void addresses(PyObject* const* a, void* (&p)[7]) {
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (PyErr_Occurred()) python_error();
            value_error("a function is missing");
        }
    }
}
// bind(addresses of the first seven C functions above, in that order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        void* p[7];
        addresses(a, p);
        g_attn_bwd = reinterpret_cast<decltype(g_attn_bwd)>(p[0]);
        g_attn_bwd_masked = reinterpret_cast<decltype(g_attn_bwd_masked)>(p[1]);
        g_attn_bwd_ws = reinterpret_cast<decltype(g_attn_bwd_ws)>(p[2]);
        g_norm_fwd = reinterpret_cast<decltype(g_norm_fwd)>(p[3]);
        g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[4]);
        g_norm_bwd_ws = reinterpret_cast<decltype(g_norm_bwd_ws)>(p[5]);
        g_rope = reinterpret_cast<decltype(g_rope)>(p[6]);
        return Py_NewRef(Py_None);
    });
}
// bind_streaming(addresses of the last seven, in that order)
PyObject* bind_streaming(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        void* p[7];
        addresses(a, p);
        g_window_fwd = reinterpret_cast<decltype(g_window_fwd)>(p[0]);
        g_window_fwd_ws = reinterpret_cast<decltype(g_window_fwd_ws)>(p[1]);
        g_window_bwd = reinterpret_cast<decltype(g_window_bwd)>(p[2]);
        g_window_bwd_ws = reinterpret_cast<decltype(g_window_bwd_ws)>(p[3]);
        g_append = reinterpret_cast<decltype(g_append)>(p[4]);
        g_paged = reinterpret_cast<decltype(g_paged)>(p[5]);
        g_paged_ws = reinterpret_cast<decltype(g_paged_ws)>(p[6]);
        return Py_NewRef(Py_None);
    });
}

#define DIT_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {DIT_METHOD(attn_bwd), DIT_METHOD(norm_fwd), DIT_METHOD(norm_bwd), DIT_METHOD(rope), DIT_METHOD(bind),
                          DIT_METHOD(window_fwd), DIT_METHOD(window_bwd), DIT_METHOD(append), DIT_METHOD(paged),
                          DIT_METHOD(bind_streaming),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "dit_calls", "calls of libditattn's operators", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_dit_calls() { return PyModule_Create(&kModule); }
