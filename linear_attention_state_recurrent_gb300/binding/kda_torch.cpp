// The calls around the recurrence for torch tensors, as a CPython module: checks of the
// arguments and nothing else, then the C entry point. These kernels run in a few microseconds,
// and the same checks in Python cost 8 us a call on the GPU machine's cores where this costs 3.
//
// Every function takes its arguments by position and returns the outputs, or the C entry
// point's status as an int where that is not KDA_OK; arguments that it does not accept raise
// ValueError.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kda.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *refuse(const char *format, ...)
{
    va_list ap;
    va_start(ap, format);
    PyErr_FormatV(PyExc_ValueError, format, ap);
    va_end(ap);
    return nullptr;
}

// A tensor argument; `none`: whether None is accepted (then *t stays null).
bool tensor(PyObject *o, const char *name, bool none, const Tensor **t)
{
    *t = nullptr;
    if (o == Py_None && none) return true;
    if (!THPVariable_Check(o)) {
        refuse("%s must be a tensor", name);
        return false;
    }
    *t = &THPVariable_Unpack(o);
    return true;
}

bool on_device(const Tensor &t, const char *name, const Tensor *first)
{
    if (!t.is_cuda()) {
        refuse("%s must be on the GPU", name);
        return false;
    }
    if (first && t.device() != first->device()) {
        refuse("%s must be on the device of the other tensors", name);
        return false;
    }
    return true;
}

bool of_type(const Tensor &t, const char *name, ScalarType type)
{
    if (t.scalar_type() == type) return true;
    refuse("%s must be %s (got %s)", name, c10::toString(type), c10::toString(t.scalar_type()));
    return false;
}

// The row stride of a [rows, cols] tensor with unit inner stride; the stride of a single row says nothing.
bool matrix(const Tensor &t, const char *name, ScalarType type, int64_t rows, int64_t cols, const Tensor *first, int64_t *ld)
{
    if (!of_type(t, name, type)) return false;
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) {
        refuse("%s must be [%lld, %lld]", name, (long long)rows, (long long)cols);
        return false;
    }
    if (cols > 1 && t.stride(1) != 1) {
        refuse("%s must have unit inner stride", name);
        return false;
    }
    *ld = rows > 1 || t.stride(0) > cols ? t.stride(0) : cols;
    return on_device(t, name, first);
}

bool scales_of(const Tensor &t, const char *name, int64_t rows, int64_t groups, const Tensor *first, int64_t *row, int64_t *group)
{
    if (!of_type(t, name, ScalarType::Float)) return false;
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != groups) {
        refuse("%s must be [%lld, %lld]", name, (long long)rows, (long long)groups);
        return false;
    }
    *row = rows > 1 ? t.stride(0) : 1;
    *group = groups > 1 ? t.stride(1) : 1;
    return on_device(t, name, first);
}

bool vector(const Tensor &t, const char *name, ScalarType type, int64_t n, const Tensor *first)
{
    if (!of_type(t, name, type)) return false;
    if (t.dim() != 1 || t.size(0) < n || !t.is_contiguous()) {
        refuse("%s must be contiguous and 1-D with at least %lld entries", name, (long long)n);
        return false;
    }
    return on_device(t, name, first);
}

bool error_word(PyObject *o, const Tensor *first, uint32_t **p)
{
    const Tensor *t;
    *p = nullptr;
    if (!tensor(o, "err_flags", true, &t)) return false;
    if (!t) return true;
    if ((t->scalar_type() != ScalarType::Int && t->scalar_type() != ScalarType::UInt32) || t->numel() < 1) {
        refuse("err_flags must be a 32-bit integer tensor");
        return false;
    }
    *p = static_cast<uint32_t *>(t->data_ptr());
    return on_device(*t, "err_flags", first);
}

bool integer(PyObject *o, int64_t *v)
{
    *v = PyLong_AsLongLong(o);
    return !(*v == -1 && PyErr_Occurred());
}

// The stream: a raw handle, or None for the device's current one.
bool stream_of(PyObject *o, const Tensor &t, void **s)
{
    if (o == Py_None) {
        *s = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
        return true;
    }
    *s = PyLong_AsVoidPtr(o);
    return !(*s == nullptr && PyErr_Occurred());
}

// KDA_BF16 .. KDA_FP32, or -1
int code_of(ScalarType t)
{
    return t == ScalarType::BFloat16 ? KDA_BF16 : t == ScalarType::Half ? KDA_FP16 : t == ScalarType::Float ? KDA_FP32 : -1;
}

constexpr ScalarType E4M3 = ScalarType::Float8_e4m3fn;

bool count(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return false;
}

// (x, weight, eps, residual, residual_out, y, q, scales, stream) -> (q, scales, residual_out)
PyObject *norm_quant(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const Tensor *x, *weight, *res, *res_out, *y, *q, *scales;
    if (!count(n, 9) || !tensor(a[0], "x", false, &x) || !tensor(a[1], "weight", true, &weight) || !tensor(a[3], "residual", true, &res) ||
        !tensor(a[4], "residual_out", true, &res_out) || !tensor(a[5], "y", true, &y) || !tensor(a[6], "q", true, &q) ||
        !tensor(a[7], "scales", true, &scales))
        return nullptr;
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const ScalarType type = x->scalar_type();
    const int code = code_of(type);
    if (x->dim() != 2 || code < 0) return refuse("x must be a 2-D bf16, fp16 or fp32 tensor");
    const int64_t N = x->size(0), D = x->size(1), groups = (D + 127) / 128;
    int64_t ld_x, ld_res = 0, ld_ro = 0, ld_y = 0, ld_q, s_row, s_group;
    if (!matrix(*x, "x", type, N, D, nullptr, &ld_x)) return nullptr;
    if (!res && res_out) return refuse("residual_out needs a residual");
    if (res && !matrix(*res, "residual", type, N, D, x, &ld_res)) return nullptr;
    if (res_out && !matrix(*res_out, "residual_out", type, N, D, x, &ld_ro)) return nullptr;
    if (y && !matrix(*y, "y", type, N, D, x, &ld_y)) return nullptr;
    if (weight && (!vector(*weight, "weight", ScalarType::Float, D, x) || weight->size(0) != D))
        return PyErr_Occurred() ? nullptr : refuse("weight must have %lld entries", (long long)D);
    if (q && !matrix(*q, "q", E4M3, N, D, x, &ld_q)) return nullptr;
    if (scales && !scales_of(*scales, "scales", N, groups, x, &s_row, &s_group)) return nullptr;
    const c10::cuda::CUDAGuard guard(x->device());
    void *stream;
    if (!stream_of(a[8], *x, &stream)) return nullptr;
    // what is allocated below belongs to the stream that the kernel runs on
    c10::cuda::OptionalCUDAStreamGuard on;
    if (a[8] != Py_None) on.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), x->device().index()));
    Tensor made_q, made_s, made_r;
    if (!q) {   // rows on 16-byte boundaries
        ld_q = (D + 15) / 16 * 16;
        made_q = at::empty({N, ld_q}, x->options().dtype(E4M3)).narrow(1, 0, D);
        q = &made_q;
    }
    if (!scales) {   // the rows of a group next to each other
        made_s = at::empty({groups, N}, x->options().dtype(ScalarType::Float)).t();
        scales = &made_s;
        s_row = 1;
        s_group = N > 1 ? N : 1;
    }
    if (res && !res_out) {
        made_r = at::empty({N, D}, x->options());
        res_out = &made_r;
        ld_ro = D;
    }
    const int status = kda_norm_quant(
        x->data_ptr(), ld_x, res ? res->data_ptr() : nullptr, ld_res, code,
        weight ? static_cast<const float *>(weight->data_ptr()) : nullptr, static_cast<float>(eps), N, D,
        res ? res_out->data_ptr() : nullptr, ld_ro, y ? y->data_ptr() : nullptr, ld_y, static_cast<uint8_t *>(q->data_ptr()), ld_q,
        static_cast<float *>(scales->data_ptr()), s_row, s_group, stream);
    if (status != KDA_OK) return PyLong_FromLong(status);
    PyObject *out = PyTuple_New(3);
    if (!out) return nullptr;
    auto give = [&](Py_ssize_t i, PyObject *given, const Tensor &made) {
        PyObject *o = made.defined() ? THPVariable_Wrap(made) : Py_NewRef(given);
        PyTuple_SET_ITEM(out, i, o);
        return o != nullptr;
    };
    if (!give(0, a[6], made_q) || !give(1, a[7], made_s) || !give(2, a[4], made_r)) {
        Py_DECREF(out);
        return nullptr;
    }
    return out;
    END_HANDLE_TH_ERRORS
}

// (a, a_scales, w, w_scales, out, err_flags, stalled, stream) -> out; stalled: None, or the self-test's
PyObject *fp8_matmul(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const Tensor *a, *sa, *w, *sw, *out;
    if (!count(n, 8) || !tensor(v[0], "a", false, &a) || !tensor(v[1], "a_scales", false, &sa) || !tensor(v[2], "w", false, &w) ||
        !tensor(v[3], "w_scales", false, &sw) || !tensor(v[4], "out", false, &out))
        return nullptr;
    if (a->dim() != 2 || w->dim() != 2) return refuse("a and w must be 2-D with the same number of columns");
    const int64_t M = a->size(0), K = a->size(1), N = w->size(0), groups = (K + 127) / 128;
    const int code = code_of(out->scalar_type());
    if (code < 0) return refuse("out must be bf16, fp16 or fp32");
    int64_t ld_a, ld_w, ld_out, sa_row, sa_group, sw_row, sw_group;
    int64_t stalled = 0;
    uint32_t *err;
    void *stream;
    if (!matrix(*a, "a", E4M3, M, K, nullptr, &ld_a) || !matrix(*w, "w", E4M3, N, K, a, &ld_w) ||
        !scales_of(*sa, "a_scales", M, groups, a, &sa_row, &sa_group) ||
        !scales_of(*sw, "w_scales", (N + 127) / 128, groups, a, &sw_row, &sw_group) ||
        !matrix(*out, "out", out->scalar_type(), M, N, a, &ld_out) || !error_word(v[5], a, &err) ||
        (v[6] != Py_None && !integer(v[6], &stalled)) || !stream_of(v[7], *a, &stream))
        return nullptr;
    if (stalled < 0 || stalled > 7) return refuse("stalled must be in [0, 7]");
    const c10::cuda::CUDAGuard guard(a->device());
    const auto pa = static_cast<const uint8_t *>(a->data_ptr()), pw = static_cast<const uint8_t *>(w->data_ptr());
    const auto psa = static_cast<const float *>(sa->data_ptr()), psw = static_cast<const float *>(sw->data_ptr());
    const int status = v[6] == Py_None ? kda_fp8_matmul(pa, ld_a, psa, sa_row, sa_group, pw, ld_w, psw, sw_row, sw_group, M, N, K,
                                                        out->data_ptr(), ld_out, code, err, stream)
                                       : kda_selftest_fp8_matmul(pa, ld_a, psa, sa_row, sa_group, pw, ld_w, psw, sw_row, sw_group, M, N,
                                                                 K, out->data_ptr(), ld_out, code, static_cast<int32_t>(stalled), err, stream);
    if (status != KDA_OK) return PyLong_FromLong(status);
    return Py_NewRef(v[4]);
    END_HANDLE_TH_ERRORS
}

// (query_lens, context_lens, state_slots, block_table, free_pages, free_count, page_size, num_pages,
//  out (tuple of seven), err_flags, stream) -> out
PyObject *batch_maps(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const Tensor *q, *c, *slots, *table, *pages, *left;
    int64_t page, num_pages;
    if (!count(n, 11) || !tensor(v[0], "query_lens", false, &q) || !tensor(v[1], "context_lens", false, &c) ||
        !tensor(v[2], "state_slots", false, &slots) || !tensor(v[3], "block_table", false, &table) ||
        !tensor(v[4], "free_pages", false, &pages) || !tensor(v[5], "free_count", false, &left) || !integer(v[6], &page) ||
        !integer(v[7], &num_pages))
        return nullptr;
    if (page < INT32_MIN || page > INT32_MAX) return refuse("page_size is out of range");
    if (!PyTuple_Check(v[8]) || PyTuple_GET_SIZE(v[8]) != 7) return refuse("out must be a BatchMaps");
    const Tensor *o[7];
    static const char *const names[7] = {"out.order", "out.cu_seqlens", "out.state_indices", "out.num_decodes", "out.positions",
                                         "out.slot_map", "out.free_left"};
    for (int i = 0; i < 7; i++)
        if (!tensor(PyTuple_GET_ITEM(v[8], i), names[i], false, &o[i])) return nullptr;
    if (q->dim() != 1) return refuse("query_lens must be 1-D");
    const ScalarType I = ScalarType::Int;
    const int64_t R = q->size(0), tokens = o[4]->dim() == 1 ? o[4]->size(0) : 0;
    const int64_t need[7] = {R, R + 1, R, 1, 0, tokens, 1};
    if (!vector(*q, "query_lens", I, R, nullptr) || !vector(*c, "context_lens", I, R, q) || !vector(*pages, "free_pages", I, 0, q) ||
        !vector(*left, "free_count", I, 1, q))
        return nullptr;
    for (int i = 0; i < 7; i++)
        if (!vector(*o[i], names[i], i == 5 ? ScalarType::Long : I, need[i], q)) return nullptr;
    if (!of_type(*slots, "state_slots", I) || !on_device(*slots, "state_slots", q)) return nullptr;
    if (slots->dim() != 1 || slots->size(0) < R) return refuse("state_slots must be 1-D with an entry per request");
    if (!of_type(*table, "block_table", I) || !on_device(*table, "block_table", q)) return nullptr;
    if (table->dim() != 2 || table->size(0) < R || (table->size(1) > 1 && table->stride(1) != 1))
        return refuse("block_table must be [num_reqs, width] with unit inner stride");
    const int64_t width = table->size(1);
    uint32_t *err;
    void *stream;
    if (!error_word(v[9], q, &err) || !stream_of(v[10], *q, &stream)) return nullptr;
    const c10::cuda::CUDAGuard guard(q->device());
    auto i32 = [](const Tensor *t) { return static_cast<int32_t *>(t->data_ptr()); };
    const int status = kda_batch_maps(i32(q), i32(c), i32(slots), R > 1 ? slots->stride(0) : 1, R, i32(table),
                                      R > 1 ? table->stride(0) : (width > 1 ? width : 1), width, i32(pages), pages->size(0), i32(left),
                                      num_pages, static_cast<int32_t>(page), tokens, i32(o[0]), i32(o[1]), i32(o[2]), i32(o[3]),
                                      i32(o[4]), static_cast<int64_t *>(o[5]->data_ptr()), i32(o[6]), err, stream);
    if (status != KDA_OK) return PyLong_FromLong(status);
    return Py_NewRef(v[8]);
    END_HANDLE_TH_ERRORS
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"norm_quant", FAST(norm_quant), nullptr},
                         {"fp8_matmul", FAST(fp8_matmul), nullptr},
                         {"batch_maps", FAST(batch_maps), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_torch() { return PyModule_Create(&module); }
