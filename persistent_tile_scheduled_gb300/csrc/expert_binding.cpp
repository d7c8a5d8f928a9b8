// The expert layer's calls from Python, as an extension module.
//
// A decoding step makes several of these calls for a few microseconds of GPU
// work each, so what a call costs the host counts: with the tensors checked in
// Python and the arguments passed through ctypes a sort takes 4.0 us, a 4-bit
// product 5.3; here they take 2.7 and 3.0, the launch being 1.5 of it.  Only
// checks and conversions live here; every rule on sizes is the C call's own.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <initializer_list>

#include "gemm_ctx.h"

namespace {

// torch.Tensor and its accessors, the dtypes, and what a refused tensor calls
// (it raises); set once by setup().
PyObject *g_tensor, *g_dtype, *g_device, *g_contiguous, *g_numel, *g_data_ptr, *g_refuse, *g_cuda_stream;
PyObject *g_elements[3], *g_i32, *g_f32, *g_u8;

PyObject *get(PyObject *accessor, PyObject *x)
{
    return Py_TYPE(accessor)->tp_descr_get(accessor, x, reinterpret_cast<PyObject *>(Py_TYPE(x)));
}

PyObject *call(PyObject *method, PyObject *x) { return PyObject_Vectorcall(method, &x, 1, nullptr); }

// The product of sizes; one below zero leaves it to the C call to refuse them.
int64_t product(std::initializer_list<int64_t> sizes)
{
    int64_t n = 1;
    for (const int64_t s : sizes) {
        if (s <= 0) return 0;
        if (__builtin_mul_overflow(n, s, &n)) n = INT64_MAX;
    }
    return n;
}

int64_t offsets_of(int64_t experts) { return experts < INT64_MAX ? experts + 1 : experts; }

// One call's arguments, taken in order; after the first that does not fit, an
// exception is set and nothing more is read.
class Args {
public:
    Args(PyObject *const *v, Py_ssize_t n, Py_ssize_t wanted) : v_(v)
    {
        ok_ = n == wanted;
        if (!ok_) PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, wanted);
    }
    bool ok() const { return ok_; }

    int64_t integer()
    {
        if (!ok_) return 0;
        const int64_t x = PyLong_AsLongLong(*v_++);
        if (x == -1 && PyErr_Occurred()) ok_ = false;
        return x;
    }

    float real()
    {
        if (!ok_) return 0.0f;
        const double x = PyFloat_AsDouble(*v_++);
        if (x == -1.0 && PyErr_Occurred()) ok_ = false;
        return static_cast<float>(x);
    }

    // a dtype of the library, and torch's for it
    gemm_dtype_t type(const char *what, PyObject **torch)
    {
        const int64_t d = integer();
        if (ok_ && (d < GEMM_F16 || d > GEMM_E4M3)) refuse(what, Py_None, Py_None, d);
        *torch = ok_ ? g_elements[d] : nullptr;
        return static_cast<gemm_dtype_t>(ok_ ? d : 0);
    }

    gemm_handle_t handle()
    {
        const auto h = static_cast<gemm_handle_t>(raw());
        if (h) device_ = h->device;
        return h;
    }

    void *raw()   // an address
    {
        if (!ok_) return nullptr;
        PyObject *x = *v_++;
        if (x == Py_None) return nullptr;
        void *p = PyLong_AsVoidPtr(x);
        if (p == nullptr && PyErr_Occurred()) ok_ = false;
        return p;
    }

    // a tensor's address; it must be contiguous, on the handle's GPU, of `dtype` and hold `count` elements
    void *array(PyObject *dtype, int64_t count, const char *what)
    {
        if (!ok_) return nullptr;
        PyObject *x = *v_;
        if (x == Py_None || PyLong_CheckExact(x)) return raw();
        ++v_;
        if (!PyObject_TypeCheck(x, reinterpret_cast<PyTypeObject *>(g_tensor))) return refuse(what, x, dtype, count);
        PyObject *type = get(g_dtype, x), *device = type ? call(g_device, x) : nullptr;
        PyObject *contiguous = device ? call(g_contiguous, x) : nullptr, *numel = contiguous ? call(g_numel, x) : nullptr;
        const int64_t at_device = numel ? PyLong_AsLongLong(device) : -1;   // (-1: on no GPU)
        const bool fits = numel && type == dtype && at_device >= 0 && (device_ < 0 || at_device == device_) && contiguous == Py_True
                          && PyLong_AsLongLong(numel) >= count;
        Py_XDECREF(type);
        Py_XDECREF(device);
        Py_XDECREF(contiguous);
        Py_XDECREF(numel);
        if (PyErr_Occurred()) return fail();
        if (!fits) return refuse(what, x, dtype, count);
        PyObject *at = call(g_data_ptr, x);
        if (!at) return fail();
        void *p = PyLong_AsVoidPtr(at);
        Py_DECREF(at);
        if (p == nullptr && PyErr_Occurred()) return fail();
        return p;
    }

    void *stream()
    {
        if (!ok_) return nullptr;
        if (*v_ == Py_None || PyLong_Check(*v_)) return raw();
        PyObject *s = PyObject_GetAttr(*v_++, g_cuda_stream);
        if (!s) return fail();
        void *p = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        if (p == nullptr && PyErr_Occurred()) return fail();
        return p;
    }

private:
    void *fail()
    {
        ok_ = false;
        return nullptr;
    }
    void *refuse(const char *what, PyObject *x, PyObject *dtype, int64_t count)
    {
        PyObject *r = PyObject_CallFunction(g_refuse, "sOOLi", what, x, dtype, static_cast<long long>(count), device_);
        Py_XDECREF(r);   // (it raises)
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, what);
        return fail();
    }

    PyObject *const *v_;
    bool ok_;
    int device_ = -1;   // the handle's
};

// Make the call without the interpreter's lock; its status as an int.
template <class F>
PyObject *run(const Args &a, F f)
{
    if (!a.ok()) return nullptr;
    gemm_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// The functions below take every argument of the C call, in its order but for
// the dtype, which comes first: the arrays' checks need it.

#define PTS_CALL(name_, count_)                                                   \
    PyObject *name_(PyObject *, PyObject *const *v, Py_ssize_t n)                 \
    {                                                                             \
        Args a(v, n, count_);

PTS_CALL(expert_sort, 9)
    const auto h = a.handle();
    const int64_t tokens = a.integer(), top_k = a.integer(), experts = a.integer(), m = product({tokens, top_k});
    const auto ids = static_cast<const int32_t *>(a.array(g_i32, m, "expert_ids"));
    const auto offsets = static_cast<int32_t *>(a.array(g_i32, offsets_of(experts), "offsets"));
    const auto row_of = static_cast<int32_t *>(a.array(g_i32, m, "row_of"));
    const auto src_of = static_cast<int32_t *>(a.array(g_i32, m, "src_of"));
    void *stream = a.stream();
    return run(a, [&] { return gemm_expert_sort(h, tokens, top_k, experts, ids, offsets, row_of, src_of, stream); });
}

PTS_CALL(expert_gather, 9)
    PyObject *t;
    const gemm_dtype_t dtype = a.type("gemm_expert_gather", &t);
    const auto h = a.handle();
    const int64_t tokens = a.integer(), top_k = a.integer(), dim = a.integer(), m = product({tokens, top_k});
    const void *X = a.array(t, product({tokens, dim}), "X");
    const auto row_of = static_cast<const int32_t *>(a.array(g_i32, m, "row_of"));
    void *Xs = a.array(t, product({m, dim}), "Xs");
    void *stream = a.stream();
    return run(a, [&] { return gemm_expert_gather(h, tokens, top_k, dim, X, row_of, Xs, dtype, stream); });
}

PTS_CALL(expert_combine, 10)
    PyObject *t;
    const gemm_dtype_t dtype = a.type("gemm_expert_combine", &t);
    const auto h = a.handle();
    const int64_t tokens = a.integer(), top_k = a.integer(), dim = a.integer(), m = product({tokens, top_k});
    const void *Ys = a.array(t, product({m, dim}), "Ys");
    const auto row_of = static_cast<const int32_t *>(a.array(g_i32, m, "row_of"));
    const auto weights = static_cast<const float *>(a.array(g_f32, m, "weights"));
    void *Y = a.array(t, product({tokens, dim}), "Y");
    void *stream = a.stream();
    return run(a, [&] { return gemm_expert_combine(h, tokens, top_k, dim, Ys, row_of, weights, Y, dtype, stream); });
}

PTS_CALL(expert_combine_grad, 12)
    PyObject *t;
    const gemm_dtype_t dtype = a.type("gemm_expert_combine_grad", &t);
    const auto h = a.handle();
    const int64_t tokens = a.integer(), top_k = a.integer(), dim = a.integer(), m = product({tokens, top_k});
    const void *dY = a.array(t, product({tokens, dim}), "dY"), *Ys = a.array(t, product({m, dim}), "Ys");
    const auto row_of = static_cast<const int32_t *>(a.array(g_i32, m, "row_of"));
    const auto weights = static_cast<const float *>(a.array(g_f32, m, "weights"));
    void *dYs = a.array(t, product({m, dim}), "dYs");
    const auto dweights = static_cast<float *>(a.array(g_f32, m, "dweights"));
    void *stream = a.stream();
    return run(a, [&] {
        return gemm_expert_combine_grad(h, tokens, top_k, dim, dY, Ys, row_of, weights, dYs, dweights, dtype, stream);
    });
}

PTS_CALL(run_experts, 13)
    PyObject *t;
    const gemm_dtype_t dtype = a.type("gemm_run_experts", &t);
    const auto h = a.handle();
    const int64_t rows = a.integer(), experts = a.integer(), N = a.integer(), K = a.integer();
    const void *A = a.array(t, product({rows, K}), "A"), *B = a.array(t, product({experts, N, K}), "B");
    const auto offsets = static_cast<const int32_t *>(a.array(g_i32, offsets_of(experts), "offsets"));
    void *C = a.array(dtype == GEMM_E4M3 ? g_elements[GEMM_BF16] : t, product({rows, N}), "C");
    const float scale_a = a.real(), scale_b = a.real();
    void *stream = a.stream();
    return run(a, [&] {
        return gemm_run_experts(h, rows, experts, N, K, A, B, offsets, C, dtype, scale_a, scale_b, stream);
    });
}

PTS_CALL(run_experts_dgrad, 11)
    PyObject *t;
    const gemm_dtype_t dtype = a.type("gemm_run_experts_dgrad", &t);
    const auto h = a.handle();
    const int64_t rows = a.integer(), experts = a.integer(), N = a.integer(), K = a.integer();
    const void *dC = a.array(t, product({rows, N}), "dC"), *B = a.array(t, product({experts, N, K}), "B");
    const auto offsets = static_cast<const int32_t *>(a.array(g_i32, offsets_of(experts), "offsets"));
    void *dA = a.array(t, product({rows, K}), "dA");
    void *stream = a.stream();
    return run(a, [&] { return gemm_run_experts_dgrad(h, rows, experts, N, K, dC, B, offsets, dA, dtype, stream); });
}

PTS_CALL(run_experts_wgrad, 11)
    PyObject *t;
    const gemm_dtype_t dtype = a.type("gemm_run_experts_wgrad", &t);
    const auto h = a.handle();
    const int64_t rows = a.integer(), experts = a.integer(), N = a.integer(), K = a.integer();
    const void *dC = a.array(t, product({rows, N}), "dC"), *A = a.array(t, product({rows, K}), "A");
    const auto offsets = static_cast<const int32_t *>(a.array(g_i32, offsets_of(experts), "offsets"));
    void *dB = a.array(t, product({experts, N, K}), "dB");
    void *stream = a.stream();
    return run(a, [&] { return gemm_run_experts_wgrad(h, rows, experts, N, K, dC, A, offsets, dB, dtype, stream); });
}

PTS_CALL(run_nibble, 14)
    PyObject *t;
    const gemm_dtype_t dtype = a.type("gemm_run_nibble", &t);
    const auto h = a.handle();
    const int64_t rows = a.integer(), experts = a.integer(), N = a.integer(), K = a.integer(), group = a.integer();
    const int64_t groups = product({experts, N, group > 0 && K > 0 ? (K - 1) / group + 1 : 0});
    const void *A = a.array(t, product({rows, K}), "A"), *B = a.array(g_u8, product({experts, N, K}) / 2, "B");
    const void *scales = a.array(t, groups, "scales");
    const auto zeros = static_cast<const uint8_t *>(a.array(g_u8, groups, "zeros"));
    const auto offsets = static_cast<const int32_t *>(a.array(g_i32, offsets_of(experts), "offsets"));
    void *C = a.array(t, product({rows, N}), "C");
    void *stream = a.stream();
    return run(a, [&] {
        return gemm_run_nibble(h, rows, experts, N, K, group, A, B, scales, zeros, offsets, C, dtype, stream);
    });
}

// setup(Tensor, refuse, float16, bfloat16, float8_e4m3fn, int32, float32, uint8)
PyObject *setup(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "setup: 8 arguments");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) Py_INCREF(v[i]);   // (kept until the process ends, as what follows)
    g_tensor = v[0];
    g_refuse = v[1];
    for (int i = 0; i < 3; ++i) g_elements[i] = v[2 + i];
    g_i32 = v[5];
    g_f32 = v[6];
    g_u8 = v[7];
    g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    const struct { PyObject **to; const char *name; } members[] = {{&g_dtype, "dtype"}, {&g_device, "get_device"},
        {&g_contiguous, "is_contiguous"}, {&g_numel, "numel"}, {&g_data_ptr, "data_ptr"}};
    for (const auto &m : members) {
        *m.to = PyObject_GetAttrString(g_tensor, m.name);
        if (!*m.to) return nullptr;
    }
    if (!PyType_Check(g_tensor) || !Py_TYPE(g_dtype)->tp_descr_get || !g_cuda_stream) {
        PyErr_SetString(PyExc_TypeError, "setup: not a tensor type");
        return nullptr;
    }
    Py_RETURN_NONE;
}

#define PTS_METHOD(name_) {#name_, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name_)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {PTS_METHOD(setup), PTS_METHOD(expert_sort), PTS_METHOD(expert_gather), PTS_METHOD(expert_combine),
                           PTS_METHOD(expert_combine_grad), PTS_METHOD(run_experts), PTS_METHOD(run_experts_dgrad),
                           PTS_METHOD(run_experts_wgrad), PTS_METHOD(run_nibble), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "pts_experts", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pts_experts() { return PyModule_Create(&g_module); }
