// pycalls.cpp -- Python module _calls: the operators around the layer as direct
// calls of the C ABI.
//
// A step of decoding makes several of them per block and their kernels take 2 to
// 5 us, while converting 11 to 18 arguments through ctypes takes 0.6 to 1.2 us of
// the host's time; here it is 0.2 to 0.4.  The library's functions are bound by
// address (the one that abi.lib() loaded); a status other than MOE_OK goes to
// abi.check, which raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <cstring>

#include "moe.h"

namespace {

decltype(&moe_rmsnorm_quant) rmsnorm_quant;
decltype(&moe_swiglu_quant) swiglu_quant;
decltype(&moe_linear_int8) linear_int8;
decltype(&moe_route_select) route_select;
decltype(&moe_quant_fp8) quant_fp8;
decltype(&moe_linear_fp8) linear_fp8;
decltype(&moe_grouped_linear) grouped_linear;
decltype(&moe_group_rows) group_rows;
decltype(&moe_combine_rows) combine_rows;
PyObject *check, *addr;                        // of abi
PyObject *name_data_ptr, *name_cuda_stream;

// The arguments in turn.  After a failure the rest are nulls and Python's error
// is set.
class Args {
public:
    Args(PyObject *const *v, Py_ssize_t n, Py_ssize_t want) : v_(v)
    {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
            ok_ = false;
        } else if (!check) {
            PyErr_SetString(PyExc_RuntimeError, "_calls.bind has not been called");
            ok_ = false;
        }
    }
    bool ok() const
    {
        return ok_;
    }
    // a tensor's data_ptr(), an integer, None, or whatever abi.addr knows
    void *ptr()
    {
        if (!ok_)
            return nullptr;
        PyObject *o = *v_++;
        if (o == Py_None)
            return nullptr;
        if (PyLong_Check(o))
            return address(o);
        PyObject *r = PyObject_CallMethodNoArgs(o, name_data_ptr);
        if (!r && PyErr_ExceptionMatches(PyExc_AttributeError)) {
            PyErr_Clear();
            r = PyObject_CallOneArg(addr, o);
        }
        return taken(r);
    }
    // None, an integer, or a torch stream
    void *stream()
    {
        if (!ok_)
            return nullptr;
        PyObject *o = *v_++;
        if (o == Py_None)
            return nullptr;
        return PyLong_Check(o) ? address(o) : taken(PyObject_GetAttr(o, name_cuda_stream));
    }
    int64_t i64()
    {
        if (!ok_)
            return 0;
        const long long x = PyLong_AsLongLong(*v_++);
        ok_ = !(x == -1 && PyErr_Occurred());
        return x;
    }
    int32_t i32()
    {
        const int64_t x = i64();
        if (ok_ && x != (int32_t)x) {
            PyErr_Format(PyExc_OverflowError, "%lld does not fit 32 bits", (long long)x);
            ok_ = false;
        }
        return (int32_t)x;
    }
    float f32()
    {
        if (!ok_)
            return 0.0f;
        const double x = PyFloat_AsDouble(*v_++);
        ok_ = !(x == -1.0 && PyErr_Occurred());
        return (float)x;
    }
    // a ctypes structure
    bool copy(void *to, Py_ssize_t bytes)
    {
        if (!ok_)
            return false;
        Py_buffer b;
        if (PyObject_GetBuffer(*v_++, &b, PyBUF_SIMPLE) != 0) {
            ok_ = false;
            return false;
        }
        if (b.len == bytes) {
            memcpy(to, b.buf, (size_t)bytes);
        } else {
            PyErr_Format(PyExc_TypeError, "a structure of %zd bytes, %zd wanted", b.len, bytes);
            ok_ = false;
        }
        PyBuffer_Release(&b);
        return ok_;
    }

private:
    void *address(PyObject *o)
    {
        void *p = PyLong_AsVoidPtr(o);
        ok_ = p || !PyErr_Occurred();
        return p;
    }
    void *taken(PyObject *o)
    {
        if (!o) {
            ok_ = false;
            return nullptr;
        }
        void *p = address(o);
        Py_DECREF(o);
        return p;
    }
    PyObject *const *v_;
    bool ok_ = true;
};

// the call without the interpreter's lock, its status through abi.check
template <typename F>
PyObject *called(const Args &a, F &&f)
{
    if (!a.ok())
        return nullptr;
    moe_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    if (st == MOE_OK)
        Py_RETURN_NONE;
    return PyObject_CallFunction(check, "i", (int)st);
}

PyObject *py_rmsnorm_quant(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 18);
    const void *x = a.ptr();
    const int32_t xd = a.i32();
    const int64_t ldx = a.i64();
    const void *res = a.ptr();
    const int32_t rd = a.i32();
    const int64_t ldr = a.i64();
    const float *gamma = (const float *)a.ptr();
    const int32_t T = a.i32(), H = a.i32();
    const float eps = a.f32();
    void *h = a.ptr();
    const int64_t ldh = a.i64();
    void *y = a.ptr();
    const int64_t ldy = a.i64();
    int8_t *q = (int8_t *)a.ptr();
    const int64_t ldq = a.i64();
    float *s = (float *)a.ptr();
    void *st = a.stream();
    return called(a, [&] {
        return rmsnorm_quant(x, xd, ldx, res, rd, ldr, gamma, T, H, eps, h, ldh, y, ldy, q, ldq, s, st);
    });
}

PyObject *py_swiglu_quant(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 11);
    const void *gu = a.ptr();
    const int32_t dt = a.i32();
    const int64_t ld = a.i64();
    const int32_t T = a.i32(), F = a.i32();
    void *y = a.ptr();
    const int64_t ldy = a.i64();
    int8_t *q = (int8_t *)a.ptr();
    const int64_t ldq = a.i64();
    float *s = (float *)a.ptr();
    void *st = a.stream();
    return called(a, [&] { return swiglu_quant(gu, dt, ld, T, F, y, ldy, q, ldq, s, st); });
}

PyObject *py_linear_int8(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 14);
    const int8_t *q = (const int8_t *)a.ptr();
    const int64_t ldq = a.i64();
    const float *s = (const float *)a.ptr();
    const int32_t T = a.i32();
    const int8_t *w = (const int8_t *)a.ptr();
    const int64_t ldw = a.i64();
    const float *ws = (const float *)a.ptr(), *bias = (const float *)a.ptr();
    const int32_t N = a.i32(), K = a.i32();
    void *out = a.ptr();
    const int32_t od = a.i32();
    const int64_t ldo = a.i64();
    void *st = a.stream();
    return called(a, [&] { return linear_int8(q, ldq, s, T, w, ldw, ws, bias, N, K, out, od, ldo, st); });
}

PyObject *py_route_select(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 9);
    moe_route_desc d;
    a.copy(&d, sizeof(d));
    const void *logits = a.ptr();
    const int32_t dt = a.i32();
    const int64_t ld = a.i64();
    const float *bias = (const float *)a.ptr();
    const int32_t T = a.i32();
    int32_t *idx = (int32_t *)a.ptr();
    float *w = (float *)a.ptr();
    void *st = a.stream();
    return called(a, [&] { return route_select(&d, logits, dt, ld, bias, T, idx, w, st); });
}

PyObject *py_quant_fp8(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 12);
    const void *x = a.ptr();
    const int32_t xd = a.i32();
    const int64_t ldx = a.i64();
    const int32_t act = a.i32(), T = a.i32(), K = a.i32();
    const int32_t *count = (const int32_t *)a.ptr();
    void *q = a.ptr();
    const int64_t ldq = a.i64();
    float *s = (float *)a.ptr();
    const int64_t lds = a.i64();
    void *st = a.stream();
    return called(a, [&] { return quant_fp8(x, xd, ldx, act, T, K, count, q, ldq, s, lds, st); });
}

PyObject *py_linear_fp8(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 16);
    const void *q = a.ptr();
    const int64_t ldq = a.i64();
    const float *s = (const float *)a.ptr();
    const int64_t lds = a.i64();
    const int32_t T = a.i32();
    const void *w = a.ptr();
    const int64_t ldw = a.i64();
    const float *ws = (const float *)a.ptr();
    const int64_t ldws = a.i64();
    const float *bias = (const float *)a.ptr();
    const int32_t N = a.i32(), K = a.i32();
    void *out = a.ptr();
    const int32_t od = a.i32();
    const int64_t ldo = a.i64();
    void *st = a.stream();
    return called(a, [&] {
        return linear_fp8(q, ldq, s, lds, T, w, ldw, ws, ldws, bias, N, K, out, od, ldo, st);
    });
}

PyObject *py_grouped_linear(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 22);
    const void *x = a.ptr();
    const int32_t xd = a.i32();
    const int64_t ldx = a.i64();
    const float *s = (const float *)a.ptr();
    const int64_t lds = a.i64();
    const int32_t R = a.i32();
    const int32_t *rows = (const int32_t *)a.ptr(), *offsets = (const int32_t *)a.ptr();
    const int32_t E = a.i32(), M = a.i32();
    const void *w = a.ptr();
    const int64_t ldw = a.i64(), w_stride = a.i64();
    const float *ws = (const float *)a.ptr();
    const int64_t ldws = a.i64(), ws_stride = a.i64();
    const int32_t N = a.i32(), K = a.i32();
    void *out = a.ptr();
    const int32_t od = a.i32();
    const int64_t ldo = a.i64();
    void *st = a.stream();
    return called(a, [&] {
        return grouped_linear(x, xd, ldx, s, lds, R, rows, offsets, E, M, w, ldw, w_stride, ws, ldws, ws_stride, N,
                              K, out, od, ldo, st);
    });
}

PyObject *py_group_rows(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 8);
    const int32_t *idx = (const int32_t *)a.ptr();
    const int32_t T = a.i32(), k = a.i32(), E = a.i32();
    int32_t *offsets = (int32_t *)a.ptr(), *rows = (int32_t *)a.ptr(), *pos = (int32_t *)a.ptr();
    void *st = a.stream();
    return called(a, [&] { return group_rows(idx, T, k, E, offsets, rows, pos, st); });
}

PyObject *py_combine_rows(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    Args a(v, n, 15);
    const void *y = a.ptr();
    const int32_t yd = a.i32();
    const int64_t ldy = a.i64();
    const int32_t R = a.i32();
    const int32_t *pos = (const int32_t *)a.ptr();
    const float *w = (const float *)a.ptr();
    const void *base = a.ptr();
    const int64_t ldb = a.i64();
    const int32_t T = a.i32(), k = a.i32(), H = a.i32();
    void *out = a.ptr();
    const int32_t od = a.i32();
    const int64_t ldo = a.i64();
    void *st = a.stream();
    return called(a, [&] { return combine_rows(y, yd, ldy, R, pos, w, base, ldb, T, k, H, out, od, ldo, st); });
}

// the functions in NAMES' order
const char *const NAMES[] = {"moe_rmsnorm_quant", "moe_swiglu_quant", "moe_linear_int8",
                             "moe_route_select",  "moe_quant_fp8",    "moe_linear_fp8",
                             "moe_grouped_linear", "moe_group_rows",  "moe_combine_rows"};
constexpr Py_ssize_t N_NAMES = sizeof(NAMES) / sizeof(NAMES[0]);

template <typename F>
void set_function(F &f, unsigned long long at)
{
    f = (F)(uintptr_t)at;
}

// bind(addresses of the functions, abi.check, abi.addr)
PyObject *py_bind(PyObject *, PyObject *args)
{
    if (PyTuple_GET_SIZE(args) != N_NAMES + 2) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", PyTuple_GET_SIZE(args), N_NAMES + 2);
        return nullptr;
    }
    unsigned long long f[N_NAMES];
    for (Py_ssize_t i = 0; i < N_NAMES; ++i) {
        f[i] = PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(args, i));
        if (PyErr_Occurred())
            return nullptr;
    }
    set_function(rmsnorm_quant, f[0]);
    set_function(swiglu_quant, f[1]);
    set_function(linear_int8, f[2]);
    set_function(route_select, f[3]);
    set_function(quant_fp8, f[4]);
    set_function(linear_fp8, f[5]);
    set_function(grouped_linear, f[6]);
    set_function(group_rows, f[7]);
    set_function(combine_rows, f[8]);
    PyObject *c = PyTuple_GET_ITEM(args, N_NAMES), *d = PyTuple_GET_ITEM(args, N_NAMES + 1);
    Py_INCREF(c);
    Py_XSETREF(check, c);
    Py_INCREF(d);
    Py_XSETREF(addr, d);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", py_bind, METH_VARARGS, "bind(addresses of NAMES, check, addr)"},
    {"moe_rmsnorm_quant", (PyCFunction)(void (*)(void))py_rmsnorm_quant, METH_FASTCALL, nullptr},
    {"moe_swiglu_quant", (PyCFunction)(void (*)(void))py_swiglu_quant, METH_FASTCALL, nullptr},
    {"moe_linear_int8", (PyCFunction)(void (*)(void))py_linear_int8, METH_FASTCALL, nullptr},
    {"moe_route_select", (PyCFunction)(void (*)(void))py_route_select, METH_FASTCALL, nullptr},
    {"moe_quant_fp8", (PyCFunction)(void (*)(void))py_quant_fp8, METH_FASTCALL, nullptr},
    {"moe_linear_fp8", (PyCFunction)(void (*)(void))py_linear_fp8, METH_FASTCALL, nullptr},
    {"moe_grouped_linear", (PyCFunction)(void (*)(void))py_grouped_linear, METH_FASTCALL, nullptr},
    {"moe_group_rows", (PyCFunction)(void (*)(void))py_group_rows, METH_FASTCALL, nullptr},
    {"moe_combine_rows", (PyCFunction)(void (*)(void))py_combine_rows, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "The operators around the layer, called directly.",
                      -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void)
{
    name_data_ptr = PyUnicode_InternFromString("data_ptr");
    name_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!name_data_ptr || !name_cuda_stream)
        return nullptr;
    PyObject *m = PyModule_Create(&module);
    if (!m)
        return nullptr;
    PyObject *names = PyTuple_New(N_NAMES);
    for (Py_ssize_t i = 0; names && i < N_NAMES; ++i) {
        PyObject *name = PyUnicode_FromString(NAMES[i]);
        if (!name)
            Py_CLEAR(names);
        else
            PyTuple_SET_ITEM(names, i, name);
    }
    if (!names || PyModule_AddObject(m, "NAMES", names) != 0) {
        Py_XDECREF(names);
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
