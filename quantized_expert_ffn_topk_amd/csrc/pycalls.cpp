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

// bind(addresses of the four in NAMES' order, abi.check, abi.addr)
PyObject *py_bind(PyObject *, PyObject *args)
{
    unsigned long long f[4];
    PyObject *c, *d;
    if (!PyArg_ParseTuple(args, "KKKKOO", &f[0], &f[1], &f[2], &f[3], &c, &d))
        return nullptr;
    rmsnorm_quant = (decltype(rmsnorm_quant))(uintptr_t)f[0];
    swiglu_quant = (decltype(swiglu_quant))(uintptr_t)f[1];
    linear_int8 = (decltype(linear_int8))(uintptr_t)f[2];
    route_select = (decltype(route_select))(uintptr_t)f[3];
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
    PyObject *names = Py_BuildValue("(ssss)", "moe_rmsnorm_quant", "moe_swiglu_quant", "moe_linear_int8",
                                    "moe_route_select");
    if (!names || PyModule_AddObject(m, "NAMES", names) != 0) {
        Py_XDECREF(names);
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
