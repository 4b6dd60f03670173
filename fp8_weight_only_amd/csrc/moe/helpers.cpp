// The tensor helpers of moe.py for calls that are right: the checks, the
// allocations and the C-ABI call without Python in between. A small call costs
// the host as long as it costs the GPU; through ctypes one token's route took
// 13 us and a weighted sum 8, of which the kernels take 5 and 2.
//
// Each function returns None for arguments that it does not take (a wrong type,
// shape, device or layout) and for a call that the library refused, which it does
// before it enqueues anything; moe.py then goes through the same call step by step
// and raises what is wrong. A call that failed in HIP may have enqueued some of its
// kernels: its status is returned, for moe.py to raise, and it is not tried again.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../../include/fp8w_moe.h"

namespace {

// A contiguous GPU tensor argument.
struct Arg {
    const at::Tensor* t = nullptr;
    bool read(PyObject* o)
    {
        if (!THPVariable_Check(o))
            return false;
        t = &THPVariable_Unpack(o);
        return t->is_cuda() && t->layout() == at::kStrided && t->is_contiguous();
    }
    at::ScalarType type() const { return t->scalar_type(); }
    int64_t dim() const { return t->dim(); }
    int64_t size(int i) const { return t->size(i); }
    void* ptr() const { return t->numel() ? t->data_ptr() : nullptr; }
    bool like(const Arg& first, at::ScalarType type_, std::initializer_list<int64_t> shape) const
    {
        return t->device() == first.t->device() && type() == type_ && t->sizes().equals(at::IntArrayRef(shape));
    }
};

// One that may be None.
struct Maybe : Arg {
    bool given = false;
    bool read(PyObject* o)
    {
        if (o == Py_None)
            return true;
        given = true;
        return Arg::read(o);
    }
    bool like(const Arg& first, at::ScalarType type_, std::initializer_list<int64_t> shape) const
    {
        return !given || Arg::like(first, type_, shape);
    }
    void* ptr() const { return given ? Arg::ptr() : nullptr; }
};

bool act_type(at::ScalarType t, fp8w_dtype_t& out)
{
    out = t == at::kBFloat16 ? FP8W_BF16 : FP8W_FP16;
    return t == at::kBFloat16 || t == at::kHalf;
}

hipStream_t stream_of(const Arg& a)
{
    return c10::hip::getCurrentHIPStream(a.t->get_device()).stream();
}

at::Tensor make(const Arg& like, at::IntArrayRef shape, at::ScalarType type)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.t->device()));
}

PyObject* none()
{
    Py_RETURN_NONE;
}

// The launches and allocations of a call go to its first tensor's device.
#define FP8W_ON_DEVICE_OF(arg) const c10::DeviceGuard on_device((arg).t->device())

// Runs f, and turns a C++ exception into the Python one that torch's own calls
// raise for it (torch.OutOfMemoryError where an allocation failed).
template <typename F>
PyObject* guarded(F&& f)
{
    try {
        return f();
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

template <typename F>
fp8w_status_t without_gil(F&& f)
{
    fp8w_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return st;
}

// What a call that did not succeed returns.
PyObject* failed(fp8w_status_t st)
{
    return st == FP8W_ERR_HIP ? PyLong_FromLong(st) : none();
}

// combine(y, weights, out)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Arg y, w;
        Maybe out;
        fp8w_dtype_t act;
        if (n != 3 || !y.read(a[0]) || !w.read(a[1]) || !out.read(a[2]) || y.dim() != 2 || w.dim() != 2 ||
            !act_type(y.type(), act))
            return none();
        const int64_t t = w.size(0), top = w.size(1), c = y.size(1);
        if (!y.like(y, y.type(), {t * top, c}) || !w.like(y, at::kFloat, {t, top}) || !out.like(y, y.type(), {t, c}))
            return none();
        FP8W_ON_DEVICE_OF(y);
        const at::Tensor made = out.given ? *out.t : make(y, {t, c}, y.type());
        const hipStream_t stream = stream_of(y);
        const fp8w_status_t st = without_gil([&] {
            return fp8w_combine(y.ptr(), act, static_cast<const float*>(w.ptr()), t, top, c,
                                made.numel() ? made.data_ptr() : nullptr, stream);
        });
        return st == FP8W_SUCCESS ? THPVariable_Wrap(made) : failed(st);
    });
}

// route(logits, top_k, renormalize) -> (weights, experts, offsets, slots, tokens), the workspace its own
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Arg l;
        if (n != 3 || !l.read(a[0]) || l.dim() != 2 || !PyLong_CheckExact(a[1]))
            return none();
        const int64_t t = l.size(0), e = l.size(1);
        const long long top = PyLong_AsLongLong(a[1]);
        if (top == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        const int renorm = PyObject_IsTrue(a[2]);
        const at::ScalarType type = l.type();
        const fp8w_dtype_t dt = type == at::kBFloat16 ? FP8W_BF16 : (type == at::kHalf ? FP8W_FP16 : FP8W_FP32);
        if (renorm < 0 || (dt == FP8W_FP32 && type != at::kFloat) || top < 1 || top > e || top > 64 || e > 1024 ||
            t > INT32_MAX / top)
            return none();
        FP8W_ON_DEVICE_OF(l);
        // one allocation: weights, experts, slots, tokens, offsets, workspace
        const int64_t s = t * top;
        const size_t need = fp8w_route_workspace_bytes(t, e, top);
        const at::Tensor buf = make(l, {4 * s + e + 1 + (int64_t)(need / 4)}, at::kInt);
        int32_t* p = static_cast<int32_t*>(buf.data_ptr());
        const hipStream_t stream = stream_of(l);
        const fp8w_status_t st = without_gil([&] {
            return fp8w_route(l.ptr(), dt, t, e, top, renorm, reinterpret_cast<float*>(p), p + s, p + 4 * s,
                              p + 2 * s, p + 3 * s, need ? p + 4 * s + e + 1 : nullptr, need, stream);
        });
        if (st != FP8W_SUCCESS)
            return failed(st);
        auto list = [&](int64_t first, int64_t count) { return buf.as_strided({count}, {1}, first); };
        auto table = [&](const at::Tensor& b, int64_t first) { return b.as_strided({t, top}, {top, 1}, first); };
        PyObject* r = PyTuple_New(5);
        if (!r)
            return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(table(buf.view(at::kFloat), 0)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(table(buf, s)));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(list(4 * s, e + 1)));
        PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(list(2 * s, s)));
        PyTuple_SET_ITEM(r, 4, THPVariable_Wrap(list(3 * s, s)));
        return r;
    });
}

// linear_experts(x, q, scale, offsets, bias, x_rows, y_rows, out)
PyObject* linear_experts(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Arg x, q, s, off;
        Maybe b, xr, yr, out;
        fp8w_dtype_t act;
        if (n != 8 || !x.read(a[0]) || !q.read(a[1]) || !s.read(a[2]) || !off.read(a[3]) || !b.read(a[4]) ||
            !xr.read(a[5]) || !yr.read(a[6]) || !out.read(a[7]) || x.dim() != 2 || q.dim() != 3 ||
            !act_type(x.type(), act))
            return none();
        const int64_t rows = x.size(0), k = x.size(1), e = q.size(0), c = q.size(1);
        const int64_t m = xr.given ? xr.t->numel() : rows;
        if (!q.like(x, at::kByte, {e, c, k}) || !s.like(x, at::kFloat, {e, c}) || !off.like(x, at::kInt, {e + 1}) ||
            !b.like(x, x.type(), {e, c}) || !xr.like(x, at::kInt, {m}) || !yr.like(x, at::kInt, {m}) ||
            !out.like(x, x.type(), {m, c}))
            return none();
        FP8W_ON_DEVICE_OF(x);
        const at::Tensor made = out.given ? *out.t : make(x, {m, c}, x.type());
        const hipStream_t stream = stream_of(x);
        const fp8w_status_t st = without_gil([&] {
            return fp8w_linear_experts(x.ptr(), act, rows, k, static_cast<const uint8_t*>(q.ptr()),
                                       static_cast<const float*>(s.ptr()), b.ptr(), e, c,
                                       static_cast<const int32_t*>(off.ptr()), m,
                                       static_cast<const int32_t*>(xr.ptr()), static_cast<const int32_t*>(yr.ptr()),
                                       made.numel() ? made.data_ptr() : nullptr, nullptr, 0, stream);
        });
        return st == FP8W_SUCCESS ? THPVariable_Wrap(made) : failed(st);
    });
}

// linear_int8(x, q, scale, bias, out), the workspace its own
PyObject* linear_int8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Arg x, q, s;
        Maybe b, out;
        fp8w_dtype_t act;
        if (n != 5 || !x.read(a[0]) || !q.read(a[1]) || !s.read(a[2]) || !b.read(a[3]) || !out.read(a[4]) ||
            x.dim() != 2 || q.dim() != 2 || !act_type(x.type(), act))
            return none();
        const int64_t m = x.size(0), k = x.size(1), c = q.size(0);
        if (!q.like(x, at::kChar, {c, k}) || !s.like(x, at::kFloat, {c}) || !b.like(x, x.type(), {c}) ||
            !out.like(x, x.type(), {m, c}))
            return none();
        const int8_t* qp = static_cast<const int8_t*>(q.ptr());
        const size_t need = fp8w_linear_int8_workspace_bytes(m, c, k, x.ptr(), qp);
        FP8W_ON_DEVICE_OF(x);
        const at::Tensor made = out.given ? *out.t : make(x, {m, c}, x.type());
        at::Tensor ws;
        if (need)
            ws = make(x, {(int64_t)need}, at::kByte);
        const hipStream_t stream = stream_of(x);
        const fp8w_status_t st = without_gil([&] {
            return fp8w_linear_int8(x.ptr(), act, m, k, qp, static_cast<const float*>(s.ptr()), b.ptr(), c,
                                    made.numel() ? made.data_ptr() : nullptr, need ? ws.data_ptr() : nullptr, need,
                                    stream);
        });
        return st == FP8W_SUCCESS ? THPVariable_Wrap(made) : failed(st);
    });
}

// linear_fp4(x, q, scale, bias, out), the workspace its own
PyObject* linear_fp4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Arg x, q, s;
        Maybe b, out;
        fp8w_dtype_t act;
        if (n != 5 || !x.read(a[0]) || !q.read(a[1]) || !s.read(a[2]) || !b.read(a[3]) || !out.read(a[4]) ||
            x.dim() != 2 || q.dim() != 2 || !act_type(x.type(), act))
            return none();
        const int64_t m = x.size(0), k = x.size(1), c = q.size(0);
        if (!q.like(x, at::kByte, {c, (k + 1) / 2}) || !s.like(x, at::kByte, {c, (k + 31) / 32}) ||
            !b.like(x, x.type(), {c}) || !out.like(x, x.type(), {m, c}))
            return none();
        const uint8_t *qp = static_cast<const uint8_t*>(q.ptr()), *sp = static_cast<const uint8_t*>(s.ptr());
        const size_t need = fp8w_linear_fp4_workspace_bytes(m, c, k, x.ptr(), qp, sp);
        FP8W_ON_DEVICE_OF(x);
        const at::Tensor made = out.given ? *out.t : make(x, {m, c}, x.type());
        at::Tensor ws;
        if (need)
            ws = make(x, {(int64_t)need}, at::kByte);
        const hipStream_t stream = stream_of(x);
        const fp8w_status_t st = without_gil([&] {
            return fp8w_linear_fp4(x.ptr(), act, m, k, qp, sp, b.ptr(), c, made.numel() ? made.data_ptr() : nullptr,
                                   need ? ws.data_ptr() : nullptr, need, stream);
        });
        return st == FP8W_SUCCESS ? THPVariable_Wrap(made) : failed(st);
    });
}

// linear_experts_fp4(x, q, scale, offsets, bias, x_rows, y_rows, out)
PyObject* linear_experts_fp4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Arg x, q, s, off;
        Maybe b, xr, yr, out;
        fp8w_dtype_t act;
        if (n != 8 || !x.read(a[0]) || !q.read(a[1]) || !s.read(a[2]) || !off.read(a[3]) || !b.read(a[4]) ||
            !xr.read(a[5]) || !yr.read(a[6]) || !out.read(a[7]) || x.dim() != 2 || q.dim() != 3 ||
            !act_type(x.type(), act))
            return none();
        const int64_t rows = x.size(0), k = x.size(1), e = q.size(0), c = q.size(1);
        const int64_t m = xr.given ? xr.t->numel() : rows;
        if (!q.like(x, at::kByte, {e, c, (k + 1) / 2}) || !s.like(x, at::kByte, {e, c, (k + 31) / 32}) ||
            !off.like(x, at::kInt, {e + 1}) || !b.like(x, x.type(), {e, c}) || !xr.like(x, at::kInt, {m}) ||
            !yr.like(x, at::kInt, {m}) || !out.like(x, x.type(), {m, c}))
            return none();
        FP8W_ON_DEVICE_OF(x);
        const at::Tensor made = out.given ? *out.t : make(x, {m, c}, x.type());
        const hipStream_t stream = stream_of(x);
        const fp8w_status_t st = without_gil([&] {
            return fp8w_linear_experts_fp4(x.ptr(), act, rows, k, static_cast<const uint8_t*>(q.ptr()),
                                           static_cast<const uint8_t*>(s.ptr()), b.ptr(), e, c,
                                           static_cast<const int32_t*>(off.ptr()), m,
                                           static_cast<const int32_t*>(xr.ptr()), static_cast<const int32_t*>(yr.ptr()),
                                           made.numel() ? made.data_ptr() : nullptr, stream);
        });
        return st == FP8W_SUCCESS ? THPVariable_Wrap(made) : failed(st);
    });
}

// moe_layer(x, logits, top_k, (q, scale), (q, scale), gate_up_bias, down_bias, renormalize, out), the workspace its own
PyObject* moe_layer(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Arg x, l, q[2], s[2];
        Maybe b[2], out;
        fp8w_dtype_t act;
        if (n != 9 || !x.read(a[0]) || !l.read(a[1]) || !PyLong_CheckExact(a[2]) || !b[0].read(a[5]) || !b[1].read(a[6]) ||
            !out.read(a[8]) || x.dim() != 2 || l.dim() != 2 || !act_type(x.type(), act))
            return none();
        for (int i = 0; i < 2; ++i) {
            PyObject* pair = a[3 + i];
            if (!PyTuple_Check(pair) || PyTuple_GET_SIZE(pair) != 2 || !q[i].read(PyTuple_GET_ITEM(pair, 0)) ||
                !s[i].read(PyTuple_GET_ITEM(pair, 1)) || q[i].dim() != 3)
                return none();
        }
        const int64_t t = x.size(0), hidden = x.size(1), e = l.size(1), inner = q[0].size(1) / 2;
        const long long top = PyLong_AsLongLong(a[2]);
        if (top == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        const int renorm = PyObject_IsTrue(a[7]);
        const at::ScalarType type = l.type();
        const fp8w_dtype_t dt = type == at::kBFloat16 ? FP8W_BF16 : (type == at::kHalf ? FP8W_FP16 : FP8W_FP32);
        const bool fp4 = s[0].type() == at::kByte;
        if (renorm < 0 || (dt == FP8W_FP32 && type != at::kFloat) || !l.like(x, type, {t, e}))
            return none();
        const int64_t rows[2] = {2 * inner, hidden}, k[2] = {hidden, inner};
        for (int i = 0; i < 2; ++i)
            if (!q[i].like(x, at::kByte, {e, rows[i], fp4 ? (k[i] + 1) / 2 : k[i]}) ||
                !(fp4 ? s[i].like(x, at::kByte, {e, rows[i], (k[i] + 31) / 32}) : s[i].like(x, at::kFloat, {e, rows[i]})) ||
                !b[i].like(x, x.type(), {e, rows[i]}))
                return none();
        if (!out.like(x, x.type(), {t, hidden}))
            return none();
        const size_t need = fp8w_moe_layer_workspace_bytes(t, e, top, hidden, inner);
        if (t > 0 && need == 0)
            return none();  // sizes that the call does not take
        FP8W_ON_DEVICE_OF(x);
        const at::Tensor made = out.given ? *out.t : make(x, {t, hidden}, x.type());
        at::Tensor ws;
        if (need)
            ws = make(x, {(int64_t)need}, at::kByte);
        const hipStream_t stream = stream_of(x);
        const fp8w_status_t st = without_gil([&] {
            return fp8w_moe_layer(x.ptr(), act, t, hidden, l.ptr(), dt, e, top, renorm,
                                  fp4 ? FP8W_WEIGHT_FP4 : FP8W_WEIGHT_E4M3, static_cast<const uint8_t*>(q[0].ptr()),
                                  s[0].ptr(), b[0].ptr(), inner, static_cast<const uint8_t*>(q[1].ptr()), s[1].ptr(),
                                  b[1].ptr(), made.numel() ? made.data_ptr() : nullptr, need ? ws.data_ptr() : nullptr,
                                  need, stream);
        });
        return st == FP8W_SUCCESS ? THPVariable_Wrap(made) : failed(st);
    });
}

PyMethodDef methods[] = {
    {"combine", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(combine)), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route)), METH_FASTCALL, nullptr},
    {"linear_experts", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_experts)), METH_FASTCALL,
     nullptr},
    {"linear_int8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_int8)), METH_FASTCALL, nullptr},
    {"linear_fp4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_fp4)), METH_FASTCALL, nullptr},
    {"linear_experts_fp4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_experts_fp4)),
     METH_FASTCALL, nullptr},
    {"moe_layer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(moe_layer)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_helpers", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_helpers()
{
    return PyModule_Create(&module);
}
