// The training operators on torch tensors: argument checks, allocation and the call into
// libbl.so's C ABI, in C++ because these operators are called with lists of hundreds of tensors
// and at sizes where the GPU's work takes a few microseconds. The same marshalling written in
// Python over ctypes took 42 us for the norm of 12 small tensors and 593 us for clipping 400.
//
// Every function returns new tensors of the stream that the work runs on; scratch memory is taken
// from, and goes back to, the allocator in that stream's order.
#include <Python.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>

#include <cstdint>
#include <vector>

#include "../../../include/bl.h"

namespace {

PyObject *g_error = nullptr;      // BLError, handed over by init()

struct Refused {};                // a Python error is set

[[noreturn]] void refuse(PyObject *type, const char *fmt, const char *name = "") {
    PyErr_Format(type, fmt, name);
    throw Refused();
}

[[noreturn]] void failed(int status) {
    PyObject *e = PyObject_CallFunction(g_error, "is", status, bl_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor", name);
    return THPVariable_Unpack(o);
}

// The device, and the stream that the call was given (None: the current one), as the allocator's
// current ones for the guard's life.
struct On {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard stream;
    cudaStream_t raw;
    On(c10::Device d, PyObject *s) : device(d) {
        if (s == Py_None) {
            raw = c10::cuda::getCurrentCUDAStream(d.index()).stream();
            return;
        }
        raw = static_cast<cudaStream_t>(PyLong_AsVoidPtr(s));
        if (PyErr_Occurred()) throw Refused();
        if (raw != c10::cuda::getCurrentCUDAStream(d.index()).stream())
            stream.reset_stream(c10::cuda::getStreamFromExternal(raw, d.index()));
    }
    bl_stream_t bl() const { return reinterpret_cast<bl_stream_t>(raw); }
};

c10::DataPtr scratch(int64_t bytes) {
    return c10::cuda::CUDACachingAllocator::get()->allocate(static_cast<size_t>(bytes));
}

// The call has written to a tensor of the caller's: autograd then knows that what it saved of it is gone.
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

at::Tensor floats(at::IntArrayRef shape, c10::Device d) {
    return at::empty(shape, at::TensorOptions().dtype(at::kFloat).device(d));
}

// ------------------------------------------------------------------ gnorm, gclip

int grad_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return BL_F32;
        case at::kDouble: return BL_F64;
        case at::kBFloat16: return BL_BF16;
        case at::kHalf: return BL_F16;
        default: refuse(PyExc_TypeError, "unsupported dtype %s", c10::toString(t));
    }
}

struct Ref {
    PyObject *o;
    explicit Ref(PyObject *p) : o(p) {
        if (!p) throw Refused();
    }
    ~Ref() { Py_DECREF(o); }
    Ref(const Ref &) = delete;
};

PyObject *grads(PyObject *list, bool clip, double max_norm, PyObject *out, PyObject *stream) {
    // Both lists are held to the end of the call: a generator's tensors may have no other owner, and the
    // norm and the workspace must not be given their memory. Iterating over one may also run anything, the
    // other list's own changes among it, so the items are looked at after that.
    Ref seq(PySequence_Fast(list, "a list of tensors is wanted"));
    const bool given = clip && out != Py_None;
    Ref outs(given ? PySequence_Fast(out, "out must be a list of tensors") : PyTuple_New(0));
    const int64_t n = PySequence_Fast_GET_SIZE(seq.o);
    PyObject **items = PySequence_Fast_ITEMS(seq.o);
    std::vector<int32_t> kinds(n + 1);
    std::vector<int64_t> sizes(n + 1);
    std::vector<const void *> x(n + 1);
    std::vector<void *> y(n + 1);
    c10::Device device(c10::kCUDA, 0);
    for (int64_t i = 0; i < n; ++i) {
        const at::Tensor &t = tensor(items[i], "every gradient");
        kinds[i] = grad_code(t.scalar_type());
        if (i == 0) device = t.device();
        if (!t.is_cuda() || t.device() != device) refuse(PyExc_ValueError, "the tensors must be on one CUDA device");
        // any memory order will do, as long as the elements fill one block of memory
        if (!t.is_non_overlapping_and_dense())
            refuse(PyExc_ValueError, "a tensor has gaps or overlaps in memory");
        sizes[i] = t.numel();
        x[i] = t.data_ptr();
        y[i] = t.data_ptr();
    }
    if (given) {
        if (PySequence_Fast_GET_SIZE(outs.o) != n) refuse(PyExc_ValueError, "out must have as many tensors");
        for (int64_t i = 0; i < n; ++i) {
            const at::Tensor &t = THPVariable_Unpack(items[i]), &o = tensor(PySequence_Fast_GET_ITEM(outs.o, i), "every output");
            if (o.scalar_type() != t.scalar_type() || o.sizes() != t.sizes() || o.device() != device)
                refuse(PyExc_ValueError, "an output must have its tensor's type, shape and device");
            if (o.strides() != t.strides() && !(o.is_contiguous() && t.is_contiguous()))
                refuse(PyExc_ValueError, "an output must have its tensor's strides");
            y[i] = o.data_ptr();
        }
    }
    if (n == 0) device = c10::Device(c10::kCUDA, c10::cuda::current_device());
    On on(device, stream);
    at::Tensor norm = floats({}, device);
    const int64_t need = bl_gnorm_workspace(n);
    if (need < 0) refuse(PyExc_ValueError, "too many tensors");
    const c10::DataPtr ws = scratch(need);
    float *const to = norm.mutable_data_ptr<float>();
    const int st = clip ? bl_gclip(n, kinds.data(), x.data(), y.data(), sizes.data(), max_norm, to, ws.get(), need, on.bl())
                        : bl_gnorm(n, kinds.data(), x.data(), sizes.data(), to, ws.get(), need, on.bl());
    if (st != BL_SUCCESS) failed(st);
    if (clip) {
        PyObject **const results = given ? PySequence_Fast_ITEMS(outs.o) : items;
        for (int64_t i = 0; i < n; ++i) written(THPVariable_Unpack(results[i]));
    }
    return THPVariable_Wrap(std::move(norm));
}

// ------------------------------------------------------------------ xent, xent_grad

// Leading dimension of a matrix whose rows are stored back to back or apart.
int64_t rows_of(const at::Tensor &m, const char *name, const at::Tensor &like) {
    if (m.dim() != 2) refuse(PyExc_ValueError, "%s must be (rows, cols)", name);
    if (!m.is_cuda() || m.device() != like.device()) refuse(PyExc_ValueError, "%s must be a CUDA tensor on H's device", name);
    if (m.scalar_type() != like.scalar_type()) refuse(PyExc_TypeError, "%s must have H's dtype", name);
    if (m.size(1) > 1 && m.stride(1) != 1) refuse(PyExc_ValueError, "%s's rows must be contiguous (stride(1) == 1)", name);
    return m.size(0) > 1 ? m.stride(0) : std::max<int64_t>(m.size(1), 1);
}

template <typename T>
T *values_of(const at::Tensor &v, const char *name, at::ScalarType type, const at::Tensor &h) {
    if (v.dim() != 1 || v.size(0) != h.size(0) || v.scalar_type() != type || v.device() != h.device())
        refuse(PyExc_ValueError, "%s must hold one value for each row of H, on its device (int64 targets, f32 values)", name);
    if (v.size(0) > 1 && v.stride(0) != 1) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T *>(v.data_ptr());
}

struct Xent {
    const at::Tensor &h, &w;
    bl_dtype code;
    int64_t ldh, ldw, rows, dim, vocab;
    const int64_t *target;

    Xent(PyObject *ho, PyObject *wo, PyObject *to) : h(tensor(ho, "H")), w(tensor(wo, "W")) {
        if (h.scalar_type() != at::kFloat && h.scalar_type() != at::kBFloat16)
            refuse(PyExc_TypeError, "unsupported dtype %s", c10::toString(h.scalar_type()));
        code = h.scalar_type() == at::kFloat ? BL_F32 : BL_BF16;
        ldh = rows_of(h, "H", h);
        ldw = rows_of(w, "W", h);
        rows = h.size(0), dim = h.size(1), vocab = w.size(0);
        if (w.size(1) != dim) refuse(PyExc_ValueError, "H and W must have as many columns");
        target = values_of<const int64_t>(tensor(to, "target"), "target", at::kLong, h);
    }
    int64_t need(int grad) const {
        const int64_t n = bl_xent_workspace(code, rows, dim, vocab, h.data_ptr(), ldh, w.data_ptr(), ldw, grad);
        if (n < 0) failed(BL_ERR_INVALID_ARGUMENT);
        return n;
    }
};

PyObject *pair(PyObject *a, PyObject *b) {
    Ref x(a), y(b);
    return PyTuple_Pack(2, a, b);
}

PyObject *do_xent(PyObject *const *a) {
    const Xent c(a[0], a[1], a[2]);
    On on(c.h.device(), a[3]);
    const int64_t need = c.need(0);
    at::Tensor loss = floats({c.rows}, c.h.device()), lse = floats({c.rows}, c.h.device());
    const c10::DataPtr ws = scratch(need);
    const int st = bl_xent(c.code, c.rows, c.dim, c.vocab, c.h.data_ptr(), c.ldh, c.w.data_ptr(), c.ldw, c.target,
                           loss.mutable_data_ptr<float>(), lse.mutable_data_ptr<float>(), ws.get(), need, on.bl());
    if (st != BL_SUCCESS) failed(st);
    return pair(THPVariable_Wrap(std::move(loss)), THPVariable_Wrap(std::move(lse)));
}

// A gradient to write: a given tensor, a new one (None), or none (False).
at::Tensor gradient(PyObject *o, const char *name, const at::Tensor &of, int64_t *ld) {
    *ld = 0;
    if (o == Py_False) return at::Tensor();
    if (o == Py_None) {
        *ld = std::max<int64_t>(of.size(1), 1);
        return at::empty(of.sizes(), of.options());
    }
    const at::Tensor &t = tensor(o, name);
    *ld = rows_of(t, name, of);
    if (t.sizes() != of.sizes()) refuse(PyExc_ValueError, "%s must have the shape of what it is the gradient of", name);
    return t;
}

PyObject *wrapped(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject *do_xent_grad(PyObject *const *a) {
    const Xent c(a[0], a[1], a[2]);
    const float *const lse = values_of<const float>(tensor(a[3], "lse"), "lse", at::kFloat, c.h);
    const float *const g = values_of<const float>(tensor(a[4], "g"), "g", at::kFloat, c.h);
    if (a[5] == Py_False && a[6] == Py_False) refuse(PyExc_ValueError, "dH and dW are both left out");
    On on(c.h.device(), a[7]);
    const int64_t need = c.need(1);
    int64_t lddh, lddw;
    at::Tensor dh = gradient(a[5], "dH", c.h, &lddh), dw = gradient(a[6], "dW", c.w, &lddw);
    const c10::DataPtr ws = scratch(need);
    const int st = bl_xent_grad(c.code, c.rows, c.dim, c.vocab, c.h.data_ptr(), c.ldh, c.w.data_ptr(), c.ldw, c.target, lse, g,
                                dh.defined() ? dh.data_ptr() : nullptr, lddh, dw.defined() ? dw.data_ptr() : nullptr, lddw,
                                ws.get(), need, on.bl());
    if (st != BL_SUCCESS) failed(st);
    if (dh.defined()) written(dh);
    if (dw.defined()) written(dw);
    return pair(wrapped(dh), wrapped(dw));
}

// ------------------------------------------------------------------ the module

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t wanted, F f) {
    HANDLE_TH_ERRORS
    if (got != wanted) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *py_init(PyObject *, PyObject *error) {
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    Py_RETURN_NONE;
}
// gnorm(tensors, stream)
PyObject *py_gnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 2, [&] { return grads(a[0], false, 0.0, Py_None, a[1]); });
}
// gclip(tensors, max_norm, out, stream)
PyObject *py_gclip(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject * {
        const double limit = PyFloat_AsDouble(a[1]);
        if (PyErr_Occurred()) throw Refused();
        return grads(a[0], true, limit, a[2], a[3]);
    });
}
// xent(H, W, target, stream)
PyObject *py_xent(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&] { return do_xent(a); });
}
// xent_grad(H, W, target, lse, g, dH, dW, stream)
PyObject *py_xent_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&] { return do_xent_grad(a); });
}

#define BL_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"init", py_init, METH_O, nullptr}, BL_METHOD(gnorm), BL_METHOD(gclip), BL_METHOD(xent),
                         BL_METHOD(xent_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
