// What the wrappers of the layer's operators do on every call, without Python between: describe the tensors'
// layouts, make an output, pass addresses and the current stream to a function of libosdn.so.
// Marshalling only. A decode token's kernel takes 2 to 4 us; through ctypes its call took 9 to 12.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <exception>
#include <string>

namespace {

bool is_tensor(PyObject* o) { return THPVariable_Check(o); }
const at::Tensor& tensor(PyObject* o) { return THPVariable_Unpack(o); }

// Runs f; a C++ exception becomes a Python one.
template <typename F> PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// layouts(tensor or None, ...) -> bytes: type, device, shape and strides of each, equal where all are equal.
PyObject* layouts(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        std::string s;
        s.reserve(64 * n);
        auto put = [&](int64_t v) { s.append(reinterpret_cast<const char*>(&v), sizeof(v)); };
        for (Py_ssize_t i = 0; i < n; ++i) {
            if (args[i] == Py_None) {
                put(-1);
                continue;
            }
            if (!is_tensor(args[i])) {
                PyErr_Format(PyExc_TypeError, "a tensor is needed, not %s", Py_TYPE(args[i])->tp_name);
                return nullptr;
            }
            const at::Tensor& t = tensor(args[i]);
            if (t.layout() != at::kStrided) {
                PyErr_SetString(PyExc_TypeError, "a strided tensor is needed");
                return nullptr;
            }
            put((int64_t)t.dim() << 32 | (int64_t)t.scalar_type() << 24 | (int64_t)t.device().type() << 16 |
                (int64_t)(uint8_t)t.device().index());
            for (int64_t v : t.sizes()) put(v);
            for (int64_t v : t.strides()) put(v);
        }
        return PyBytes_FromStringAndSize(s.data(), (Py_ssize_t)s.size());
    });
}

// here(tensor) -> whether it is on the current CUDA device.
PyObject* here(PyObject*, PyObject* arg) {
    return guarded([&]() -> PyObject* {
        if (!is_tensor(arg)) return PyBool_FromLong(0);
        const at::Device d = tensor(arg).device();
        return PyBool_FromLong(d.is_cuda() && d.index() == c10::cuda::current_device());
    });
}

// like(tensor) -> an uninitialised dense tensor of its shape, type and device.
PyObject* like(PyObject*, PyObject* arg) {
    return guarded([&]() -> PyObject* {
        if (!is_tensor(arg)) {
            PyErr_SetString(PyExc_TypeError, "a tensor is needed");
            return nullptr;
        }
        const at::Tensor& t = tensor(arg);
        return THPVariable_Wrap(at::empty(t.sizes(), t.options().requires_grad(false)));
    });
}

// floats(tensor, size, ...) -> an uninitialised dense fp32 tensor of these sizes on the tensor's device.
PyObject* floats(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n < 1 || n > 5 || !is_tensor(args[0])) {
            PyErr_SetString(PyExc_TypeError, "a tensor and up to 4 sizes are needed");
            return nullptr;
        }
        int64_t sizes[4];
        for (Py_ssize_t i = 1; i < n; ++i) sizes[i - 1] = PyLong_AsLongLong(args[i]);
        if (PyErr_Occurred()) return nullptr;
        return THPVariable_Wrap(at::empty(at::IntArrayRef(sizes, (size_t)(n - 1)),
                                          at::TensorOptions().dtype(at::kFloat).device(tensor(args[0]).device())));
    });
}

// Addresses of the arguments after the first two (the function's and the parameter block's): tensors, None (NULL)
// or addresses.
constexpr int kMost = 16;
struct Call {
    void* fn = nullptr;
    void* params = nullptr;
    void* at[kMost] = {};
    void* stream = nullptr;
    bool ok = false;
};
Call parse(PyObject* const* args, Py_ssize_t n, int want) {
    Call c;
    if (n != want + 2) {
        PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", want + 2, n);
        return c;
    }
    c.fn = PyLong_AsVoidPtr(args[0]);
    c.params = PyLong_AsVoidPtr(args[1]);
    for (int i = 0; i < want; ++i) {
        PyObject* o = args[i + 2];
        if (o == Py_None) c.at[i] = nullptr;
        else if (is_tensor(o)) c.at[i] = tensor(o).data_ptr();
        else c.at[i] = PyLong_AsVoidPtr(o);
    }
    if (PyErr_Occurred()) return c;
    c.stream = c10::cuda::getCurrentCUDAStream().stream();
    c.ok = true;
    return c;
}

size_t bytes_of(PyObject* o) {
    if (o == Py_None || !is_tensor(o)) return 0;
    return (size_t)tensor(o).numel() * tensor(o).element_size();
}

using P = void*;
#define CALL(NAME, WANT, TYPE, ...)                                           \
    PyObject* NAME(PyObject*, PyObject* const* args, Py_ssize_t n) {          \
        return guarded([&]() -> PyObject* {                                   \
            const Call c = parse(args, n, WANT);                              \
            if (!c.ok) return nullptr;                                        \
            auto fn = reinterpret_cast<TYPE>(c.fn);                           \
            auto a = c.at;                                                    \
            int rc;                                                           \
            Py_BEGIN_ALLOW_THREADS rc = fn(c.params, __VA_ARGS__, c.stream);  \
            Py_END_ALLOW_THREADS return PyLong_FromLong(rc);                  \
        });                                                                   \
    }

// recur_fwd(fn, params, x, gate, h0, lengths, h, final_h, checkpoints)
CALL(recur_fwd, 7, int (*)(P, P, P, P, P, P, P, P, P), a[0], a[1], a[2], a[3], a[4], a[5], a[6])
// recur_bwd(fn, params, x, gate, h0, lengths, dh, dfinal_h, checkpoints, dx, dgate, dh0, workspace)
CALL(recur_bwd, 11, int (*)(P, P, P, P, P, P, P, P, P, P, P, P, size_t, P), a[0], a[1], a[2], a[3], a[4], a[5], a[6],
     a[7], a[8], a[9], a[10], bytes_of(args[12]))
// recur_step(fn, params, x, gate, state, h)
CALL(recur_step, 4, int (*)(P, P, P, P, P, P), a[0], a[1], a[2], a[3])
// qk_fwd(fn, params, q, k, wq, wk, positions, freqs, lengths, q_out, k_out)
CALL(qk_fwd, 9, int (*)(P, P, P, P, P, P, P, P, P, P, P), a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8])
// qk_bwd(fn, params, q, k, wq, wk, positions, freqs, lengths, dq_out, dk_out, dq, dk, dwq, dwk, workspace)
CALL(qk_bwd, 14, int (*)(P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, size_t, P), a[0], a[1], a[2], a[3], a[4], a[5], a[6],
     a[7], a[8], a[9], a[10], a[11], a[12], a[13], bytes_of(args[15]))
// rope(fn, params, x, positions, freqs, lengths, out, inverse)
CALL(rope, 6, int (*)(P, P, P, P, P, P, int, P), a[0], a[1], a[2], a[3], a[4], a[5] ? 1 : 0)

#define FAST(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(layouts), {"here", here, METH_O, nullptr}, {"like", like, METH_O, nullptr}, FAST(floats),
                         FAST(recur_fwd), FAST(recur_bwd), FAST(recur_step), FAST(qk_fwd), FAST(qk_bwd), FAST(rope),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "Calls into libosdn.so without Python between.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&module); }
