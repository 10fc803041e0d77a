// What the parts of the Python module _rows share: the session, tensors taken
// from Python and made for it, errors.
#pragma once

#include <Python.h>

#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdarg>
#include <exception>
#include <string>
#include <vector>

#include "rc.h"

namespace rows_binding {

using at::ScalarType;
using at::Tensor;

inline PyObject* g_error = nullptr;  // CollectiveError

struct Raised {};  // a Python error is set

[[noreturn]] inline void raise(int code, const char* what, const char* f, ...) {
    char text[400];
    va_list args;
    va_start(args, f);
    vsnprintf(text, sizeof text, f, args);
    va_end(args);
    const std::string msg = std::string(what) + ": " + text;
    PyObject* e = PyObject_CallFunction(g_error, "is", code, msg.c_str());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// The status of a library call, made without the interpreter's lock: the
// library's own may be held by a thread that waits for the GPU.
template <class F>
void call(F f) {
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = f();
    Py_END_ALLOW_THREADS
    if (code == RC_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", code, rc_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// The open session; `id` goes with the call, so that another session, opened by
// another thread in the meantime, is not taken for it.
struct Session {
    int64_t id = 0;
    int ranks = 0, device = -1;
    Session() {
        thread_local Session seen{0, 0, -1};  // a number is of one session only
        call([&] {
            int64_t open = 0;
            int e = rc_session_id(&open);
            if (!e && open != seen.id) {
                e = rc_session_info(&seen.ranks, &seen.device);
                seen.id = e ? 0 : open;
            }
            return e;
        });
        *this = seen;
    }

  private:
    Session(int64_t i, int r, int d) : id(i), ranks(r), device(d) {}
};

inline const char* type_name(ScalarType t) { return at::toString(t); }

inline at::TensorOptions options(ScalarType type, const at::Device& device) { return at::TensorOptions().dtype(type).device(device); }

// A dense tensor within another's storage, from element `at` on: what
// as_strided gives, without a pass through the dispatcher for each.
inline Tensor part_of(const Tensor& all, int64_t at, at::IntArrayRef sizes) {
    auto impl = c10::make_intrusive<at::TensorImpl>(at::Storage(all.storage()), all.key_set(), all.dtype());
    impl->set_storage_offset(at);
    impl->set_sizes_contiguous(sizes);
    return Tensor(std::move(impl));
}

// One tensor per rank.
struct Tensors {
    PyObject* list = nullptr;  // what Python gave or gets
    int n = 0;
    Tensor made[RC_MAX_RANKS];
    PyObject* given[RC_MAX_RANKS] = {};  // owned: the list may change while the call is made
    const Tensor* t[RC_MAX_RANKS] = {};
    void* p[RC_MAX_RANKS] = {};

    Tensors() = default;
    Tensors(const Tensors&) = delete;
    Tensors& operator=(const Tensors&) = delete;
    ~Tensors() {
        for (int r = 0; r < n && given[r]; ++r) Py_DECREF(given[r]);
        Py_XDECREF(list);
    }

    // A list or tuple of `ranks` tensors.
    void take(PyObject* seq, int ranks, const char* what) {
        Py_INCREF(seq);
        list = seq;
        if (!PyList_Check(seq) && !PyTuple_Check(seq)) raise(RC_ERR_INVALID_ARGUMENT, what, "not a list of tensors");
        const Py_ssize_t size = PySequence_Fast_GET_SIZE(seq);
        if (size != ranks) raise(RC_ERR_INVALID_ARGUMENT, what, "%lld tensors for %d ranks", (long long)size, ranks);
        n = ranks;
        for (int r = 0; r < n; ++r) {
            PyObject* o = PySequence_Fast_GET_ITEM(seq, r);
            if (!THPVariable_Check(o)) raise(RC_ERR_INVALID_ARGUMENT, what, "no tensor for rank %d", r);
            hold(r, o);
        }
    }
    void hold(int r, PyObject* o) {
        Py_INCREF(o);
        given[r] = o;
        t[r] = &THPVariable_Unpack(o);
    }
    void take_one(PyObject* o) {
        n = 1;
        hold(0, o);
    }

    // Tensors made here, given to Python with give().
    void make(int ranks) {
        n = ranks;
        for (int r = 0; r < n; ++r) t[r] = &made[r];
    }
    // The same, [rows[r], cols] each; small ones as parts of one allocation (and
    // one fill), on boundaries of 256 bytes: eight ranks' calls on a token each
    // take 5.6 to 9.6 us that way, and took 10 to 39.  Large ones stand alone, so
    // that each can be freed.
    static constexpr int64_t kTogether = int64_t(1) << 24;  // bytes of all
    void make(int ranks, const int64_t* rows, int64_t cols, ScalarType type, const at::Device& device, const char* what,
              bool zeros = false) {
        make(ranks);
        const int64_t es = (int64_t)c10::elementSize(type), step = 256 / es;
        auto padded = [&](int r) { return (rows[r] * cols + step - 1) / step * step; };
        int64_t size = 0, from = 0;
        for (int r = 0; r < n; ++r) {
            if (rows[r] > INT32_MAX || cols > INT32_MAX / 2)
                raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d: %lld rows of %lld", r, (long long)rows[r], (long long)cols);
            size = std::min(kTogether + 1, size + std::min(kTogether + 1, padded(r) * es));
        }
        auto fresh = [&](at::IntArrayRef sizes) {
            return zeros ? at::zeros(sizes, options(type, device)) : at::empty(sizes, options(type, device));
        };
        if (size > kTogether) {
            for (int r = 0; r < n; ++r) made[r] = fresh({rows[r], cols});
        } else {
            const Tensor all = fresh({size / es});
            for (int r = 0; r < n; from += padded(r++)) made[r] = part_of(all, from, {rows[r], cols});
        }
    }
    PyObject* give() {
        if (!list) {
            list = PyList_New(n);
            if (!list) throw Raised{};
            for (int r = 0; r < n; ++r) {
                PyObject* o = THPVariable_Wrap(made[r]);
                if (!o) throw Raised{};
                PyList_SET_ITEM(list, r, o);
            }
        }
        Py_INCREF(list);
        return list;
    }

    void dims(int want, const char* what, const char* shape) const {
        for (int r = 0; r < n; ++r)
            if (t[r]->dim() != want)
                raise(RC_ERR_SHAPE_MISMATCH, what, "rank %d has %lld dimensions, expected %s", r, (long long)t[r]->dim(), shape);
    }

    // Rank r's [rows[r]] (cols < 0) or [rows[r], cols] tensor; fills p.
    void expect(ScalarType type, const at::Device& device, const int64_t* rows, int64_t cols, const char* what) {
        for (int r = 0; r < n; ++r) {
            const Tensor& x = *t[r];
            if (x.scalar_type() != type)
                raise(RC_ERR_DTYPE_MISMATCH, what, "rank %d has dtype %s, expected %s", r, type_name(x.scalar_type()), type_name(type));
            const bool ok = cols < 0 ? x.dim() == 1 && x.size(0) == rows[r]
                                     : x.dim() == 2 && x.size(0) == rows[r] && x.size(1) == cols;
            if (!ok) {
                std::string has;
                for (int64_t d : x.sizes()) has += (has.empty() ? "" : ", ") + std::to_string(d);
                if (cols < 0) raise(RC_ERR_SHAPE_MISMATCH, what, "rank %d has shape (%s), expected (%lld)", r, has.c_str(), (long long)rows[r]);
                raise(RC_ERR_SHAPE_MISMATCH, what, "rank %d has shape (%s), expected (%lld, %lld)", r, has.c_str(), (long long)rows[r], (long long)cols);
            }
            if (x.device() != device)
                raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d on %s, others on %s", r, x.device().str().c_str(), device.str().c_str());
            if (x.layout() != at::kStrided || !x.is_contiguous()) raise(RC_ERR_INVALID_ARGUMENT, what, "rank %d is not contiguous", r);
            p[r] = x.data_ptr();
        }
    }
};

inline int row_type(const Tensor& x, const char* what) {
    switch (x.scalar_type()) {
        case ScalarType::Float: return RC_F32;
        case ScalarType::Half: return RC_F16;
        case ScalarType::BFloat16: return RC_BF16;
        default: break;
    }
    PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %s; float32, float16 and bfloat16 are supported", what, type_name(x.scalar_type()));
    throw Raised{};
}

// The call's stream: the current one of the tensors' GPU, which has to be the
// session's.
inline void* stream_on(const Session& s, const at::Device& device, const char* what) {
    if (!device.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "tensors must be on a CUDA (HIP) device");
        throw Raised{};
    }
    if (s.device >= 0 && device.index() != s.device)
        raise(RC_ERR_INVALID_ARGUMENT, what, "tensors on %s, the session on GPU %d", device.str().c_str(), s.device);
    return c10::hip::getCurrentHIPStream(device.index()).stream();
}

// ---------------------------------------------------------------- arguments

inline long long to_int(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
inline int32_t to_int32(PyObject* o, const char* what) {
    const long long v = to_int(o);
    if (v < INT32_MIN || v > INT32_MAX) raise(RC_ERR_INVALID_ARGUMENT, what, "%lld is out of range", v);
    return (int32_t)v;
}
inline double to_double(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}
inline float to_float(PyObject* o) { return (float)to_double(o); }
inline bool to_bool(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v;
}
// A pair (list, list), or None.
inline bool pair_of(PyObject* o, const char* what, PyObject** a, PyObject** b) {
    if (o == Py_None) return false;
    if ((!PyTuple_Check(o) && !PyList_Check(o)) || PySequence_Fast_GET_SIZE(o) != 2)
        raise(RC_ERR_INVALID_ARGUMENT, what, "out is not a pair of lists");
    *a = PySequence_Fast_GET_ITEM(o, 0);
    *b = PySequence_Fast_GET_ITEM(o, 1);
    return true;
}
inline PyObject* pack(PyObject* a, PyObject* b) {
    PyObject* t = PyTuple_Pack(2, a, b);
    Py_DECREF(a);
    Py_DECREF(b);
    if (!t) throw Raised{};
    return t;
}

struct Arity {
    const char* name;
    Py_ssize_t n;
};
inline void arity(Py_ssize_t got, Arity want) {
    if (got == want.n) return;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", want.name, want.n, got);
    throw Raised{};
}

// torch's exceptions become the Python ones that torch's own functions raise
// (OutOfMemoryError among them).
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Raised&) {
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

}  // namespace rows_binding
