// What the Python entry points of the compiled operators share: checks of torch tensors,
// allocation of results and the way errors become Python exceptions.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <utility>

#include "fp8_ops.h"

namespace wstma_bind {

using at::Tensor;

struct Refused {
    PyObject *type;
    std::string what;
};

struct Failed {
    PyObject *type;  // raised as type(status, call)
    int status;
    const char *call;
};

[[noreturn]] inline void type_error(std::string what) { throw Refused{PyExc_TypeError, std::move(what)}; }
[[noreturn]] inline void value_error(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }

inline const Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o))
        type_error(std::string(what) + " must be a tensor");
    const Tensor &t = THPVariable_Unpack(o);
    // the result would be detached from it without a word
    if (t.requires_grad() && at::GradMode::is_enabled())
        value_error(std::string(what) + " requires a gradient, which these operators do not record: call them under "
                                        "torch.no_grad(), or in the forward of a torch.autograd.Function");
    // and so from its tangent (undefined where forward-mode derivatives are not recorded)
    if (t._fw_grad(/* level */ 0).defined())
        value_error(std::string(what) + " has a forward-mode tangent, which these operators do not carry on: call them on "
                                        "its primal, or in the forward of a torch.autograd.Function with a jvp");
    return t;
}

inline const Tensor *maybe_tensor(PyObject *o, const char *what) { return o == Py_None ? nullptr : &tensor(o, what); }

inline int element_type(const Tensor &t, const char *what)
{
    if (t.scalar_type() == at::kBFloat16)
        return FP8_BF16;
    if (t.scalar_type() == at::kFloat)
        return FP8_FP32;
    type_error(std::string(what) + " must be bf16 or fp32");
}

inline std::string size_text(int64_t r, int64_t c) { return std::to_string(r) + " x " + std::to_string(c); }

// Elements from one row of a matrix to the next.
inline int64_t pitch_of(const Tensor &t, const char *what)
{
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
        value_error(std::string(what) + " must be a matrix with contiguous rows");
    const int64_t ld = t.size(0) > 1 ? t.stride(0) : t.size(1);
    if (ld < t.size(1))
        value_error(std::string(what) + ": its rows overlap");
    return ld;
}

inline int64_t padded(int64_t cols) { return (cols + 127) / 128 * 128; }

inline bool is_codes(const Tensor &t) { return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte; }

inline int64_t codes_pitch(const Tensor &t, const char *what)
{
    if (!is_codes(t))
        type_error(std::string(what) + " must be float8_e4m3fn (or its bytes)");
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
        value_error(std::string(what) + " must be a matrix with contiguous rows");
    if (t.size(1) == 0)
        return 0;
    // a single row has no pitch that matters: any that the library accepts
    return t.size(0) > 1 ? t.stride(0) : padded(t.size(1));
}

inline void need_scales(const Tensor &s, const Tensor &codes, const char *what)
{
    if (s.scalar_type() != at::kFloat8_e8m0fnu && s.scalar_type() != at::kByte)
        type_error(std::string(what) + " must be float8_e8m0fnu (or its bytes)");
    if (s.dim() != 3 || s.size(0) != (codes.size(1) + 511) / 512 || s.size(1) != codes.size(0) || s.size(2) != 4 ||
        !s.is_contiguous())
        value_error(std::string(what) + " must be a contiguous ceil(K / 512) x rows x 4 tensor");
}

inline int64_t need_bf16(const Tensor &t, int64_t R, int64_t C, const char *what)
{
    if (t.scalar_type() != at::kBFloat16)
        type_error(std::string(what) + " must be bf16");
    if (t.dim() != 2 || t.size(0) != R || t.size(1) != C)
        value_error(std::string(what) + " must be " + size_text(R, C));
    return pitch_of(t, what);
}

inline void need_vector(const Tensor &t, int64_t n, const char *what)
{
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        value_error(std::string(what) + " must be a contiguous vector of " + std::to_string(n));
}

// The current stream of the tensors' device; allocations and the call run there.
struct Place {
    std::optional<c10::cuda::CUDAGuard> guard;
    std::optional<c10::Device> on;
    void *stream;
    int index;

    explicit Place(const Tensor &first)
    {
        const c10::Device dev = first.device();
        if (!dev.is_cuda())
            value_error("tensors must be on a CUDA device (got " + dev.str() + ")");
        index = dev.index();
        if (c10::cuda::current_device() != index)
            guard.emplace(dev);
        on = dev;
        stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }

    void same(const Tensor *t) const
    {
        if (t && (!t->is_cuda() || t->get_device() != index))
            value_error("tensors must be on one device (cuda:" + std::to_string(index) + " and " + t->device().str() +
                        ")");
    }

    // Uninitialised tensors straight from the allocator: the dispatcher takes longer
    // than the allocation.
    Tensor empty(at::IntArrayRef size, at::ScalarType type) const
    {
        return at::detail::empty_cuda(size, type, on, std::nullopt);
    }

    // codes (rows at multiples of 128 bytes) and scales of a rows x cols matrix
    std::pair<Tensor, Tensor> quantized(int64_t rows, int64_t cols) const
    {
        return {at::detail::empty_strided_cuda({rows, cols}, {padded(cols), 1}, at::kFloat8_e4m3fn, on),
                empty({(cols + 511) / 512, rows, 4}, at::kFloat8_e8m0fnu)};
    }
};

inline void *data(const Tensor &t) { return const_cast<void *>(t.const_data_ptr()); }
inline void *data(const Tensor *t) { return t ? data(*t) : nullptr; }

// The caller's tensor has been written to: autograd finds by its version that a tensor saved for a backward
// pass is no longer what was saved.  (A tensor of inference mode is never saved, and has no version.)
inline void written(const Tensor *t)
{
    if (t && !t->is_inference())
        t->unsafeGetTensorImpl()->bump_version();
}

inline PyObject *tuple_of(std::initializer_list<PyObject *> items)
{
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (t && o)
            PyTuple_SET_ITEM(t, i++, o);
        else
            Py_XDECREF(o);
    }
    if (t && i != (Py_ssize_t)items.size()) {
        Py_DECREF(t);
        return nullptr;
    }
    return t;
}

inline PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// Calls f and turns what it throws into a Python exception: no C++ exception
// leaves an entry point.
template <typename F>
PyObject *guarded(F f)
{
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const Failed &e) {
        PyObject *args = Py_BuildValue("(is)", e.status, e.call);
        if (args) {
            PyErr_SetObject(e.type, args);
            Py_DECREF(args);
        }
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

inline void need_args(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want)
        type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}

template <typename F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace wstma_bind
