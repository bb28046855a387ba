// Python entry points of the 8-bit operators: torch tensors in, the C ABI of
// include/fp8_ops.h called on their device's current stream, torch tensors out.
// It checks arguments, allocates outputs and marshals; the work is done by
// libfp8_ops.so.  It is compiled, rather than written over ctypes, because
// the smallest calls (one token) take 2-3 us on the GPU and the marshalling of
// four outputs and sixteen arguments in Python took 23 us (8 us here, measured
// on the Grace host).
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <optional>
#include <string>
#include <utility>

#include "fp8_ops.h"
#include "fp8_overlap.h"

namespace {

using at::Tensor;

PyObject *fp8_error = nullptr;  // raised for a status code: Fp8Error(status, call)

struct Refused {
    PyObject *type;
    std::string what;
};

struct Failed {
    int status;
    const char *call;
};

[[noreturn]] void type_error(std::string what) { throw Refused{PyExc_TypeError, std::move(what)}; }
[[noreturn]] void value_error(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }

void check(int status, const char *call)
{
    if (status != FP8_OK)
        throw Failed{status, call};
}

const Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o))
        type_error(std::string(what) + " must be a tensor");
    const Tensor &t = THPVariable_Unpack(o);
    // the result would be detached from it without a word
    if (t.requires_grad() && at::GradMode::is_enabled())
        value_error(std::string(what) + " requires a gradient, which these operators do not record: call them under "
                                        "torch.no_grad(), or in the forward of a torch.autograd.Function");
    return t;
}

const Tensor *maybe_tensor(PyObject *o, const char *what) { return o == Py_None ? nullptr : &tensor(o, what); }

int element_type(const Tensor &t, const char *what)
{
    if (t.scalar_type() == at::kBFloat16)
        return FP8_BF16;
    if (t.scalar_type() == at::kFloat)
        return FP8_FP32;
    type_error(std::string(what) + " must be bf16 or fp32");
}

std::string size_text(int64_t r, int64_t c) { return std::to_string(r) + " x " + std::to_string(c); }

// Elements from one row of a matrix to the next.
int64_t pitch_of(const Tensor &t, const char *what)
{
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
        value_error(std::string(what) + " must be a matrix with contiguous rows");
    const int64_t ld = t.size(0) > 1 ? t.stride(0) : t.size(1);
    if (ld < t.size(1))
        value_error(std::string(what) + ": its rows overlap");
    return ld;
}

int64_t padded(int64_t cols) { return (cols + 127) / 128 * 128; }

bool is_codes(const Tensor &t) { return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte; }

int64_t codes_pitch(const Tensor &t, const char *what)
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

void need_scales(const Tensor &s, const Tensor &codes, const char *what)
{
    if (s.scalar_type() != at::kFloat8_e8m0fnu && s.scalar_type() != at::kByte)
        type_error(std::string(what) + " must be float8_e8m0fnu (or its bytes)");
    if (s.dim() != 3 || s.size(0) != (codes.size(1) + 511) / 512 || s.size(1) != codes.size(0) || s.size(2) != 4 ||
        !s.is_contiguous())
        value_error(std::string(what) + " must be a contiguous ceil(K / 512) x rows x 4 tensor");
}

int64_t need_bf16(const Tensor &t, int64_t R, int64_t C, const char *what)
{
    if (t.scalar_type() != at::kBFloat16)
        type_error(std::string(what) + " must be bf16");
    if (t.dim() != 2 || t.size(0) != R || t.size(1) != C)
        value_error(std::string(what) + " must be " + size_text(R, C));
    return pitch_of(t, what);
}

void need_vector(const Tensor &t, int64_t n, const char *what)
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

void *data(const Tensor &t) { return const_cast<void *>(t.const_data_ptr()); }
void *data(const Tensor *t) { return t ? data(*t) : nullptr; }

PyObject *tuple_of(std::initializer_list<PyObject *> items)
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

PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

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
            PyErr_SetObject(fp8_error, args);
            Py_DECREF(args);
        }
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

void need_args(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want)
        type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}

// The product's handles by device, for their plans: a call's workspace is its own.
// Guarded by the interpreter lock; they live as long as the process.
std::map<int, fp8_gemm_t> handles;

fp8_gemm_t kept_handle(int device)
{
    fp8_gemm_t &kept = handles[device];
    if (!kept)
        check(fp8_gemm_create(device, &kept), "fp8_gemm_create");
    return kept;
}

// run(handle or 0, a, a_scales, b, b_scales, out or None, out_dtype) -> out
PyObject *bind_gemm(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 7);
        fp8_gemm_t h = static_cast<fp8_gemm_t>(PyLong_AsVoidPtr(args[0]));
        if (PyErr_Occurred())
            throw python_error();
        const Tensor &a = tensor(args[1], "a"), &as = tensor(args[2], "a_scales");
        const Tensor &b = tensor(args[3], "b"), &bs = tensor(args[4], "b_scales");
        const Tensor *given = maybe_tensor(args[5], "out");
        const int64_t lda = codes_pitch(a, "a"), ldb = codes_pitch(b, "b");
        const int64_t M = a.size(0), N = b.size(0), K = a.size(1);
        if (b.size(1) != K)
            value_error("a and b contract over " + std::to_string(K) + " and " + std::to_string(b.size(1)) + " columns");
        need_scales(as, a, "a_scales");
        need_scales(bs, b, "b_scales");
        Place at(a);
        at.same(&as), at.same(&b), at.same(&bs), at.same(given);
        Tensor out;
        if (given) {
            out = *given;
            if (out.dim() != 2 || out.size(0) != M || out.size(1) != N)
                value_error("out must be " + size_text(M, N));
        } else {
            if (!THPDtype_Check(args[6]))
                type_error("out_dtype must be a torch.dtype");
            const at::ScalarType st = reinterpret_cast<THPDtype *>(args[6])->scalar_type;
            if (st != at::kBFloat16 && st != at::kFloat)
                type_error("out_dtype must be bf16 or fp32");
            out = at.empty({M, N}, st);
        }
        const int type = element_type(out, "out");
        if (!h)
            h = kept_handle(at.index);
        check(fp8_gemm_plan(h, M, N, K, lda, ldb, pitch_of(out, "out"), type), "fp8_gemm_plan");
        int64_t need = 0;
        check(fp8_gemm_workspace(h, &need), "fp8_gemm_workspace");
        Tensor work;  // freed on return, to this stream's (or this graph's) later allocations: they run after it
        if (need)
            work = at.empty({need}, at::kByte);
        check(fp8_gemm_run_in(h, data(a), data(as), data(b), data(bs), data(out), need ? data(work) : nullptr, need,
                              at.stream),
              "fp8_gemm_run");
        return wrap(std::move(out));
    });
}

// quantize(x, tile, rows, columns, row_factor or None, column_factor or None) -> tuple
PyObject *bind_quantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 6);
        const Tensor &x = tensor(args[0], "x");
        const int tile = PyObject_IsTrue(args[1]), rows = PyObject_IsTrue(args[2]), cols = PyObject_IsTrue(args[3]);
        if (tile < 0 || rows < 0 || cols < 0)
            throw python_error();
        const Tensor *rf = maybe_tensor(args[4], "row_factor"), *cf = maybe_tensor(args[5], "column_factor");
        const int type = element_type(x, "x");
        const int64_t ldx = pitch_of(x, "x"), R = x.size(0), C = x.size(1);
        Place at(x);
        at.same(rf), at.same(cf);
        if (rf) {
            need_vector(*rf, R, "row_factor");
            if (rf->scalar_type() != at::kFloat)
                type_error("row_factor must be fp32");
        }
        if (cf)
            need_vector(*cf, C, "column_factor");
        const int ctype = cf ? element_type(*cf, "column_factor") : FP8_BF16;
        Tensor q, s, qt, st;
        if (rows)
            std::tie(q, s) = at.quantized(R, C);
        if (cols)
            std::tie(qt, st) = at.quantized(C, R);
        check(fp8_quantize(data(x), type, ldx, R, C, tile, static_cast<const float *>(data(rf)), data(cf), ctype,
                           rows ? data(q) : nullptr, padded(C), rows ? data(s) : nullptr, cols ? data(qt) : nullptr,
                           padded(R), cols ? data(st) : nullptr, at.stream),
              "fp8_quantize");
        if (rows && cols)
            return tuple_of({wrap(q), wrap(s), wrap(qt), wrap(st)});
        return rows ? tuple_of({wrap(q), wrap(s)}) : tuple_of({wrap(qt), wrap(st)});
    });
}

// rmsnorm(x, weight, residual or None, eps, out_h or None) -> (codes, scales, h, rstd)
PyObject *bind_rmsnorm(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 5);
        const Tensor &x = tensor(args[0], "x"), &w = tensor(args[1], "weight");
        const Tensor *res = maybe_tensor(args[2], "residual"), *out_h = maybe_tensor(args[4], "out_h");
        const double eps = PyFloat_AsDouble(args[3]);
        if (eps == -1.0 && PyErr_Occurred())
            throw python_error();
        if (x.dim() != 2)
            value_error("x must be a matrix");
        const int64_t R = x.size(0), C = x.size(1);
        const int64_t ldx = need_bf16(x, R, C, "x");
        need_vector(w, C, "weight");
        const int wtype = element_type(w, "weight");
        if (out_h && !res)
            value_error("out_h needs a residual: without one, h is x");
        const int64_t ldr = res ? need_bf16(*res, R, C, "residual") : 0;
        Place at(x);
        at.same(&w), at.same(res), at.same(out_h);
        int64_t ldh = 0;
        Tensor h;
        if (res) {
            h = out_h ? *out_h : at.empty({R, C}, at::kBFloat16);
            ldh = need_bf16(h, R, C, "out_h");
            if (out_h && (wstma::rows_clash(data(x), 2 * ldx, data(h), 2 * ldh, R, 2 * C) ||
                          wstma::rows_clash(data(res), 2 * ldr, data(h), 2 * ldh, R, 2 * C)))
                value_error("out_h lies over part of x or residual: it may be one of them, or apart");
        }
        auto [q, s] = at.quantized(R, C);
        Tensor rstd = at.empty({R}, at::kFloat);
        check(fp8_rmsnorm(data(x), ldx, data(res), ldr, data(w), wtype, R, C, (float)eps, res ? data(h) : nullptr, ldh,
                          data(q), padded(C), data(s), static_cast<float *>(data(rstd)), at.stream),
              "fp8_rmsnorm");
        PyObject *hp = args[0];  // without a residual h is x itself
        if (out_h)
            hp = args[4];
        if (!res || out_h)
            Py_INCREF(hp);
        else
            hp = wrap(h);
        return tuple_of({wrap(q), wrap(s), hp, wrap(rstd)});
    });
}

// rmsnorm_backward(dy, h, weight, rstd, dresidual or None) -> (dx, dweight)
PyObject *bind_rmsnorm_backward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 5);
        const Tensor &dy = tensor(args[0], "dy"), &h = tensor(args[1], "h"), &w = tensor(args[2], "weight"),
                     &rstd = tensor(args[3], "rstd");
        const Tensor *dres = maybe_tensor(args[4], "dresidual");
        if (dy.dim() != 2)
            value_error("dy must be a matrix");
        const int64_t R = dy.size(0), C = dy.size(1);
        const int64_t lddy = need_bf16(dy, R, C, "dy"), ldh = need_bf16(h, R, C, "h");
        need_vector(w, C, "weight");
        const int wtype = element_type(w, "weight");
        const int64_t lddr = dres ? need_bf16(*dres, R, C, "dresidual") : 0;
        need_vector(rstd, R, "rstd");
        if (rstd.scalar_type() != at::kFloat)
            type_error("rstd must be fp32");
        Place at(dy);
        at.same(&h), at.same(&w), at.same(&rstd), at.same(dres);
        int64_t need = 0;
        check(fp8_rmsnorm_backward_workspace(R, C, &need), "fp8_rmsnorm_backward_workspace");
        Tensor dx = at.empty({R, C}, at::kBFloat16), dw = at.empty({C}, at::kFloat);
        // freed on return, to this stream's later allocations: they run after it
        Tensor work = at.empty({need}, at::kByte);
        check(fp8_rmsnorm_backward(data(dy), lddy, data(h), ldh, data(w), wtype, static_cast<const float *>(data(rstd)),
                                   data(dres), lddr, data(dx), C, static_cast<float *>(data(dw)), R, C, data(work),
                                   need, at.stream),
              "fp8_rmsnorm_backward");
        return tuple_of({wrap(dx), wrap(dw)});
    });
}

// kept_handle(device) -> the address of the handle that gemm() runs on there
PyObject *bind_kept_handle(PyObject *, PyObject *device)
{
    return guarded([&]() -> PyObject * {
        const long index = PyLong_AsLong(device);
        if (index == -1 && PyErr_Occurred())
            throw python_error();
        if (index < 0 || index > 0xFFFF)
            value_error("no such device");
        return PyLong_FromVoidPtr(kept_handle((int)index));
    });
}

PyObject *bind_set_error(PyObject *, PyObject *type)
{
    Py_INCREF(type);
    Py_XSETREF(fp8_error, type);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"gemm", fast(&bind_gemm), METH_FASTCALL, nullptr},
    {"quantize", fast(&bind_quantize), METH_FASTCALL, nullptr},
    {"rmsnorm", fast(&bind_rmsnorm), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", fast(&bind_rmsnorm_backward), METH_FASTCALL, nullptr},
    {"kept_handle", &bind_kept_handle, METH_O, nullptr},
    {"set_error", &bind_set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_bind() { return PyModule_Create(&module); }
