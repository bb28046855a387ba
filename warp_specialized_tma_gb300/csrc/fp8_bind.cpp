// Python entry points of the 8-bit operators (the feed-forward operators' are in ffn_bind.h): torch tensors in, the C ABI of
// include/fp8_ops.h called on their device's current stream, torch tensors out.
// It checks arguments, allocates outputs and marshals; the work is done by
// libfp8_ops.so.  It is compiled, rather than written over ctypes, because
// the smallest calls (one token) take 2-3 us on the GPU and the marshalling of
// four outputs and sixteen arguments in Python took 23 us (8 us here, measured
// on the Grace host).
#include "bind_tensors.h"

#include <map>

#include "ffn_bind.h"
#include "fp8_overlap.h"

namespace {

using namespace wstma_bind;

PyObject *fp8_error = nullptr;  // Fp8Error

void check(int status, const char *call)
{
    if (status != FP8_OK)
        throw Failed{fp8_error, status, call};
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
        written(given);
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
        written(out_h);
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

PyMethodDef methods[] = {
    {"gemm", fast(&bind_gemm), METH_FASTCALL, nullptr},
    {"quantize", fast(&bind_quantize), METH_FASTCALL, nullptr},
    {"rmsnorm", fast(&bind_rmsnorm), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", fast(&bind_rmsnorm_backward), METH_FASTCALL, nullptr},
    {"kept_handle", &bind_kept_handle, METH_O, nullptr},
    {"set_error", &bind_set_error, METH_O, nullptr},
    {"ffn_linear", fast(&ffn_bind::linear), METH_FASTCALL, nullptr},
    {"ffn_linear_backward", fast(&ffn_bind::linear_backward), METH_FASTCALL, nullptr},
    {"ffn_gated", fast(&ffn_bind::gated), METH_FASTCALL, nullptr},
    {"ffn_gated_backward", fast(&ffn_bind::gated_backward), METH_FASTCALL, nullptr},
    {"ffn_set_error", &ffn_bind::set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_bind() { return PyModule_Create(&module); }
