// Python entry points of the feed-forward operators (include/ffn_ops.h), beside the 8-bit
// operators' in the module that fp8_bind.cpp makes: torch tensors in, the C ABI called on
// their device's current stream, torch tensors out.
#pragma once

#include "bind_tensors.h"
#include "ffn_ops.h"
#include "ffn_overlap.h"

namespace ffn_bind {

using namespace wstma_bind;

inline PyObject *error = nullptr;  // FfnError

inline void check(int status, const char *call)
{
    if (status != FFN_OK)
        throw Failed{error, status, call};
}

inline ffn_matrix matrix(const Tensor &t, int64_t R, int64_t C, const char *what)
{
    return {data(t), need_bf16(t, R, C, what)};
}

// An R x C result whose rows start at multiples of 128 bytes.
inline Tensor whole_rows(const Place &at, int64_t R, int64_t C, at::ScalarType type)
{
    const int64_t per = type == at::kFloat ? 32 : 64, ld = (C + per - 1) / per * per;
    return ld == C ? at.empty({R, C}, type) : at::detail::empty_strided_cuda({R, C}, {ld, 1}, type, at.on);
}

inline ffn_matrix result(const Tensor &t) { return {data(t), t.size(0) > 1 ? t.stride(0) : t.size(1)}; }

inline int32_t activation(PyObject *o)
{
    const long a = PyLong_AsLong(o);
    if (a == -1 && PyErr_Occurred())
        throw python_error();
    return (int32_t)a;
}

inline at::ScalarType result_type(PyObject *o, const char *what)
{
    if (!THPDtype_Check(o))
        type_error(std::string(what) + " must be a torch.dtype");
    const at::ScalarType st = reinterpret_cast<THPDtype *>(o)->scalar_type;
    if (st != at::kBFloat16 && st != at::kFloat)
        type_error(std::string(what) + " must be bf16 or fp32");
    return st;
}

inline wstma::Span span(const Tensor &t)
{
    const int64_t size = t.element_size();
    return {data(t), (t.size(0) > 1 ? t.stride(0) : t.size(1)) * size, t.size(1) * size, t.size(0)};
}

inline void need_apart(const Tensor &out, const Tensor &in, const char *what)
{
    if (wstma::touch(span(out), span(in)))
        value_error(std::string("out lies over ") + what + ": it may be the residual itself, or apart");
}

inline int truth(PyObject *o)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0)
        throw python_error();
    return t;
}

// An 8-bit matrix of R rows and C columns.
inline ffn_quantized quantized(const Tensor &codes, const Tensor &scales, int64_t R, int64_t C, const char *what)
{
    const int64_t ld = codes_pitch(codes, what);
    if (codes.size(0) != R || codes.size(1) != C)
        value_error(std::string(what) + " must be " + size_text(R, C));
    need_scales(scales, codes, what);
    return {data(codes), ld, data(scales)};
}

// Runs a call with a workspace of its own, freed on return to this stream's (or this graph's)
// later allocations: they run after it.
template <typename Args>
void run(const Place &at, const Args &args, int (*measure)(const Args *, int64_t *),
         int (*call)(const Args *, void *, int64_t, void *), const char *name)
{
    int64_t need = 0;
    check(measure(&args, &need), name);
    Tensor work;
    if (need)
        work = at.empty({need}, at::kByte);
    check(call(&args, need ? data(work) : nullptr, need, at.stream), name);
}

// linear(x, weight, bias or None, activation, residual or None, save, out or None, out_dtype or None) -> y or (y, z)
inline PyObject *linear(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 8);
        const Tensor &x = tensor(args[0], "x"), &w = tensor(args[1], "weight");
        const Tensor *bias = maybe_tensor(args[2], "bias"), *res = maybe_tensor(args[4], "residual"),
                     *given = maybe_tensor(args[6], "out");
        if (x.dim() != 2 || w.dim() != 2)
            value_error("x and weight must be matrices");
        ffn_linear_args a = {};
        const int64_t M = a.M = x.size(0), K = a.K = x.size(1), N = a.N = w.size(0);
        a.x = matrix(x, M, K, "x");
        a.weight = matrix(w, N, K, "weight");
        if (bias) {
            need_vector(*bias, N, "bias");
            a.bias = data(*bias);
            a.bias_type = element_type(*bias, "bias");
        }
        a.activation = activation(args[3]);
        if (res)
            a.residual = matrix(*res, M, N, "residual");
        const int save = truth(args[5]);
        const at::ScalarType type = args[7] != Py_None ? result_type(args[7], "out_dtype")
                                    : given            ? given->scalar_type()
                                                       : at::kBFloat16;
        if (given && given->scalar_type() != type)
            value_error("out is not of out_dtype");
        Place at(x);
        at.same(&w), at.same(bias), at.same(res), at.same(given);
        Tensor y, z;
        if (given) {
            y = *given;
            if (y.dim() != 2 || y.size(0) != M || y.size(1) != N)
                value_error("out must be " + size_text(M, N));
            a.y = {data(y), pitch_of(y, "out")};
            need_apart(y, x, "x");
            need_apart(y, w, "weight");
            if (bias)
                need_apart(y, bias->unsqueeze(0), "bias");
            const bool same = res && data(res) == data(y) && res->scalar_type() == y.scalar_type() &&
                              (M <= 1 || a.residual.ld == a.y.ld);
            if (res && !same)
                need_apart(y, *res, "residual");
        } else {
            y = whole_rows(at, M, N, type);
            a.y = result(y);
        }
        a.y_type = element_type(y, "out");
        if (save) {
            z = whole_rows(at, M, N, at::kBFloat16);
            a.z = result(z);
        }
        run(at, a, &ffn_linear_workspace, &ffn_linear, "ffn_linear");
        written(given);
        if (!save)
            return wrap(std::move(y));
        return tuple_of({wrap(std::move(y)), wrap(std::move(z))});
    });
}

// linear_backward(dy, x, weight, z or None, activation, bias, dweight_dtype) -> (dx, dweight, dbias or None)
inline PyObject *linear_backward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 7);
        const Tensor &dy = tensor(args[0], "dy"), &x = tensor(args[1], "x"), &w = tensor(args[2], "weight");
        const Tensor *z = maybe_tensor(args[3], "z");
        if (x.dim() != 2 || w.dim() != 2)
            value_error("x and weight must be matrices");
        ffn_linear_backward_args a = {};
        const int64_t M = a.M = x.size(0), K = a.K = x.size(1), N = a.N = w.size(0);
        a.dy = matrix(dy, M, N, "dy");
        a.x = matrix(x, M, K, "x");
        a.weight = matrix(w, N, K, "weight");
        a.activation = activation(args[4]);
        if (z)
            a.z = matrix(*z, M, N, "z");
        else if (a.activation != FFN_ACT_NONE)
            value_error("the gradient of an activation needs z, which linear saves");
        const int bias = truth(args[5]);
        const at::ScalarType wtype = result_type(args[6], "grad_dtype");
        a.dweight_type = wtype == at::kFloat ? FFN_FP32 : FFN_BF16;
        Place at(dy);
        at.same(&x), at.same(&w), at.same(z);
        Tensor dx = whole_rows(at, M, K, at::kBFloat16), dw = whole_rows(at, N, K, wtype), db;
        a.dx = result(dx);
        a.dweight = result(dw);
        if (bias) {
            db = at.empty({N}, at::kFloat);
            a.dbias = static_cast<float *>(data(db));
        }
        run(at, a, &ffn_linear_backward_workspace, &ffn_linear_backward, "ffn_linear_backward");
        PyObject *third = Py_None;
        if (bias)
            third = wrap(std::move(db));
        else
            Py_INCREF(third);
        return tuple_of({wrap(std::move(dx)), wrap(std::move(dw)), third});
    });
}

// gated(x, w_gate, w_up, activation, save: 0, 1 = bf16, 2 = e4m3) -> h, or (h, g, u), or (h, codes, scales, codes, scales)
inline PyObject *gated(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 5);
        const Tensor &x = tensor(args[0], "x"), &wg = tensor(args[1], "w_gate"), &wu = tensor(args[2], "w_up");
        if (x.dim() != 2 || wg.dim() != 2)
            value_error("x and w_gate must be matrices");
        ffn_gated_args a = {};
        const int64_t M = a.M = x.size(0), C = a.C = x.size(1), F = a.F = wg.size(0);
        a.x = matrix(x, M, C, "x");
        a.w_gate = matrix(wg, F, C, "w_gate");
        a.w_up = matrix(wu, F, C, "w_up");
        a.activation = activation(args[3]);
        const int32_t save = activation(args[4]);
        Place at(x);
        at.same(&wg), at.same(&wu);
        Tensor h = whole_rows(at, M, F, at::kBFloat16), g, u, gs, us;
        a.h = result(h);
        if (save == 1) {
            g = whole_rows(at, M, F, at::kBFloat16), u = whole_rows(at, M, F, at::kBFloat16);
            a.g = result(g), a.u = result(u);
        } else if (save == 2) {
            std::tie(g, gs) = at.quantized(M, F);
            std::tie(u, us) = at.quantized(M, F);
            a.qg = {data(g), padded(F), data(gs)};
            a.qu = {data(u), padded(F), data(us)};
        }
        run(at, a, &ffn_gated_workspace, &ffn_gated, "ffn_gated");
        if (save == 1)
            return tuple_of({wrap(h), wrap(g), wrap(u)});
        if (save == 2)
            return tuple_of({wrap(h), wrap(g), wrap(gs), wrap(u), wrap(us)});
        return wrap(std::move(h));
    });
}

// gated_backward(dy, x, saved: (g, u) or (codes, scales, codes, scales), w_gate, w_up, w_down, activation,
//                dweight_dtype) -> (dx, dw_gate, dw_up, dw_down)
inline PyObject *gated_backward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        need_args(n, 8);
        const Tensor &dy = tensor(args[0], "dy"), &x = tensor(args[1], "x");
        const Tensor &wg = tensor(args[3], "w_gate"), &wu = tensor(args[4], "w_up"), &wd = tensor(args[5], "w_down");
        if (x.dim() != 2 || wg.dim() != 2 || dy.dim() != 2)
            value_error("dy, x and w_gate must be matrices");
        ffn_gated_backward_args a = {};
        const int64_t M = a.M = x.size(0), C = a.C = x.size(1), F = a.F = wg.size(0), N = a.N = dy.size(1);
        a.dy = matrix(dy, M, N, "dy");
        a.x = matrix(x, M, C, "x");
        a.w_gate = matrix(wg, F, C, "w_gate");
        a.w_up = matrix(wu, F, C, "w_up");
        a.w_down = matrix(wd, N, F, "w_down");
        a.activation = activation(args[6]);
        Place at(dy);
        at.same(&x), at.same(&wg), at.same(&wu), at.same(&wd);
        if (!PyTuple_Check(args[2]) || (PyTuple_GET_SIZE(args[2]) != 2 && PyTuple_GET_SIZE(args[2]) != 4))
            type_error("saved must be what gated() saved: (g, u), or two pairs of codes and scales");
        if (PyTuple_GET_SIZE(args[2]) == 2) {
            const Tensor &g = tensor(PyTuple_GET_ITEM(args[2], 0), "g"), &u = tensor(PyTuple_GET_ITEM(args[2], 1), "u");
            at.same(&g), at.same(&u);
            a.g = matrix(g, M, F, "g");
            a.u = matrix(u, M, F, "u");
        } else {
            const Tensor &g = tensor(PyTuple_GET_ITEM(args[2], 0), "g"), &gs = tensor(PyTuple_GET_ITEM(args[2], 1), "g's scales"),
                         &u = tensor(PyTuple_GET_ITEM(args[2], 2), "u"), &us = tensor(PyTuple_GET_ITEM(args[2], 3), "u's scales");
            at.same(&g), at.same(&gs), at.same(&u), at.same(&us);
            a.qg = quantized(g, gs, M, F, "g");
            a.qu = quantized(u, us, M, F, "u");
        }
        const at::ScalarType wtype = result_type(args[7], "grad_dtype");
        a.dweight_type = wtype == at::kFloat ? FFN_FP32 : FFN_BF16;
        Tensor dx = whole_rows(at, M, C, at::kBFloat16), dwg = whole_rows(at, F, C, wtype), dwu = whole_rows(at, F, C, wtype),
               dwd = whole_rows(at, N, F, wtype);
        a.dx = result(dx);
        a.dw_gate = result(dwg);
        a.dw_up = result(dwu);
        a.dw_down = result(dwd);
        run(at, a, &ffn_gated_backward_workspace, &ffn_gated_backward, "ffn_gated_backward");
        return tuple_of({wrap(dx), wrap(dwg), wrap(dwu), wrap(dwd)});
    });
}

inline PyObject *set_error(PyObject *, PyObject *type)
{
    Py_INCREF(type);
    Py_XSETREF(error, type);
    Py_RETURN_NONE;
}

}  // namespace ffn_bind
