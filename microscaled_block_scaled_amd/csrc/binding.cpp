// binding.cpp -- the native half of block.py: one call that checks the
// tensors of a row, routing or epilogue operator, allocates its outputs and
// launches it through the C ABI (include/mxgemm.h).  In a decode step these
// operators run for 3 to 5 us on the GPU, and the same marshalling in Python
// takes 9 to 14 us a call; this takes about half.
//
// Each function takes the operator's arguments, the current device's index
// and the current stream's handle, and returns
//   * a tuple of the outputs (None for what was not wanted);
//   * an int, the library's error code, if the library refused the call;
//   * None for anything but plain tensors of the expected types, shapes and
//     device: block.py then says what is wrong.
// The library's functions are handed over by address (bind), so that this
// module and the ctypes binding always call the same library.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "mxgemm.h"

namespace {

struct Library {
    decltype(&mx_rmsnorm_quantize) rmsnorm_quantize;
    decltype(&mx_rmsnorm_backward_workspace) rmsnorm_backward_workspace;
    decltype(&mx_rmsnorm_backward) rmsnorm_backward;
    decltype(&mx_swiglu_quantize) swiglu_quantize;
    decltype(&mx_swiglu_backward) swiglu_backward;
    decltype(&mx_moe_sort_workspace) moe_sort_workspace;
    decltype(&mx_moe_sort) moe_sort;
    decltype(&mx_moe_gather) moe_gather;
    decltype(&mx_moe_combine) moe_combine;
    decltype(&mx_moe_combine_backward) moe_combine_backward;
    decltype(&mx_gemm_fused) gemm_fused;
    decltype(&mx_gemm_bf16_fused) gemm_bf16_fused;
    decltype(&mx_gemm_fused_plan) gemm_fused_plan;
    decltype(&mx_gemm_bf16_fused_plan) gemm_bf16_fused_plan;
} lib;
constexpr int kFunctions = sizeof(lib) / sizeof(void *);

// Thrown where an argument is not what the fast path takes.
struct Other {};

// The arguments of one call; device and stream are its last two.
struct Call {
    PyObject *const *args;
    int n, at = 0;
    int64_t device = -1;
    void *stream = nullptr;

    Call(PyObject *const *a, Py_ssize_t count, int want) : args(a), n((int)count)
    {
        if (n != want + 2 || !lib.gemm_fused) throw Other{};
        device = number(args[n - 2]);
        stream = reinterpret_cast<void *>(static_cast<uintptr_t>(number(args[n - 1])));
    }
    static int64_t number(PyObject *o)
    {
        if (!PyLong_CheckExact(o)) throw Other{};
        const int64_t v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Other{};
        }
        return v;
    }
    int64_t integer() { return number(args[at++]); }
    // Whether the next argument is None, which is passed over then.
    bool none()
    {
        if (args[at] != Py_None) return false;
        ++at;
        return true;
    }
    bool flag()
    {
        const int v = PyObject_IsTrue(args[at++]);
        if (v < 0) {
            PyErr_Clear();
            throw Other{};
        }
        return v == 1;
    }
    double real()
    {
        const double v = PyFloat_AsDouble(args[at++]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Other{};
        }
        return v;
    }
    // A tensor on the call's device, or with `none` allowed a null pointer.
    const at::Tensor *tensor(bool none = false)
    {
        PyObject *o = args[at++];
        if (none && o == Py_None) return nullptr;
        if (!THPVariable_CheckExact(o)) throw Other{};
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.get_device() != device) throw Other{};
        return &t;
    }
    at::Tensor make(at::IntArrayRef size, at::ScalarType type) const
    {
        return at::empty(size, at::TensorOptions().dtype(type).device(at::kCUDA, (int8_t)device));
    }
};

int dtype_code(const at::Tensor &t)
{
    if (t.scalar_type() == at::kBFloat16) return MX_IN_BF16;
    if (t.scalar_type() == at::kFloat) return MX_IN_FP32;
    throw Other{};
}

// Rows with contiguous elements that do not overlap: length and pitch.
struct Rows { int64_t n, width, ld; };
Rows rows_of(const at::Tensor &t, int64_t n = -1, int64_t width = -1)
{
    if (t.dim() != 2) throw Other{};
    const Rows r{t.size(0), t.size(1), t.size(0) <= 1 ? t.size(1) : t.stride(0)};
    if ((n >= 0 && r.n != n) || (width >= 0 && r.width != width) || r.ld < r.width ||
        (r.width > 1 && t.stride(1) != 1))
        throw Other{};
    return r;
}
Rows rows_like(const at::Tensor &t, const at::Tensor &like, int64_t n, int64_t width)
{
    if (t.scalar_type() != like.scalar_type()) throw Other{};
    return rows_of(t, n, width);
}

void dense(const at::Tensor &t, at::IntArrayRef size, at::ScalarType type)
{
    if (t.scalar_type() != type || t.sizes() != size || !t.is_contiguous()) throw Other{};
}

int vector_code(const at::Tensor &t, int64_t n)
{
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) throw Other{};
    return dtype_code(t);
}

int64_t row_bytes(int64_t fmt, int64_t k)
{
    if (fmt < MX_FMT_E2M1 || fmt > MX_FMT_E3M2) throw Other{};
    return fmt == MX_FMT_E2M1 ? k / 2 : fmt >= MX_FMT_E2M3 ? k / 4 * 3 : k;
}

void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }
void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

template <typename... T>
PyObject *outputs(int rc, const T &...t)
{
    if (rc != MX_OK) return PyLong_FromLong(rc);
    PyObject *r = PyTuple_New(sizeof...(t));
    if (!r) return nullptr;
    int i = 0;
    bool whole = true;
    auto put = [&](const at::Tensor &v) {
        if (!v.defined()) Py_INCREF(Py_None);
        PyObject *o = v.defined() ? THPVariable_Wrap(v) : Py_None;
        whole = whole && o;
        PyTuple_SET_ITEM(r, i++, o);
    };
    (put(t), ...);
    if (whole) return r;
    Py_DECREF(r);
    return nullptr;
}

PyObject *rmsnorm_quantize(Call c)
{
    const at::Tensor &x = *c.tensor(), &w = *c.tensor(), *res = c.tensor(true);
    const bool quantized = !c.none();                      // fmt None: no quantized output
    const int64_t fmt = quantized ? c.integer() : 0;
    const float eps = (float)c.real();
    const bool need_y = c.flag(), need_rstd = c.flag();
    const int dt = dtype_code(x);
    const Rows r = rows_of(x);
    const int wt = vector_code(w, r.width);
    const int64_t ldr = res ? rows_like(*res, x, r.n, r.width).ld : 0;
    at::Tensor h, q, qs, y, rstd;
    if (res) h = c.make({r.n, r.width}, x.scalar_type());
    if (quantized) {
        q = c.make({r.n, row_bytes(fmt, r.width)}, at::kByte);
        qs = c.make({r.n, r.width / 32}, at::kByte);
    }
    if (need_y) y = c.make({r.n, r.width}, x.scalar_type());
    if (need_rstd) rstd = c.make({r.n}, at::kFloat);
    const int rc = lib.rmsnorm_quantize((int)fmt, dt, wt, r.n, r.width, ptr(x), r.ld, ptr(res), ldr,
                                        ptr(w), eps, ptr(h), ptr(y), ptr(q), ptr(qs),
                                        (float *)ptr(rstd), c.stream);
    return outputs(rc, q, qs, h, y, rstd);
}

PyObject *rmsnorm_backward(Call c)
{
    const at::Tensor &dy = *c.tensor(), &h = *c.tensor(), &rstd = *c.tensor(), &w = *c.tensor();
    const at::Tensor *dh = c.tensor(true);
    const bool need_dw = c.flag();
    const int dt = dtype_code(h);
    const Rows r = rows_of(h);
    const int64_t lddy = rows_like(dy, h, r.n, r.width).ld;
    const int64_t lddh = dh ? rows_like(*dh, h, r.n, r.width).ld : 0;
    const int wt = vector_code(w, r.width);
    dense(rstd, {r.n}, at::kFloat);
    at::Tensor dx = c.make({r.n, r.width}, h.scalar_type()), dw, ws;
    int64_t bytes = 0;
    if (need_dw) {
        bytes = lib.rmsnorm_backward_workspace(r.n, r.width);
        if (bytes < 0) return PyLong_FromLongLong(bytes);
        dw = c.make({r.width}, at::kFloat);
        ws = c.make({bytes}, at::kByte);
    }
    const int rc = lib.rmsnorm_backward(dt, wt, r.n, r.width, ptr(dy), lddy, ptr(h), r.ld,
                                        (const float *)ptr(rstd), ptr(w), ptr(dh), lddh, ptr(dx),
                                        (float *)ptr(dw), ptr(ws), bytes, c.stream);
    return outputs(rc, dx, dw);
}

PyObject *swiglu_quantize(Call c)
{
    const at::Tensor &gu = *c.tensor();
    const int64_t fmt = c.integer();
    const Rows r = rows_of(gu);
    if (r.width % 2) throw Other{};
    const int64_t width = r.width / 2;
    at::Tensor q = c.make({r.n, row_bytes(fmt, width)}, at::kByte);
    at::Tensor qs = c.make({r.n, width / 32}, at::kByte);
    const int rc = lib.swiglu_quantize((int)fmt, dtype_code(gu), r.n, width, ptr(gu), r.ld, ptr(q),
                                       ptr(qs), c.stream);
    return outputs(rc, q, qs);
}

PyObject *swiglu_backward(Call c)
{
    const at::Tensor &dy = *c.tensor(), &gu = *c.tensor();
    const Rows r = rows_of(gu);
    if (r.width % 2) throw Other{};
    const int64_t lddy = rows_like(dy, gu, r.n, r.width / 2).ld;
    const int dt = dtype_code(gu);
    at::Tensor dgu = c.make({r.n, r.width}, gu.scalar_type());
    const int rc = lib.swiglu_backward(dt, r.n, r.width / 2, ptr(dy), lddy, ptr(gu), r.ld, ptr(dgu),
                                       c.stream);
    return outputs(rc, dgu);
}

PyObject *moe_sort(Call c)
{
    const at::Tensor &ids = *c.tensor();
    const int64_t experts = c.integer();
    if (ids.dim() != 2 || !ids.is_contiguous() ||
        (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong))
        throw Other{};
    const int64_t tokens = ids.size(0), top = ids.size(1);
    const int64_t bytes = lib.moe_sort_workspace(tokens, top, experts);
    if (bytes < 0) return PyLong_FromLongLong(bytes);
    at::Tensor group_rows = c.make({experts}, at::kLong), row_of = c.make({tokens, top}, at::kInt), ws;
    if (bytes) ws = c.make({bytes}, at::kByte);
    const int rc = lib.moe_sort((int)ids.element_size(), tokens, top, experts, ptr(ids),
                                (int64_t *)ptr(group_rows), (int32_t *)ptr(row_of), ptr(ws), bytes,
                                c.stream);
    return outputs(rc, group_rows, row_of);
}

// A plan's row_of: tokens x top int32.
struct Plan { const int32_t *row_of; int64_t tokens, top; };
Plan plan_of(const at::Tensor &t)
{
    if (t.dim() != 2 || t.scalar_type() != at::kInt || !t.is_contiguous()) throw Other{};
    return {(const int32_t *)t.data_ptr(), t.size(0), t.size(1)};
}

PyObject *moe_gather(Call c)
{
    const Plan p = plan_of(*c.tensor());
    const at::Tensor &x = *c.tensor(), *s = c.tensor(true);
    const Rows r = rows_of(x, p.tokens);
    const int64_t size = (int64_t)x.element_size();
    at::Tensor xs = c.make({p.tokens * p.top, r.width}, x.scalar_type()), ss;
    int64_t sbytes = 0, lds = 0;
    if (s) {
        const Rows rs = rows_of(*s, p.tokens);
        sbytes = rs.width * (int64_t)s->element_size();
        lds = rs.ld * (int64_t)s->element_size();
        ss = c.make({p.tokens * p.top, rs.width}, s->scalar_type());
    }
    const int rc = lib.moe_gather(p.tokens, p.top, p.row_of, ptr(x), r.width * size, r.ld * size,
                                  ptr(s), sbytes, lds, ptr(xs), ptr(ss), c.stream);
    return outputs(rc, xs, ss);
}

PyObject *moe_combine(Call c)
{
    const Plan p = plan_of(*c.tensor());
    const at::Tensor &y = *c.tensor(), *w = c.tensor(true), *res = c.tensor(true);
    const Rows r = rows_of(y);
    const int dt = dtype_code(y);
    if (w) dense(*w, {p.tokens, p.top}, at::kFloat);
    const int64_t ldr = res ? rows_like(*res, y, p.tokens, r.width).ld : 0;
    at::Tensor out = c.make({p.tokens, r.width}, y.scalar_type());
    const int rc = lib.moe_combine(dt, p.tokens, p.top, r.width, p.row_of, ptr(y), r.n, r.ld,
                                   (const float *)ptr(w), ptr(res), ldr, ptr(out), c.stream);
    return outputs(rc, out);
}

PyObject *moe_combine_backward(Call c)
{
    const Plan p = plan_of(*c.tensor());
    const at::Tensor &dout = *c.tensor(), &y = *c.tensor(), &w = *c.tensor();
    const Rows r = rows_of(y);
    const int dt = dtype_code(y);
    const int64_t lddo = rows_like(dout, y, p.tokens, r.width).ld;
    dense(w, {p.tokens, p.top}, at::kFloat);
    at::Tensor dy = c.make({r.n, r.width}, y.scalar_type());
    at::Tensor dw = c.make({p.tokens, p.top}, at::kFloat);
    const int rc = lib.moe_combine_backward(dt, p.tokens, p.top, r.width, p.row_of, ptr(dout), lddo,
                                            ptr(y), r.n, r.ld, (const float *)ptr(w), ptr(dy),
                                            (float *)ptr(dw), c.stream);
    return outputs(rc, dy, dw);
}

// Bytes of packed elements or scales: n rows.
int64_t bytes_of(const at::Tensor &t, int64_t n, int64_t width = -1)
{
    if (t.dim() != 2 || t.scalar_type() != at::kByte || !t.is_contiguous() || t.size(0) != n ||
        (width >= 0 && t.size(1) != width))
        throw Other{};
    return t.size(1);
}

// bias, act, residual and output type of a fused epilogue; makes C.
struct Ep {
    const at::Tensor *bias, *res;
    int bias_code = 0, out_code;
    int64_t act, ldr = 0;
    at::Tensor out;
    Ep(Call &c, int64_t M, int64_t N)
    {
        bias = c.tensor(true);
        act = c.integer();
        if (act < MX_ACT_NONE || act > MX_ACT_GELU_TANH) throw Other{};   // before it is an int
        res = c.tensor(true);
        out_code = (int)c.integer();
        if (out_code != MX_OUT_FP32 && out_code != MX_OUT_BF16) throw Other{};
        const at::ScalarType type = out_code == MX_OUT_FP32 ? at::kFloat : at::kBFloat16;
        if (bias) bias_code = vector_code(*bias, N);
        if (res) {
            if (res->scalar_type() != type) throw Other{};
            ldr = rows_of(*res, M, N).ld;
        }
        const at::Tensor *given = c.tensor(true);
        if (given) {
            dense(*given, {M, N}, type);
            out = *given;
        } else {
            out = c.make({M, N}, type);
        }
    }
};

PyObject *gemm_fused(Call c)
{
    const int64_t fa = c.integer(), fb = c.integer();
    const at::Tensor &a = *c.tensor(), &as = *c.tensor(), &b = *c.tensor(), &bs = *c.tensor();
    if (a.dim() != 2 || b.dim() != 2) throw Other{};
    const int64_t M = a.size(0), N = b.size(0), ra = bytes_of(a, M);
    const int64_t K = fa == MX_FMT_E2M1 ? 2 * ra : ra;
    // the formats this GEMM takes have whole elements in any number of bytes
    if ((fa != MX_FMT_E2M1 && fa != MX_FMT_E4M3) || (fb != MX_FMT_E2M1 && fb != MX_FMT_E4M3))
        throw Other{};
    bytes_of(b, N, row_bytes(fb, K));
    bytes_of(as, M, K / 32);
    bytes_of(bs, N, K / 32);
    Ep e(c, M, N);
    mx_plan_t plan;
    int rc = lib.gemm_fused_plan((int)fa, (int)fb, M, N, K, e.out_code, &plan);
    if (rc != MX_OK) return PyLong_FromLong(rc);
    at::Tensor ws;
    if (plan.workspace_bytes) ws = c.make({plan.workspace_bytes}, at::kByte);
    rc = lib.gemm_fused((int)fa, (int)fb, M, N, K, ptr(a), ptr(as), ptr(b), ptr(bs), ptr(e.bias),
                        e.bias_code, (int)e.act, ptr(e.res), e.ldr, ptr(e.out), e.out_code, ptr(ws),
                        plan.workspace_bytes, c.stream);
    return outputs(rc, e.out);
}

PyObject *gemm_bf16_fused(Call c)
{
    const at::Tensor &a = *c.tensor(), &b = *c.tensor();
    if (a.dim() != 2 || b.dim() != 2) throw Other{};
    const int64_t M = a.size(0), N = b.size(0), K = a.size(1);
    dense(a, {M, K}, at::kBFloat16);
    dense(b, {N, K}, at::kBFloat16);
    Ep e(c, M, N);
    mx_plan_t plan;
    int rc = lib.gemm_bf16_fused_plan(M, N, K, e.out_code, &plan);
    if (rc != MX_OK) return PyLong_FromLong(rc);
    at::Tensor ws;
    if (plan.workspace_bytes) ws = c.make({plan.workspace_bytes}, at::kByte);
    rc = lib.gemm_bf16_fused(M, N, K, ptr(a), ptr(b), ptr(e.bias), e.bias_code, (int)e.act, ptr(e.res),
                             e.ldr, ptr(e.out), e.out_code, ptr(ws), plan.workspace_bytes, c.stream);
    return outputs(rc, e.out);
}

// Every entry: the fast path, None where it does not apply.  No C++ exception
// passes the interpreter: one of torch's (no memory for an output) comes
// before anything is launched, and block.py, which tries the same, meets it
// again and raises it as torch does.
template <PyObject *(*F)(Call), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        return F(Call(args, n, N));
    } catch (const Other &) {
    } catch (const std::exception &) {
    }
    Py_RETURN_NONE;
}

// bind(addresses): the library's functions, in the order of struct Library.
PyObject *bind(PyObject *, PyObject *arg)
{
    if (!PyTuple_Check(arg) || PyTuple_GET_SIZE(arg) != kFunctions) {
        PyErr_SetString(PyExc_ValueError, "bind takes the addresses of all library functions");
        return nullptr;
    }
    uintptr_t at[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
        at[i] = (uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(arg, i));
        if (PyErr_Occurred()) return nullptr;
    }
    __builtin_memcpy(&lib, at, sizeof(lib));
    Py_RETURN_NONE;
}

#define ENTRY(name, args) \
    {#name, (PyCFunction)(void (*)(void))entry<name, args>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    ENTRY(rmsnorm_quantize, 7),
    ENTRY(rmsnorm_backward, 6),
    ENTRY(swiglu_quantize, 2),
    ENTRY(swiglu_backward, 2),
    ENTRY(moe_sort, 2),
    ENTRY(moe_gather, 3),
    ENTRY(moe_combine, 4),
    ENTRY(moe_combine_backward, 4),
    ENTRY(gemm_fused, 11),
    ENTRY(gemm_bf16_fused, 7),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr,
                      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
