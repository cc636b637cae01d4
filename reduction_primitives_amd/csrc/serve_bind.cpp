// serve_bind.cpp -- the serving operators' calls from Python: checks torch
// tensors and passes their addresses to the C ABI.
//
// A decode step makes these calls with kernels of 3 to 5 us; looking at each
// tensor from Python and passing twenty arguments through ctypes took 4 us of
// a call, here it is under half of one.  The module holds no
// arithmetic and links nothing of librk.so: bind() is given the addresses of
// its functions, as the package has loaded them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "rk.h"

namespace {

// Addresses of the C ABI's functions, in bind()'s order.
decltype(&rk_softmax) p_softmax;
decltype(&rk_draft_verify) p_draft_verify;
decltype(&rk_block_tables) p_block_tables;
decltype(&rk_slot_map) p_slot_map;

// Thrown with a Python error set.
struct Refused {};

[[noreturn]] void refuse(const char *format, const char *call, const char *what, const char *more = "")
{
    PyErr_Format(PyExc_ValueError, format, call, what, more);
    throw Refused();
}

const char *type_name(at::ScalarType t) { return c10::toString(t); }

struct Buffer {
    void *at;
    size_t bytes;
};

// One call: its name, and the device of its first operand, made the current
// one for the call.
struct Call {
    const char *name;
    c10::Device device;
    c10::DeviceGuard guard;

    Call(const char *n, const char *what, PyObject *first) : name(n), device(device_of(n, what, first)), guard(device) {}

    static const at::Tensor &tensor(const char *name, const char *what, PyObject *o)
    {
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s: %s takes a tensor", name, what);
            throw Refused();
        }
        return THPVariable_Unpack(o);
    }

    static c10::Device device_of(const char *name, const char *what, PyObject *o)
    {
        if (!p_slot_map) {
            PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
            throw Refused();
        }
        const at::Tensor &t = tensor(name, what, o);
        if (!t.is_cuda())
            refuse("%s: %s is not on a GPU", name, what);
        return t.device();
    }

    const at::Tensor &here(const char *what, PyObject *o) const
    {
        const at::Tensor &t = tensor(name, what, o);
        if (!t.is_cuda())
            refuse("%s: %s is not on a GPU", name, what);
        if (t.device() != device)
            refuse("%s: %s is on another device", name, what);
        return t;
    }

    // A contiguous tensor of n elements of a dtype.
    void *flat(const char *what, PyObject *o, int64_t n, at::ScalarType dtype) const
    {
        const at::Tensor &t = here(what, o);
        if (t.scalar_type() != dtype || t.numel() != n || !t.is_contiguous()) {
            PyErr_Format(PyExc_ValueError, "%s: %s takes %lld contiguous %s", name, what, (long long)n, type_name(dtype));
            throw Refused();
        }
        return t.data_ptr();
    }

    void *flat_or_null(const char *what, PyObject *o, int64_t n, at::ScalarType dtype) const
    {
        return o == Py_None ? nullptr : flat(what, o, n, dtype);
    }

    // A 2-d tensor whose lines are contiguous.
    const at::Tensor &lines(const char *what, PyObject *o) const
    {
        const at::Tensor &t = here(what, o);
        if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
            refuse("%s: %s takes two dims, the second contiguous", name, what);
        return t;
    }

    // None: none is needed.
    Buffer workspace(PyObject *o) const
    {
        if (o == Py_None)
            return Buffer{nullptr, 0};
        const at::Tensor &t = here("workspace", o);
        if (!t.is_contiguous())
            refuse("%s: %s takes a contiguous tensor", name, "workspace");
        return Buffer{t.data_ptr(), t.nbytes()};
    }

    int prob_code(const char *what, const at::Tensor &t) const
    {
        switch (t.scalar_type()) {
        case at::kFloat: return RK_F32;
        case at::kBFloat16: return RK_BF16;
        case at::kHalf: return RK_F16;
        default: refuse("%s: %s cannot be %s", name, what, type_name(t.scalar_type()));
        }
    }

    int id_code(const char *what, const at::Tensor &t) const
    {
        switch (t.scalar_type()) {
        case at::kInt: return RK_I32;
        case at::kLong: return RK_I64;
        default: refuse("%s: %s cannot be %s", name, what, type_name(t.scalar_type()));
        }
    }

    // An int32 block table with a line for each of n requests.
    const at::Tensor &table(PyObject *o, int64_t n) const
    {
        const at::Tensor &t = lines("table", o);
        if (t.size(0) != n || t.scalar_type() != at::kInt)
            refuse("%s: %s takes an int32 line for every request", name, "table");
        return t;
    }
};

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Refused();
    return v;
}

// A C int: what does not fit one, the library refuses as -1.
int small_integer(PyObject *o)
{
    const int64_t v = integer(o);
    return v < -0x7fffffffLL - 1 || v > 0x7fffffffLL ? -1 : int(v);
}

void *handle(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw Refused();
    return p;
}

PyObject *status(int rc) { return PyLong_FromLong(rc); }

// Softmax has no backward pass: where gradients are recorded, what requires
// them is refused rather than left without.
void no_gradient(const char *name, const char *what, PyObject *o)
{
    if (THPVariable_Check(o) && c10::GradMode::is_enabled() && THPVariable_Unpack(o).requires_grad())
        refuse("%s: %s requires grad and the call has no gradient: detach it, or call under no_grad", name, what);
}

PyObject *softmax(PyObject *const *a)
{
    no_gradient("softmax", "x", a[1]);
    no_gradient("softmax", "temperature", a[2]);
    no_gradient("softmax", "out", a[3]);
    Call c("softmax", "x", a[1]);
    const at::Tensor &x = c.lines("x", a[1]);
    const int in = c.prob_code("x", x);
    const int64_t n = x.size(1), lines = x.size(0);
    const at::Tensor &out = c.lines("out", a[3]);
    if (out.size(0) != lines || out.size(1) != n)
        refuse("%s: %s takes x's shape and out_dtype", c.name, "out");
    const Buffer ws = c.workspace(a[4]);
    const int to = c.prob_code("out", out);
    const auto *tp = static_cast<const float *>(c.flat_or_null("temperature", a[2], lines, at::kFloat));
    return status(p_softmax(in, to, x.data_ptr(), n, lines, x.stride(0), tp, out.data_ptr(), out.stride(0), ws.at,
                            ws.bytes, handle(a[0])));
}

PyObject *draft_verify(PyObject *const *a)
{
    Call c("draft_verify", "p", a[1]);
    const at::Tensor &p = c.lines("p", a[1]);
    const int code = c.prob_code("p", p);
    const at::Tensor &drafted = c.here("drafted", a[3]);
    const at::Tensor &r = c.here("r", a[5]);
    const int tok = c.id_code("drafted", drafted);
    const int64_t vocab = p.size(1), req = r.numel(), drafts = drafted.numel();
    const int max_draft = small_integer(a[7]);
    if (p.size(0) != drafts + req)
        refuse("%s: %s takes a line for every draft and one for every request", c.name, "p");
    const void *q = nullptr;
    int64_t qs = 0;
    if (a[2] != Py_None) {
        const at::Tensor &t = c.lines("q", a[2]);
        if (t.scalar_type() != p.scalar_type() || t.size(0) != drafts || t.size(1) != vocab)
            refuse("%s: %s takes p's dtype and vocabulary, a line for every draft", c.name, "q");
        q = t.data_ptr();
        qs = t.stride(0);
    }
    const Buffer ws = c.workspace(a[10]);
    const at::ScalarType ids = drafted.scalar_type();
    const auto *xp = c.flat("drafted", a[3], drafts, ids);
    const auto *up = static_cast<const float *>(c.flat("u", a[4], drafts, at::kFloat));
    const auto *rp = static_cast<const float *>(c.flat("r", a[5], req, at::kFloat));
    const auto *sp = static_cast<const int32_t *>(c.flat_or_null("starts", a[6], req + 1, at::kInt));
    auto *tp = c.flat("tokens", a[8], req * (int64_t(max_draft) + 1), ids);
    auto *ap = static_cast<int32_t *>(c.flat("accepted", a[9], req, at::kInt));
    return status(p_draft_verify(code, tok, p.data_ptr(), p.stride(0), q, qs, vocab, req, drafts, max_draft, sp, xp, up, rp,
                                 tp, ap, ws.at, ws.bytes, handle(a[0])));
}

PyObject *block_tables(PyObject *const *a)
{
    Call c("block_tables", "lens", a[1]);
    const int64_t req = c.here("lens", a[1]).numel(), places = c.here("ring", a[5]).numel();
    const at::Tensor &table = c.table(a[4], req);
    const at::Tensor &state = c.here("state", a[6]);
    if (state.scalar_type() != at::kLong || !state.is_contiguous() || state.numel() < 2)
        refuse("%s: %s takes int64 head and tail", c.name, "state");
    const Buffer ws = c.workspace(a[9]);
    const int64_t width = table.size(1);
    if (width > 0x7fffffff)
        return status(RK_ERR_UNSUPPORTED);
    const auto *lp = static_cast<const int32_t *>(c.flat("lens", a[1], req, at::kInt));
    const int block = small_integer(a[2]);
    const auto *hp = static_cast<const int32_t *>(c.flat("held", a[3], req, at::kInt));
    auto *rp = static_cast<int32_t *>(c.flat("ring", a[5], places, at::kInt));
    auto *op = static_cast<int32_t *>(c.flat("held_out", a[7], req, at::kInt));
    auto *sp = static_cast<int64_t *>(c.flat("state_out", a[8], 4, at::kLong));
    return status(p_block_tables(lp, req, block, hp, op, static_cast<int32_t *>(table.data_ptr()), table.stride(0), int(width),
                                 rp, places, static_cast<const int64_t *>(state.data_ptr()), sp, ws.at, ws.bytes,
                                 handle(a[0])));
}

PyObject *slot_map(PyObject *const *a)
{
    Call c("slot_map", "lens", a[1]);
    const int64_t req = c.here("lens", a[1]).numel();
    const at::Tensor &table = c.table(a[4], req);
    const at::Tensor &slots = c.here("slots", a[8]);
    const int64_t capacity = integer(a[7]), width = table.size(1);
    const int code = c.id_code("slots", slots);
    if (width > 0x7fffffff)
        return status(RK_ERR_UNSUPPORTED);
    const auto *lp = static_cast<const int32_t *>(c.flat("lens", a[1], req, at::kInt));
    const auto *fp = static_cast<const int32_t *>(c.flat("fresh", a[2], req, at::kInt));
    const int block = small_integer(a[3]);
    const auto *hp = static_cast<const int32_t *>(c.flat("held", a[5], req, at::kInt));
    auto *sp = c.flat("slots", a[8], capacity, slots.scalar_type());
    auto *pp = static_cast<int32_t *>(c.flat("positions", a[9], capacity, at::kInt));
    auto *qp = static_cast<int32_t *>(c.flat("requests", a[10], capacity, at::kInt));
    auto *tp = static_cast<int32_t *>(c.flat("starts", a[11], req + 1, at::kInt));
    return status(p_slot_map(lp, fp, req, block, static_cast<const int32_t *>(table.data_ptr()), table.stride(0), int(width), hp,
                             integer(a[6]), code, capacity, sp, pp, qp, tp, handle(a[0])));
}

// bind(softmax, draft_verify, block_tables, slot_map): the library's functions.
PyObject *bind(PyObject *const *a)
{
    p_softmax = reinterpret_cast<decltype(p_softmax)>(handle(a[0]));
    p_draft_verify = reinterpret_cast<decltype(p_draft_verify)>(handle(a[1]));
    p_block_tables = reinterpret_cast<decltype(p_block_tables)>(handle(a[2]));
    p_slot_map = reinterpret_cast<decltype(p_slot_map)>(handle(a[3]));
    Py_RETURN_NONE;
}

// No C++ exception leaves a call.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name)
{
    PyMethodDef m{};
    m.ml_name = name;
    m.ml_meth = reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<F, N>));
    m.ml_flags = METH_FASTCALL;
    return m;
}

PyMethodDef methods[] = {method<bind, 4>("bind"), method<softmax, 5>("softmax"), method<draft_verify, 11>("draft_verify"),
                         method<block_tables, 10>("block_tables"), method<slot_map, 12>("slot_map"), PyMethodDef{}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", "Calls of the serving operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
