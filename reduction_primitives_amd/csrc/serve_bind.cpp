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

#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <vector>

#include "rk.h"

namespace {

// Addresses of the C ABI's functions, in bind()'s order.
decltype(&rk_softmax) p_softmax;
decltype(&rk_draft_verify) p_draft_verify;
decltype(&rk_block_tables) p_block_tables;
decltype(&rk_slot_map) p_slot_map;
decltype(&rk_beam_select) p_beam_select;
decltype(&rk_fork_blocks) p_fork_blocks;
decltype(&rk_compact_blocks) p_compact_blocks;
decltype(&rk_copy_blocks) p_copy_blocks;
decltype(&rk_linear_recurrence) p_recurrence;
decltype(&rk_linear_recurrence_backward) p_recurrence_backward;

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
        if (!p_recurrence_backward) {
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

    // A 2-d tensor whose lines are contiguous (of no elements: of any strides).
    const at::Tensor &lines(const char *what, PyObject *o) const
    {
        const at::Tensor &t = here(what, o);
        if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1 && t.numel() > 0))
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

// The tokens of a recurrence: (sequences, tokens, channels), or (tokens,
// channels) where the sequences are packed, channels contiguous.
struct Tokens {
    rk_rows rows;
    const at::Tensor *t;
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

// What a call has written counts as changed in place, as with torch's own calls: a
// graph that has saved it refuses to go backward, rather than taking the new values.
void written(PyObject *o)
{
    if (!THPVariable_Check(o))
        return;                                // (None)
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_inference())                     // (which have no counters)
        t.unsafeGetTensorImpl()->bump_version();
}

PyObject *status(int rc, std::initializer_list<PyObject *> tensors)
{
    if (rc == RK_OK)
        for (PyObject *o : tensors)
            written(o);
    return status(rc);
}

// No call has a forward derivative: what carries a tangent is refused rather than
// left without.  (no_grad does not turn these off, an autograd function's forward
// does.)
void no_tangent(const char *name, const char *what, PyObject *o)
{
    if (THPVariable_Check(o) && c10::AutogradState::get_tls_state().get_fw_grad_mode() &&
        THPVariable_Unpack(o)._fw_grad(0).defined())
        refuse("%s: %s carries a tangent and the call has no forward derivative: unpack it", name, what);
}

// Calls without a backward pass: where gradients are recorded, what requires
// them is refused rather than left without.
void no_gradient(const char *name, const char *what, PyObject *o)
{
    no_tangent(name, what, o);
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
                            ws.bytes, handle(a[0])), {a[3]});
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
                                 tp, ap, ws.at, ws.bytes, handle(a[0])), {a[8], a[9]});
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
                                 handle(a[0])), {a[4], a[5], a[7], a[8]});
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
                             integer(a[6]), code, capacity, sp, pp, qp, tp, handle(a[0])), {a[8], a[9], a[10], a[11]});
}

Tokens tokens_of(const Call &c, const char *what, PyObject *o, const at::Tensor *like, at::ScalarType dtype, bool packed)
{
    const at::Tensor &t = c.here(what, o);
    if (t.dim() != (packed ? 2 : 3) || (t.size(-1) > 1 && t.stride(-1) != 1))
        refuse("%s: %s takes %s", c.name, what,
               packed ? "two dims, tokens and contiguous channels" : "three dims, sequences, tokens and contiguous channels");
    if (like && t.sizes() != like->sizes())
        refuse("%s: %s takes the gate's shape", c.name, what);
    if (t.scalar_type() != dtype)
        refuse("%s: %s takes %s", c.name, what, type_name(dtype));
    return Tokens{rk_rows{t.data_ptr(), packed ? 0 : t.stride(0), t.stride(-2)}, &t};
}

// What a recurrence's calls share: their extents, gates, inputs and offsets.
struct Recurrence {
    Tokens gate, x;
    int x_code, gate_code, kind, blend;
    at::ScalarType x_dtype;
    bool packed;
    int64_t n_seq, tokens, channels;
    const int32_t *starts;

    Recurrence(const Call &c, PyObject *gate_o, PyObject *x_o, PyObject *kind_o, PyObject *blend_o, PyObject *starts_o)
    {
        packed = starts_o != Py_None;
        const at::Tensor &g = c.here("gate", gate_o), &v = c.here("x", x_o);
        gate_code = c.prob_code("gate", g);
        x_code = c.prob_code("x", v);
        x_dtype = v.scalar_type();
        gate = tokens_of(c, "gate", gate_o, nullptr, g.scalar_type(), packed);
        x = tokens_of(c, "x", x_o, gate.t, x_dtype, packed);
        kind = small_integer(kind_o);
        blend = small_integer(blend_o);
        tokens = g.size(-2);
        channels = g.size(-1);
        n_seq = packed ? c.here("starts", starts_o).numel() - 1 : g.size(0);
        if (n_seq < 0)
            refuse("%s: %s takes an offset more than sequences", c.name, "starts");
        starts = static_cast<const int32_t *>(c.flat_or_null("starts", starts_o, n_seq + 1, at::kInt));
    }

    // A float32 line of channels for each of n sequences.
    float *states(const Call &c, const char *what, PyObject *o, int64_t n) const
    {
        if (o == Py_None)
            return nullptr;
        const at::Tensor &t = c.here(what, o);
        if (t.dim() != 2 || t.size(0) != n || t.size(1) != channels || t.scalar_type() != at::kFloat || !t.is_contiguous()) {
            PyErr_Format(PyExc_ValueError, "%s: %s takes %lld contiguous float32 lines of %lld channels", c.name, what,
                         (long long)n, (long long)channels);
            throw Refused();
        }
        return static_cast<float *>(t.data_ptr());
    }
};

// linear_recurrence(stream, gate, x, state, kind, blend, starts, sources, out, state_out, workspace)
PyObject *linear_recurrence(PyObject *const *a)
{
    // (gradients of the inputs are recorded around the call)
    no_gradient("linear_recurrence", "gate", a[1]);
    no_gradient("linear_recurrence", "x", a[2]);
    no_gradient("linear_recurrence", "state", a[3]);
    no_gradient("linear_recurrence", "out", a[8]);
    no_gradient("linear_recurrence", "state_out", a[9]);
    Call c("linear_recurrence", "gate", a[1]);
    const Recurrence r(c, a[1], a[2], a[4], a[5], a[6]);
    const Tokens out = tokens_of(c, "out", a[8], r.gate.t, r.x_dtype, r.packed);
    const auto *sources = static_cast<const int32_t *>(c.flat_or_null("sources", a[7], r.n_seq, at::kInt));
    int64_t lines = r.n_seq;
    if (sources && a[3] != Py_None) {
        const at::Tensor &t = c.here("state", a[3]);
        lines = t.dim() > 0 ? t.size(0) : 0;
    }
    const float *state = r.states(c, "state", a[3], lines);
    float *last = r.states(c, "state_out", a[9], r.n_seq);
    const Buffer ws = c.workspace(a[10]);
    return status(p_recurrence(r.x_code, r.gate_code, r.kind, r.blend, &r.gate.rows, &r.x.rows, state, lines, sources,
                               r.starts, r.n_seq, r.tokens, r.channels, &out.rows, last, ws.at, ws.bytes, handle(a[0])),
                  {a[8], a[9]});
}

// linear_recurrence_backward(stream, gate, x, out, dout, state, dstate_out, kind, blend, starts, dgate, dx, dstate, workspace)
PyObject *linear_recurrence_backward(PyObject *const *a)
{
    static constexpr const char *inputs[] = {"gate", "x", "out", "dout", "state", "dstate_out"},
                                *outputs[] = {"dgate", "dx", "dstate"};
    for (int i = 0; i < 6; ++i)
        no_gradient("linear_recurrence_backward", inputs[i], a[i + 1]);
    for (int i = 0; i < 3; ++i)
        no_gradient("linear_recurrence_backward", outputs[i], a[i + 10]);
    Call c("linear_recurrence_backward", "gate", a[1]);
    const Recurrence r(c, a[1], a[2], a[7], a[8], a[9]);
    const Tokens out = tokens_of(c, "out", a[3], r.gate.t, r.x_dtype, r.packed),
                 dout = tokens_of(c, "dout", a[4], r.gate.t, r.x_dtype, r.packed),
                 dgate = tokens_of(c, "dgate", a[10], r.gate.t, r.gate.t->scalar_type(), r.packed),
                 dx = tokens_of(c, "dx", a[11], r.gate.t, r.x_dtype, r.packed);
    const float *state = r.states(c, "state", a[5], r.n_seq), *dlast = r.states(c, "dstate_out", a[6], r.n_seq);
    float *dstate = r.states(c, "dstate", a[12], r.n_seq);
    const Buffer ws = c.workspace(a[13]);
    return status(p_recurrence_backward(r.x_code, r.gate_code, r.kind, r.blend, &r.gate.rows, &r.x.rows, &out.rows, &dout.rows,
                                        state, dlast, r.starts, r.n_seq, r.tokens, r.channels, &dgate.rows, &dx.rows, dstate,
                                        ws.at, ws.bytes, handle(a[0])), {a[10], a[11], a[12]});
}

// beam_select(stream, logits, scores, count, ended, end_token, best, tokens, parents, workspace)
PyObject *beam_select(PyObject *const *a)
{
    no_gradient("beam_select", "logits", a[1]);
    no_gradient("beam_select", "scores", a[2]);
    no_gradient("beam_select", "best", a[6]);
    Call c("beam_select", "logits", a[1]);
    const at::Tensor &x = c.lines("logits", a[1]), &scores = c.here("scores", a[2]);
    const int code = c.prob_code("logits", x);
    if (scores.dim() != 2 || scores.numel() != x.size(0))
        refuse("%s: %s takes requests times beams, a score for every line", c.name, "scores");
    const int64_t req = scores.size(0), beams = scores.size(1);
    const int count = small_integer(a[3]);
    if (beams > 0x7fffffff)
        return status(RK_ERR_UNSUPPORTED);
    if (beams == 0 || count < 1)
        return status(RK_ERR_INVALID_ARGUMENT);
    const at::Tensor &tokens = c.here("tokens", a[7]);
    const int tok = c.id_code("tokens", tokens);
    const auto *sp = static_cast<const float *>(c.flat("scores", a[2], req * beams, at::kFloat));
    const uint8_t *ep = nullptr;
    if (a[4] != Py_None) {
        const at::Tensor &e = c.here("ended", a[4]);
        ep = static_cast<const uint8_t *>(c.flat("ended", a[4], req * beams, e.scalar_type() == at::kByte ? at::kByte : at::kBool));
    }
    auto *bp = static_cast<float *>(c.flat("best", a[6], req * count, at::kFloat));
    auto *tp = c.flat("tokens", a[7], req * count, tokens.scalar_type());
    auto *pp = static_cast<int32_t *>(c.flat("parents", a[8], req * count, at::kInt));
    const Buffer ws = c.workspace(a[9]);
    return status(p_beam_select(code, tok, x.data_ptr(), x.stride(0), x.size(1), req, int(beams), sp, ep, integer(a[5]), count,
                                bp, tp, pp, ws.at, ws.bytes, handle(a[0])), {a[6], a[7], a[8]});
}

int64_t *state_out_of(const Call &c, PyObject *o) { return static_cast<int64_t *>(c.flat("state_out", o, 4, at::kLong)); }

// fork_blocks(stream, parents, lens, block_size, held, table, ring, state, n_blocks, table_out, held_out, lens_out, pairs,
//             state_out, workspace)
PyObject *fork_blocks(PyObject *const *a)
{
    Call c("fork_blocks", "parents", a[1]);
    const int64_t out = c.here("parents", a[1]).numel(), rows = c.here("lens", a[2]).numel(), places = c.here("ring", a[6]).numel();
    const at::Tensor &table = c.table(a[5], rows), &to = c.lines("table_out", a[9]);
    if (to.size(0) != out || to.size(1) != table.size(1) || to.scalar_type() != at::kInt)
        refuse("%s: %s takes an int32 line of the table's width for every parent", c.name, "table_out");
    const at::Tensor &state = c.here("state", a[7]);
    if (state.scalar_type() != at::kLong || !state.is_contiguous() || state.numel() < 2)
        refuse("%s: %s takes int64 head and tail", c.name, "state");
    const int64_t width = table.size(1);
    if (width > 0x7fffffff)
        return status(RK_ERR_UNSUPPORTED);
    const auto *par = static_cast<const int32_t *>(c.flat("parents", a[1], out, at::kInt));
    const auto *lens = static_cast<const int32_t *>(c.flat("lens", a[2], rows, at::kInt));
    const auto *held = static_cast<const int32_t *>(c.flat("held", a[4], rows, at::kInt));
    auto *ring = static_cast<int32_t *>(c.flat("ring", a[6], places, at::kInt));
    auto *ho = static_cast<int32_t *>(c.flat("held_out", a[10], out, at::kInt));
    auto *lo = static_cast<int32_t *>(c.flat("lens_out", a[11], out, at::kInt));
    auto *pairs = static_cast<int32_t *>(c.flat("pairs", a[12], 2 * out, at::kInt));
    auto *so = state_out_of(c, a[13]);
    const Buffer ws = c.workspace(a[14]);
    return status(p_fork_blocks(par, out, lens, rows, small_integer(a[3]), held, static_cast<const int32_t *>(table.data_ptr()),
                                table.stride(0), int(width), ring, places, static_cast<const int64_t *>(state.data_ptr()),
                                integer(a[8]), static_cast<int32_t *>(to.data_ptr()), to.stride(0), ho, lo, pairs, so, ws.at,
                                ws.bytes, handle(a[0])), {a[6], a[9], a[10], a[11], a[12], a[13]});
}

// compact_blocks(stream, held, table, ring, n_blocks, table_out, pairs, state_out, workspace)
PyObject *compact_blocks(PyObject *const *a)
{
    Call c("compact_blocks", "held", a[1]);
    const int64_t rows = c.here("held", a[1]).numel(), places = c.here("ring", a[3]).numel();
    const at::Tensor &table = c.table(a[2], rows), &to = c.lines("table_out", a[5]), &pairs = c.here("pairs", a[6]);
    if (to.sizes() != table.sizes() || to.scalar_type() != at::kInt)
        refuse("%s: %s takes the table's shape, int32", c.name, "table_out");
    if (pairs.numel() % 2)
        refuse("%s: %s takes pairs", c.name, "pairs");
    const int64_t width = table.size(1), most = pairs.numel() / 2;
    if (width > 0x7fffffff)
        return status(RK_ERR_UNSUPPORTED);
    const auto *held = static_cast<const int32_t *>(c.flat("held", a[1], rows, at::kInt));
    auto *ring = static_cast<int32_t *>(c.flat("ring", a[3], places, at::kInt));
    auto *pp = static_cast<int32_t *>(c.flat("pairs", a[6], 2 * most, at::kInt));
    auto *so = state_out_of(c, a[7]);
    const Buffer ws = c.workspace(a[8]);
    return status(p_compact_blocks(held, rows, static_cast<const int32_t *>(table.data_ptr()), table.stride(0), int(width),
                                   integer(a[4]), static_cast<int32_t *>(to.data_ptr()), to.stride(0), ring, places, pp, most, so,
                                   ws.at, ws.bytes, handle(a[0])), {a[3], a[5], a[6], a[7]});
}

// copy_blocks(stream, caches, pairs)
PyObject *copy_blocks(PyObject *const *a)
{
    Call c("copy_blocks", "pairs", a[2]);
    const int64_t n = c.here("pairs", a[2]).numel();
    if (n % 2)
        refuse("%s: %s takes pairs", c.name, "pairs");
    const auto *pairs = static_cast<const int32_t *>(c.flat("pairs", a[2], n, at::kInt));
    if (!PyList_Check(a[1]) && !PyTuple_Check(a[1])) {
        PyErr_Format(PyExc_TypeError, "%s: caches takes a list or tuple of tensors", c.name);
        throw Refused();
    }
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[1]);
    std::vector<rk_block_cache> caches;
    caches.reserve(size_t(count));
    for (Py_ssize_t i = 0; i < count; ++i) {
        no_gradient("copy_blocks", "caches", PySequence_Fast_GET_ITEM(a[1], i));
        const at::Tensor &t = c.here("caches", PySequence_Fast_GET_ITEM(a[1], i));
        if (t.dim() < 1)
            refuse("%s: %s takes tensors of blocks", c.name, "caches");
        int64_t whole = 1;                    // elements of a block, contiguous
        for (int64_t d = t.dim() - 1; d > 0; --d) {
            if (t.size(d) > 1 && t.stride(d) != whole)
                refuse("%s: %s takes tensors whose blocks are contiguous", c.name, "caches");
            whole *= t.size(d);
        }
        const int64_t size = int64_t(t.element_size());
        caches.push_back(rk_block_cache{t.data_ptr(), t.stride(0) * size, whole * size, t.size(0)});
    }
    const int rc = p_copy_blocks(caches.data(), int(count), pairs, n / 2, handle(a[0]));
    for (Py_ssize_t i = 0; i < count && rc == RK_OK; ++i)
        written(PySequence_Fast_GET_ITEM(a[1], i));
    return status(rc);
}

// bind(softmax, draft_verify, ...): the library's functions, in the order above.
PyObject *bind(PyObject *const *a)
{
    p_softmax = reinterpret_cast<decltype(p_softmax)>(handle(a[0]));
    p_draft_verify = reinterpret_cast<decltype(p_draft_verify)>(handle(a[1]));
    p_block_tables = reinterpret_cast<decltype(p_block_tables)>(handle(a[2]));
    p_slot_map = reinterpret_cast<decltype(p_slot_map)>(handle(a[3]));
    p_beam_select = reinterpret_cast<decltype(p_beam_select)>(handle(a[4]));
    p_fork_blocks = reinterpret_cast<decltype(p_fork_blocks)>(handle(a[5]));
    p_compact_blocks = reinterpret_cast<decltype(p_compact_blocks)>(handle(a[6]));
    p_copy_blocks = reinterpret_cast<decltype(p_copy_blocks)>(handle(a[7]));
    p_recurrence = reinterpret_cast<decltype(p_recurrence)>(handle(a[8]));
    p_recurrence_backward = reinterpret_cast<decltype(p_recurrence_backward)>(handle(a[9]));
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

PyMethodDef methods[] = {method<bind, 10>("bind"), method<beam_select, 10>("beam_select"),
                         method<fork_blocks, 15>("fork_blocks"), method<compact_blocks, 9>("compact_blocks"),
                         method<copy_blocks, 3>("copy_blocks"), method<linear_recurrence, 11>("linear_recurrence"),
                         method<linear_recurrence_backward, 14>("linear_recurrence_backward"), method<softmax, 5>("softmax"), method<draft_verify, 11>("draft_verify"),
                         method<block_tables, 10>("block_tables"), method<slot_map, 12>("slot_map"), PyMethodDef{}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", "Calls of the serving operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
