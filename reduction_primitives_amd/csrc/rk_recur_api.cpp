// rk_recur_api.cpp -- the gated linear recurrence of the C ABI (include/rk.h):
// argument checks, plan, launch.
#include "rk.h"

#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>

#include "rk_checks.hpp"
#include "rk_host.hpp"
#include "rk_recur.hpp"

namespace rk {
size_t round_up_256(size_t b);
}

using namespace rk;
using namespace rk::checks;

namespace {

// The extents that all of a call's tensors share.
struct Extents {
    int64_t seqs, tokens, channels;   // with offsets one sequence of all tokens
    bool empty() const { return seqs == 0 || tokens == 0 || channels == 0; }
};

bool fits(const rk_rows &t, const Extents &e)
{
    constexpr int64_t most = int64_t(1) << 48;
    const int64_t s = t.seq_stride, r = t.token_stride;
    return s >= 0 && r >= 0 && s <= most && r <= most && (e.seqs <= 1 || s == 0 || e.seqs <= most / s) &&
           (e.tokens <= 1 || r == 0 || e.tokens <= most / r);
}

Span span_of(const rk_rows &t, const Extents &e, int size)
{
    return span(t.data, e.empty() ? 0
                                  : ((e.seqs > 1 ? (e.seqs - 1) * t.seq_stride : 0) +
                                     (e.tokens > 1 ? (e.tokens - 1) * t.token_stride : 0) + e.channels) * size);
}

// No two elements of a written tensor share a place: one stride steps over all the other one covers.
bool unfolded(const rk_rows &t, const Extents &e)
{
    const int64_t s = e.seqs > 1 ? t.seq_stride : 0, r = e.tokens > 1 ? t.token_stride : 0;
    const bool sequences = e.seqs <= 1 || s >= (e.tokens - 1) * r + e.channels;
    const bool tokens = e.tokens <= 1 || r >= (e.seqs - 1) * s + e.channels;
    return (sequences && (e.tokens <= 1 || r >= e.channels)) || (tokens && (e.seqs <= 1 || s >= e.channels));
}

bool same_strides(const rk_rows &a, int a_size, const rk_rows &b, int b_size, const Extents &e)
{
    return (e.seqs <= 1 || a.seq_stride * a_size == b.seq_stride * b_size) &&
           (e.tokens <= 1 || a.token_stride * a_size == b.token_stride * b_size);
}

// Whether `w`, which is written, may stand beside `o`: apart from it, in other
// columns of the same rows, or (`same`) in its very place.
bool may_stand(const rk_rows &w, int w_size, const rk_rows &o, int o_size, const Extents &e, bool same)
{
    if (!o.data || !overlap(span_of(w, e, w_size), span_of(o, e, o_size)))
        return true;
    if (!same_strides(w, w_size, o, o_size, e))
        return false;
    if (w.data == o.data)
        return same && w_size == o_size;
    const int64_t s = e.seqs > 1 ? w.seq_stride * w_size : 0, r = e.tokens > 1 ? w.token_stride * w_size : 0;
    const int64_t low = s && r ? (s < r ? s : r) : s + r, high = s < r ? r : s;
    if (low == 0 || high % low)
        return false;
    const int64_t d = int64_t(reinterpret_cast<uintptr_t>(w.data) - reinterpret_cast<uintptr_t>(o.data));
    const int64_t off = (d % low + low) % low;
    return off >= e.channels * o_size && off + e.channels * w_size <= low;
}

RecurTensor flat(const rk_rows *t, const Extents &e)
{
    if (!t)
        return RecurTensor{nullptr, 0, 0};
    // one token a sequence: the sequences are the rows
    return RecurTensor{t->data, t->seq_stride, e.tokens == 1 && e.seqs > 1 ? t->seq_stride : t->token_stride};
}

// Sequences follow each other at the tokens' own stride.
bool follows(const rk_rows *t, const Extents &e)
{
    return !t || e.seqs <= 1 || e.tokens == 1 || t->seq_stride == e.tokens * t->token_stride;
}

struct Request {
    int x_dtype, gate_dtype, kind, blend;
    const rk_rows *gate, *x, *h, *dout, *out, *dgate;
    const float *state, *dlast;
    float *state_out;
    const int32_t *sources, *starts;
    int64_t n_states, n_seq, tokens, channels;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
};

bool states_fit(int64_t n, int64_t channels) { return channels == 0 || n <= (int64_t(1) << 44) / channels; }

// Room for the first states, behind the records.  Where the last ones take their
// place and states pass from tile to tile, the tiles read a copy: one that is
// computed late, or once more by a block that helps, would find a last state there.
size_t kept_states(int64_t n_seq, int64_t channels) { return round_up_256(size_t(n_seq) * size_t(channels) * 4); }

size_t workspace_size(int x_dtype, int gate_dtype, int64_t n_seq, int64_t tokens, int64_t channels, bool packed)
{
    if (n_seq < 0 || tokens < 0 || n_seq > 0x7fffffff || tokens > 0x7fffffff)
        return 0;
    const int cus = host::device_cus();
    size_t most = 0;
    RecurPlan p;
    for (const bool backward : {false, true}) {
        if ((packed || n_seq * tokens <= 0x7fffffff) &&
            plan_recur(x_dtype, gate_dtype, packed ? tokens : n_seq * tokens, 1, packed ? 0 : tokens, channels, backward, cus, &p) == ST_OK &&
            p.ws_bytes > most)
            most = p.ws_bytes;
        if (!packed && plan_recur(x_dtype, gate_dtype, tokens, n_seq, tokens, channels, backward, cus, &p) == ST_OK &&
            p.ws_bytes > most)
            most = p.ws_bytes;
    }
    return most && states_fit(n_seq, channels) ? most + kept_states(n_seq, channels) : 0;
}

int recur(const char *name, const Request &q, bool backward)
{
    if (!dtype_known(q.x_dtype) || !dtype_known(q.gate_dtype) || q.kind < RK_GATE_VALUE || q.kind > RK_GATE_SIGMOID ||
        (q.blend != 0 && q.blend != 1) || q.n_seq < 0 || q.tokens < 0 || q.channels < 0 || q.n_states < 0)
        return RK_ERR_INVALID_ARGUMENT;
    if ((q.x_dtype != F32 && q.x_dtype != BF16 && q.x_dtype != F16) || (q.gate_dtype != q.x_dtype && q.gate_dtype != F32))
        return RK_ERR_UNSUPPORTED;
    if (q.n_seq > 0x7ffffffe || q.tokens > 0x7fffffff || q.channels > 0x7fffffff)
        return RK_ERR_UNSUPPORTED;
    if (!q.gate || !q.out || (!q.x && (!backward || q.blend)) || (backward && (!q.h || !q.dout || !q.dgate)))
        return RK_ERR_INVALID_ARGUMENT;
    const int xs = dtype_size(q.x_dtype), gs = dtype_size(q.gate_dtype);
    const Extents e{q.starts ? 1 : q.n_seq, q.tokens, q.channels};
    struct { const rk_rows *t; int size; } in[] = {{q.gate, gs}, {q.x, xs}, {q.h, xs}, {q.dout, xs}},
                                           out[] = {{q.out, xs}, {q.dgate, gs}};
    for (const auto &t : in)
        if (t.t && !fits(*t.t, e))
            return RK_ERR_INVALID_ARGUMENT;
    for (const auto &t : out)
        if (t.t && (!fits(*t.t, e) || (!e.empty() && !unfolded(*t.t, e))))
            return RK_ERR_INVALID_ARGUMENT;
    if (q.n_seq == 0 || q.channels == 0)
        return RK_OK;
    const int64_t states = q.sources ? q.n_states : q.n_seq;
    if (!states_fit(states, q.channels) || !states_fit(q.n_seq, q.channels))
        return RK_ERR_INVALID_ARGUMENT;
    for (const auto &t : in)
        if (t.t && !e.empty() && (!t.t->data || !aligned(t.t->data, t.size)))
            return RK_ERR_INVALID_ARGUMENT;
    for (const auto &t : out)
        if (t.t && !e.empty() && (!t.t->data || !aligned(t.t->data, t.size)))
            return RK_ERR_INVALID_ARGUMENT;
    if ((!backward && !q.state_out) || (q.sources && !q.state) || !aligned(q.state, 4) || !aligned(q.dlast, 4) ||
        !aligned(q.state_out, 4) || !aligned(q.sources, 4) || !aligned(q.starts, 4))
        return RK_ERR_INVALID_ARGUMENT;

    // rows: all tokens one after the other, or a sequence's, the sequences apart
    // (several tiles of a sequence: apart, so that its neighbours on the device are other sequences' and not the
    // ones it waits for)
    const bool one = q.starts || (e.seqs * e.tokens <= 0x7fffffff && follows(q.gate, e) && follows(q.x, e) &&
                                  follows(q.h, e) && follows(q.dout, e) && follows(q.out, e) && follows(q.dgate, e) &&
                                  (e.tokens < tune::kRecurApart || e.seqs > tune::kRecurApartMost));
    RecurPlan p;
    const int rc = plan_recur(q.x_dtype, q.gate_dtype, one ? e.seqs * e.tokens : e.tokens, one ? 1 : e.seqs,
                              q.starts ? 0 : e.tokens, q.channels, backward, host::device_cus(), &p);
    if (rc)
        return rc;
    const bool in_place = !backward && !q.sources && q.state == q.state_out, keep = in_place && q.state && p.linked;
    const size_t ws = p.ws_bytes + (keep ? kept_states(q.n_seq, q.channels) : 0);
    if (ws > 0 && (!q.workspace || !aligned(q.workspace, 8) || q.workspace_bytes < ws))
        return RK_ERR_INVALID_ARGUMENT;

    // what is written: the rows may take the place of an input's or stand beside them; the forward pass's
    // last states may be its first ones
    const Span sw = span(q.workspace, int64_t(ws)), so = span(q.state_out, q.n_seq * q.channels * 4),
               ss = span(q.state, states * q.channels * 4), sd = span(q.dlast, q.n_seq * q.channels * 4),
               sc = span(q.sources, q.n_seq * 4), st = span(q.starts, (q.n_seq + 1) * 4);
    if ((overlap(so, ss) && !in_place) || overlap(so, sd) || overlap(so, sc) || overlap(so, st) || overlap(so, sw))
        return RK_ERR_INVALID_ARGUMENT;
    for (const Span &s : {ss, sd, sc, st})
        if (overlap(sw, s))
            return RK_ERR_INVALID_ARGUMENT;
    for (const auto &t : in)
        if (t.t && (overlap(sw, span_of(*t.t, e, t.size)) || overlap(so, span_of(*t.t, e, t.size))))
            return RK_ERR_INVALID_ARGUMENT;
    for (const auto &o : out) {
        if (!o.t)
            continue;
        const Span s = span_of(*o.t, e, o.size);
        for (const Span &v : {sw, so, ss, sd, sc, st})
            if (overlap(s, v))
                return RK_ERR_INVALID_ARGUMENT;
        for (const auto &t : in)
            if (t.t && !may_stand(*o.t, o.size, *t.t, t.size, e, t.t != q.h))
                return RK_ERR_INVALID_ARGUMENT;
    }
    if (q.dgate && !may_stand(*q.dgate, gs, *q.out, xs, e, false))
        return RK_ERR_INVALID_ARGUMENT;
    if (p.launches == 0 || (p.tiles == 0 && !q.state_out))
        return RK_OK;
    if (host::debug_enabled())
        std::fprintf(stderr, "%s: sequences=%lld tokens=%lld channels=%lld tiles=%lld strips=%d tokens a lane=%d ws=%zu\n", name,
                     (long long)q.n_seq, (long long)q.tokens, (long long)q.channels, (long long)p.tiles, p.strips, p.per_lane,
                     ws);
    RecurLaunch L;
    std::memset(static_cast<void *>(&L), 0, sizeof L);
    L.plan = p;
    L.a.gate = flat(q.gate, e);
    L.a.x = flat(q.x, e);
    L.a.h = flat(q.h, e);
    L.a.dout = flat(q.dout, e);
    L.a.out = flat(q.out, e);
    L.a.dgate = flat(q.dgate, e);
    L.a.state = q.state;
    if (keep) {
        L.state = q.state;
        L.kept = reinterpret_cast<float *>(static_cast<char *>(q.workspace) + p.ws_bytes);
        L.a.state = L.kept;
    }
    L.a.dlast = q.dlast;
    L.a.state_out = q.state_out;
    L.a.sources = q.sources;
    L.a.n_states = states;
    L.a.starts = q.starts;
    L.a.n_seq = q.n_seq;
    L.a.rows = one ? e.seqs * e.tokens : e.tokens;
    L.a.segs = one ? 1 : e.seqs;
    L.a.period = make_divider(uint32_t(e.tokens > 0 ? e.tokens : 1));
    L.a.channels = q.channels;
    L.a.kind = q.kind;
    L.a.blend = q.blend != 0;
    L.a.lanes_log2 = p.lanes_log2;
    L.a.strips = p.strips;
    L.a.tiles = p.tiles;
    L.a.tile_rows = p.tile_rows;
    L.a.linked = p.linked;
    L.a.ws = static_cast<uint32_t *>(q.workspace);
    L.a.patience = tune::kRecurPatience;
    L.a.force_help = host::forced_wait() >= 0;
    L.gate_dtype = q.gate_dtype;
    L.backward = backward;
    L.stream = q.stream;
    host::launch_events(&L.ev_begin, &L.ev_end);
    if (host::injected_launch_failure())
        return RK_ERR_HIP;
    return q.x_dtype == F32 ? launch_recur_f32(L) : q.x_dtype == BF16 ? launch_recur_bf16(L) : launch_recur_f16(L);
}

}  // namespace

extern "C" {

size_t rk_linear_recurrence_workspace_size(int x_dtype, int gate_dtype, int64_t n_seq, int64_t tokens, int64_t channels,
                                           int packed)
{
    return workspace_size(x_dtype, gate_dtype, n_seq, tokens, channels, packed != 0);
}

int rk_linear_recurrence(int x_dtype, int gate_dtype, int kind, int blend, const rk_rows *gate, const rk_rows *x,
                         const float *state, int64_t n_states, const int32_t *sources, const int32_t *starts,
                         int64_t n_seq, int64_t tokens, int64_t channels, const rk_rows *out, float *state_out,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    Request q{};
    q.x_dtype = x_dtype;
    q.gate_dtype = gate_dtype;
    q.kind = kind;
    q.blend = blend;
    q.gate = gate;
    q.x = x;
    q.out = out;
    q.state = state;
    q.state_out = state_out;
    q.sources = sources;
    q.starts = starts;
    q.n_states = n_states;
    q.n_seq = n_seq;
    q.tokens = tokens;
    q.channels = channels;
    q.workspace = workspace;
    q.workspace_bytes = workspace_bytes;
    q.stream = stream;
    return recur("rk_linear_recurrence", q, false);
}

int rk_linear_recurrence_backward(int x_dtype, int gate_dtype, int kind, int blend, const rk_rows *gate, const rk_rows *x,
                                  const rk_rows *out, const rk_rows *dout, const float *state, const float *dstate_out,
                                  const int32_t *starts, int64_t n_seq, int64_t tokens, int64_t channels,
                                  const rk_rows *dgate, const rk_rows *dx, float *dstate, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    Request q{};
    q.x_dtype = x_dtype;
    q.gate_dtype = gate_dtype;
    q.kind = kind;
    q.blend = blend;
    q.gate = gate;
    q.x = blend ? x : nullptr;
    q.h = out;
    q.dout = dout;
    q.out = dx;
    q.dgate = dgate;
    q.state = state;
    q.dlast = dstate_out;
    q.state_out = dstate;
    q.starts = starts;
    q.n_seq = n_seq;
    q.tokens = tokens;
    q.channels = channels;
    q.workspace = workspace;
    q.workspace_bytes = workspace_bytes;
    q.stream = stream;
    return recur("rk_linear_recurrence_backward", q, true);
}

}  // extern "C"
