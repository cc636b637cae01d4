"""Serving operators: the reductions and scans around a language model's step.

``softmax`` turns logits into probabilities, ``draft_verify`` verifies drafted
tokens against them, ``block_tables`` brings block tables to the requests'
lengths and ``slot_map`` lays out the next batch.  Like the reductions and scans
of the package they marshal torch tensors into the C ABI (include/rk.h has
each call's definition); everything stays on the device, so a step of them
can be captured into a HIP graph.

Buffers that are not given are allocated with torch on the call's stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import _native as N

_lib = N.load()

_CODES = {torch.float32: N.RK_F32, torch.bfloat16: N.RK_BF16, torch.float16: N.RK_F16, torch.float64: N.RK_F64,
          torch.int32: N.RK_I32, torch.int64: N.RK_I64}


_PROBS = (N.RK_F32, N.RK_BF16, N.RK_F16)
_IDS = (N.RK_I32, N.RK_I64)
_f32, _i32, _i64 = torch.float32, torch.int32, torch.int64
_current_stream = torch._C._cuda_getCurrentRawStream


# The checks below run on every call of a decode step, where the kernels take
# a few microseconds: each looks at a tensor once, in one expression, and says
# what is wrong only when something is.

def _flat(name, what, t, n, dtype, dev):
    """t's address, for a contiguous tensor of n elements of dtype on dev."""
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        _wrong(name, what, t, dev)
        raise ValueError(f"{name}: {what} takes {n} contiguous {dtype}")
    return t.data_ptr()


def _lines(name, what, t, dev):
    """Stride of a 2-d tensor on dev whose lines are contiguous."""
    if t.dim() != 2 or t.get_device() != dev:
        _wrong(name, what, t, dev)
        raise ValueError(f"{name}: {what} takes two dims, the second contiguous")
    stride, one = t.stride()
    if one != 1 and t.size(1) > 1:
        raise ValueError(f"{name}: {what} takes two dims, the second contiguous")
    return stride


def _wrong(name, what, t, dev):
    if not t.is_cuda:
        raise ValueError(f"{name}: {what} is not on a GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name}: {what} is on another device")


def _device(name, what, t):
    dev = t.get_device()
    if dev < 0:
        _wrong(name, what, t, dev)
    return dev


def _code(name, what, dtype, allowed):
    c = _CODES.get(dtype)
    if c not in allowed:
        raise ValueError(f"{name}: {what} cannot be {dtype}")
    return c


def _launch(name, dev, stream, call, *args):
    """call(*args, stream handle) with dev the current device."""
    if stream is None:
        stream = _current_stream(dev)
    else:
        if stream.device_index != dev:
            raise ValueError(f"{name}: the stream belongs to another device")
        stream = stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        rc = call(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, stream)
    if rc:
        raise N.RkError(rc, "rk_" + name)


def _empty(shape, dtype, dev, stream):
    """A tensor that belongs to the call's stream, so that the caching allocator
    hands its bytes to no other stream's work too early."""
    with torch.cuda.device(dev), (contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)):
        return torch.empty(shape, dtype=dtype, device="cuda")


def _workspace(name, given, size, dev, stream):
    """The caller's workspace, or one of size() bytes."""
    if given is None:
        with torch.cuda.device(dev):
            n = size()
        return _empty(max(n, 256), torch.uint8, dev, stream)
    if given.get_device() != dev or not given.is_contiguous():
        _wrong(name, "workspace", given, dev)
        raise ValueError(f"{name}: workspace takes a contiguous tensor")
    return given


def softmax(x, temperature=None, out_dtype=None, out=None, workspace=None, stream=None):
    """softmax(x / temperature) along the lines of the 2-d tensor x
    (rk_softmax).  temperature: float32, one per line; a value <= 0 picks the
    first largest entry.  `out` defaults to a new tensor of out_dtype (x's
    dtype); it may be x itself.  Returns out."""
    dev = _device("softmax", "x", x)
    in_code = _code("softmax", "x", x.dtype, _PROBS)
    xs = _lines("softmax", "x", x, dev)
    lines, n = x.shape
    t = None if temperature is None else _flat("softmax", "temperature", temperature, lines, _f32, dev)
    if out is None:
        out = _empty((lines, n), out_dtype or x.dtype, dev, stream)
    elif out.shape != x.shape or (out_dtype is not None and out.dtype is not out_dtype):
        raise ValueError("softmax: out takes x's shape and out_dtype")
    out_code = _code("softmax", "out", out.dtype, _PROBS)
    ws = _workspace("softmax", workspace, lambda: N.rk_softmax_workspace_size(in_code, out_code, n, lines), dev, stream)
    _launch("softmax", dev, stream, _lib.rk_softmax, in_code, out_code, x.data_ptr(), n, lines, xs, t, out.data_ptr(),
            _lines("softmax", "out", out, dev), ws.data_ptr(), ws.nbytes)
    return out


def draft_verify(p, q, drafted, u, r, starts=None, max_draft=None, tokens=None, accepted=None, workspace=None,
                 stream=None):
    """Verify drafted tokens (rk_draft_verify).  p: the target's probabilities,
    a line for every draft and one more after each request's last; q: the
    draft's, a line for every draft, or None; drafted, u: the tokens and
    their uniform numbers; r: a uniform number per request; starts: int32
    offsets of the requests' drafts (None: max_draft each).  Returns (tokens,
    accepted): per request the kept tokens, the drawn one and -1 behind it,
    and how many drafts were kept."""
    name = "draft_verify"
    dev = _device(name, "p", p)
    code = _code(name, "p", p.dtype, _PROBS)
    tok = _code(name, "drafted", drafted.dtype, _IDS)
    ps = _lines(name, "p", p, dev)
    rows, vocab = p.shape
    req, drafts = r.numel(), drafted.numel()
    if max_draft is None:
        if starts is not None:
            raise ValueError("draft_verify: starts needs max_draft, the most drafts of a request")
        max_draft = drafts // max(req, 1)
    if rows != drafts + req:
        raise ValueError("draft_verify: p takes a line for every draft and one for every request")
    q_ptr, qs = None, 0
    if q is not None:
        qs = _lines(name, "q", q, dev)
        if q.dtype is not p.dtype or q.shape != (drafts, vocab):
            raise ValueError("draft_verify: q takes p's dtype and vocabulary, a line for every draft")
        q_ptr = q.data_ptr()
    x_ptr = _flat(name, "drafted", drafted, drafts, drafted.dtype, dev)
    u_ptr = _flat(name, "u", u, drafts, _f32, dev)
    r_ptr = _flat(name, "r", r, req, _f32, dev)
    s_ptr = None if starts is None else _flat(name, "starts", starts, req + 1, _i32, dev)
    if tokens is None:
        tokens = _empty((req, max_draft + 1), drafted.dtype, dev, stream)
    if accepted is None:
        accepted = _empty((req,), _i32, dev, stream)
    t_ptr = _flat(name, "tokens", tokens, req * (max_draft + 1), drafted.dtype, dev)
    a_ptr = _flat(name, "accepted", accepted, req, _i32, dev)
    ws = _workspace(name, workspace, lambda: N.rk_draft_verify_workspace_size(code, vocab, req), dev, stream)
    _launch(name, dev, stream, _lib.rk_draft_verify, code, tok, p.data_ptr(), ps, q_ptr, qs, vocab, req, drafts, max_draft,
            s_ptr, x_ptr, u_ptr, r_ptr, t_ptr, a_ptr, ws.data_ptr(), ws.nbytes)
    return tokens, accepted


def block_tables(lens, block_size, held, table, ring, state, held_out=None, state_out=None, workspace=None,
                 stream=None):
    """Bring block tables to the requests' lengths (rk_block_tables), table and
    ring in place.  state: int64 (head, tail) of the ring, and two places more
    (4 in all) where it is updated in place; held and state are, unless held_out and state_out
    (4 int64) are given.  Returns (held_out, state_out)."""
    name = "block_tables"
    dev = _device(name, "lens", lens)
    req, blocks = lens.numel(), ring.numel()
    ts = _table(name, table, req, dev)
    held_out = held if held_out is None else held_out
    state_out = state if state_out is None else state_out
    l_ptr = _flat(name, "lens", lens, req, _i32, dev)
    h_ptr = _flat(name, "held", held, req, _i32, dev)
    o_ptr = h_ptr if held_out is held else _flat(name, "held_out", held_out, req, _i32, dev)
    r_ptr = _flat(name, "ring", ring, blocks, _i32, dev)
    so_ptr = _flat(name, "state_out", state_out, 4, _i64, dev)
    if state is state_out:
        s_ptr = so_ptr
    else:
        s_ptr = _flat(name, "state", state, max(state.numel(), 2), _i64, dev)
    ws = _workspace(name, workspace, lambda: N.rk_block_tables_workspace_size(req), dev, stream)
    _launch(name, dev, stream, _lib.rk_block_tables, l_ptr, req, block_size, h_ptr, o_ptr, table.data_ptr(), ts,
            table.size(1), r_ptr, blocks, s_ptr, so_ptr, ws.data_ptr(), ws.nbytes)
    return held_out, state_out


def _table(name, table, req, dev):
    """Line stride of a block table."""
    ts = _lines(name, "table", table, dev)
    if table.size(0) != req or table.dtype is not _i32:
        raise ValueError(f"{name}: table takes an int32 line for every request")
    return ts


def slot_map(lens, fresh, block_size, table, held, n_blocks, capacity=None, slot_dtype=None, slots=None,
             positions=None, requests=None, starts=None, stream=None):
    """Slots, positions, requests and starts of a batch's new tokens
    (rk_slot_map): the last fresh[b] of each request's lens[b] tokens.  n_blocks:
    the blocks of the pool; capacity: entries of the outputs (slots' own
    when slots is given).  Returns (slots, positions, requests, starts)."""
    name = "slot_map"
    dev = _device(name, "lens", lens)
    req = lens.numel()
    ts = _table(name, table, req, dev)
    l_ptr = _flat(name, "lens", lens, req, _i32, dev)
    f_ptr = _flat(name, "fresh", fresh, req, _i32, dev)
    h_ptr = _flat(name, "held", held, req, _i32, dev)
    if capacity is None:
        if slots is None:
            raise ValueError("slot_map: needs capacity or slots")
        capacity = slots.numel()
    if slots is None:
        slots = _empty((capacity,), slot_dtype or _i64, dev, stream)
    code = _code(name, "slots", slots.dtype, _IDS)
    if positions is None:
        positions = _empty((capacity,), _i32, dev, stream)
    if requests is None:
        requests = _empty((capacity,), _i32, dev, stream)
    if starts is None:
        starts = _empty((req + 1,), _i32, dev, stream)
    _launch(name, dev, stream, _lib.rk_slot_map, l_ptr, f_ptr, req, block_size, table.data_ptr(), ts, table.size(1), h_ptr,
            n_blocks, code, capacity, _flat(name, "slots", slots, capacity, slot_dtype or slots.dtype, dev),
            _flat(name, "positions", positions, capacity, _i32, dev), _flat(name, "requests", requests, capacity, _i32, dev),
            _flat(name, "starts", starts, req + 1, _i32, dev))
    return slots, positions, requests, starts
