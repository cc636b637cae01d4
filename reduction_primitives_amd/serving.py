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

import torch

from . import _native as N

_CODES = {torch.float32: N.RK_F32, torch.bfloat16: N.RK_BF16, torch.float16: N.RK_F16, torch.float64: N.RK_F64,
          torch.int32: N.RK_I32, torch.int64: N.RK_I64}


class _Call:
    """The device and stream of one call: the operands' device is made the
    current one, and what the call allocates belongs to its stream."""

    __slots__ = ("device", "stream", "handle", "_guards")

    def __init__(self, name, stream, **operands):
        first = None
        for what, t in operands.items():
            if t is None:
                continue
            if not t.is_cuda:
                raise ValueError(f"{name}: {what} is not on a GPU")
            if first is None:
                first = t.get_device()
            elif t.get_device() != first:
                raise ValueError(f"{name}: {what} is on another device")
        if stream is not None and stream.device_index != first:
            raise ValueError(f"{name}: the stream belongs to another device")
        self.device = first
        self.stream = stream
        self.handle = torch._C._cuda_getCurrentRawStream(first) if stream is None else stream.cuda_stream
        self._guards = ()

    def __enter__(self):
        guards = []
        if self.device != torch.cuda.current_device():
            guards.append(torch.cuda.device(self.device))
        if self.stream is not None:
            guards.append(torch.cuda.stream(self.stream))
        for g in guards:
            g.__enter__()
        self._guards = guards
        return self

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)

    def empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.device))

    def workspace(self, given, size):
        """The caller's workspace, or one of size() bytes."""
        return self.empty(max(int(size()), 256), torch.uint8) if given is None else given


def _code(name, what, t, allowed):
    c = _CODES.get(t if isinstance(t, torch.dtype) else t.dtype)
    if c not in allowed:
        raise ValueError(f"{name}: {what} cannot be {t if isinstance(t, torch.dtype) else t.dtype}")
    return c


def _lines(name, what, t):
    """(lines, entries, stride) of a 2-d tensor whose lines are contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: {what} takes two dims, the second contiguous")
    return t.shape[0], t.shape[1], t.stride(0)


def _flat(name, what, t, n, dtype):
    if t.dtype != dtype or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name}: {what} takes {n} contiguous {dtype}")


def _check(rc, what):
    if rc:
        raise N.RkError(rc, what)


_PROBS = (N.RK_F32, N.RK_BF16, N.RK_F16)
_IDS = (N.RK_I32, N.RK_I64)


def softmax(x, temperature=None, out_dtype=None, out=None, workspace=None, stream=None):
    """softmax(x / temperature) along the lines of the 2-d tensor x
    (rk_softmax).  temperature: float32, one per line; a value <= 0 picks the
    first largest entry.  `out` defaults to a new tensor of out_dtype (x's
    dtype); it may be x itself.  Returns out."""
    name = "softmax"
    in_code = _code(name, "x", x, _PROBS)
    lines, n, xs = _lines(name, "x", x)
    with _Call(name, stream, x=x, temperature=temperature, out=out, workspace=workspace) as call:
        if temperature is not None:
            _flat(name, "temperature", temperature, lines, torch.float32)
        if out is None:
            out = call.empty((lines, n), out_dtype or x.dtype)
        elif out.shape != x.shape or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("softmax: out takes x's shape and out_dtype")
        out_code = _code(name, "out", out, _PROBS)
        ws = call.workspace(workspace, lambda: N.rk_softmax_workspace_size(in_code, out_code, n, lines))
        _check(N.rk_softmax(in_code, out_code, x.data_ptr(), n, lines, xs,
                            None if temperature is None else temperature.data_ptr(), out.data_ptr(),
                            _lines(name, "out", out)[2], ws.data_ptr(), ws.nbytes, call.handle), "rk_softmax")
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
    code = _code(name, "p", p, _PROBS)
    tok = _code(name, "drafted", drafted, _IDS)
    rows, vocab, ps = _lines(name, "p", p)
    req, drafts = r.numel(), drafted.numel()
    if max_draft is None:
        if starts is not None:
            raise ValueError("draft_verify: starts needs max_draft, the most drafts of a request")
        max_draft = drafts // max(req, 1)
    if rows != drafts + req:
        raise ValueError("draft_verify: p takes a line for every draft and one for every request")
    qs = 0
    if q is not None:
        if q.dtype != p.dtype or q.shape[0] != drafts or q.shape[1] != vocab:
            raise ValueError("draft_verify: q takes p's dtype and vocabulary, a line for every draft")
        qs = _lines(name, "q", q)[2]
    _flat(name, "drafted", drafted, drafts, drafted.dtype)
    _flat(name, "u", u, drafts, torch.float32)
    _flat(name, "r", r, req, torch.float32)
    if starts is not None:
        _flat(name, "starts", starts, req + 1, torch.int32)
    with _Call(name, stream, p=p, q=q, drafted=drafted, u=u, r=r, starts=starts, tokens=tokens, accepted=accepted,
               workspace=workspace) as call:
        if tokens is None:
            tokens = call.empty((req, max_draft + 1), drafted.dtype)
        else:
            _flat(name, "tokens", tokens, req * (max_draft + 1), drafted.dtype)
        if accepted is None:
            accepted = call.empty(req, torch.int32)
        else:
            _flat(name, "accepted", accepted, req, torch.int32)
        ws = call.workspace(workspace, lambda: N.rk_draft_verify_workspace_size(code, vocab, req))
        _check(N.rk_draft_verify(code, tok, p.data_ptr(), ps, None if q is None else q.data_ptr(), qs, vocab, req,
                                 drafts, max_draft, None if starts is None else starts.data_ptr(),
                                 drafted.data_ptr(), u.data_ptr(), r.data_ptr(), tokens.data_ptr(),
                                 accepted.data_ptr(), ws.data_ptr(), ws.nbytes, call.handle), "rk_draft_verify")
    return tokens, accepted


def block_tables(lens, block_size, held, table, ring, state, held_out=None, state_out=None, workspace=None,
                 stream=None):
    """Bring block tables to the requests' lengths (rk_block_tables), table and
    ring in place.  state: int64 (head, tail) of the ring, and two places more
    (4 in all) where it is updated in place; held and state are, unless held_out and state_out
    (4 int64) are given.  Returns (held_out, state_out)."""
    name = "block_tables"
    req = lens.numel()
    _, width, ts = _lines(name, "table", table)
    if table.shape[0] != req or table.dtype != torch.int32:
        raise ValueError("block_tables: table takes an int32 line for every request")
    held_out = held if held_out is None else held_out
    state_out = state if state_out is None else state_out
    _flat(name, "lens", lens, req, torch.int32)
    _flat(name, "held", held, req, torch.int32)
    _flat(name, "held_out", held_out, req, torch.int32)
    _flat(name, "ring", ring, ring.numel(), torch.int32)
    _flat(name, "state_out", state_out, 4, torch.int64)
    if state.dtype != torch.int64 or not state.is_contiguous() or state.numel() < 2:
        raise ValueError("block_tables: state takes int64 head and tail")
    with _Call(name, stream, lens=lens, held=held, table=table, ring=ring, state=state, held_out=held_out,
               state_out=state_out, workspace=workspace) as call:
        ws = call.workspace(workspace, lambda: N.rk_block_tables_workspace_size(req))
        _check(N.rk_block_tables(lens.data_ptr(), req, block_size, held.data_ptr(), held_out.data_ptr(),
                                 table.data_ptr(), ts, width, ring.data_ptr(), ring.numel(), state.data_ptr(),
                                 state_out.data_ptr(), ws.data_ptr(), ws.nbytes, call.handle), "rk_block_tables")
    return held_out, state_out


def slot_map(lens, fresh, block_size, table, held, n_blocks, capacity=None, slot_dtype=None, slots=None,
             positions=None, requests=None, starts=None, stream=None):
    """Slots, positions, requests and starts of a batch's new tokens
    (rk_slot_map): the last fresh[b] of each request's lens[b] tokens.  n_blocks:
    the blocks of the pool; capacity: entries of the outputs (slots' own
    when slots is given).  Returns (slots, positions, requests, starts)."""
    name = "slot_map"
    req = lens.numel()
    _, width, ts = _lines(name, "table", table)
    if table.shape[0] != req or table.dtype != torch.int32:
        raise ValueError("slot_map: table takes an int32 line for every request")
    _flat(name, "lens", lens, req, torch.int32)
    _flat(name, "fresh", fresh, req, torch.int32)
    _flat(name, "held", held, req, torch.int32)
    if slots is not None:
        capacity = slots.numel() if capacity is None else capacity
        _flat(name, "slots", slots, capacity, slot_dtype or slots.dtype)
    elif capacity is None:
        raise ValueError("slot_map: needs capacity or slots")
    with _Call(name, stream, lens=lens, fresh=fresh, table=table, held=held, slots=slots, positions=positions,
               requests=requests, starts=starts) as call:
        if slots is None:
            slots = call.empty(capacity, slot_dtype or torch.int64)
        code = _code(name, "slots", slots, _IDS)
        if positions is None:
            positions = call.empty(capacity, torch.int32)
        else:
            _flat(name, "positions", positions, capacity, torch.int32)
        if requests is None:
            requests = call.empty(capacity, torch.int32)
        else:
            _flat(name, "requests", requests, capacity, torch.int32)
        if starts is None:
            starts = call.empty(req + 1, torch.int32)
        else:
            _flat(name, "starts", starts, req + 1, torch.int32)
        _check(N.rk_slot_map(lens.data_ptr(), fresh.data_ptr(), req, block_size, table.data_ptr(), ts, width,
                             held.data_ptr(), n_blocks, code, capacity, slots.data_ptr(), positions.data_ptr(),
                             requests.data_ptr(), starts.data_ptr(), call.handle), "rk_slot_map")
    return slots, positions, requests, starts
