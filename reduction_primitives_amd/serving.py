"""Serving operators: the reductions and scans around a language model's step.

``softmax`` turns logits into probabilities, ``draft_verify`` verifies drafted
tokens against them, ``block_tables`` brings block tables to the requests'
lengths and ``slot_map`` lays out the next batch.  ``beam_select`` chooses the
beams a search goes on with, ``fork_blocks`` gives them the block tables of the
beams they come from, ``copy_blocks`` copies the blocks that are then theirs alone,
and ``compact_blocks`` brings the blocks in use together.  Like the reductions and scans
of the package they marshal torch tensors into the C ABI (include/rk.h has
each call's definition); everything stays on the device, so a step of them
can be captured into a HIP graph.

Buffers that are not given are allocated with torch on the call's stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _native as N

_lib = N.load()

from . import _serving as _calls  # noqa: E402  (checks tensors and passes their addresses to the library)

_calls.bind(*(ctypes.cast(getattr(_lib, f), ctypes.c_void_p).value
              for f in ("rk_softmax", "rk_draft_verify", "rk_block_tables", "rk_slot_map", "rk_beam_select", "rk_fork_blocks",
                        "rk_compact_blocks", "rk_copy_blocks", "rk_linear_recurrence", "rk_linear_recurrence_backward")))

_CODES = {torch.float32: N.RK_F32, torch.bfloat16: N.RK_BF16, torch.float16: N.RK_F16}
_current_stream = torch._C._cuda_getCurrentRawStream


def _handle(name, what, t, stream):
    """hipStream_t of a call on t's device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: {what} is not on a GPU")
    if stream is None:
        return _current_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"{name}: the stream belongs to another device")
    return stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """A tensor on like's device that belongs to the call's stream, so that the
    caching allocator hands its bytes to no other stream's work too early."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _workspace(size, args, like, stream):
    """A workspace of size(*args) bytes on like's device, None where that is 0."""
    if like.get_device() == torch.cuda.current_device():
        n = size(*args)
    else:
        with torch.cuda.device(like.device):
            n = size(*args)
    return _empty(n, torch.uint8, like, stream) if n else None


def _code(name, what, dtype):
    if dtype not in _CODES:
        raise ValueError(f"{name}: {what} cannot be {dtype}")
    return _CODES[dtype]


def softmax(x, temperature=None, out_dtype=None, out=None, workspace=None, stream=None):
    """softmax(x / temperature) along the lines of the 2-d tensor x
    (rk_softmax).  temperature: float32, one per line; a value <= 0 picks the
    first largest entry.  `out` defaults to a new tensor of out_dtype (x's
    dtype); it may be x itself.  Returns out.  There is no backward pass:
    tensors that require grad are refused where gradients are recorded."""
    handle = _handle("softmax", "x", x, stream)
    if out is None:
        out = _empty(x.shape, out_dtype or x.dtype, x, stream)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError("softmax: out takes x's shape and out_dtype")
    if workspace is None and x.dim() == 2:        # (other dims are refused below)
        codes = _code("softmax", "x", x.dtype), _code("softmax", "out", out.dtype)
        workspace = _workspace(N.rk_softmax_workspace_size, (*codes, x.shape[-1], x.shape[0]), x, stream)
    rc = _calls.softmax(handle, x, temperature, out, workspace)
    if rc:
        raise N.RkError(rc, "rk_softmax")
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
    handle = _handle("draft_verify", "p", p, stream)
    if max_draft is None:
        if starts is not None:
            raise ValueError("draft_verify: starts needs max_draft, the most drafts of a request")
        max_draft = drafted.numel() // max(r.numel(), 1)
    if tokens is None:
        tokens = _empty((r.numel(), max_draft + 1), drafted.dtype, p, stream)
    if accepted is None:
        accepted = _empty((r.numel(),), torch.int32, p, stream)
    if workspace is None and p.dim() == 2:
        workspace = _workspace(N.rk_draft_verify_workspace_size,
                               (_code("draft_verify", "p", p.dtype), p.shape[-1], r.numel()), p, stream)
    rc = _calls.draft_verify(handle, p, q, drafted, u, r, starts, max_draft, tokens, accepted, workspace)
    if rc:
        raise N.RkError(rc, "rk_draft_verify")
    return tokens, accepted


def block_tables(lens, block_size, held, table, ring, state, held_out=None, state_out=None, workspace=None,
                 stream=None):
    """Bring block tables to the requests' lengths (rk_block_tables), table and
    ring in place.  state: int64 (head, tail) of the ring, and two places more
    (4 in all) where it is updated in place; held and state are, unless held_out and state_out
    (4 int64) are given.  Returns (held_out, state_out)."""
    handle = _handle("block_tables", "lens", lens, stream)
    held_out = held if held_out is None else held_out
    state_out = state if state_out is None else state_out
    if workspace is None:
        workspace = _workspace(N.rk_block_tables_workspace_size, (lens.numel(),), lens, stream)
    rc = _calls.block_tables(handle, lens, block_size, held, table, ring, state, held_out, state_out, workspace)
    if rc:
        raise N.RkError(rc, "rk_block_tables")
    return held_out, state_out


def slot_map(lens, fresh, block_size, table, held, n_blocks, capacity=None, slot_dtype=None, slots=None,
             positions=None, requests=None, starts=None, stream=None):
    """Slots, positions, requests and starts of a batch's new tokens
    (rk_slot_map): the last fresh[b] of each request's lens[b] tokens.  n_blocks:
    the blocks of the pool; capacity: entries of the outputs (slots' own
    when slots is given).  Returns (slots, positions, requests, starts)."""
    handle = _handle("slot_map", "lens", lens, stream)
    if capacity is None:
        if slots is None:
            raise ValueError("slot_map: needs capacity or slots")
        capacity = slots.numel()
    if slots is None:
        slots = _empty((capacity,), slot_dtype or torch.int64, lens, stream)
    elif slot_dtype is not None and slots.dtype is not slot_dtype:
        raise ValueError("slot_map: slots takes slot_dtype")
    if positions is None:
        positions = _empty((capacity,), torch.int32, lens, stream)
    if requests is None:
        requests = _empty((capacity,), torch.int32, lens, stream)
    if starts is None:
        starts = _empty((lens.numel() + 1,), torch.int32, lens, stream)
    rc = _calls.slot_map(handle, lens, fresh, block_size, table, held, n_blocks, capacity, slots, positions, requests, starts)
    if rc:
        raise N.RkError(rc, "rk_slot_map")
    return slots, positions, requests, starts


def beam_select(logits, scores, count=None, ended=None, end_token=None, token_dtype=None, best=None, tokens=None,
                parents=None, workspace=None, stream=None):
    """The best continuations of every request's beams (rk_beam_select).
    logits: a line for each beam, those of a request one after the other;
    scores: float32 (requests, beams); count: how many to keep (None: as many
    as there are beams, at most 64); ended: bool (requests, beams), beams that
    go on as they are, by end_token.  Returns (best, tokens, parents), each
    (requests, count), best first: scores, tokens and the lines they continue.
    There is no backward pass: tensors that require grad are refused where
    gradients are recorded."""
    handle = _handle("beam_select", "logits", logits, stream)
    if ended is not None and end_token is None:
        raise ValueError("beam_select: ended needs end_token, the token an ended beam goes on with")
    if scores.dim() != 2:
        raise ValueError("beam_select: scores takes requests times beams, a score for every line")
    req, beams = scores.shape
    if count is None:
        count = beams
    if count < 1 or beams < 1:
        raise ValueError("beam_select: takes one beam and one candidate to keep at least")
    if best is None:
        best = _empty((req, count), torch.float32, logits, stream)
    if tokens is None:
        tokens = _empty((req, count), token_dtype or torch.int64, logits, stream)
    elif token_dtype is not None and tokens.dtype is not token_dtype:
        raise ValueError("beam_select: tokens takes token_dtype")
    if parents is None:
        parents = _empty((req, count), torch.int32, logits, stream)
    if workspace is None and logits.dim() == 2:
        workspace = _workspace(N.rk_beam_select_workspace_size,
                               (_code("beam_select", "logits", logits.dtype), logits.shape[-1], req, beams, count), logits, stream)
    rc = _calls.beam_select(handle, logits, scores, count, ended, 0 if end_token is None else end_token, best, tokens, parents,
                            workspace)
    if rc:
        raise N.RkError(rc, "rk_beam_select")
    return best, tokens, parents


def fork_blocks(parents, lens, block_size, held, table, ring, state, n_blocks, table_out=None, held_out=None, lens_out=None,
                pairs=None, state_out=None, workspace=None, stream=None):
    """Make the rows of a block table those of their parents (rk_fork_blocks),
    ring in place.  parents: int32, the old row each new one goes on from, -1 for
    an empty one; lens, held: tokens and blocks of the old rows; n_blocks: the
    blocks of the pool; state: int64 (head, tail) of the ring, and two places
    more (4 in all) where it is updated in place, as it is unless state_out (4
    int64) is given.  Returns (table_out, held_out, lens_out, pairs, state_out);
    pairs: (source, fresh block) of the rows whose last block is to be copied
    (copy_blocks)."""
    handle = _handle("fork_blocks", "parents", parents, stream)
    n = parents.numel()
    width = table.shape[-1] if table.dim() == 2 else 0
    if table_out is None:
        table_out = _empty((n, width), torch.int32, parents, stream)
    if held_out is None:
        held_out = _empty((n,), torch.int32, parents, stream)
    if lens_out is None:
        lens_out = _empty((n,), torch.int32, parents, stream)
    if pairs is None:
        pairs = _empty((n, 2), torch.int32, parents, stream)
    state_out = state if state_out is None else state_out
    if workspace is None:
        workspace = _workspace(N.rk_fork_blocks_workspace_size, (lens.numel(), n, min(width, 2 ** 31 - 1), n_blocks), parents, stream)
    rc = _calls.fork_blocks(handle, parents, lens, block_size, held, table, ring, state, n_blocks, table_out, held_out, lens_out,
                            pairs, state_out, workspace)
    if rc:
        raise N.RkError(rc, "rk_fork_blocks")
    return table_out, held_out, lens_out, pairs, state_out


def compact_blocks(held, table, ring, n_blocks, table_out=None, pairs=None, state_out=None, workspace=None, stream=None):
    """Bring the blocks that block tables name to the lowest ids
    (rk_compact_blocks), table (unless table_out is given) and ring in place:
    every block no row names is free afterwards.  Returns (table_out, pairs,
    state_out): pairs, of n_blocks // 2, holds the moves (copy_blocks) and -1
    behind them; state_out the ring's head and tail, and the number of moves."""
    handle = _handle("compact_blocks", "held", held, stream)
    table_out = table if table_out is None else table_out
    if pairs is None:
        pairs = _empty((max(n_blocks, 0) // 2, 2), torch.int32, held, stream)
    if state_out is None:
        state_out = _empty((4,), torch.int64, held, stream)
    if workspace is None:
        workspace = _workspace(N.rk_compact_blocks_workspace_size, (n_blocks,), held, stream)
    rc = _calls.compact_blocks(handle, held, table, ring, n_blocks, table_out, pairs, state_out, workspace)
    if rc:
        raise N.RkError(rc, "rk_compact_blocks")
    return table_out, pairs, state_out


def copy_blocks(caches, pairs, stream=None):
    """Copy blocks inside caches (rk_copy_blocks): block pairs[i, 1] becomes
    what block pairs[i, 0] is; pairs with an id outside a cache are left out.
    caches: a list of tensors whose first dim counts the blocks, each block
    contiguous; pairs: int32.  Returns caches.  Caches that require grad are
    refused where gradients are recorded."""
    handle = _handle("copy_blocks", "pairs", pairs, stream)
    rc = _calls.copy_blocks(handle, caches, pairs)
    if rc:
        raise N.RkError(rc, "rk_copy_blocks")
    return caches
