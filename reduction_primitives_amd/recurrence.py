"""The scan of a recurrent layer: ``linear_recurrence`` and its gradient.

They marshal torch tensors into the C ABI (include/rk.h has the definitions) as
the serving operators do.  Where gradients are recorded and an input requires
one, ``linear_recurrence`` takes part in torch's autograd.

Buffers that are not given are allocated with torch on the call's stream.
"""
from __future__ import annotations

import functools

import torch

from . import _native as N
from .serving import _calls, _code, _empty, _handle

KINDS = {"value": N.RK_GATE_VALUE, "log": N.RK_GATE_LOG, "sigmoid": N.RK_GATE_SIGMOID}


def _kind(name, kind):
    if kind not in KINDS:
        raise ValueError(f"{name}: kind takes one of {', '.join(KINDS)}")
    return KINDS[kind]


def _scratch(name, gate, x, starts, stream):
    """A workspace for tokens like x's (None where none is needed, or where the call refuses them)."""
    if x.dim() != (3 if starts is None else 2):
        return None
    if starts is None and x.shape[1] <= 1:     # (none is needed: the size would take as long as the call)
        return None
    n_seq = x.shape[0] if starts is None else max(starts.numel() - 1, 0)
    n = _size(x.get_device(), _code(name, "x", x.dtype), _code(name, "gate", gate.dtype), n_seq, x.shape[-2], x.shape[-1],
              int(starts is not None))
    return _empty(n, torch.uint8, x, stream) if n else None


@functools.lru_cache(maxsize=1024)
def _size(device, *args):
    """rk_linear_recurrence_workspace_size on a device (through ctypes it takes longer than a short sequence's call)."""
    with torch.cuda.device(device):
        return N.rk_linear_recurrence_workspace_size(*args)


def _sequences(gate, starts):
    return max(starts.numel() - 1, 0) if starts is not None else gate.shape[0] if gate.dim() else 0


def linear_recurrence(gate, x, state=None, kind="value", blend=False, starts=None, sources=None, out=None, state_out=None,
                      workspace=None, stream=None):
    """h_t = a_t h_(t-1) + w_t x_t along the tokens of every sequence
    (rk_linear_recurrence), a the gate, its exponential or its logistic
    function (kind: "value", "log", "sigmoid") and w = 1, or 1 - a with blend.
    gate and x: (sequences, tokens, channels), or (tokens, channels) packed,
    sequence b the tokens [starts[b], starts[b + 1]).  state: float32
    (sequences, channels), zeros where it is None; with sources (int32),
    sequence b starts from line sources[b] of it.  Returns (out, state_out): every
    token's h, of x's dtype, and the last ones in float32; state_out may be state
    where there are no sources.  Up to 2048 gates in a row are folded into one
    float32 factor: with gates above 1, one that leaves float32's range makes a
    state infinite or NaN that need not be.

    Where gradients are recorded and gate, x or state requires one, the outputs
    have them (of the first order, computed on the stream that was current;
    sources, out, state_out and stream are then refused, and tokens of no
    sequence get zeros).  There are no forward derivatives: tensors that carry
    a tangent are refused.  Not while the stream is captured: a captured backward
    pass that meets an eager graph of the same leaves ends the process inside
    torch; linear_recurrence_backward can be captured."""
    code = _kind("linear_recurrence", kind)
    if torch.is_grad_enabled() and (gate.requires_grad or x.requires_grad or (state is not None and state.requires_grad)):
        if sources is not None or out is not None or state_out is not None or stream is not None:
            raise ValueError("linear_recurrence: sources, out, state_out and stream have no gradient: detach the inputs, "
                             "or call under no_grad")
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("linear_recurrence: records no gradients while the stream is captured: call it and "
                             "linear_recurrence_backward under no_grad")
        return _Recurrence.apply(gate, x, state, kind, blend, starts, workspace)
    handle = _handle("linear_recurrence", "gate", gate, stream)
    if out is None:
        out = _empty(x.shape, x.dtype, x, stream)
    if state_out is None:
        state_out = _empty((_sequences(gate, starts), gate.shape[-1] if gate.dim() else 0), torch.float32, x, stream)
    if workspace is None:
        workspace = _scratch("linear_recurrence", gate, x, starts, stream)
    rc = _calls.linear_recurrence(handle, gate, x, state, code, int(bool(blend)), starts, sources, out, state_out, workspace)
    if rc:
        raise N.RkError(rc, "rk_linear_recurrence")
    return out, state_out


def linear_recurrence_backward(gate, x, out, dout, state=None, dstate_out=None, kind="value", blend=False, starts=None,
                               dgate=None, dx=None, dstate=None, workspace=None, stream=None):
    """Gradients of linear_recurrence's gate, x and first states from those of
    its outputs (rk_linear_recurrence_backward): out is what it returned, dout
    the gradient of that, dstate_out the last states' (None: zeros).  Returns
    (dgate, dx, dstate).  Where they are not given, tokens of no sequence get
    zeros.  There is no second derivative: tensors that require grad are refused
    where gradients are recorded."""
    code = _kind("linear_recurrence_backward", kind)
    handle = _handle("linear_recurrence_backward", "gate", gate, stream)
    if dgate is None:
        dgate = _gradient(gate, gate, starts, stream)
    if dx is None:
        dx = _gradient(x, gate, starts, stream)
    if dstate is None:
        dstate = _empty((_sequences(gate, starts), gate.shape[-1] if gate.dim() else 0), torch.float32, x, stream)
    if workspace is None:
        workspace = _scratch("linear_recurrence_backward", gate, x, starts, stream)
    rc = _calls.linear_recurrence_backward(handle, gate, x, out, dout, state, dstate_out, code, int(bool(blend)), starts, dgate,
                                           dx, dstate, workspace)
    if rc:
        raise N.RkError(rc, "rk_linear_recurrence_backward")
    return dgate, dx, dstate


def _gradient(t, like, starts, stream):
    g = _empty(t.shape, t.dtype, like, stream)
    if starts is None:
        return g
    if stream is None:
        return g.zero_()
    with torch.cuda.stream(stream):
        return g.zero_()


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, x, state, kind, blend, starts, workspace):
        out = None if starts is None else torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        out, last = linear_recurrence(gate, x, state, kind, blend, starts, out=out, workspace=workspace)
        ctx.save_for_backward(gate, x, state, starts, out)
        ctx.how = kind, blend
        return out, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dlast):
        gate, x, state, starts, out = ctx.saved_tensors
        kind, blend = ctx.how
        dgate, dx, dstate = linear_recurrence_backward(gate, x, out, dout.contiguous(), state, dlast.contiguous(), kind, blend,
                                                       starts)
        return dgate, dx, dstate if state is not None else None, None, None, None, None
