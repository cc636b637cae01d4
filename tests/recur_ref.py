"""Plain sequential forms of the gated linear recurrence in 64 bits, for the
tests, and how far a float32 evaluation may be from them.

They follow the definitions in include/rk.h one token at a time and share
nothing with the kernels' order of work.
"""
import numpy as np


def gates(gate, kind):
    """a and 1 - a of gates in float64."""
    with np.errstate(over="ignore"):
        if kind == "value":
            return gate, 1.0 - gate
        if kind == "log":
            return np.exp(gate), -np.expm1(gate)
        return 1.0 / (1.0 + np.exp(-gate)), 1.0 / (1.0 + np.exp(gate))


def sequences(shape, starts):
    """(first, behind the last) token of every sequence in the flat tokens."""
    if starts is None:
        return [(b * shape[1], (b + 1) * shape[1]) for b in range(shape[0])]
    n = shape[0]
    lo = [min(max(int(s), 0), n) for s in starts]
    return [(i, max(i, j)) for i, j in zip(lo[:-1], lo[1:])]


def first_state(state, sources, b, channels):
    i = b if sources is None else int(sources[b])
    return state[i].copy() if state is not None and 0 <= i < len(state) else np.zeros(channels)


# Rounding of one step, in units of 2^-24 of the sum of magnitudes M that the
# step's result is made of.  exp: a power of two good to an ulp (2), its
# correction (1); 1 + e (1) and a reciprocal good to an ulp (2), e r (1): a and
# 1 - a of a logistic gate are off by up to 7, a of a logarithm by 3, 1 - a by 3
# a / (1 - a) + 1 < 12 where it is a difference (gates from -1/4 down) and 8
# where it is a polynomial.  A gate is used in a step once, in its product with
# the state or with the other gates of its run (1 more each); w x rounds once,
# the sum once, joining two runs once.  Under 12 + 4.
STEP = 16 * 2.0 ** -24
# What is below 2^-126 may be flushed, a gate among it: its product with a state (or
# gradient) of magnitude M is then off by 2^-126 M, and the product may be flushed itself.
TINY = 2.0 ** -126


def forward(gate, x, kind, blend, starts=None, state=None, sources=None):
    """float64 (out, last, error bound of out, of last) of float64 gate and x;
    tokens of no sequence are NaN."""
    shape = x.shape
    a, w = gates(gate.reshape(-1, shape[-1]), kind)
    x = x.reshape(a.shape)
    out, err = np.full((2,) + a.shape, np.nan)
    seqs = sequences(shape, starts)
    last, last_err = np.zeros((2, len(seqs), shape[-1]))
    with np.errstate(invalid="ignore", over="ignore"):
        for b, (lo, hi) in enumerate(seqs):
            h = first_state(state, sources, b, shape[-1])
            m, e = np.abs(h), np.zeros_like(h)
            for t in range(lo, hi):
                v = w[t] * x[t] if blend else x[t]
                h = a[t] * h + v
                e = np.abs(a[t]) * e + TINY * (1 + m)
                m = np.abs(a[t]) * m + np.abs(v)
                e += STEP * m
                out[t], err[t] = h, e
            last[b], last_err[b] = h, e
    return out.reshape(shape), last, err.reshape(shape), last_err


def backward(gate, x, h, dout, kind, blend, starts=None, state=None, dlast=None):
    """float64 (dgate, dx, dstate) and their error bounds.  The final products
    add a few roundings more: a (1 - a) is off by up to 14, three products."""
    shape = x.shape
    flat = lambda v: v.reshape(-1, shape[-1])  # noqa: E731
    a, w = gates(flat(gate), kind)
    x, h, dout = flat(x), flat(h), flat(dout)
    dgate, dx, eg, ex = np.full((4,) + a.shape, np.nan)
    seqs = sequences(shape, starts)
    du, eu = np.zeros((2, len(seqs), shape[-1]))
    more = 2 * STEP
    with np.errstate(invalid="ignore", over="ignore"):
        for b, (lo, hi) in enumerate(seqs):
            u = np.zeros(shape[-1]) if dlast is None else dlast[b].copy()
            m, e = np.abs(u), np.zeros_like(u)
            for t in range(hi - 1, lo - 1, -1):
                g, mg = dout[t] + u, np.abs(dout[t]) + m
                ge = e + more * mg
                before = h[t - 1] if t > lo else first_state(state, None, b, shape[-1])
                da = g * (before - x[t]) if blend else g * before
                size = np.abs(before) + (np.abs(x[t]) if blend else 0.0)
                f = {"value": 1.0, "log": a[t], "sigmoid": a[t] * w[t]}[kind]
                dgate[t], eg[t] = da * f, np.abs(f) * size * ge + TINY * (1 + size * mg)
                dx[t], ex[t] = (g * w[t], ge * np.abs(w[t]) + TINY * (1 + mg)) if blend else (g, ge)
                u, m = a[t] * g, np.abs(a[t]) * mg
                e = np.abs(a[t]) * e + STEP * m + TINY * (1 + mg)
            du[b], eu[b] = u, e
    return (dgate.reshape(shape), dx.reshape(shape), du), (eg.reshape(shape), ex.reshape(shape), eu)
