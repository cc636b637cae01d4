"""Plain sequential forms of the serving operators in 64 bits, for the tests.

They follow the definitions in include/rk.h one element at a time and share
nothing with the kernels' order of work.
"""
import numpy as np


def softmax(x, t):
    """float64 softmax of the lines of x (float64) at temperatures t."""
    out = np.zeros_like(x)
    for i in range(x.shape[0]):
        v, temp = x[i], float(t[i])
        if v.size == 0:
            continue
        if np.isnan(v).any() or np.isnan(temp):
            out[i] = np.nan
            continue
        m = v.max()
        if m == -np.inf:
            continue
        if temp <= 0.0:
            out[i, int(np.argmax(v))] = 1.0
        elif m == np.inf:
            out[i] = np.nan
        else:
            live = v > -np.inf
            e = np.exp(np.maximum(v[live] - m, -1e300) / temp) if np.isfinite(temp) else np.ones(live.sum())
            out[i, live] = e / e.sum()
    return out


def softmax_error(x, t, want, eps_out, tiny_out):
    """How far a float32 evaluation, rounded once more to the output's type,
    may be from `want`.  With z = (x - m) log2(e) / t: the difference, the
    factor (a rounded constant and a division) and the product round once each,
    so z is off by at most 4 * 2^-24 |z| and its power of two by ln 2 times
    that, under 3 |z| 2^-24 relative; the power itself by 2^-23.  The sum is
    off by the mean of its terms' errors (sum p |z| <= log2 n < 20, so under
    60 * 2^-24) and by its additions: 32 in a row in a thread, 6 levels of a
    wave, 4 of a block, up to 8 tiles of a split line in a row and 8 levels for
    these, under 64 * 2^-24 together.  Reciprocal and product add 2 * 2^-24.
    Results under 2^-126 are flushed."""
    with np.errstate(all="ignore"):
        m = np.max(np.where(np.isnan(x), -np.inf, x), axis=1, keepdims=True, initial=-np.inf)
        z = np.abs(x - m) / np.abs(np.asarray(t, np.float64))[:, None] * np.log2(np.e)
    z = np.where(np.isfinite(z), z, 0.0)
    return want * ((3 * z + 130) * 2.0 ** -24 + eps_out) + tiny_out + 2.0 ** -126


def weights(w):
    return np.where((w > 0) & (w < np.inf), w, 0.0)


def pick(w, r):
    """First index whose running float64 sum passes r * (whole sum)."""
    c = np.cumsum(w)
    if not c[-1] > 0:
        return -1
    r = min(r, 1.0) if r > 0 else 0.0
    over = np.nonzero(c > r * c[-1])[0]
    return int(over[0]) if over.size else int(np.nonzero(w)[0][-1])


def draft_verify(p, q, drafted, u, r, starts, max_draft):
    """p, q: float64 lines; returns (tokens, accepted)."""
    req, n, drafts = len(r), p.shape[1], len(drafted)
    tokens = np.full((req, max_draft + 1), -1, np.int64)
    accepted = np.zeros(req, np.int64)
    with np.errstate(invalid="ignore"):
        for b in range(req):
            lo = min(max(int(starts[b]), 0), drafts)
            hi = min(max(int(starts[b + 1]), lo), drafts, lo + max_draft)
            i = lo
            while i < hi:
                x = int(drafted[i])
                if not 0 <= x < n:
                    break
                qx = q[i, x] if q is not None else 1.0
                if not float(u[i]) * qx < weights(p[i + b, x]):
                    break
                tokens[b, i - lo] = x
                i += 1
            w = weights(p[i + b])
            if i < hi:
                if q is not None:
                    less = weights(p[i + b] - q[i])
                else:
                    less = w.copy()
                    if 0 <= drafted[i] < n:
                        less[drafted[i]] = weights(p[i + b, drafted[i]] - 1.0)
                w = less if less.sum() > 0 else w
            tokens[b, i - lo] = pick(w, float(r[b]))
            accepted[b] = i - lo
    return tokens, accepted


def block_tables(lens, block, held, table, ring, state):
    """Returns (held, table, ring, state of 4) afterwards."""
    table, ring = table.copy(), ring.copy()
    width, size = table.shape[1], ring.size
    head, tail = int(state[0]), int(state[1])
    held = [min(max(int(h), 0), width) for h in held]
    want = [-(-max(int(n), 0) // block) for n in lens]
    after, missing, lost = list(held), 0, 0
    given = []
    for b, n in enumerate(want):
        for j in range(min(n, width), held[b]):
            given.append(table[b, j])
        after[b] = min(after[b], n)
    free = [ring[(head + i) % size] for i in range(tail - head)]
    room = size - len(free)
    lost = max(0, len(given) - room)
    given = given[:room]
    for i, g in enumerate(given):
        ring[(tail + i) % size] = g
    free += given
    taken = 0
    for b, n in enumerate(want):
        missing += max(0, n - width)
        for j in range(held[b], min(n, width)):
            if taken < len(free):
                table[b, j] = free[taken]
                taken += 1
                after[b] += 1
            else:
                missing += 1
    return np.array(after), table, ring, np.array([head + taken, tail + len(given), missing, lost])


def slot_map(lens, fresh, block, table, held, n_blocks, capacity):
    """Returns (slots, positions, requests, starts)."""
    slots, positions, requests = (np.full(capacity, v, np.int64) for v in (-1, 0, -1))
    starts, t = [0], 0
    for b in range(len(lens)):
        n = max(int(lens[b]), 0)
        m = min(max(int(fresh[b]), 0), n)
        for pos in range(n - m, n) if t < capacity else ():
            if t < capacity:
                requests[t], positions[t] = b, pos
                j = pos // block
                if j < held[b] and j < table.shape[1] and 0 <= table[b, j] < n_blocks:
                    slots[t] = int(table[b, j]) * block + pos % block
            t += 1
        t = starts[-1] + m
        starts.append(min(t, 2 ** 31 - 1))
    return slots, positions, requests, np.array(starts)
