"""Plain sequential forms of the beam and block operators in 64 bits, for the
tests.

They follow the definitions in include/rk.h one row at a time and share nothing
with the kernels' order of work.
"""
import numpy as np


def beam_select(x, scores, ended, end_token, count):
    """x: float64 lines; returns (best, tokens, parents, candidates' scores of every request)."""
    req, beams = scores.shape
    n = x.shape[1]
    best, tokens, parents, all_s = (np.full((req, count), v) for v in (-np.inf, -1, -1, 0.0))
    whole = []
    for b in range(req):
        found, odd = [], False
        for j in range(beams):
            line, score = b * beams + j, scores[b, j]
            odd |= not score < np.inf
            if ended is not None and ended[b, j]:
                if score > -np.inf:
                    found.append((score, line, 0.0, end_token))
                continue
            if not score > -np.inf:
                continue
            m = x[line].max()
            odd |= not m < np.inf
            if m == -np.inf or odd:
                continue
            z = x[line] - m
            s = z - np.log(np.exp(z).sum()) + score
            found += [(s[v], line, x[line, v], v) for v in np.nonzero(x[line] > -np.inf)[0]]
        found.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        whole.append(found)
        if odd:
            best[b] = np.nan
            continue
        for i, (s, line, _, v) in enumerate(found[:count]):
            best[b, i], tokens[b, i], parents[b, i] = s, v, line
    return best, tokens, parents, whole


def fork_blocks(parents, lens, block, held, table, ring, state, n_blocks, table_out):
    """Returns (table_out, held_out, lens_out, pairs, state of 4, ring) afterwards."""
    ring, out = ring.copy(), table_out.copy()
    rows, width = table.shape
    size = ring.size
    held = [min(max(int(h), 0), width) for h in held]
    head, tail = int(state[0]), int(state[1])
    free = [ring[(head + i) % size] for i in range(min(max(tail - head, 0), size))]
    room = size - len(free)
    live = [p for p in parents if 0 <= p < rows]
    named = {int(i) for p in live for i in table[p, : held[p]]}
    given = []
    for p in range(rows):
        if p not in live:
            for i in table[p, : held[p]]:
                if 0 <= i < n_blocks and int(i) not in named:
                    named.add(int(i))
                    given.append(i)
    lost = max(0, len(given) - room)
    given = given[:room]
    for i, g in enumerate(given):
        ring[(head + len(free) + i) % size] = g
    free += given
    n = len(parents)
    held_out, lens_out, pairs = np.zeros(n, np.int64), np.zeros(n, np.int64), np.full((n, 2), -1, np.int64)
    taken = missing = 0
    seen = set()
    for r, p in enumerate(parents):
        if not 0 <= p < rows:
            continue
        p = int(p)
        lens_out[r] = max(int(lens[p]), 0)
        row, h = table[p].copy(), held[p]
        if p in seen:
            full = int(lens_out[r]) // block
            wants = lens_out[r] % block != 0 and full < h
            h = min(h, full)
            if wants:
                if taken < len(free):
                    pairs[r] = row[full], free[taken]
                    row[full] = free[taken]
                    taken += 1
                    h += 1
                else:
                    missing += 1
        seen.add(p)
        out[r, :h] = row[:h]
        held_out[r] = h
    return out, held_out, lens_out, pairs, np.array([head + taken, tail + len(given), missing, lost]), ring


def compact_blocks(held, table, ring, n_blocks, max_pairs):
    """Returns (table, pairs, state of 4, ring) afterwards."""
    table, ring = table.copy(), ring.copy()
    width = table.shape[1]
    held = [min(max(int(h), 0), width) for h in held]
    used = sorted({int(i) for r, h in enumerate(held) for i in table[r, :h] if 0 <= i < n_blocks})
    u = len(used)
    src = [i for i in used if i >= u]
    dst = sorted(set(range(u)) - set(used))
    to = dict(zip(src, dst))
    for r, h in enumerate(held):
        table[r, :h] = [to.get(int(i), i) for i in table[r, :h]]
    pairs = np.full((max_pairs, 2), -1, np.int64)
    pairs[: len(src)] = np.array(list(zip(src, dst))).reshape(-1, 2)
    ring[: n_blocks - u] = np.arange(u, n_blocks)
    return table, pairs, np.array([0, n_blocks - u, len(src), 0]), ring
