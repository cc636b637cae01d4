"""GPU tests of beam selection and of forked, compacted and copied blocks against
the plain forms of tests/beams_ref.py, and of a beam search's step made of them
and the other serving operators, captured and replayed."""
import numpy as np
import pytest
import torch

from tests import beams_ref as ref
from tests import recur_ref
from tests import serving_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")


def _rk():
    import reduction_primitives_amd as rk
    rk.load()
    return rk


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def np64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ selection

def check_beams(x, scores, count, ended=None, end_token=0, ids=torch.int64, **more):
    """The float32 sum is off by at most 2^-24 (|z| of its terms, at most 60 in
    their mean; 3 roundings each; 32 additions of a tile in a row), under 2^-17
    relative, and so a score by that and its own rounding.  Where two candidates
    are nearer than that, either order is right: what must agree is every
    score, each candidate's own score, and that no candidate stands twice."""
    rk = _rk()
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    best, tokens, parents = rk.beam_select(dev(x), dev(scores), count, ended=dev(ended), end_token=end_token, token_dtype=ids, **more)
    assert best.dtype == F32 and tokens.dtype == ids and parents.dtype == torch.int32
    want, want_t, want_p, whole = ref.beam_select(np64(x), np64(scores), None if ended is None else ended.numpy(), end_token, count)
    b, t, p = np64(best), tokens.cpu().numpy(), parents.cpu().numpy()
    with np.errstate(over="ignore"):
        low = np.isneginf(want.astype(np.float32))     # a difference beyond float32's range rounds to -inf
    assert np.array_equal(np.isnan(b), np.isnan(want)) and np.array_equal(np.isneginf(b), low)
    fine = np.isfinite(want)
    tol = 2.0 ** -17 + 2.0 ** -24 * np.abs(want)
    assert (np.abs(b - want)[fine & ~low] <= tol[fine & ~low]).all()
    assert (t[~fine] == -1).all() and (p[~fine] == -1).all()
    for r in range(scores.shape[0]):
        own = {(line, v): s for s, line, _, v in whole[r]}
        got = [(int(line), int(v)) for line, v in zip(p[r][fine[r]], t[r][fine[r]])]
        assert len(set(got)) == len(got)
        for i, c in enumerate(got):
            assert abs(own[c] - want[r, i]) <= 2 * (2.0 ** -17 + 2.0 ** -24 * abs(want[r, i])), (r, i, c)
    return t, p, want_t, want_p


@pytest.mark.parametrize("n", [1, 2, 7, 63, 64, 257, 2047, 2048, 2049, 4100, 32768, 50001])
@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("beams,count", [(1, 1), (4, 8), (3, 64), (7, 5)])
def test_beam_sizes(n, dt, beams, count):
    g = gen(n + beams)
    req = 2 if n > 3000 else 5
    x = (torch.randn(req * beams, n, generator=g) * 3).to(dt)
    t, p, wt, wp = check_beams(x, torch.randn(req, beams, generator=g) * 2 - 20, count, ids=torch.int32 if n % 2 else torch.int64)
    if dt == F32:                                   # far from ties
        assert np.array_equal(t, wt) and np.array_equal(p, wp)


@pytest.mark.parametrize("req,beams,n,count", [(40, 8, 9001, 16), (300, 4, 700, 8), (1, 16, 140001, 33), (2500, 2, 100, 4), (1, 300, 50, 64), (2, 4096, 70, 64)])
def test_beam_counts(req, beams, n, count):
    g = gen(req)
    x = torch.randn(req * beams, n, generator=g) * 2
    t, p, wt, wp = check_beams(x, torch.randn(req, beams, generator=g), count)
    assert np.array_equal(t, wt) and np.array_equal(p, wp)


@pytest.mark.parametrize("n", [3, 100, 5000, 40000])
@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_beam_masks_and_odd_values(n, dt):
    g = gen(n)
    beams = 3
    x = (torch.randn(14 * beams, n, generator=g) * 3).to(dt)
    scores = torch.randn(14, beams, generator=g)
    low = torch.finfo(dt).min
    line = lambda r, j: r * beams + j  # noqa: E731
    x[line(0, 0)] = -INF                            # a line with nothing left
    x[line(1, 0): line(2, 0)] = -INF                # a request with nothing left
    x[line(2, 0): line(3, 0), 1:] = -INF            # three candidates in all
    x[line(3, 1), : n - 1] = low                    # masked by the lowest value
    x[line(4, 2)] = low
    x[line(5, 0), n // 2] = NAN
    x[line(6, 1), n - 1] = INF
    scores[7, 1] = -INF
    x[line(7, 1)] = NAN                             # not read
    scores[8, 2] = NAN
    scores[9, 0] = INF
    scores[10] = -INF
    x[line(11, 0): line(12, 0), ::2] = -INF
    x[line(12, 0)] = 0.0                            # everything the same
    x[line(12, 0), ::3] = -0.0
    scores[12, 1:] = -INF
    x[line(13, 0), 0], x[line(13, 0), n - 1] = low, torch.finfo(dt).max
    ended = torch.zeros(14, beams, dtype=torch.bool)
    t, p, wt, wp = check_beams(x, scores, 6)
    assert np.array_equal(t[12], wt[12]) and np.array_equal(p[12], wp[12])     # the lowest tokens
    assert (t[1] == -1).all() and (t[10] == -1).all()
    ended[5, 0] = ended[6, 1] = ended[0, 1] = ended[10, 0] = True              # the odd lines are not read
    ended[11] = True
    t, p, wt, wp = check_beams(x, scores, 6, ended=ended, end_token=n - 1)
    assert np.array_equal(t[11], wt[11]) and (t[11, :3] == n - 1).all() and (t[11, 3:] == -1).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("beams", [1, 4])
def test_beam_ties_and_orders(dt, beams):
    """Equal logits go by line and token; rising and falling lines, and the largest in one lane's places."""
    n = 6000
    up = torch.arange(n, dtype=F32).div(64).floor().repeat(beams, 1)
    for x in (up, up.flip(1), torch.zeros(beams, n), (torch.arange(n) % 7 == 3).float().repeat(beams, 1) * 5,
              (torch.arange(n) % 256 < 4).float().repeat(beams, 1) * (torch.arange(n) % 11 + 1)):
        for count in (1, 5, 64):
            t, p, wt, wp = check_beams(x.to(dt), torch.zeros(1, beams), count)
            assert np.array_equal(t, wt) and np.array_equal(p, wp)
            t, p, wt, wp = check_beams(x.to(dt), -torch.arange(beams, dtype=F32).view(1, beams).flip(1) * 0.0, count, ended=torch.ones(1, beams, dtype=torch.bool))
            assert np.array_equal(p, wp)


def test_beam_strides_offsets_and_buffers():
    rk = _rk()
    g = gen(3)
    for n, pad, dt in ((5003, 3, BF16), (301, 0, F16), (4099, 1, F32)):
        buf = torch.randn(1 + 6 * (n + pad), generator=g).to(dt).to(DEV)
        x = buf.as_strided((6, n), (n + pad, 1), 1)
        scores = torch.randn(2, 3, generator=g)
        check_beams(x.cpu(), scores, 4)
        want = rk.beam_select(x.contiguous(), scores.to(DEV), 4)
        best, tokens, parents = torch.zeros(2, 4, device=DEV), torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, 4, dtype=torch.int32, device=DEV)
        got = rk.beam_select(x, scores.to(DEV), 4, best=best, tokens=tokens, parents=parents,
                             ended=torch.zeros(2, 3, dtype=torch.uint8, device=DEV), end_token=0)
        assert got[0] is best and got[1] is tokens and got[2] is parents
        for a, b in zip(got, want):
            assert torch.equal(a.double(), b.double())
    one = torch.randn(1, 900, generator=g).to(DEV).expand(4, 900)      # one line for all beams
    check_beams(one.cpu(), torch.tensor([[0.0, -1.0, -1.0, -3.0]]), 10)


def test_beam_of_nothing_and_refusals():
    rk = _rk()
    z = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    best, tokens, parents = rk.beam_select(z(0, 9), z(0, 3))
    assert best.shape == (0, 3)
    bad = [dict(logits=z(6, 9, 1)), dict(logits=z(6, 9, dtype=torch.float64)), dict(scores=z(2, 4)), dict(scores=z(6)),
           dict(scores=z(2, 3, dtype=BF16)), dict(ended=z(2, 3, dtype=torch.bool)), dict(ended=z(2, 3, dtype=torch.int32), end_token=0),
           dict(ended=z(2, 4, dtype=torch.bool), end_token=0), dict(count=0), dict(tokens=z(2, 3)), dict(best=z(2, 4)),
           dict(parents=z(2, 3, dtype=torch.int64)), dict(logits=z(9, 6).t()), dict(token_dtype=F32), dict(scores=z(2, 0), logits=z(0, 9)),
           dict(logits=z(6, 9).requires_grad_()), dict(tokens=z(2, 3, dtype=torch.int32), token_dtype=torch.int64)]
    for b in bad:
        with pytest.raises(ValueError):
            rk.beam_select(**{**dict(logits=z(6, 9), scores=z(2, 3)), **b})
    for b, what in ((dict(count=65), "unsupported"), (dict(ended=z(2, 3, dtype=torch.bool), end_token=9), "invalid"),
                    (dict(ended=z(2, 3, dtype=torch.bool), end_token=-1), "invalid"), (dict(logits=z(6, 0)), "invalid"),
                    (dict(best=z(2, 3).expand(2, 3), workspace=z(4, dtype=torch.uint8)), "invalid")):
        with pytest.raises(rk.RkError, match=what):
            rk.beam_select(**{**dict(logits=z(6, 9), scores=z(2, 3)), **b})
    with torch.no_grad():
        rk.beam_select(z(6, 9).requires_grad_(), z(2, 3))


def test_beam_past_2_31_elements():
    rk = _rk()
    lines, n = 16, 200_000_001
    x = torch.zeros(lines, n, dtype=BF16, device=DEV)
    at = [(15, n - 1), (15, 5), (14, n - 3), (0, 7)]
    for line, v in at:
        x[line, v] = 30.0
    best, tokens, parents = rk.beam_select(x, torch.zeros(1, lines, device=DEV), 5)
    assert parents[0, :4].tolist() == [0, 14, 15, 15] or sorted(zip(parents[0, :4].tolist(), tokens[0, :4].tolist())) == sorted(at)
    assert sorted(zip(parents[0, :4].tolist(), tokens[0, :4].tolist())) == sorted(at)


# ----------------------------------------------------------------------- fork

def tables(seed, groups, beams, longest, block, spare, width=None):
    """Rows in groups that share their first blocks."""
    rng = np.random.default_rng(seed)
    width = width or longest // block + 2
    rows = groups * beams
    lens, table, held = np.zeros(rows, np.int64), rng.integers(-5, 5, (rows, width)), np.zeros(rows, np.int64)
    ids = iter(rng.permutation(rows * width + spare))
    pool = rows * width + spare
    for g in range(groups):
        n = int(rng.integers(0, longest + 1))
        h = -(-n // block)
        common = [next(ids) for _ in range(int(rng.integers(0, h + 1)))] if h else []
        for b in range(beams):
            r = g * beams + b
            lens[r], held[r] = n, h
            table[r, :h] = common + [next(ids) for _ in range(h - len(common))]
    free = list(ids)
    return lens, held, table, free, pool


def run_fork(parents, lens, block, held, table, ring, state, n_blocks, in_place=False, **more):
    rk = _rk()
    n = len(parents)
    out0 = np.random.default_rng(1).integers(-9, -5, (n, table.shape[1]))
    d = lambda v: torch.from_numpy(np.asarray(v)).to(torch.int32).to(DEV)  # noqa: E731
    dr, ds = d(ring), torch.tensor([int(v) for v in state] + [7, 7], device=DEV)
    out = d(out0)
    so = None if in_place else torch.zeros(4, dtype=torch.int64, device=DEV)
    dt = d(table)
    got = rk.fork_blocks(d(parents), d(lens), block, d(held), dt, dr, ds, n_blocks, table_out=out, state_out=so, **more)
    assert got[0] is out and (not in_place or got[4] is ds) and torch.equal(dt, d(table))
    want = ref.fork_blocks(parents, lens, block, held, table, ring, state, n_blocks, out0)
    for name, g, w in zip(("table", "held", "lens", "pairs", "state", "ring"), (*got, dr), want):
        assert np.array_equal(g.cpu().numpy(), w), (name, g.cpu().numpy(), w)
    return got


def make_ring(rng, free, size, head):
    ring = rng.integers(-9, 0, size)
    for i, f in enumerate(free):
        ring[(head + i) % size] = f
    return ring, (head, head + len(free))


@pytest.mark.parametrize("groups,beams,longest,block", [(1, 1, 40, 16), (1, 4, 100, 16), (5, 4, 1000, 7), (40, 8, 300, 16), (3, 3, 40000, 16),
                                                        (300, 4, 60, 8), (1, 600, 500, 32), (2, 2, 5, 1), (700, 6, 200, 16), (1500, 4, 90, 24)])
@pytest.mark.parametrize("kind", ["beams", "same", "gone", "any", "fewer", "more"])
def test_fork(groups, beams, longest, block, kind):
    rng = np.random.default_rng(groups * 10 + beams)
    lens, held, table, free, pool = tables(groups + beams, groups, beams, longest, block, 3000)
    rows = groups * beams
    row = np.arange(rows)
    own = row // beams * beams + rng.integers(0, beams, rows)
    parents = {"beams": own, "same": row, "gone": np.where(rng.random(groups)[row // beams] < 0.6, -1, own),
               "any": rng.integers(-2, rows + 2, rows), "fewer": row[::3], "more": rng.integers(0, rows, 2 * rows + 3)}[kind]
    size = pool + int(rng.integers(0, 50))
    ring, state = make_ring(rng, free, size, int(rng.integers(0, 5 * size)))
    run_fork(parents, lens, block, held, table, ring, state, pool, in_place=kind == "any")


@pytest.mark.parametrize("free,room", [(0, 0), (0, 3), (2, 0), (5, 1000), (1, 100)])
def test_fork_short_rings(free, room):
    """Blocks given back are taken in the same call; some find none, or no place."""
    rng = np.random.default_rng(free)
    for groups, beams, longest in ((6, 4, 200), (2, 5, 30000)):
        lens, held, table, ids, pool = tables(3, groups, beams, longest, 16, 50)
        size = max(1, free + room)
        ring, state = make_ring(rng, ids[:free], size, int(rng.integers(0, 100)))
        row = np.arange(groups * beams)
        parents = row // beams * beams + rng.integers(0, beams, row.size)
        run_fork(parents, lens, 16, held, table, ring, state, pool)
        parents = np.where(row // beams == 1, -1, row // beams * beams + beams - 1)
        run_fork(parents, lens, 16, held, table, ring, state, pool)


def test_fork_odd_data():
    """Lengths, blocks, parents and ids a host cannot check; the same block at several places and in rows far apart."""
    rng = np.random.default_rng(4)
    rows, width = 60, 9
    for seed in range(6):
        table = rng.integers(-3, 40, (rows, width))
        table[rng.random((rows, width)) < 0.05] = 2 ** 31 - 1
        lens, held = rng.integers(-20, 200, rows), rng.integers(-2, width + 3, rows)
        lens[0], held[1] = 2 ** 31 - 1, 2 ** 31 - 1
        parents = rng.integers(-2, rows + 3, 70)
        parents[3], parents[4] = 2 ** 31 - 1, -2 ** 31
        ring, state = make_ring(rng, list(range(40, 40 + 30)), 100, int(rng.integers(0, 300)))
        run_fork(parents, lens, 8, held, table, ring, state, 38)
    for state in ((5, 2), (0, 1000), (-7, 3), (2 ** 40, 2 ** 40 + 4), (-2 ** 40, -2 ** 40 + 100)):
        run_fork(parents, lens, 8, held, table, ring, state, 38)


def test_fork_sizes_at_the_borders():
    """Rows and lines around what one wave, one segment and the planning in LDS take."""
    rng = np.random.default_rng(8)
    for groups, beams, longest, width in ((1024, 4, 64, None), (1025, 4, 64, None), (2, 3, 16 * 1024, 1024), (2, 3, 16 * 1023, 1025), (1, 2, 16 * 2047, 2048)):
        lens, held, table, free, pool = tables(groups, groups, beams, longest, 16, 500, width)
        row = np.arange(groups * beams)
        parents = row // beams * beams + rng.integers(0, beams, row.size)
        ring, state = make_ring(rng, free, pool + 1, 3)
        run_fork(parents, lens, 16, held, table, ring, state, pool)


def test_fork_of_nothing():
    rng = np.random.default_rng(8)
    lens, held, table, free, pool = tables(1, 4, 2, 100, 16, 9)
    ring, state = make_ring(rng, free, pool, 0)
    run_fork(np.zeros(0, np.int64), lens, 16, held, table, ring, state, pool)                      # every row is given up
    none = np.zeros(0, np.int64)
    run_fork(np.array([0, -1]), none, 16, none, np.zeros((0, 5), np.int64), ring, state, pool)     # no row was there
    run_fork(np.arange(8), lens, 16, held, table[:, :0], ring, state, pool)                        # no table


def test_fork_wide_lines():
    """Table lines that lie apart."""
    rk = _rk()
    rng = np.random.default_rng(2)
    lens, held, table, free, pool = tables(5, 6, 4, 300, 16, 100)
    ring, state = make_ring(rng, free, pool, 11)
    parents = np.arange(24) // 4 * 4 + rng.integers(0, 4, 24)
    d = lambda v: torch.from_numpy(np.asarray(v)).to(torch.int32).to(DEV)  # noqa: E731
    wide, out = torch.full((24, 50), 77, dtype=torch.int32, device=DEV), torch.full((24, 61), 77, dtype=torch.int32, device=DEV)
    w = table.shape[1]
    wide[:, 3: 3 + w] = d(table)
    ds = torch.tensor([*state, 0, 0], device=DEV)
    got = rk.fork_blocks(d(parents), d(lens), 16, d(held), wide[:, 3: 3 + w], d(ring), ds, pool, table_out=out[:, 1: 1 + w])
    want = ref.fork_blocks(parents, lens, 16, held, table, ring, state, pool, np.full((24, w), 77))
    for g, v in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), v)
    assert (out[:, 0] == 77).all() and (out[:, 1 + w:] == 77).all()


# -------------------------------------------------------------------- compact

@pytest.mark.parametrize("groups,beams,longest,spare", [(1, 1, 10, 0), (3, 4, 500, 40), (40, 8, 300, 5000), (2, 2, 40000, 0), (500, 4, 100, 20000), (3, 1, 0, 70)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(groups, beams, longest, spare, in_place):
    rk = _rk()
    rng = np.random.default_rng(groups)
    _, held, table, _, pool = tables(groups, groups, beams, longest, 16, spare)
    table[0, -1] = 2 ** 31 - 1
    if groups == 3:
        held[0], held[-1] = 2 ** 31 - 1, -4
    d = lambda v: torch.from_numpy(np.asarray(v)).to(torch.int32).to(DEV)  # noqa: E731
    ring = rng.integers(-9, 0, pool + 7)
    dt, dr = d(table), d(ring)
    out = None if in_place else dt.clone()
    got, pairs, state = rk.compact_blocks(d(held), dt, dr, pool, table_out=out)
    assert got is (dt if in_place else out) and (in_place or torch.equal(dt, d(table)))
    want = ref.compact_blocks(held, table, ring, pool, pool // 2)
    for name, g, w in zip(("table", "pairs", "state", "ring"), (got, pairs, state, dr), want):
        assert np.array_equal(g.cpu().numpy(), w), name
    again = rk.compact_blocks(d(held), got, dr, pool, table_out=got.clone())       # nothing is left to move
    assert again[2][2] == 0 and (again[1] == -1).all()


@pytest.mark.parametrize("pool", [1, 2, 63, 64, 65, 4095, 4096, 4097, 65535, 65536, 65537, 70000])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.5, 1.0])
def test_compact_pools(pool, share):
    rk = _rk()
    rng = np.random.default_rng(pool)
    n = int(pool * share)
    for ids in (rng.permutation(pool)[:n], np.arange(pool - n, pool), np.arange(n)):
        table = np.concatenate([ids, [-1, pool]])[None]
        d = lambda v: torch.from_numpy(np.asarray(v)).to(torch.int32).to(DEV)  # noqa: E731
        dr, ring = d(np.full(pool, -3)), np.full(pool, -3)
        more = torch.full((pool // 2 + 5, 2), 9, dtype=torch.int32, device=DEV)
        got, pairs, state = rk.compact_blocks(i32([n + 2]), d(table), dr, pool, pairs=more)
        want = ref.compact_blocks([n + 2], table, ring, pool, pool // 2 + 5)
        for name, g, w in zip(("table", "pairs", "state", "ring"), (got, pairs, state, dr), want):
            assert np.array_equal(g.cpu().numpy(), w), name


def test_compact_pool_of_many_chunks():
    """More than 4096 chunks of 4096 ids: their counts are summed by a launch of its own."""
    rk = _rk()
    rng = np.random.default_rng(8)
    pool = 4096 * 4097 + 13
    ids = np.unique(np.concatenate([rng.integers(0, pool, 6000), [0, 4095, 4096, pool - 1, pool - 14, pool // 2]]))
    table = np.concatenate([rng.permutation(ids), rng.permutation(ids)]).reshape(2, -1)
    d = lambda v: torch.from_numpy(np.asarray(v)).to(torch.int32).to(DEV)  # noqa: E731
    dr, ring = d(np.full(pool, -3)), np.full(pool, -3)
    got, pairs, state = rk.compact_blocks(i32([len(ids)] * 2), d(table), dr, pool)
    want = ref.compact_blocks([len(ids)] * 2, table, ring, pool, pool // 2)
    for name, g, w in zip(("table", "pairs", "state", "ring"), (got, pairs, state, dr), want):
        assert np.array_equal(g.cpu().numpy(), w), name


def test_compact_of_nothing():
    rk = _rk()
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    ring = i32([5, 5, 5])
    _, pairs, state = rk.compact_blocks(z, torch.zeros(0, 4, dtype=torch.int32, device=DEV), ring, 3)
    assert state.tolist() == [0, 3, 0, 0] and ring.tolist() == [0, 1, 2] and pairs.shape == (1, 2)
    _, pairs, state = rk.compact_blocks(z, torch.zeros(0, 4, dtype=torch.int32, device=DEV), ring, 0)
    assert state.tolist() == [0, 0, 0, 0] and pairs.shape == (0, 2)


# ----------------------------------------------------------------------- copy

def copied(caches, pairs):
    want = [c.clone() for c in caches]
    for c, w in zip(caches, want):
        for s, t in pairs.tolist():
            if 0 <= s < len(c) and 0 <= t < len(c):
                w[t] = c[s]
    return want


@pytest.mark.parametrize("shape,dt", [((40, 16, 8, 64), BF16), ((40, 1), torch.uint8), ((40, 3), torch.uint8), ((40, 15), torch.uint8), ((40, 17), torch.int8),
                                      ((40, 16401), torch.uint8), ((40, 8191), F16), ((40, 100000), F32), ((40,), torch.int64)])
@pytest.mark.parametrize("count", [1, 3])
def test_copy(shape, dt, count):
    rk = _rk()
    g = gen(len(shape))
    caches = [torch.randint(-100, 100, shape, generator=g).to(dt) for _ in range(count)]
    pairs = torch.tensor([[0, 20], [1, 21], [-1, -1], [1, 22], [19, 39], [5, 40], [40, 25], [-1, 26], [3, 3], [7, -2], [2 ** 31 - 1, 27]], dtype=torch.int32)
    dev = [c.to(DEV) for c in caches]
    assert rk.copy_blocks(dev, pairs.to(DEV)) is dev
    for d, w in zip(dev, copied(caches, pairs)):
        assert torch.equal(d.cpu(), w)


def test_copy_many_pairs_caches_and_strides():
    rk = _rk()
    g = gen(1)
    n = 1500
    ids = torch.randperm(2 * n, generator=g).to(torch.int32)
    pairs = torch.stack([ids[:n], ids[n:]], 1)
    pairs[torch.rand(n, generator=g) < 0.4] = -1
    for count in (1, 64, 65, 130):
        caches = [torch.randint(-100, 100, (2 * n, 10 + i), generator=g).to(torch.int16) for i in range(count)]
        dev = [c.to(DEV) for c in caches]
        rk.copy_blocks(tuple(dev), pairs.to(DEV))
        for d, w in zip(dev, copied(caches, pairs)):
            assert torch.equal(d.cpu(), w)
    both = torch.randint(-100, 100, (2 * n, 2, 6, 5), generator=g).to(torch.int16)       # keys and values of a block side by side
    d = both.to(DEV)
    rk.copy_blocks([d[:, 0], d[:, 1, :, :]], pairs.to(DEV))
    assert torch.equal(d.cpu(), copied([both], pairs)[0])
    d = both.to(DEV)
    rk.copy_blocks([d[:, 1]], pairs.to(DEV))
    assert torch.equal(d[:, 0].cpu(), both[:, 0]) and torch.equal(d[:, 1].cpu(), copied([both[:, 1]], pairs)[0])
    byte = torch.randint(0, 100, (1 + 60 * 37,), generator=g).to(torch.uint8)             # blocks at odd addresses
    view = lambda t: t[1:].view(60, 37)  # noqa: E731
    d, few = byte.to(DEV), pairs[(pairs < 60).all(1)][:1] * 0 + torch.tensor([[2, 59]], dtype=torch.int32)
    rk.copy_blocks([view(d)], few.to(DEV))
    assert torch.equal(view(d).cpu(), copied([view(byte)], few)[0]) and d[0].cpu() == byte[0]


def test_copy_of_nothing_and_refusals():
    rk = _rk()
    c = torch.ones(4, 6, device=DEV)
    pairs = i32([[0, 1]])
    assert rk.copy_blocks([], pairs) == []
    rk.copy_blocks([c], torch.zeros(0, 2, dtype=torch.int32, device=DEV))
    rk.copy_blocks([c[:0], torch.ones(4, 0, device=DEV)], pairs)
    for caches, p in (([c.t()], pairs), ([c.cpu()], pairs), ([c[0, 0]], pairs), ([c], pairs.long()), ([c], i32([0, 1, 2])), ([c], pairs.cpu())):
        with pytest.raises(ValueError):
            rk.copy_blocks(caches, p)
    with pytest.raises(TypeError):
        rk.copy_blocks(c, pairs)
    with pytest.raises(TypeError):
        rk.copy_blocks([3], pairs)
    with pytest.raises(rk.RkError, match="invalid"):
        rk.copy_blocks([c[:1].expand(4, 6)], pairs)
    with pytest.raises(rk.RkError, match="invalid"):
        rk.copy_blocks([pairs.view(-1)], pairs)


def test_copy_past_2_31_bytes():
    rk = _rk()
    c = torch.zeros(70000, 65536, dtype=torch.uint8, device=DEV)
    c[69998], c[3] = 5, 6
    rk.copy_blocks([c], i32([[69998, 69999], [3, 40000]]))
    assert (c[69999] == 5).all() and (c[40000] == 6).all() and not c[40001].any() and not c[39999].any()


# ---------------------------------------------------------------- refusals

def test_block_calls_check_tensors():
    rk = _rk()
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    state = z(4, dtype=torch.int64)
    base = dict(parents=z(3), lens=z(4), block_size=16, held=z(4), table=z(4, 5), ring=z(9), state=state, n_blocks=9)
    for b in (dict(parents=z(3, dtype=torch.int64)), dict(lens=z(5)), dict(held=z(3)), dict(table=z(3, 5)), dict(table=z(5, 4).t()),
              dict(table=z(4, 5, dtype=torch.int64)), dict(state=z(2, dtype=torch.int64)), dict(state=z(4)), dict(table_out=z(3, 4)),
              dict(table_out=z(4, 5)), dict(held_out=z(4)), dict(lens_out=z(2)), dict(pairs=z(3)), dict(state_out=z(3, dtype=torch.int64)),
              dict(ring=torch.zeros(9, dtype=torch.int32)), dict(parents=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            rk.fork_blocks(**{**base, **b})
    t = z(7, 5)
    for b, what in ((dict(block_size=0), "invalid"), (dict(n_blocks=-1), "invalid"), (dict(table=t[:4], table_out=t[3:6]), "invalid"),
                    (dict(workspace=z(8, dtype=torch.uint8)), "invalid"), (dict(ring=z(0)), "invalid"), (dict(n_blocks=1 << 40), "unsupported"),
                    (dict(held_out=base["parents"]), "invalid")):
        with pytest.raises(rk.RkError, match=what):
            rk.fork_blocks(**{**base, **b})
    base = dict(held=z(4), table=z(4, 5), ring=z(9), n_blocks=9)
    for b in (dict(held=z(3)), dict(table=z(4, 5, dtype=torch.int64)), dict(table_out=z(4, 6)), dict(pairs=z(9)), dict(state_out=z(4)),
              dict(ring=z(9, dtype=torch.int64)), dict(held=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            rk.compact_blocks(**{**base, **b})
    for b, what in ((dict(ring=z(8)), "invalid"), (dict(pairs=z(3, 2)), "invalid"), (dict(n_blocks=-1), "invalid"),
                    (dict(workspace=z(8, dtype=torch.uint8)), "invalid"), (dict(held=t.view(-1)[:4], table=t[:4]), "invalid")):
        with pytest.raises(rk.RkError, match=what):
            rk.compact_blocks(**{**base, **b})
    rk.rk_debug_fail_launches(1)
    with pytest.raises(rk.RkError, match="HIP"):
        rk.copy_blocks([z(4, 4)], z(1, 2))


# --------------------------------------------------- a step of a beam search

def test_search_step():
    """Selection, forked tables, copied blocks, one more token for each beam, its slots, and a recurrent layer's
    states from the beams' parents: eagerly and captured, step after step, against the plain forms."""
    rk = _rk()
    req, beams, vocab, block, width, ch = 3, 4, 1000, 4, 12, 40
    rows, pool = req * beams, 200
    g = gen(1)
    prompt = np.array([5, 8, 11])
    lens = np.repeat(prompt, beams)
    table, held = np.full((rows, width), -1), np.zeros(rows, np.int64)
    ids = list(np.random.default_rng(3).permutation(pool))
    for b in range(req):                            # a prompt's blocks are its beams' at first, but the last one
        h = -(-prompt[b] // block)
        common = [ids.pop() for _ in range(prompt[b] // block)]
        for j in range(beams):
            r = b * beams + j
            held[r] = h
            table[r, :h] = common + [ids.pop() for _ in range(h - len(common))]
    ring = np.array(ids + [-1] * (pool - len(ids)))
    state = np.array([0, len(ids), 0, 0])
    cache = torch.randn(pool, block, 6, generator=g)
    hidden = torch.randn(rows, ch, generator=g)
    scores = torch.full((req, beams), -INF)
    scores[:, 0] = 0.0
    d = lambda v: torch.from_numpy(np.array(v)).to(torch.int32).to(DEV)  # noqa: E731
    s = dict(lens=d(lens), held=d(held), table=d(table), ring=d(ring), state=torch.from_numpy(state).to(DEV), cache=cache.to(DEV), hidden=hidden.to(DEV), scores=scores.to(DEV))
    buf = dict(logits=torch.zeros(rows, vocab, device=DEV), gate=torch.zeros(rows, 1, ch, device=DEV), x=torch.zeros(rows, 1, ch, device=DEV),
               one=torch.ones(rows, dtype=torch.int32, device=DEV))
    new = {k: torch.zeros_like(v) for k, v in s.items()}
    new["table"].fill_(-1)
    ended = torch.zeros(req, beams, dtype=torch.bool, device=DEV)

    def step():
        best, tokens, parents = rk.beam_select(buf["logits"], s["scores"], ended=ended, end_token=1)
        table, held, lens, pairs, _ = rk.fork_blocks(parents.view(-1), s["lens"], block, s["held"], s["table"], s["ring"], s["state"], pool, table_out=new["table"])
        rk.copy_blocks([s["cache"]], pairs)
        lens = lens + buf["one"]
        held, _ = rk.block_tables(lens, block, held, table, s["ring"], s["state"])
        slots, positions, _, _ = rk.slot_map(lens, buf["one"], block, table, held, pool, capacity=rows)
        out, hidden = rk.linear_recurrence(buf["gate"], buf["x"], state=s["hidden"], kind="sigmoid", blend=True, sources=parents.view(-1), state_out=new["hidden"])
        for k, v in (("scores", best), ("lens", lens), ("held", held), ("table", table), ("hidden", hidden)):
            s[k].copy_(v)
        return tokens, parents, slots, out

    first = {k: v.clone() for k, v in s.items()}
    ins = [dict(logits=torch.randn(rows, vocab, generator=g) * 3, gate=torch.randn(rows, 1, ch, generator=g), x=torch.randn(rows, 1, ch, generator=g)) for _ in range(6)]

    def plain(inputs):
        st = dict(lens=lens.copy(), held=held.copy(), table=table.copy(), ring=ring.copy(), state=state.copy(), cache=cache.numpy().copy(), hidden=np64(hidden), scores=np64(scores))
        outs = []
        for i in inputs:
            best, tokens, parents, _ = ref.beam_select(np64(i["logits"]), st["scores"].astype(np.float32).astype(np.float64), None, 0, beams)
            par = parents.reshape(-1)
            t, h, n, pairs, state2, ring2 = ref.fork_blocks(par, st["lens"], block, st["held"], st["table"], st["ring"], st["state"], pool, np.full((rows, width), -1))
            for a, b in pairs:
                if a >= 0:
                    st["cache"][b] = st["cache"][a]
            n = n + 1
            h, t, ring2, state2 = serving_ref.block_tables(n, block, h, t, ring2, state2)
            slots, _, _, _ = serving_ref.slot_map(n, np.ones(rows, np.int64), block, t, h, pool, rows)
            _, st["hidden"], _, st["err"] = recur_ref.forward(np64(i["gate"]), np64(i["x"]), "sigmoid", True, state=st["hidden"], sources=par)
            st.update(lens=n, held=h, table=t, ring=ring2, state=state2, scores=best)
            outs.append((tokens, parents, slots))
        return st, outs

    want, outs = plain(ins)
    for captured in (False, True):
        for k in s:
            s[k].copy_(first[k])
        if captured:
            graph = torch.cuda.CUDAGraph()
            new["table"].fill_(-1)
            with torch.cuda.graph(graph):
                got = step()
            for k in s:
                s[k].copy_(first[k])
        for i, o in zip(ins, outs):
            for k in i:
                buf[k].copy_(i[k])
            new["table"].fill_(-1)
            if captured:
                graph.replay()
            else:
                got = step()
            torch.cuda.synchronize()
            for v, w in zip(got, o):
                assert np.array_equal(v.cpu().numpy(), w)
        for k in ("lens", "held", "ring", "state"):
            assert np.array_equal(s[k].cpu().numpy(), want[k]), k
        for r in range(rows):
            assert np.array_equal(s["table"][r, : want["held"][r]].cpu().numpy(), want["table"][r, : want["held"][r]])
        assert np.array_equal(s["cache"].cpu().numpy(), want["cache"])
        assert np.abs(np64(s["hidden"]) - want["hidden"]).max() <= 6 * recur_ref.STEP * 8      # six steps, magnitudes under 8
        assert np.abs(np64(s["scores"]) - want["scores"]).max() <= 6 * (2.0 ** -17 + 2.0 ** -24 * 60)


def test_two_streams_and_other_graphs():
    """Calls on two streams at once, and two captured graphs replayed in turn, keep apart."""
    rk = _rk()
    rng = np.random.default_rng(5)
    d = lambda v: torch.from_numpy(np.asarray(v)).to(torch.int32).to(DEV)  # noqa: E731
    sets = []
    for seed in range(2):
        lens, held, table, free, pool = tables(seed, 30, 4, 900, 16, 500)
        ring, state = make_ring(rng, free, pool, 5)
        parents = np.arange(120) // 4 * 4 + rng.integers(0, 4, 120)
        x, sc = torch.randn(120, 9000, generator=gen(seed)).to(DEV), torch.randn(30, 4, generator=gen(seed)).to(DEV)
        sets.append((d(parents), d(lens), d(held), d(table), d(ring), torch.tensor([*state, 0, 0], device=DEV), pool, x, sc))

    def work(q, stream=None):
        parents, lens, held, table, ring, state, pool, x, sc = q
        out, so = torch.full_like(table, -1), torch.empty_like(state)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        a = rk.fork_blocks(parents, lens, 16, held, table, ring, state, pool, table_out=out, state_out=so, stream=stream)
        b = rk.compact_blocks(a[1], a[0], torch.empty_like(ring) if stream is None else spare[stream], pool, stream=stream)
        c = rk.beam_select(x, sc, 9, stream=stream)
        return (*a, *b, *c)

    streams = [torch.cuda.Stream() for _ in sets]
    spare = {s: torch.empty_like(q[4]) for s, q in zip(streams, sets)}
    want = [[t.clone() for t in work(q)] for q in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [work(q, s) for q, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    graphs = []
    for q in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(q)
        graphs.append((graph, out))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, a), b in zip(graphs, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
