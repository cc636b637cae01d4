"""CPU tests of beam selection and of forked, compacted and copied blocks:
refusals, workspace sizes, and the plain forms the GPU tests compare with."""
import itertools

import numpy as np
import pytest
import torch

from tests import beams_ref as ref

FAKE = 0x1000000        # never dereferenced: every call below fails validation
MB = 1 << 20


def _rk():
    import reduction_primitives_amd as rk
    rk.load()
    return rk


@pytest.mark.parametrize("args,code", [
    (dict(dtype=9), 1), (dict(dtype=3), 2), (dict(dtype=4), 2), (dict(token=9), 1), (dict(token=0), 2), (dict(vocab=0), 1),
    (dict(vocab=1 << 31), 2), (dict(req=-1), 1), (dict(beams=0), 1), (dict(beams=4097), 2), (dict(count=0), 1), (dict(count=65), 2),
    (dict(req=1 << 31), 2), (dict(stride=-1), 1), (dict(stride=1 << 60), 1), (dict(end=-1), 1), (dict(end=1000), 1),
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(best=None), 1), (dict(tokens=None), 1), (dict(parents=None), 1),
    (dict(logits=FAKE + 2), 1), (dict(scores=FAKE + MB + 1), 1), (dict(best=FAKE + 3 * MB + 2), 1), (dict(tokens=FAKE + 4 * MB + 4), 1),
    (dict(parents=FAKE + 5 * MB + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 6 * MB + 4), 1), (dict(ws_bytes=100), 1),
    (dict(best=FAKE), 1), (dict(best=FAKE + MB), 1), (dict(tokens=FAKE + 2 * MB), 1), (dict(parents=FAKE + 3 * MB + 8), 1),
    (dict(tokens=FAKE + 3 * MB), 1), (dict(ws=FAKE + MB), 1), (dict(ws=FAKE + 4 * MB), 1),
])
def test_beam_select_refusals(args, code):
    a = dict(dtype=0, token=4, logits=FAKE, stride=1000, vocab=1000, req=3, beams=4, scores=FAKE + MB, ended=FAKE + 2 * MB, end=7,
             count=8, best=FAKE + 3 * MB, tokens=FAKE + 4 * MB, parents=FAKE + 5 * MB, ws=FAKE + 6 * MB, ws_bytes=MB)
    rk = _rk()
    a["token"] = rk.RK_I64
    if args.get("token") == 0:
        args = dict(token=rk.RK_F32)
    a.update(args)
    assert rk.rk_beam_select(a["dtype"], a["token"], a["logits"], a["stride"], a["vocab"], a["req"], a["beams"], a["scores"], a["ended"],
                             a["end"], a["count"], a["best"], a["tokens"], a["parents"], a["ws"], a["ws_bytes"], None) == code


@pytest.mark.parametrize("args,code", [
    (dict(n_out=-1), 1), (dict(rows=-1), 1), (dict(block=0), 1), (dict(max_blocks=-1), 1), (dict(size=0), 1), (dict(pool=-1), 1),
    (dict(size=1 << 31), 2), (dict(pool=1 << 31), 2), (dict(n_out=1 << 31), 2), (dict(rows=1 << 31), 2),
    (dict(rows=1 << 20, max_blocks=1 << 11, ts=1 << 11, tos=1 << 11), 2), (dict(ts=-1), 1), (dict(tos=3), 1), (dict(tos=-1), 1),
    (dict(parents=None), 1), (dict(lens=None), 1), (dict(held=None), 1), (dict(table=None), 1), (dict(ring=None), 1), (dict(state=None), 1),
    (dict(table_out=None), 1), (dict(held_out=None), 1), (dict(lens_out=None), 1), (dict(pairs=None), 1), (dict(state_out=None), 1),
    (dict(ws=None), 1), (dict(ws_bytes=64), 1), (dict(ws=FAKE + 11 * MB + 4), 1), (dict(parents=FAKE + 1), 1), (dict(lens=FAKE + MB + 2), 1),
    (dict(held=FAKE + 2 * MB + 2), 1), (dict(table=FAKE + 3 * MB + 2), 1), (dict(ring=FAKE + 4 * MB + 2), 1), (dict(state=FAKE + 5 * MB + 4), 1),
    (dict(state_out=FAKE + 10 * MB + 4), 1), (dict(pairs=FAKE + 9 * MB + 2), 1),
    (dict(table_out=FAKE + 3 * MB), 1),                            # table: never in place
    (dict(held_out=FAKE + 2 * MB), 1), (dict(lens_out=FAKE + MB), 1), (dict(pairs=FAKE), 1), (dict(pairs=FAKE + 8 * MB), 1),
    (dict(ring=FAKE + 3 * MB), 1), (dict(state_out=FAKE + 5 * MB + 8), 1), (dict(state_out=FAKE + 4 * MB), 1), (dict(ws=FAKE + 3 * MB), 1),
])
def test_fork_blocks_refusals(args, code):
    a = dict(parents=FAKE, n_out=6, lens=FAKE + MB, rows=5, block=16, held=FAKE + 2 * MB, table=FAKE + 3 * MB, ts=4, max_blocks=4,
             ring=FAKE + 4 * MB, size=100, state=FAKE + 5 * MB, pool=90, table_out=FAKE + 6 * MB, tos=4, held_out=FAKE + 7 * MB,
             lens_out=FAKE + 8 * MB, pairs=FAKE + 9 * MB, state_out=FAKE + 10 * MB, ws=FAKE + 11 * MB, ws_bytes=MB)
    a.update(args)
    assert _rk().rk_fork_blocks(a["parents"], a["n_out"], a["lens"], a["rows"], a["block"], a["held"], a["table"], a["ts"],
                                a["max_blocks"], a["ring"], a["size"], a["state"], a["pool"], a["table_out"], a["tos"], a["held_out"],
                                a["lens_out"], a["pairs"], a["state_out"], a["ws"], a["ws_bytes"], None) == code


@pytest.mark.parametrize("args,code", [
    (dict(rows=-1), 1), (dict(max_blocks=-1), 1), (dict(pool=-1), 1), (dict(size=0), 1), (dict(size=89), 1), (dict(max_pairs=44), 1),
    (dict(rows=1 << 31), 2), (dict(pool=1 << 31, size=1 << 31, max_pairs=1 << 30), 2), (dict(size=1 << 31), 2), (dict(max_pairs=1 << 31), 2),
    (dict(ts=-1), 1), (dict(tos=3), 1), (dict(held=None), 1), (dict(table=None), 1), (dict(table_out=None), 1), (dict(ring=None), 1),
    (dict(pairs=None), 1), (dict(state_out=None), 1), (dict(ws=None), 1), (dict(ws_bytes=64), 1), (dict(ws=FAKE + 6 * MB + 8), 1),
    (dict(held=FAKE + 2), 1), (dict(table=FAKE + MB + 1), 1), (dict(table_out=FAKE + 2 * MB + 2), 1), (dict(ring=FAKE + 3 * MB + 2), 1),
    (dict(pairs=FAKE + 4 * MB + 2), 1), (dict(state_out=FAKE + 5 * MB + 4), 1),
    (dict(table_out=FAKE + MB + 4), 1), (dict(table_out=FAKE + MB, tos=5), 1),     # neither the table itself nor beside it
    (dict(ring=FAKE + MB), 1), (dict(pairs=FAKE + 3 * MB), 1), (dict(state_out=FAKE), 1), (dict(ws=FAKE), 1), (dict(ws=FAKE + 4 * MB), 1),
])
def test_compact_blocks_refusals(args, code):
    a = dict(held=FAKE, rows=5, table=FAKE + MB, ts=4, max_blocks=4, pool=90, table_out=FAKE + 2 * MB, tos=4, ring=FAKE + 3 * MB, size=90,
             pairs=FAKE + 4 * MB, max_pairs=45, state_out=FAKE + 5 * MB, ws=FAKE + 6 * MB, ws_bytes=MB)
    a.update(args)
    assert _rk().rk_compact_blocks(a["held"], a["rows"], a["table"], a["ts"], a["max_blocks"], a["pool"], a["table_out"], a["tos"],
                                   a["ring"], a["size"], a["pairs"], a["max_pairs"], a["state_out"], a["ws"], a["ws_bytes"], None) == code


@pytest.mark.parametrize("cache,args,code", [
    (dict(data=None), {}, 1), (dict(stride=-1), {}, 1), (dict(stride=99), {}, 1), (dict(size=-1), {}, 1), (dict(blocks=-1), {}, 1),
    (dict(blocks=1 << 31, stride=1 << 10), {}, 2), (dict(size=(1 << 29) + 1, stride=1 << 30), {}, 2), (dict(stride=1 << 60), {}, 1),
    ({}, dict(n_pairs=-1), 1), ({}, dict(n_pairs=1 << 31), 2), ({}, dict(pairs=None), 1), ({}, dict(pairs=FAKE - MB + 2), 1),
    ({}, dict(pairs=FAKE + 96), 1),
])
def test_copy_blocks_refusals(cache, args, code):
    rk = _rk()
    c = dict(data=FAKE, stride=100, size=100, blocks=7)
    c.update(cache)
    a = dict(pairs=FAKE - MB, n_pairs=5)
    a.update(args)
    caches = [(FAKE + 2 * MB, 100, 100, 7), (c["data"], c["stride"], c["size"], c["blocks"])]
    assert rk.rk_copy_blocks(caches, a["pairs"], a["n_pairs"], None) == code


def test_calls_of_nothing():
    rk = _rk()
    assert rk.rk_beam_select(0, rk.RK_I32, None, 5, 5, 0, 2, None, None, 0, 2, None, None, None, None, 0, None) == 0
    assert rk.load().rk_copy_blocks(None, 0, None, 0, None) == 0 and rk.load().rk_copy_blocks(None, 1, None, 0, None) == 1
    assert rk.load().rk_copy_blocks(None, -1, None, 0, None) == 1
    assert rk.rk_copy_blocks([(None, 0, 0, 0)], FAKE, 4, None) == 0


def test_workspace_sizes():
    rk = _rk()
    beam, fork, compact = rk.rk_beam_select_workspace_size, rk.rk_fork_blocks_workspace_size, rk.rk_compact_blocks_workspace_size
    for vocab, req, beams, count in ((1, 1, 1, 1), (32768, 1, 4, 8), (131072, 64, 8, 16), (50257, 300, 5, 64)):
        assert beam(0, vocab, req, beams, count) >= req * beams * (12 + 8 * count) and beam(1, vocab, req, beams, count) % 256 == 0
    assert beam(3, 5, 1, 1, 1) == 0 and beam(0, 0, 1, 1, 1) == 0 and beam(0, 5, 1, 1, 65) == 0
    # what the kernels of a call keep: a bit an entry, a word a block, three a row
    for rows, out, width, pool in ((0, 0, 0, 0), (1, 1, 1, 1), (256, 256, 257, 70000), (5000, 3, 64, 2 ** 24)):
        assert fork(rows, out, width, pool) >= 32 + rows * -(-width // 64) * 8 + 4 * (2 * rows + out + pool)
    assert fork(-1, 1, 1, 1) == 0 and fork(1 << 20, 1, 1 << 12, 1) == 0 and fork(1, 1, 1, 1 << 31) == 0
    for pool in (0, 1, 4096, 4097, 2 ** 24, 2 ** 31 - 1):
        assert compact(pool) >= pool + -(-pool // 64) * 16 and compact(pool) % 256 == 0
    assert compact(-1) == 0 and compact(1 << 31) == 0


def test_tensor_refusals():
    """What the Python calls refuse before the library sees it (CPU tensors
    among it: there is no fallback)."""
    rk = _rk()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64)  # noqa: E731
    for call in (lambda: rk.beam_select(torch.zeros(4, 8), torch.zeros(2, 2)),
                 lambda: rk.fork_blocks(i32(3), i32(3), 16, i32(3), i32(3, 4), i32(9), i64(4), 12),
                 lambda: rk.compact_blocks(i32(3), i32(3, 4), i32(12), 12),
                 lambda: rk.copy_blocks([torch.zeros(5, 3)], i32(2, 2))):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_plain_beams_are_the_best_paths():
    """Two steps of selection with as many beams as there are paths keep all of
    them: their scores are the sums of log probabilities, by enumeration."""
    rng = np.random.default_rng(0)
    n = 3
    first, second = rng.standard_normal(n), rng.standard_normal((n, n))
    log = lambda x: x - np.log(np.exp(x).sum(-1, keepdims=True))  # noqa: E731
    best, tokens, parents, _ = ref.beam_select(first[None], np.zeros((1, 1)), None, 0, n)
    assert (np.sort(tokens[0]) == np.arange(n)).all() and (parents[0] == 0).all()
    again, last, lines, _ = ref.beam_select(second[tokens[0]], best, None, 0, n * n)
    got = {(int(tokens[0][p]), int(t)): s for s, t, p in zip(again[0], last[0], lines[0])}
    for i, j in itertools.product(range(n), range(n)):
        assert got[i, j] == pytest.approx(log(first)[i] + log(second[i])[j], abs=1e-12)
    assert (np.diff(again[0]) <= 0).all()


def test_plain_forks_and_compaction_keep_what_rows_read():
    """Copied and renamed blocks hold what the rows named before, and no block is
    free and named at once."""
    rng = np.random.default_rng(1)
    block, width, pool = 4, 6, 60
    for _ in range(20):
        rows = 6
        lens = rng.integers(0, block * width + 1, rows)
        held = -(-lens // block)
        ids = rng.permutation(pool)
        table, at = np.full((rows, width), -7), 0
        for r in range(rows):
            table[r, : held[r]] = ids[at: at + held[r]]
            at += held[r]
        free = ids[at:]
        ring, state = np.full(pool, -1), [0, len(free)]
        ring[: len(free)] = free
        data = rng.integers(0, 1 << 30, (pool, block))
        read = lambda d, t, h, n: d[t[:h]].reshape(-1)[:n]  # noqa: E731
        parents = rng.integers(0, rows, rows)
        out, h2, l2, pairs, st, ring2 = ref.fork_blocks(parents, lens, block, held, table, ring, state, pool, table)
        moved = data.copy()
        for s, d in pairs:
            if s >= 0:
                moved[d] = data[s]
        left = {int(ring2[i % pool]) for i in range(st[0], st[1])}
        named = {int(i) for r in range(rows) for i in out[r, : h2[r]]}
        assert st[2] == 0 and not left & named and left | named == set(range(pool))
        for r in range(rows):
            p = parents[r]
            assert (read(moved, out[r], h2[r], l2[r]) == read(data, table[p], held[p], lens[p])).all()
        t3, p3, s3, ring3 = ref.compact_blocks(h2, out, ring2, pool, pool // 2)
        packed = moved.copy()
        for s, d in p3:
            if s >= 0:
                packed[d] = moved[s]
        assert {int(i) for r in range(rows) for i in t3[r, : h2[r]]} == set(range(len(named))) and s3[1] == pool - len(named)
        for r in range(rows):
            assert (read(packed, t3[r], h2[r], l2[r]) == read(moved, out[r], h2[r], l2[r])).all()
