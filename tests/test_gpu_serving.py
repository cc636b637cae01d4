"""GPU tests of the serving operators against the plain 64-bit forms of
tests/serving_ref.py: softmax of lines, draft verification, block tables, slot
maps, and a step made of all of them, captured and replayed."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref

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
    return t.detach().cpu().to(torch.float64).numpy()


# ------------------------------------------------------------------ softmax

def half_step(dt):
    """(relative, absolute) rounding of a store to dt: half a step, below the
    smallest normal value half of its last place."""
    f = torch.finfo(dt)
    return f.eps / 2, (0.0 if dt == F32 else f.tiny * f.eps / 2)


def check_softmax(got, x, t):
    x64 = np64(x)
    want = ref.softmax(x64, t)
    got64 = np64(got)
    assert np.array_equal(np.isnan(got64), np.isnan(want))
    w = np.nan_to_num(want)
    tol = ref.softmax_error(x64, t, w, *half_step(got.dtype))
    err = np.abs(np.nan_to_num(got64) - w)
    assert (err <= tol).all(), (err.max(), np.argwhere(err > tol)[:4])
    for i, temp in enumerate(t):
        if temp <= 0:
            assert np.array_equal(got64[i], want[i], equal_nan=True)


SOFT_N = [1, 2, 7, 8, 63, 65, 255, 256, 257, 511, 2047, 2048, 2049, 4097, 8191, 8192, 8193, 16383, 16385, 32767, 32768, 32769, 50001, 65536, 65537, 131072, 200003]


@pytest.mark.parametrize("n", SOFT_N)
@pytest.mark.parametrize("din,dout", [(F32, F32), (BF16, F32), (F16, F16), (F32, BF16), (BF16, BF16), (F16, F32), (F32, F16)])
def test_softmax_sizes(n, din, dout):
    rk = _rk()
    lines = 3 if n > 20000 else 5
    g = gen(n + 7)
    x = (torch.randn(lines, n, generator=g) * 4).to(din)
    t = [1.0, 0.5, 2.5, 0.0, 1.3][:lines]
    got = rk.softmax(x.to(DEV), temperature=torch.tensor(t).to(DEV), out_dtype=dout)
    check_softmax(got, x, t)


@pytest.mark.parametrize("lines,n", [(1, 1), (17, 256), (63, 255), (1001, 16), (130, 257), (1, 131072), (2, 50000), (64, 300), (700, 33), (513, 4097), (300, 9000), (260, 20000)])
def test_softmax_line_counts(lines, n):
    rk = _rk()
    x = torch.randn(lines, n, generator=gen(lines)) * 2
    check_softmax(rk.softmax(x.to(DEV)), x, [1.0] * lines)


@pytest.mark.parametrize("n", [5, 200, 1000, 9001, 40000, 140001])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_softmax_masks_and_odd_values(n, dt):
    rk = _rk()
    x = (torch.randn(16, n, generator=gen(3 * n)) * 3).to(dt)
    t = [1.0] * 16
    low, high = torch.finfo(dt).min, torch.finfo(dt).max
    x[0] = -INF                                    # nothing left
    x[1, 1:] = -INF
    x[2, : n - 1] = -INF
    x[3, ::2] = low                                # masked by the lowest value
    x[4] = low                                     # ... everywhere: all the same
    x[5, n // 2] = NAN
    x[6, n - 1] = INF
    x[7, n // 2] = INF
    t[7] = 0.0                                     # the infinity is the largest
    x[8], t[8] = -INF, 0.0
    x[9], t[9] = 1.0, 0.0                          # a tie: the first
    x[10, 0], t[10] = NAN, 0.0
    t[11] = INF                                    # the same for all that are left
    x[11, ::3] = -INF
    t[12] = 1e-38                                  # next to nothing but the largest
    t[13] = NAN
    x[14, 0], x[14, n - 1] = high, low
    t[15] = -1.0
    got = rk.softmax(x.to(DEV), temperature=torch.tensor(t).to(DEV))
    check_softmax(got, x, t)
    assert got[0].count_nonzero() == 0 and got[8].count_nonzero() == 0
    assert got[9, 0] == 1


@pytest.mark.parametrize("n", [5, 200, 1000, 9001, 40000, 140001])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_softmax_differences_past_the_largest_float(n, dt):
    """x - m is -inf in float32, (x - m) / t is not."""
    rk = _rk()
    low, high = torch.finfo(dt).min, torch.finfo(dt).max
    t = [INF, 2.0 ** 127, 2.0 ** 124, 1.0, INF]
    x = torch.zeros(len(t), n, dtype=dt)
    x[:, ::2] = low
    x[:, n // 2] = high
    x[:, n - 1] = low
    x[4, 1] = -INF
    check_softmax(rk.softmax(x.to(DEV), temperature=torch.tensor(t).to(DEV)), x, t)
    check_softmax(rk.softmax(x.to(DEV), temperature=torch.tensor(t).to(DEV), out_dtype=F32), x, t)


@pytest.mark.parametrize("n", [77, 8200, 33333, 70003])
@pytest.mark.parametrize("din,dout", [(F32, F32), (F16, F32), (BF16, BF16), (F32, F16)])
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (0, 24)])
def test_softmax_strides_and_offsets(n, din, dout, offset, pad):
    rk = _rk()
    lines, stride = 4, n + pad
    buf = (torch.randn(offset + lines * stride, generator=gen(n)) * 2).to(din)
    view = buf[offset:].as_strided((lines, n), (stride, 1))
    x = buf.to(DEV)[offset:].as_strided((lines, n), (stride, 1), offset)
    obuf = torch.full((offset + lines * (stride + 1),), 7.0, dtype=dout, device=DEV)
    out = obuf.as_strided((lines, n), (stride + 1, 1), offset)
    x_dev = buf.to(DEV).as_strided((lines, n), (stride, 1), offset)
    del x
    assert rk.softmax(x_dev, out=out) is out
    check_softmax(out, view, [1.0] * lines)
    touched = torch.zeros_like(obuf, dtype=torch.bool)
    touched.as_strided((lines, n), (stride + 1, 1), offset).fill_(True)
    assert (obuf[~touched] == 7.0).all()           # between the lines and outside them


@pytest.mark.parametrize("n", [100, 9000, 70000])
def test_softmax_in_place_and_broadcast(n):
    rk = _rk()
    x = torch.randn(3, n, generator=gen(n))
    y = x.to(DEV)
    assert rk.softmax(y, out=y) is y
    check_softmax(y, x, [1.0] * 3)
    both = torch.zeros(3, 2 * n, device=DEV)       # the other half of the same rows
    both[:, :n] = x.to(DEV)
    rk.softmax(both[:, :n], out=both[:, n:])
    check_softmax(both[:, n:], x, [1.0] * 3)
    assert torch.equal(both[:, :n].cpu(), x)
    one = x[:1].to(DEV).expand(4, n)               # one line, four temperatures
    t = [1.0, 0.3, 0.0, 7.0]
    check_softmax(rk.softmax(one, temperature=torch.tensor(t).to(DEV)), x[:1].expand(4, n), t)


@pytest.mark.parametrize("n", [1048576, 1048577, 3000001])
def test_softmax_lines_of_many_tiles(n):
    rk = _rk()
    x = (torch.randn(4, n, generator=gen(n)) * 3).to(BF16)
    x[1, : n - 7] = -INF
    x[3, n // 2] = 60.0
    t = [0.9, 1.0, 1.7, 0.0]
    got = rk.softmax(x.to(DEV), temperature=torch.tensor(t).to(DEV), out_dtype=F32)
    check_softmax(got, x, t)


def test_softmax_of_nothing():
    rk = _rk()
    assert rk.softmax(torch.zeros(0, 9, device=DEV)).shape == (0, 9)
    assert rk.softmax(torch.zeros(9, 0, device=DEV)).shape == (9, 0)


def test_verify_of_nothing():
    rk = _rk()
    z = torch.zeros(0, device=DEV)
    t, a = rk.draft_verify(torch.zeros(0, 9, device=DEV), None, torch.zeros(0, dtype=torch.int64, device=DEV), z, z, max_draft=3)
    assert t.shape == (0, 4) and a.shape == (0,)
    with pytest.raises(rk.RkError, match="invalid"):
        rk.draft_verify(torch.zeros(1, 0, device=DEV), None, torch.zeros(0, dtype=torch.int64, device=DEV), z,
                        torch.zeros(1, device=DEV))


def test_softmax_same_bits_every_time():
    rk = _rk()
    x = torch.randn(9, 60001, generator=gen(1)).to(DEV)
    a = rk.softmax(x)
    for _ in range(3):
        assert torch.equal(a, rk.softmax(x))


# ------------------------------------------------------------- verification

def drafts(seed, req, k, n, dt, q=True, ragged=True, ids=torch.int64, peak=15.0):
    g = gen(seed)
    counts = torch.randint(0, k + 1, (req,), generator=g) if ragged else torch.full((req,), k)
    starts = torch.zeros(req + 1, dtype=torch.int32)
    starts[1:] = counts.cumsum(0)
    rows = int(starts[-1])
    z = torch.randn(rows + req, n, generator=g) * 2
    top = torch.randint(0, n, (rows + req, 1), generator=g)
    z.scatter_(1, top, peak)
    p = torch.softmax(z, 1).to(dt)
    at = torch.arange(rows) + torch.repeat_interleave(torch.arange(req), counts)
    qq = torch.softmax(z[at] + 0.5 * torch.randn(rows, n, generator=g), 1)
    drafted = torch.multinomial(qq, 1, generator=g).view(-1) if rows else torch.zeros(0, dtype=torch.int64)
    return dict(p=p, q=qq.to(dt) if q else None, starts=starts, drafted=drafted.to(ids), k=k,
                u=torch.rand(rows, generator=g), r=torch.rand(req, generator=g))


def run_verify(d, **kw):
    rk = _rk()
    to = lambda v: None if v is None else v.to(DEV)  # noqa: E731
    return rk.draft_verify(to(d["p"]), to(d["q"]), to(d["drafted"]), to(d["u"]), to(d["r"]), starts=to(d["starts"]),
                           max_draft=d["k"], **kw)


def check_verify(d, got):
    starts = d["starts"].tolist() if d["starts"] is not None else [i * d["k"] for i in range(len(d["r"]) + 1)]
    t, a = ref.draft_verify(np64(d["p"]), None if d["q"] is None else np64(d["q"]), d["drafted"].tolist(), np64(d["u"]),
                            np64(d["r"]), starts, d["k"])
    assert got[0].dtype == d["drafted"].dtype
    assert np.array_equal(got[1].cpu().numpy(), a)
    assert np.array_equal(got[0].cpu().numpy(), t)
    return t, a


VERIFY = [(1, 4, 1), (2, 3, 2), (3, 1, 31), (5, 4, 2047), (5, 4, 2048), (5, 4, 2049), (4, 7, 8192), (4, 2, 8193), (3, 3, 50001),
          (2, 2, 131072), (70, 3, 3001), (300, 2, 517), (1, 100, 40), (2, 0, 999), (1, 1, 600000)]


@pytest.mark.parametrize("req,k,n", VERIFY)
@pytest.mark.parametrize("dt,ids,q", [(F32, torch.int64, True), (F16, torch.int32, True), (BF16, torch.int64, True),
                                      (F32, torch.int32, False), (BF16, torch.int32, False)])
def test_verify_sizes(req, k, n, dt, ids, q):
    d = drafts(req * 1000 + n, req, k, n, dt, q=q, ids=ids)
    check_verify(d, run_verify(d))


def test_verify_every_place_is_reached():
    """Whatever is kept: none, some, all of the drafts."""
    d = drafts(5, 200, 6, 300, F32, ragged=False, peak=3.0)
    t, a = check_verify(d, run_verify(d))
    assert set(a.tolist()) == set(range(7))
    d["starts"] = None                             # the same without offsets
    check_verify(d, run_verify(d))


@pytest.mark.parametrize("n", [64, 4096, 16384])
def test_verify_borders_are_exact(n):
    """Equal dyadic weights: every running sum and every bar is exact, so a bar
    on a border takes the entry behind it."""
    req = 64
    d = dict(p=torch.full((req, n), 1.0 / n), q=None, starts=torch.zeros(req + 1, dtype=torch.int32),
             drafted=torch.zeros(0, dtype=torch.int64), k=0, u=torch.zeros(0), r=torch.arange(req) / req)
    got = run_verify(d)
    assert got[0].view(-1).tolist() == [i * n // req for i in range(req)]
    check_verify(d, got)


def test_verify_accepts_exactly():
    """u q < p as real numbers: u = p / q itself is turned down, the float32
    below it kept."""
    n, req = 50, 40
    g = gen(9)
    q = torch.rand(req, n, generator=g) + 0.5
    u = torch.randint(1, 2 ** 12, (req,), generator=g) / 2.0 ** 12
    q = (q * 2 ** 10).round() / 2 ** 10            # 12 bits times 11 bits: exact in float32
    p = torch.zeros(2 * req, n) + 0.001
    x = torch.randint(0, n, (req,), generator=g)
    for b in range(req):
        p[2 * b, x[b]] = u[b] * q[b, x[b]]
    d = dict(p=p, q=q, starts=None, drafted=x, k=1, u=u, r=torch.rand(req, generator=g))
    t, a = check_verify(d, run_verify(d))
    assert a.sum() == 0
    d["u"] = torch.nextafter(u, torch.zeros(()))
    t, a = check_verify(d, run_verify(d))
    assert a.sum() == req


@pytest.mark.parametrize("n", [40, 5000])
def test_verify_odd_values(n):
    req = 12
    d = drafts(4, req, 1, n, F32, ragged=False)
    p, q = d["p"], d["q"]
    x = d["drafted"]
    p[0::2, :][0] = 0.0                            # request 0: turned down, the target's line empty
    p[2] = q[1]                                    # request 1: the draft leaves nothing; u = 1 turns it down
    d["u"][1] = 1.0
    x[2], x[3], x[4] = -1, n, 2 ** 40              # no such tokens
    d["r"][5], d["r"][6] = 0.0, 1.0
    p[14], p[15] = 0.0, 0.0                        # request 7: one entry left
    p[14, n - 1] = p[15, n - 1] = 1.0
    p[16, ::2] = NAN                               # request 8
    p[17, ::3], p[17, 1::3] = INF, -1.0
    d["u"][9] = NAN
    d["r"][10], d["r"][11] = NAN, -0.5
    q[11, : n // 2] = INF
    check_verify(d, run_verify(d))
    p[1] = 0.0                                     # kept, and nothing to draw from
    x[0], d["u"][0] = 3, 0.0
    p[0, 3] = 1.0
    t, a = check_verify(d, run_verify(d))
    assert t[0].tolist() == [3, -1]


def test_verify_clamps_bad_offsets():
    d = drafts(11, 6, 3, 700, F32, ragged=False)
    d["starts"] = torch.tensor([-5, 3, 1, 40, 7, 18, 1000], dtype=torch.int32)
    check_verify(d, run_verify(d))
    d["starts"] = torch.tensor([0, 18, 18, 18, 18, 18, 18], dtype=torch.int32)   # more than max_draft for the first
    check_verify(d, run_verify(d))


@pytest.mark.parametrize("dt", [F32, F16])
@pytest.mark.parametrize("n,pad,offset", [(2049, 1, 1), (9001, 7, 3), (4096, 64, 0)])
def test_verify_strides(dt, n, pad, offset):
    d = drafts(n, 5, 3, n, dt)

    def spread(t):
        buf = torch.full((offset + t.shape[0] * (n + pad) + pad,), NAN, dtype=t.dtype)
        v = buf.as_strided(t.shape, (n + pad, 1), offset)
        v.copy_(t)
        return buf.to(DEV).as_strided(t.shape, (n + pad, 1), offset)
    rk = _rk()
    rest = [d[k].to(DEV) for k in ("drafted", "u", "r")]
    check_verify(d, rk.draft_verify(spread(d["p"]), spread(d["q"]), *rest, starts=d["starts"].to(DEV), max_draft=d["k"]))


def test_verify_second_launch_gives_the_same():
    rk = _rk()
    for seed, (req, k, n) in enumerate([(6, 4, 30000), (600, 2, 9000), (3000, 1, 8500)]):
        d = drafts(seed, req, k, 97, F32)          # small to make, then spread over n
        big = {"p": torch.zeros(d["p"].shape[0], n), "q": torch.zeros(d["q"].shape[0], n)}
        for name in big:
            big[name][:, :97 * 80:80] = d[name]
        d.update(big, drafted=d["drafted"] * 80)
        want = run_verify(d)
        prev = rk.rk_debug_set_fused_finish(0)
        try:
            got = run_verify(d)
        finally:
            rk.rk_debug_set_fused_finish(prev)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        if req == 6:
            check_verify(d, got)


# --------------------------------------------------------------- block tables

def check_tables(lens, block, held, table, ring, state, in_place=True):
    rk = _rk()
    want = ref.block_tables(lens.tolist(), block, held.tolist(), table.numpy(), ring.numpy(), state[:2].tolist())
    dl, dh, dt, dr, ds = (v.to(DEV) for v in (lens, held, table, ring, state))
    if in_place:
        ho, so = rk.block_tables(dl, block, dh, dt, dr, ds)
        assert ho is dh and so is ds
    else:
        ho, so = torch.full_like(dh, -7), torch.full((4,), -7, dtype=torch.int64, device=DEV)
        rk.block_tables(dl, block, dh, dt, dr, ds, held_out=ho, state_out=so)
        assert torch.equal(dh.cpu(), held) and torch.equal(ds.cpu(), state)
    for got, w in zip((ho, dt, dr, so), want):
        assert np.array_equal(got.cpu().numpy(), w)
    return ho.cpu(), dt.cpu(), dr.cpu(), so.cpu()


def pool(seed, req, width, block, spare, turnover=0.5, head=None, size=None):
    g = gen(seed)
    held = torch.randint(0, width + 1, (req,), generator=g)
    lens = (held - 1) * block + torch.randint(1, 2 * block + 1, (req,), generator=g)
    move = torch.rand(req, generator=g)
    lens = torch.where(move < turnover / 2, torch.zeros_like(lens), lens)
    lens = torch.where(move > 1 - turnover / 2, torch.randint(0, width * block + 1, (req,), generator=g), lens).clamp(min=0, max=width * block)
    used = int(held.sum())
    size = used + spare if size is None else size
    ids = torch.randperm(used + spare, generator=g).to(torch.int32)
    table = torch.full((req, width), -1, dtype=torch.int32)
    at = 0
    for b in range(req):
        table[b, :held[b]] = ids[at:at + int(held[b])]
        at += int(held[b])
    head = int(torch.randint(0, 5 * size + 1, (1,), generator=g)) if head is None else head
    ring = torch.full((size,), -1, dtype=torch.int32)
    ring[(head + torch.arange(spare)) % size] = ids[used:]
    return lens.to(torch.int32), block, held.to(torch.int32), table, ring, torch.tensor([head, head + spare, 0, 0])


@pytest.mark.parametrize("req,width,block,spare", [(1, 1, 1, 1), (1, 5, 16, 9), (3, 4, 7, 20), (64, 12, 16, 900), (65, 33, 24, 0),
                                                   (1023, 9, 8, 5000), (1024, 3, 128, 4000), (1025, 17, 16, 100), (5000, 6, 32, 20000),
                                                   (7, 3000, 16, 9000)])
@pytest.mark.parametrize("in_place", [True, False])
def test_tables_sizes(req, width, block, spare, in_place):
    check_tables(*pool(req + width, req, width, block, spare), in_place=in_place)


def test_tables_run_out_and_go_on():
    """Too few free blocks: what is missing is said, and a later call, with
    blocks given back, goes on from there."""
    lens = torch.tensor([64, 64, 64, 64], dtype=torch.int32)
    held = torch.tensor([4, 0, 1, 0], dtype=torch.int32)
    table = torch.full((4, 5), -1, dtype=torch.int32)
    table[0, :4], table[2, 0] = torch.tensor([1, 2, 3, 4]).int(), 5
    ring = torch.tensor([9, 8, 7, 6, 10, 11, 12], dtype=torch.int32)
    h, t, r, s = check_tables(lens, 16, held, table, ring, torch.tensor([12, 17, 0, 0]))
    assert h.tolist() == [4, 4, 2, 0] and s.tolist() == [17, 17, 6, 0]
    lens[0] = 0
    h, t, r, s = check_tables(lens, 16, h, t, r, s)
    assert h.tolist() == [0, 4, 4, 2] and s.tolist() == [21, 21, 2, 0]


def test_tables_ring_too_small_and_bad_values():
    # more blocks come back than the ring has room for
    check_tables(*pool(3, 40, 8, 16, 30, turnover=1.0, size=33))
    # lengths over the table's width, negative ones, held out of range
    lens, block, held, table, ring, state = pool(4, 30, 6, 16, 400)
    lens[::3], lens[1::7] = 16 * 6 + 33, -5
    lens[5] = 2 ** 31 - 1
    held[2], held[9] = -3, 77
    check_tables(lens, block, held, table, ring, state)
    # head far along, and the state of an empty ring
    check_tables(*pool(5, 30, 6, 16, 200, head=2 ** 40 + 17))
    check_tables(*pool(6, 30, 6, 16, 0))
    # nothing to do
    lens, block, held, table, ring, state = pool(7, 20, 6, 16, 50)
    check_tables((held * block).to(torch.int32), block, held, table, ring, state)


def test_tables_leave_the_rest_alone():
    rk = _rk()
    lens, block, held, table, ring, state = pool(8, 50, 9, 16, 500)
    wide = torch.full((60, 13), -77, dtype=torch.int32)
    wide[:50, 2:11] = table
    d = wide.to(DEV)
    want = ref.block_tables(lens.tolist(), block, held.tolist(), table.numpy(), ring.numpy(), state[:2].tolist())
    rk.block_tables(lens.to(DEV), block, held.to(DEV), d[:50, 2:11], ring.to(DEV), state.to(DEV))
    wide[:50, 2:11] = torch.from_numpy(want[1])
    assert torch.equal(d.cpu(), wide)


def test_tables_of_no_requests():
    rk = _rk()
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    ring, state = torch.arange(5, dtype=torch.int32, device=DEV), torch.tensor([3, 7, 9, 9], device=DEV)
    rk.block_tables(z, 16, z, torch.zeros(0, 4, dtype=torch.int32, device=DEV), ring, state)
    assert state.tolist() == [3, 7, 0, 0] and ring.tolist() == [0, 1, 2, 3, 4]


# ------------------------------------------------------------------ slot maps

def check_slots(lens, fresh, block, table, held, n_blocks, capacity, dtype=torch.int64, **kw):
    rk = _rk()
    want = ref.slot_map(lens.tolist(), fresh.tolist(), block, table.numpy(), held.tolist(), n_blocks, capacity)
    got = rk.slot_map(lens.to(DEV), fresh.to(DEV), block, table.to(DEV), held.to(DEV), n_blocks, capacity=capacity,
                      slot_dtype=dtype, **kw)
    assert got[0].dtype == dtype
    for name, g, w in zip(("slots", "positions", "requests", "starts"), got, want):
        assert np.array_equal(g.cpu().numpy(), w), name
    return got


def batch(seed, req, longest, block, new):
    g = gen(seed)
    lens = torch.randint(1, longest + 1, (req,), generator=g)
    fresh = torch.minimum(torch.randint(0, new + 1, (req,), generator=g), lens)
    width = -(-longest // block)
    table = torch.randperm(req * width, generator=g).to(torch.int32).view(req, width)
    held = (lens + block - 1) // block
    return lens.to(torch.int32), fresh.to(torch.int32), block, table, held.to(torch.int32), req * width


@pytest.mark.parametrize("req,longest,block,new", [(1, 1, 1, 1), (1, 5000, 16, 5000), (3, 70, 7, 70), (255, 40, 16, 1), (256, 99, 24, 5),
                                                   (257, 300, 128, 300), (1025, 64, 8, 8), (4096, 12, 4, 3), (4097, 12, 4, 3), (1023, 700, 3, 700),
                                                   (20000, 9, 16, 2)])
@pytest.mark.parametrize("spare,dtype", [(0, torch.int64), (37, torch.int32)])
def test_slots_sizes(req, longest, block, new, spare, dtype):
    b = batch(req, req, longest, block, new)
    check_slots(*b, capacity=int(b[1].sum()) + spare, dtype=dtype)


def test_slots_odd_values():
    lens, fresh, block, table, held, n = batch(2, 90, 200, 16, 200)
    total = int(fresh.sum())
    check_slots(lens, fresh, block, table, held, n, total // 2)        # the batch is longer than the outputs
    check_slots(lens, fresh, block, table, held, n, 0)
    check_slots(lens, torch.zeros_like(fresh), block, table, held, n, 5)
    lens[3], lens[4], lens[5] = 0, -9, 2 ** 31 - 1
    fresh[3], fresh[5], fresh[6], fresh[7] = 4, 50, -2, 2 ** 31 - 1    # more new ones than tokens, fewer than none
    lens[7] = 60
    held[8], held[9], held[10] = 0, 1000, -4
    table[11, 0], table[12, 0], table[13, 0] = -1, n, 2 ** 31 - 1      # ids of no block
    fresh[8:14] = lens[8:14]
    check_slots(lens, fresh, block, table, held, n, total + 500)


def test_slots_saturating_starts():
    """Token counts whose sum passes 2^31."""
    for req in (5, 9000):
        lens = torch.full((req,), 2 ** 31 - 1, dtype=torch.int32)
        fresh = lens.clone()
        fresh[0] = 3
        table = torch.zeros(req, 2, dtype=torch.int32)
        rk = _rk()
        s, p, r, st = rk.slot_map(lens.to(DEV), fresh.to(DEV), 16, table.to(DEV), torch.full((req,), 2, dtype=torch.int32, device=DEV),
                                  1, capacity=10)
        assert st.tolist() == [0, 3] + [2 ** 31 - 1] * (req - 1)
        assert r.tolist() == [0] * 3 + [1] * 7
        assert p.tolist() == [2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2] + list(range(7))
        assert s.tolist() == [-1] * 3 + list(range(7))


def test_slots_pass_32_bits():
    table = torch.tensor([[2 ** 31 - 2, 5]], dtype=torch.int32)
    i = lambda v: torch.tensor([v], dtype=torch.int32)  # noqa: E731
    got = check_slots(i(200), i(200), 128, table, i(2), 2 ** 31 - 1, 200)
    assert int(got[0][0]) == (2 ** 31 - 2) * 128


def test_slots_of_no_requests_and_given_outputs():
    rk = _rk()
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    s, p, r, st = rk.slot_map(z, z, 16, torch.zeros(0, 3, dtype=torch.int32, device=DEV), z, 10, capacity=7)
    assert s.tolist() == [-1] * 7 and p.tolist() == [0] * 7 and r.tolist() == [-1] * 7 and st.tolist() == [0]
    b = batch(5, 9, 50, 16, 9)
    cap = int(b[1].sum()) + 3
    # outputs that start at any element
    bufs = [torch.full((cap + 9,), -5, dtype=t, device=DEV) for t in (torch.int64, torch.int32, torch.int32)]
    starts = torch.full((16,), -5, dtype=torch.int32, device=DEV)
    check_slots(*b, capacity=cap, slots=bufs[0][1:cap + 1], positions=bufs[1][3:cap + 3], requests=bufs[2][2:cap + 2],
                starts=starts[1:11])
    for t, lo in zip(bufs, (1, 3, 2)):
        assert (t[:lo] == -5).all() and (t[lo + cap:] == -5).all()
    assert starts[0] == -5 and (starts[11:] == -5).all()


# ------------------------------------------------------- far addresses

def test_lines_past_2_31_elements():
    """Lines whose places pass 2^31 elements and 2^32 bytes: strides are 64-bit."""
    rk = _rk()
    n, far = 40001, (1 << 31) + 77
    buf = torch.empty(far + n, dtype=BF16, device=DEV)
    x = (torch.randn(2, n, generator=gen(1)) * 3).to(BF16)
    view = buf.as_strided((2, n), (far, 1))
    view.copy_(x)
    check_softmax(rk.softmax(view, out_dtype=F32), x, [1.0] * 2)
    short = buf.as_strided((2, 300), (far, 1))
    check_softmax(rk.softmax(short, out=short), x[:, :300], [1.0] * 2)
    d = drafts(2, 1, 1, n, BF16, ragged=False)
    view.copy_(d["p"])
    on = [d[k].to(DEV) for k in ("q", "drafted", "u", "r")]
    for u in (0.0, 1.0):                            # the near line, the far one
        d["u"].fill_(u)
        on[2].fill_(u)
        check_verify(d, rk.draft_verify(view, *on))
    del view, short
    table = buf.view(torch.int32)[: far // 2 + 9].as_strided((2, 4), (far // 2, 1))
    table.copy_(torch.tensor([[5, 6, -1, -1], [7, -1, -1, -1]]).int())
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    lens, held, ring, state = i(16, 64), i(2, 1), i(1, 2, 3, 4, -1), torch.tensor([0, 4, 0, 0])
    want = ref.block_tables(lens.tolist(), 16, held.tolist(), table.cpu().numpy(), ring.numpy(), [0, 4])
    dev = [t.to(DEV) for t in (held, ring, state)]
    rk.block_tables(lens.to(DEV), 16, dev[0], table, dev[1], dev[2])
    for got, w in zip((dev[0], table, dev[1], dev[2]), want):
        assert np.array_equal(got.cpu().numpy(), w)
    s = rk.slot_map(lens.to(DEV), i(3, 20).to(DEV), 16, table, dev[0], 100, capacity=23)
    w = ref.slot_map(lens.tolist(), [3, 20], 16, want[1], want[0], 100, 23)
    assert all(np.array_equal(g.cpu().numpy(), v) for g, v in zip(s, w))


def test_tables_of_many_entries():
    """A table of over 2^31 entries takes two launches with 64-bit sums."""
    rk = _rk()
    req, width = 2100, 1 << 20
    lens = torch.full((req,), 5, dtype=torch.int32)
    lens[7], lens[9] = width, 0
    held = torch.zeros(req, dtype=torch.int32)
    table = torch.empty(req, width, dtype=torch.int32, device=DEV)
    size = req + width + 10
    ring = torch.arange(size, dtype=torch.int32, device=DEV)
    ho, so = torch.empty_like(held, device=DEV), torch.empty(4, dtype=torch.int64, device=DEV)
    rk.block_tables(lens.to(DEV), 1, held.to(DEV), table, ring, torch.tensor([0, size], device=DEV), held_out=ho, state_out=so)
    taken = min(size, int(lens.sum()))
    assert so.tolist() == [taken, size, int(lens.sum()) - taken, 0]
    off = torch.cat([torch.zeros(1, dtype=torch.int64), lens.long().cumsum(0)])
    got = (torch.minimum(off[1:], torch.tensor(size)) - torch.minimum(off[:-1], torch.tensor(size))).int()
    assert torch.equal(ho.cpu(), got)
    for b in (0, 7, 8, 10, req - 1):
        n = int(got[b])
        assert torch.equal(table[b, :n].cpu(), torch.arange(int(off[b]), int(off[b]) + n, dtype=torch.int32))


# ------------------------------------------------------- streams and a whole step

def test_other_stream_and_injected_failure():
    rk = _rk()
    s = torch.cuda.Stream()
    x = torch.randn(4, 9000, generator=gen(2))
    y = x.to(DEV)
    torch.cuda.synchronize()
    got = rk.softmax(y, stream=s)
    d = drafts(3, 9, 3, 20000, F32)
    on = {k: v.to(DEV) for k, v in d.items() if isinstance(v, torch.Tensor)}
    torch.cuda.synchronize()
    v = rk.draft_verify(on["p"], on["q"], on["drafted"], on["u"], on["r"], starts=on["starts"], max_draft=d["k"], stream=s)
    s.synchronize()
    check_softmax(got, x, [1.0] * 4)
    check_verify(d, v)
    rk.rk_debug_fail_launches(4)
    out = torch.full_like(y, 5.0)
    b = batch(5, 9, 50, 16, 9)
    p = pool(7, 20, 6, 16, 50)
    tables = [t.to(DEV) if isinstance(t, torch.Tensor) else t for t in p]
    try:
        with pytest.raises(rk.RkError, match="HIP"):
            rk.softmax(y, out=out)
        with pytest.raises(rk.RkError, match="HIP"):
            run_verify(d)
        with pytest.raises(rk.RkError, match="HIP"):
            rk.block_tables(*tables)
        with pytest.raises(rk.RkError, match="HIP"):
            rk.slot_map(*[t.to(DEV) if isinstance(t, torch.Tensor) else t for t in b], capacity=9)
    finally:
        rk.rk_debug_fail_launches(0)
    assert (out == 5.0).all()
    for t, was in zip(tables, p):
        assert not isinstance(t, torch.Tensor) or torch.equal(t.cpu(), was)
    with pytest.raises(rk.RkError, match="invalid"):
        rk.softmax(torch.zeros(2, 200000, device=DEV), workspace=torch.empty(8, dtype=torch.uint8, device=DEV))


def test_tensor_refusals():
    """What the Python calls refuse before the library sees it."""
    rk = _rk()
    x = torch.zeros(2, 8, device=DEV)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, device=DEV)  # noqa: E731
    f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731

    def refused(match, call, *args, **kw):
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)
    refused("two dims", rk.softmax, x.t())
    refused("two dims", rk.softmax, x[0])
    refused("cannot be", rk.softmax, x.double())
    refused("cannot be", rk.softmax, x, out=torch.zeros_like(x).double())
    refused("shape", rk.softmax, x, out=f(2, 9))
    refused("shape", rk.softmax, x, out=f(2, 8), out_dtype=BF16)
    refused("two dims", rk.softmax, x, out=f(8, 2).t())
    refused("temperature", rk.softmax, x, temperature=f(3))
    refused("temperature is not on a GPU", rk.softmax, x, temperature=torch.zeros(2))
    refused("workspace is not on a GPU", rk.softmax, x, workspace=torch.zeros(9))
    v = rk.draft_verify
    refused("every draft", v, f(5, 8), None, i32(4), f(4), f(2), max_draft=2)
    refused("max_draft", v, f(6, 8), None, i32(4), f(4), f(2), starts=i32(3))
    refused("takes p's dtype", v, f(6, 8), f(4, 7), i32(4), f(4), f(2))
    refused("takes p's dtype", v, f(6, 8), f(4, 8).half(), i32(4), f(4), f(2))
    refused("drafted cannot be", v, f(6, 8), None, f(4), f(4), f(2))
    refused("u takes", v, f(6, 8), None, i32(4), f(3), f(2))
    refused("r takes", v, f(6, 8), None, i32(4), f(4), f(4)[::2])
    refused("starts takes", v, f(6, 8), None, i32(4), f(4), f(2), starts=i64(3), max_draft=2)
    refused("tokens takes", v, f(6, 8), None, i32(4), f(4), f(2), tokens=i64(2, 3))
    refused("accepted takes", v, f(6, 8), None, i32(4), f(4), f(2), accepted=i32(3))
    t = rk.block_tables
    refused("table", t, i32(3), 16, i32(3), i32(2, 4), i32(9), i64(4))
    refused("table", t, i32(3), 16, i32(3), i64(3, 4), i32(9), i64(4))
    refused("state_out", t, i32(3), 16, i32(3), i32(3, 4), i32(9), i64(2))
    refused("state takes", t, i32(3), 16, i32(3), i32(3, 4), i32(9), i64(1), state_out=i64(4))
    with pytest.raises(TypeError, match="held takes a tensor"):
        t(i32(3), 16, [1, 2, 3], i32(3, 4), i32(9), i64(4))
    refused("held takes", t, i32(3), 16, i32(4), i32(3, 4), i32(9), i64(4))
    refused("ring takes", t, i32(3), 16, i32(3), i32(3, 4), i64(9), i64(4))
    m = rk.slot_map
    refused("capacity", m, i32(3), i32(3), 16, i32(3, 4), i32(3), 10)
    refused("slots takes", m, i32(3), i32(3), 16, i32(3, 4), i32(3), 10, capacity=5, slots=i64(4))
    refused("slots takes", m, i32(3), i32(3), 16, i32(3, 4), i32(3), 10, slots=i64(5), slot_dtype=torch.int32)
    refused("slots cannot be", m, i32(3), i32(3), 16, i32(3, 4), i32(3), 10, slots=f(5))
    refused("positions takes", m, i32(3), i32(3), 16, i32(3, 4), i32(3), 10, capacity=5, positions=i32(4))
    refused("starts takes", m, i32(3), i32(3), 16, i32(3, 4), i32(3), 10, capacity=5, starts=i32(3))
    refused("fresh takes", m, i32(3), i32(6)[::2], 16, i32(3, 4), i32(3), 10, capacity=5)
    with pytest.raises(rk.RkError, match="rk_slot_map"):
        m(i32(3), i32(3), 0, i32(3, 4), i32(3), 10, capacity=5)


class Step:
    """A serving step with drafts: room for the drafts, their slots, the
    target's probabilities, the verification, and the tables cut back to what
    was kept.  All of it on the device, in buffers of its own."""

    def __init__(self, req=6, k=3, n=9001, block=4, width=40, seed=0):
        g = gen(seed)
        self.req, self.k, self.n, self.block, self.width = req, k, n, block, width
        size = req * width
        self.lens = torch.randint(1, 30, (req,), generator=g).int().to(DEV)
        self.held = torch.zeros(req, dtype=torch.int32, device=DEV)
        self.table = torch.full((req, width), -1, dtype=torch.int32, device=DEV)
        self.ring = torch.randperm(size, generator=g).int().to(DEV)
        self.state = torch.tensor([0, size, 0, 0], device=DEV)
        self.size = size
        self.logits = torch.zeros(req * (k + 1), n, dtype=BF16, device=DEV)
        self.q = torch.zeros(req * k, n, device=DEV)
        self.temp = torch.ones(req * (k + 1), device=DEV)
        self.drafted = torch.zeros(req * k, dtype=torch.int64, device=DEV)
        self.u = torch.zeros(req * k, device=DEV)
        self.r = torch.zeros(req, device=DEV)
        self.fresh = torch.full((req,), k + 1, dtype=torch.int32, device=DEV)
        rk = _rk()
        self.p = torch.zeros(req * (k + 1), n, device=DEV)
        self.tokens = torch.zeros(req, k + 1, dtype=torch.int64, device=DEV)
        self.accepted = torch.zeros(req, dtype=torch.int32, device=DEV)
        cap = req * (k + 1) + 5
        self.maps = dict(slots=torch.zeros(cap, dtype=torch.int64, device=DEV), positions=torch.zeros(cap, dtype=torch.int32, device=DEV),
                         requests=torch.zeros(cap, dtype=torch.int32, device=DEV), starts=torch.zeros(req + 1, dtype=torch.int32, device=DEV))
        ws = lambda b: torch.empty(max(b, 256), dtype=torch.uint8, device=DEV)  # noqa: E731
        self.ws = [ws(rk.rk_softmax_workspace_size(rk.RK_BF16, rk.RK_F32, n, req * (k + 1))),
                   ws(rk.rk_draft_verify_workspace_size(rk.RK_F32, n, req)), ws(rk.rk_block_tables_workspace_size(req))]

    def inputs(self, seed):
        g = gen(seed)
        z = torch.randn(self.logits.shape, generator=g) * 2
        z.scatter_(1, torch.randint(0, self.n, (z.shape[0], 1), generator=g), 14.0)
        self.logits.copy_(z)
        zq = z.view(self.req, self.k + 1, self.n)[:, :self.k].reshape(-1, self.n) + 0.5 * torch.randn(self.q.shape, generator=g)
        q = torch.softmax(zq, 1)
        self.q.copy_(q)
        self.drafted.copy_(torch.multinomial(q, 1, generator=g).view(-1))
        self.u.copy_(torch.rand(self.u.shape, generator=g))
        self.r.copy_(torch.rand(self.r.shape, generator=g))
        t = torch.rand(self.temp.shape, generator=g) + 0.5
        t[: self.k + 1] = 0.0                      # one request decodes greedily
        self.temp.copy_(t)

    def run(self):
        rk = _rk()
        self.lens.add_(self.k + 1)
        rk.block_tables(self.lens, self.block, self.held, self.table, self.ring, self.state, workspace=self.ws[2])
        rk.slot_map(self.lens, self.fresh, self.block, self.table, self.held, self.size, **self.maps)
        rk.softmax(self.logits, temperature=self.temp, out=self.p, workspace=self.ws[0])
        rk.draft_verify(self.p, self.q, self.drafted, self.u, self.r, tokens=self.tokens, accepted=self.accepted,
                        workspace=self.ws[1])
        self.lens.sub_(self.k - self.accepted)     # drafts turned down are forgotten
        rk.block_tables(self.lens, self.block, self.held, self.table, self.ring, self.state, workspace=self.ws[2])

    def cpu(self):
        return {k: v.cpu().clone() for k, v in vars(self).items() if isinstance(v, torch.Tensor)}

    def check(self, was):
        """The buffers after run(), from those before it."""
        now = self.cpu()
        n, k = self.req * (self.k + 1), self.k
        lens = was["lens"].numpy() + k + 1
        held, table, ring, state = ref.block_tables(lens, self.block, was["held"].tolist(), was["table"].numpy(),
                                                    was["ring"].numpy(), was["state"].tolist())
        want = ref.slot_map(lens, [k + 1] * self.req, self.block, table, held, self.size, n + 5)
        for name, w in zip(("slots", "positions", "requests", "starts"), want):
            assert np.array_equal(self.maps[name].cpu().numpy(), w), name
        check_softmax(now["p"], was["logits"], was["temp"].tolist())
        tokens, kept = ref.draft_verify(np64(now["p"]), np64(was["q"]), was["drafted"].tolist(), np64(was["u"]), np64(was["r"]),
                                        [i * k for i in range(self.req + 1)], k)
        assert np.array_equal(now["tokens"].numpy(), tokens) and np.array_equal(now["accepted"].numpy(), kept)
        lens = lens - k + kept
        assert np.array_equal(now["lens"].numpy(), lens)
        held, table, ring, state = ref.block_tables(lens, self.block, held.tolist(), table, ring, state.tolist())
        for name, w in (("held", held), ("table", table), ("ring", ring), ("state", state)):
            assert np.array_equal(now[name].numpy(), w), name
        # every block is in one place: a request's table or the ring
        own = [now["table"][b, :held[b]].tolist() for b in range(self.req)]
        free = [now["ring"][i % self.size].item() for i in range(int(state[0]), int(state[1]))]
        assert sorted(sum(own, free)) == list(range(self.size))


def test_a_serving_step():
    s = Step()
    for i in range(4):
        s.inputs(50 + i)
        was = s.cpu()
        s.run()
        torch.cuda.synchronize()
        s.check(was)


def test_captured_steps():
    """Two graphs captured on one stream and replayed on two at once, each with
    buffers of its own, with eager steps and synchronisations between."""
    steps = [Step(seed=1), Step(req=9, k=2, n=20011, block=16, width=9, seed=2)]
    for s in steps:
        s.inputs(1)
        s.run()                                    # modules load outside the capture
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.run()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    eager = Step(seed=3)
    for rep in range(4):
        was = []
        for s in steps:
            s.inputs(100 + rep)
            was.append(s.cpu())
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip(steps, was):
            s.check(w)
        eager.inputs(rep)
        w = eager.cpu()
        eager.run()
        torch.cuda.synchronize()
        eager.check(w)


def test_two_threads_on_two_streams():
    """Steps of two host threads at once, each on a stream of its own: calls of
    different streams share no counters, and no workspace here."""
    import threading
    steps = [Step(req=40, k=3, n=20011, block=16, width=30, seed=4), Step(req=33, k=5, n=33333, block=8, width=30, seed=5)]
    failed = []

    def work(s, seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(6):
                    s.inputs(seed + i)
                    torch.cuda.current_stream().synchronize()
                    was = s.cpu()
                    first = None
                    for _ in range(20):                # the same verification again and again, beside the other thread's
                        t, a = _rk().draft_verify(s.p, s.q, s.drafted, s.u, s.r, workspace=s.ws[1])
                        first = (t, a) if first is None else first
                        if not (torch.equal(t, first[0]) and torch.equal(a, first[1])):
                            failed.append("results differ")
                    s.run()
                    torch.cuda.current_stream().synchronize()
                    s.check(was)
        except BaseException as e:                     # noqa: BLE001  (shown by the test's own thread)
            failed.append(repr(e))
    threads = [threading.Thread(target=work, args=(s, 100 * i)) for i, s in enumerate(steps)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
