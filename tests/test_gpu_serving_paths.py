"""GPU tests of the serving operators' launch paths: each path that a rule on
sizes picks is run and compared with the plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.test_gpu_serving import (BF16, DEV, F16, F32, INF, _rk, check_softmax, check_tables, drafts, gen, np64, pool,
                                    run_verify)

pytestmark = pytest.mark.gpu


def spread_drafts(seed, req, k, n, empty, dt=F32, q=True, m=150):
    """Drafts over m tokens for the plain form, and the same over a vocabulary
    of n, the m tokens spread over it in order (the others weigh nothing and
    are never drawn).  empty: two requests in three have a draft that leaves
    nothing of the target."""
    d = drafts(seed, req, k, m, dt, q=q)
    starts = d["starts"].tolist()
    if empty:
        for b in range(req):
            lo, hi = starts[b], starts[b + 1]
            if b % 3 == 2 or lo == hi:
                continue
            if q:                                  # the target's own line, or twice that
                d["q"][lo:hi] = d["p"][lo + b:hi + b] * (1 if b % 3 else 2)
                d["u"][lo:hi] = 1.0
            else:                                  # one token, and under the 1 that it loses
                d["p"][lo + b] = 0.0
                d["p"][lo + b, d["drafted"][lo]] = 0.5
                d["u"][lo] = 0.75
    at = torch.randperm(n - 2, generator=gen(seed + 1))[:m - 2] + 1
    at = torch.cat([at, torch.tensor([0, n - 1])]).sort().values
    big = dict(d, drafted=at[d["drafted"].long()].to(d["drafted"].dtype))
    for name in ("p", "q"):
        if d[name] is not None:
            big[name] = torch.zeros(d[name].shape[0], n, dtype=dt, device=DEV)
            big[name][:, at.to(DEV)] = d[name].to(DEV)
    return d, big, at


def check_spread(d, at, got):
    t, a = ref.draft_verify(np64(d["p"]), None if d["q"] is None else np64(d["q"]), d["drafted"].tolist(), np64(d["u"]),
                            np64(d["r"]), d["starts"].tolist(), d["k"])
    t = np.where(t < 0, -1, at.numpy()[np.maximum(t, 0)])
    assert np.array_equal(got[1].cpu().numpy(), a)
    assert np.array_equal(got[0].cpu().numpy(), t)


@pytest.mark.parametrize("req,n", [(250, 9000), (64, 40001), (600, 9000), (4200, 8200), (1500, 18001)])
@pytest.mark.parametrize("dt,q", [(F32, True), (F32, False), (BF16, True)])
def test_verify_draws_from_the_target_where_the_draft_leaves_nothing(req, n, dt, q):
    """Many requests whose residual is empty: their sums are taken a second
    time, by the request's last block, by a second launch's, by its only one."""
    rk = _rk()
    d, big, at = spread_drafts(req + n, req, 2, n, True, dt=dt, q=q)
    check_spread(d, at, run_verify(big))
    prev = rk.rk_debug_set_fused_finish(0)
    try:
        check_spread(d, at, run_verify(big))
    finally:
        rk.rk_debug_set_fused_finish(prev)


def verify_paths(req, n):
    """(blocks a request, tiles, launches with the fused finish and without)."""
    rk = _rk()
    plan = rk.rk_plan_draft_verify(rk.RK_F32, n, req)
    prev = rk.rk_debug_set_fused_finish(0)
    try:
        apart = rk.rk_plan_draft_verify(rk.RK_F32, n, req).launches
    finally:
        rk.rk_debug_set_fused_finish(prev)
    return plan.split, -(-n // plan.tile_outputs), plan.launches, apart


@pytest.mark.parametrize("req,n,paths", [
    (64, 9000, (2, 5, 1, 2)), (250, 9000, (2, 5, 1, 2)), (20, 40001, (5, 20, 1, 2)),    # the last block finishes, or a second launch
    (1, 100000, (13, 49, 1, 2)),
    (600, 9000, (2, 5, 2, 2)), (256, 70001, (9, 35, 2, 2)),                             # a second launch by itself
    (4200, 8200, (1, 5, 1, 1)),                                                         # one block, a wave with two tiles
    (1500, 18001, (2, 9, 2, 2)), (900, 33000, (4, 17, 2, 2)),                           # several blocks, the same
])
def test_verify_launch_paths(req, n, paths):
    rk = _rk()
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert verify_paths(req, n) == paths
    d, big, at = spread_drafts(req * 7 + n, req, 2, n, False, m=80 if req > 1000 else 400)
    check_spread(d, at, run_verify(big))
    prev = rk.rk_debug_set_fused_finish(0)
    try:
        check_spread(d, at, run_verify(big))
    finally:
        rk.rk_debug_set_fused_finish(prev)


# ------------------------------------------------------------------ slot maps

def slots_of(lens, fresh, block, table, held, n_blocks, capacity):
    """The plain slot map of valid inputs, all tokens at once."""
    lens, fresh, table, held = (t.numpy().astype(np.int64) for t in (lens, fresh, table, held))
    starts = np.concatenate([[0], fresh.cumsum()])
    total = min(int(starts[-1]), capacity)
    who = np.repeat(np.arange(len(lens)), fresh)[:total]
    pos = (lens - fresh)[who] + np.arange(total) - starts[who]
    j = pos // block
    entry = table[who, np.minimum(j, table.shape[1] - 1)]
    there = (j < held[who]) & (j < table.shape[1]) & (entry >= 0) & (entry < n_blocks)
    slots, positions, requests = (np.full(capacity, v, np.int64) for v in (-1, 0, -1))
    slots[:total], positions[:total], requests[:total] = np.where(there, entry * block + pos % block, -1), pos, who
    return slots, positions, requests, starts


def prompts(seed, req, tokens, block, spare):
    """A batch of at least `tokens` new tokens, every 50th request without any
    and some table entries that name no block."""
    g = gen(seed)
    mean = tokens // req
    fresh = torch.randint(mean // 2, 2 * mean + 2, (req,), generator=g)
    fresh[::50] = 0
    lens = fresh + torch.randint(0, 70, (req,), generator=g)
    width = -(-int(lens.max()) // block)
    table = torch.randint(-1, req * width, (req, width), generator=g)
    held = (lens + block - 1) // block - (torch.rand(req, generator=g) < 0.1).long()
    n_blocks = req * width - 5
    cap = int(fresh.sum()) + spare
    assert cap > tokens
    return lens.int(), fresh.int(), block, table.int(), held.clamp(min=0).int(), n_blocks, cap


@pytest.mark.parametrize("req", [70, 4096, 4097, 9001])
@pytest.mark.parametrize("dtype,tokens", [(torch.int64, 2_200_000), (torch.int32, 2_900_000)])
def test_slots_past_the_caches(req, dtype, tokens):
    """Outputs of more than 32 MB, at any element, behind which nothing is
    written, ended inside a vector."""
    rk = _rk()
    lens, fresh, block, table, held, n_blocks, cap = prompts(req, req, tokens, 16, 1001)
    cap += 1 - cap % 2
    size = torch.empty(0, dtype=dtype).element_size()
    assert cap * (size + 8) > 32 << 20
    bufs = [torch.full((cap + 9,), -5, dtype=t, device=DEV) for t in (dtype, torch.int32, torch.int32)]
    at = (1, 3, 2)
    slots, positions, requests = (b[i:i + cap] for b, i in zip(bufs, at))
    got = rk.slot_map(lens.to(DEV), fresh.to(DEV), block, table.to(DEV), held.to(DEV), n_blocks, slots=slots,
                      positions=positions, requests=requests)
    for name, g, w in zip(("slots", "positions", "requests", "starts"), got,
                          slots_of(lens, fresh, block, table, held, n_blocks, cap)):
        assert np.array_equal(g.cpu().numpy(), w), name
    for b, i in zip(bufs, at):
        assert (b[:i] == -5).all() and (b[i + cap:] == -5).all()


@pytest.mark.parametrize("req,tokens,dtype", [(9, 300, torch.int64), (9, 300, torch.int32), (5000, 20000, torch.int64),
                                              (300, 4_300_000, torch.int64), (4500, 8_500_000, torch.int32)])
@pytest.mark.parametrize("given", ["", "positions", "requests"])
def test_slots_without_positions_or_requests(req, tokens, dtype, given):
    """The C call takes NULL for either."""
    rk = _rk()
    lens, fresh, block, table, held, n_blocks, cap = prompts(req, req, tokens, 16, 5)
    on = [t.to(DEV) for t in (lens, fresh, table, held)]
    slots = torch.full((cap + 1,), -5, dtype=dtype, device=DEV)
    more = {k: torch.full((cap + 1,), -5, dtype=torch.int32, device=DEV) for k in ("positions", "requests")}
    starts = torch.empty(req + 1, dtype=torch.int32, device=DEV)
    rc = rk.rk_slot_map(on[0].data_ptr(), on[1].data_ptr(), req, block, on[2].data_ptr(), table.shape[1], table.shape[1],
                        on[3].data_ptr(), n_blocks, rk.RK_I64 if dtype == torch.int64 else rk.RK_I32, cap, slots.data_ptr(),
                        *(more[k].data_ptr() if k == given else None for k in ("positions", "requests")), starts.data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    assert rc == rk.RK_OK
    want = dict(zip(("slots", "positions", "requests", "starts"), slots_of(lens, fresh, block, table, held, n_blocks, cap)))
    assert np.array_equal(slots[:cap].cpu().numpy(), want["slots"]) and slots[cap] == -5
    assert np.array_equal(starts.cpu().numpy(), want["starts"])
    for k, t in more.items():
        assert np.array_equal(t[:cap].cpu().numpy(), want[k]) if k == given else (t == -5).all()
        assert t[cap] == -5


# --------------------------------------------------------------- block tables

@pytest.mark.parametrize("in_place", [True, False])
def test_tables_odd_values_in_either_form(in_place):
    """What the one-launch form (outputs apart) has code of its own for."""
    # more blocks come back than the ring has room for
    check_tables(*pool(3, 40, 8, 16, 30, turnover=1.0, size=33), in_place=in_place)
    check_tables(*pool(13, 700, 8, 16, 0, turnover=1.0, size=1), in_place=in_place)
    # too few free ones, so that blocks given back are taken in the same call
    check_tables(*pool(14, 900, 21, 16, 7, turnover=0.8), in_place=in_place)
    check_tables(*pool(15, 4096, 5, 8, 100, turnover=0.9), in_place=in_place)
    # lengths over the table's width, negative ones, held out of range
    for seed, req in ((4, 30), (16, 1500)):
        lens, block, held, table, ring, state = pool(seed, req, 6, 16, 400)
        lens[::3], lens[1::7] = 16 * 6 + 33, -5
        lens[5] = 2 ** 31 - 1
        held[2], held[9] = -3, 77
        check_tables(lens, block, held, table, ring, state, in_place=in_place)
    lens, block, held, table, ring, state = pool(17, 30, 6, 1, 400)
    lens[:] = 2 ** 31 - 1                          # the blocks beyond the tables' width pass 2^32
    check_tables(lens, block, held, table, ring, state, in_place=in_place)
    # head far along, and the state of an empty ring
    for head in (2 ** 32 - 3, 2 ** 40 + 17):
        check_tables(*pool(5, 30, 6, 16, 200, head=head), in_place=in_place)
    check_tables(*pool(6, 30, 6, 16, 0), in_place=in_place)
    # nothing to do
    lens, block, held, table, ring, state = pool(7, 20, 6, 16, 50)
    check_tables((held * block).to(torch.int32), block, held, table, ring, state, in_place=in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("req", [50, 4097])
def test_tables_inside_wider_rows_in_either_form(in_place, req):
    rk = _rk()
    lens, block, held, table, ring, state = pool(8, req, 9, 16, 10 * req)
    wide = torch.full((req + 10, 13), -77, dtype=torch.int32)
    wide[:req, 2:11] = table
    d, dh, dr, ds = wide.to(DEV), held.to(DEV), ring.to(DEV), state.to(DEV)
    want = ref.block_tables(lens.tolist(), block, held.tolist(), table.numpy(), ring.numpy(), state[:2].tolist())
    apart = {} if in_place else dict(held_out=torch.empty_like(dh), state_out=torch.empty_like(ds))
    after, now = rk.block_tables(lens.to(DEV), block, dh, d[:req, 2:11], dr, ds, **apart)
    wide[:req, 2:11] = torch.from_numpy(want[1])
    assert torch.equal(d.cpu(), wide)
    for got, w in zip((after, dr, now), (want[0], want[2], want[3])):
        assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("in_place", [True, False])
def test_tables_run_out_and_go_on_in_either_form(in_place):
    lens = torch.tensor([64, 64, 64, 64], dtype=torch.int32)
    held = torch.tensor([4, 0, 1, 0], dtype=torch.int32)
    table = torch.full((4, 5), -1, dtype=torch.int32)
    table[0, :4], table[2, 0] = torch.tensor([1, 2, 3, 4]).int(), 5
    ring = torch.tensor([9, 8, 7, 6, 10, 11, 12], dtype=torch.int32)
    h, t, r, s = check_tables(lens, 16, held, table, ring, torch.tensor([12, 17, 0, 0]), in_place=in_place)
    assert h.tolist() == [4, 4, 2, 0] and s.tolist() == [17, 17, 6, 0]
    lens[0] = 0
    h, t, r, s = check_tables(lens, 16, h, t, r, s, in_place=in_place)
    assert h.tolist() == [0, 4, 4, 2] and s.tolist() == [21, 21, 2, 0]


# -------------------------------------------------------------------- softmax

@pytest.mark.parametrize("n,lines", [(131071, 68), (40003, 215), (2100001, 5)])
@pytest.mark.parametrize("din,dout,in_place", [(F32, F32, False), (BF16, F32, False), (F16, F16, False), (F32, BF16, False),
                                               (F32, F32, True), (BF16, BF16, True)])
def test_softmax_past_the_caches(n, lines, din, dout, in_place):
    """Outputs of more than 32 MB, lines at any element, between which nothing
    is written; masked and greedy lines among them."""
    rk = _rk()
    lines *= 4 // torch.empty(0, dtype=dout).element_size()
    assert lines * n * torch.empty(0, dtype=dout).element_size() > 32 << 20
    x = torch.randn(lines, n, generator=gen(n)).mul_(3).to(din)
    x[1, : n - 5] = -INF
    x[2, ::2] = torch.finfo(din).min
    x[lines - 1] = -INF
    t = [(1.0, 0.7, 2.0, 0.0)[i % 4] for i in range(lines)]
    buf = torch.full((lines * (n + 3) + 1,), 7.0, dtype=din, device=DEV)
    view = buf.as_strided((lines, n), (n + 3, 1), 1)
    view.copy_(x)
    if in_place:
        obuf, out = buf, view
    else:
        obuf = torch.full((lines * (n + 1) + 3,), 7.0, dtype=dout, device=DEV)
        out = obuf.as_strided((lines, n), (n + 1, 1), 3)
    assert rk.softmax(view, temperature=torch.tensor(t).to(DEV), out=out) is out
    for i in range(0, lines, 40):                  # (the plain form's float64 lines, a few at a time)
        check_softmax(out[i:i + 40], x[i:i + 40], t[i:i + 40])
    touched = torch.zeros_like(obuf, dtype=torch.bool)
    touched.as_strided(out.shape, out.stride(), out.storage_offset()).fill_(True)
    assert (obuf[~touched] == 7.0).all()


@pytest.mark.parametrize("n", [5, 200, 1000, 9001, 40000, 1048577])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_softmax_nan_temperature(n, dt):
    """A NaN temperature makes any line NaN, one whose mask leaves nothing too."""
    x = torch.full((4, n), -INF, dtype=dt)
    x[1, n // 2] = 1.0
    x[2] = torch.randn(n, generator=gen(n)).to(dt)
    t = [float("nan")] * 3 + [1.0]
    check_softmax(_rk().softmax(x.to(DEV), temperature=torch.tensor(t).to(DEV)), x, t)


def test_softmax_refuses_to_drop_gradients():
    rk = _rk()
    x = torch.zeros(2, 8, device=DEV).requires_grad_()
    t = torch.ones(2, device=DEV)
    y = torch.zeros(2, 8, device=DEV)
    for call in (lambda: rk.softmax(x), lambda: rk.softmax(x * 2, temperature=t), lambda: rk.softmax(y, out=x),
                 lambda: rk.softmax(y, temperature=t.clone().requires_grad_())):
        with pytest.raises(ValueError, match="no gradient"):
            call()
        with torch.no_grad():
            assert torch.equal(call(), torch.full_like(y, 0.125))
    assert torch.equal(rk.softmax(x.detach()), torch.full_like(y, 0.125))
    with torch.inference_mode():
        assert torch.equal(rk.softmax(x), torch.full_like(y, 0.125))


def test_tensors_of_no_dims_are_refused():
    rk = _rk()
    x, i, f = torch.zeros((), device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV)
    with pytest.raises(ValueError, match="two dims"):
        rk.softmax(x)
    with pytest.raises(ValueError, match="two dims"):
        rk.draft_verify(x, None, i, f[:0], f)


# ---------------------------------------------------------------- workspaces

def guarded(n):
    """A workspace of n bytes and the buffer of twos around it."""
    buf = torch.full((n + 1024,), 2, dtype=torch.uint8, device=DEV)
    return buf[512:512 + n], lambda: bool((buf[:512] == 2).all()) and bool((buf[512 + n:] == 2).all())


def test_workspaces_are_as_large_as_said():
    """Sizes whose bytes fill the multiple of 256 that is asked for."""
    rk = _rk()
    for req in (20, 148, 1300):                    # 32 + 24 req: 512, 3584, 31232
        assert (32 + 24 * req) % 256 == 0
        ws, whole = guarded(rk.rk_block_tables_workspace_size(req))
        lens, block, held, table, ring, state = (t.to(DEV) if isinstance(t, torch.Tensor) else t for t in pool(req, req, 9, 16, 5 * req))
        want = ref.block_tables(lens.tolist(), block, held.tolist(), table.cpu().numpy(), ring.cpu().numpy(), state[:2].tolist())
        rk.block_tables(lens, block, held, table, ring, state, workspace=ws)
        for got, w in zip((held, table, ring, state), want):
            assert np.array_equal(got.cpu().numpy(), w)
        assert whole()
    for req, n in ((16, 9000), (600, 9000), (4200, 8200), (64, 40001)):
        d, big, at = spread_drafts(n + req, req, 1, n, True, m=60)
        ws, whole = guarded(rk.rk_draft_verify_workspace_size(rk.RK_F32, n, req))
        check_spread(d, at, run_verify(big, workspace=ws))
        assert whole()
    for lines, n in ((64, 64 * 2048), (64, 40000), (2, 513 * 2048), (3, 1048577)):
        x = torch.randn(lines, n, generator=gen(n))
        ws, whole = guarded(rk.rk_softmax_workspace_size(rk.RK_F32, rk.RK_F32, n, lines))
        check_softmax(rk.softmax(x.to(DEV), workspace=ws), x, [1.0] * lines)
        assert whole()
