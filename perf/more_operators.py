"""Cases and plain forms of operators for beams and recurrent layers: beam
selection, forking, compacting and copying blocks of a paged cache, and a gated
linear recurrence in both directions.

`listed()` and `draw()` give cases, `prepare()` their inputs, `run()` one pass
(the plain form below, or with `own` the library's calls), `work()` the bytes
and operations a pass cannot do without, `exact()` the results in 64 bits.

Plain forms:
  recur    a = gate, exp(gate) or sigmoid(gate); w = 1 or 1 - a; h_t = a_t h_(t-1) + w_t x_t, every
           sequence from its own state (of line sources[b] where given)
  back     its gradient: g_t = dout_t + a_(t+1) g_(t+1); dx_t = w_t g_t; with da_t = g_t h_(t-1), or
           g_t (h_(t-1) - x_t) where w = 1 - a, dgate_t = da_t * (1, a or a (1 - a)); dstate = a_1 g_1
  beam     s = score + x - log sum exp(x) over a line; a request's `count` largest, ties to the lowest
           (line, token); an ended line has one candidate, the end token at its score as it is
  fork     row r of a block table becomes what row parents[r] was; its first child keeps a parent's
           last, partly filled block, the others take a fresh one from the ring of free blocks (a pair
           to copy); blocks no row names any more go to the ring's end
  compact  blocks in use move to the lowest ids: the k-th used id beyond their number to the k-th
           unused one below it
  copy     block dst of every cache becomes what block src is, for every pair
"""
import numpy as np
import torch

own = False

F32, BF16, F16 = "f32", "bf16", "f16"
DT = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
SIZE = {F32: 4, BF16: 2, F16: 2}


def listed():
    return [
        # one token for each of 64 lines (16 requests of four beams), states taken from the beams' parents: latency
        dict(name="recur_step_64x2048_bf16", op="recur", batch=64, tokens=1, channels=2048, ragged=False, dtype=BF16, gate=BF16, kind="sigmoid", blend=True, state=True, sources=True),
        # one long document, read from its start
        dict(name="recur_long_65536x2048_bf16", op="recur", batch=1, tokens=65536, channels=2048, ragged=False, dtype=BF16, gate=BF16, kind="sigmoid", blend=True, state=False, sources=False),
        # a training batch
        dict(name="back_8x4096x2048_bf16", op="back", batch=8, tokens=4096, channels=2048, ragged=False, dtype=BF16, gate=BF16, kind="sigmoid", blend=True, state=False),
        # documents of odd lengths packed into one line of tokens, odd channels, decays in float32 given by their logarithm
        dict(name="back_packed_20011x1001_f32", op="back", batch=37, tokens=20011, channels=1001, ragged=True, dtype=F32, gate=F32, kind="log", blend=False, state=True),
        # one request's four beams, twice as many kept so that some may end: latency
        dict(name="beam_1x4x32768_f32", op="beam", req=1, beams=4, n=32768, pad=0, dtype=F32, count=8, masked=0.0, ended=0.0, ids="i64"),
        # a serving batch of eight beams, logits as the model's last product leaves them
        dict(name="beam_64x8x131072_bf16", op="beam", req=64, beams=8, n=131072, pad=0, dtype=BF16, count=16, masked=0.0, ended=0.1, ids="i64"),
        # a decode step of 64 requests of four beams
        dict(name="fork_decode_64x4", op="fork", req=64, beams=4, block=16, longest=4096, ended=0.05),
        # many beams over long contexts
        dict(name="fork_long_256x8", op="fork", req=256, beams=8, block=16, longest=65536, ended=0.02),
        # a small pool
        dict(name="compact_64x4", op="compact", req=64, beams=4, block=16, longest=4096, spare=1.5),
        # a whole card's pool, two thirds of it free
        dict(name="compact_1024x4", op="compact", req=1024, beams=4, block=16, longest=16384, spare=3.0),
        # the last blocks of one request's new beams in eight layers: latency
        dict(name="copy_4x8_32k", op="copy", blocks=64, rows=4, pairs=3, caches=8, bytes=32768),
        # a batch's new beams in 32 caches
        dict(name="copy_512x32_32k", op="copy", blocks=1024, rows=512, pairs=256, caches=32, bytes=32768),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["recur", "recur", "back", "back", "beam", "beam", "fork", "compact", "copy"])
    if op in ("recur", "back"):
        dtype = rng.choice([F32, BF16, F16])
        channels = _log(rng, 16, 8192)
        most = (1 << 26) // (channels * (2 if op == "back" else 1))
        ragged = rng.random() < 0.5
        step = op == "recur" and rng.random() < 0.3
        tokens = 1 if step else _log(rng, 2, min(65536, most))
        batch = _log(rng, 1, max(1, min(512, tokens if ragged else most // tokens)))
        c = dict(op=op, batch=batch, tokens=tokens, channels=channels, ragged=ragged and not step, dtype=dtype,
                 gate=rng.choice([dtype, dtype, F32]), kind=rng.choice(["value", "log", "sigmoid"]), blend=rng.random() < 0.6,
                 state=step or rng.random() < 0.5)
        if op == "recur":
            c["sources"] = c["state"] and rng.random() < 0.5
        return c
    if op == "beam":
        n, beams = _log(rng, 500, 200000), _log(rng, 1, 16)
        return dict(op=op, req=_log(rng, 1, max(1, min(256, (1 << 26) // (n * beams)))), beams=beams, n=n, pad=rng.choice([0, 0, 1, 24]),
                    dtype=rng.choice([F32, BF16, F16]), count=rng.choice([beams, 2 * beams, 2 * beams + 1]),
                    masked=rng.choice([0.0, 0.0, 0.5, 0.97]), ended=rng.choice([0.0, 0.3]), ids=rng.choice(["i32", "i64"]))
    beams = _log(rng, 1, 16)
    block, req = rng.choice([8, 16, 24, 32, 64]), _log(rng, 1, 2048 // beams)
    if op == "fork":
        return dict(op=op, req=req, beams=beams, block=block, longest=_log(rng, 32, 65536 * block // 64), ended=rng.choice([0.0, 0.1, 0.5]))
    if op == "compact":
        return dict(op=op, req=req, beams=beams, block=block, longest=_log(rng, 32, 8192), spare=rng.choice([0.0, 0.2, 1.0, 3.0]))
    size = rng.choice([512, 1000, 4096, 9216, 32768, 65536 + 16])
    caches = _log(rng, 1, 32)
    pairs = _log(rng, 1, max(1, min(400, (1 << 28) // (size * caches))))
    return dict(op=op, blocks=2 * pairs + rng.randint(1, 100), rows=pairs + rng.randint(0, 300), pairs=pairs, caches=caches, bytes=size)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _ints(g, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    return {"recur": _prepare_recur, "back": _prepare_back, "beam": _prepare_beam, "fork": _prepare_fork, "compact": _prepare_compact,
            "copy": _prepare_copy}[case["op"]](case, g)


def _prepare_recur(c, g):
    b, t, ch = c["batch"], c["tokens"], c["channels"]
    shape = (t, ch) if c["ragged"] else (b, t, ch)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if c["kind"] == "sigmoid":
        gate = n(*shape).mul_(1.5).add_(2.0)               # logits of forget gates
    elif c["kind"] == "log":
        gate = n(*shape).sub_(3.0).exp_().neg_()           # decays of a few tokens up to hundreds
    else:
        gate = 1 - torch.rand(*shape, generator=g, device="cuda").square_()
    s = dict(op=c["op"], kind=c["kind"], blend=c["blend"], gate=gate.to(DT[c["gate"]]), x=n(*shape).to(DT[c["dtype"]]), longest=t)
    s["starts"] = None
    if c["ragged"]:
        cuts = _ints(g, (b - 1,), 0, t).sort().values
        s["starts"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), t)]).to(torch.int32)
    s["state"] = n(b, ch) if c["state"] else None
    s["sources"] = None
    if c.get("sources"):
        s["sources"] = (torch.arange(b, device="cuda") // 4 * 4 + _ints(g, (b,), 0, 3)).clamp(max=b - 1).to(torch.int32)
    s["out"] = torch.empty(shape, dtype=s["x"].dtype, device="cuda")
    s["state_out"] = torch.empty(b, ch, device="cuda")
    return s


def _prepare_back(c, g):
    s = _prepare_recur(c, g)
    shape = s["x"].shape
    s["out"] = torch.randn(shape, generator=g, device="cuda").to(s["x"].dtype)     # what the forward pass left
    s["dout"] = torch.randn(shape, generator=g, device="cuda").to(s["x"].dtype)
    s["dstate_out"] = torch.randn(s["state_out"].shape, generator=g, device="cuda") if c["state"] else None
    s["dgate"], s["dx"], s["dstate"] = torch.empty_like(s["gate"]), torch.empty_like(s["x"]), s["state_out"]
    return s


def _prepare_beam(c, g):
    lines, n = c["req"] * c["beams"], c["n"]
    x = torch.randn(lines, n, generator=g, device="cuda").mul_(3.0)
    if c["masked"]:
        x.masked_fill_(torch.rand(lines, n, generator=g, device="cuda") < c["masked"], float("-inf"))
        x[lines - 1, n // 2:] = torch.finfo(DT[c["dtype"]]).min   # another way to mask
    buf = torch.zeros(lines, n + c["pad"], dtype=DT[c["dtype"]], device="cuda")
    buf[:, :n] = x
    scores = torch.randn(c["req"], c["beams"], generator=g, device="cuda").mul_(2.0).sub_(20.0)
    scores[torch.rand(c["req"], generator=g, device="cuda") < 0.05, 1:] = float("-inf")   # a request's first step
    ended = torch.rand(c["req"], c["beams"], generator=g, device="cuda") < c["ended"] if c["ended"] else None
    k, i = c["count"], torch.int64 if c["ids"] == "i64" else torch.int32
    return dict(op="beam", logits=buf[:, :n], scores=scores, ended=ended, end=2, count=k, best=torch.empty(c["req"], k, device="cuda"),
                tokens=torch.empty(c["req"], k, dtype=i, device="cuda"), parents=torch.empty(c["req"], k, dtype=torch.int32, device="cuda"))


def _lengths(c):
    """(tokens, blocks that its beams share) of each request, shortest first: up to the longest, from half to all of them shared."""
    n = [1 + (c["longest"] - 1) * (i + 1) // c["req"] for i in range(c["req"])]
    return [(v, int(v * (0.5 + 0.5 * (i * 0.618 % 1)) / c["block"])) for i, v in enumerate(n)]


def _used(c):
    """Blocks in use by all requests' beams."""
    return sum(s + c["beams"] * (-(-n // c["block"]) - s) for n, s in _lengths(c))


def _beam_tables(c, g):
    """Tables of requests whose beams share their first blocks, the rest each beam's own: lens, held, and table entries numbered from 0."""
    req, beams, block = c["req"], c["beams"], c["block"]
    of = torch.tensor(_lengths(c), device="cuda")[torch.randperm(req, generator=g, device="cuda")].repeat_interleave(beams, 0)
    lens, shared = of[:, 0], of[:, 1]
    held = (lens + block - 1) // block
    width = -(-c["longest"] // block) + 1
    row = torch.arange(req * beams, device="cuda")
    own_from = torch.where(row % beams == 0, 0, shared)     # the first beam's row names the shared blocks
    fresh = held - own_from
    base = fresh.cumsum(0) - fresh
    j = torch.arange(width, device="cuda")
    place = torch.where(j < shared[:, None], base[row // beams * beams][:, None] + j, base[:, None] + j - own_from[:, None])
    return lens.to(torch.int32), held.to(torch.int32), torch.where(j < held[:, None], place, -1), width


def _prepare_fork(c, g):
    lens, held, place, width = _beam_tables(c, g)
    rows, used = lens.numel(), _used(c)
    pool = used + rows + 1000
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.where(place >= 0, ids[place.clamp(min=0)], -1)
    head = int(_ints(g, (1,), 0, 10 * pool))
    ring = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(pool - used, device="cuda")) % pool] = ids[used:]
    row = torch.arange(rows, device="cuda")
    parents = row // c["beams"] * c["beams"] + _ints(g, (rows,), 0, c["beams"] - 1)
    gone = torch.rand(c["req"], generator=g, device="cuda") < c["ended"]
    parents = torch.where(gone.repeat_interleave(c["beams"]), -1, parents)
    i32 = lambda *s: torch.full(s, -1, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(op="fork", block=c["block"], pool=pool, parents=parents.to(torch.int32), lens=lens, held=held, table=table, ring=ring,
                state=torch.tensor([head, head + pool - used, 0, 0], device="cuda"), table_out=i32(rows, width), held_out=i32(rows),
                lens_out=i32(rows), pairs=i32(rows, 2), state_out=torch.zeros(4, dtype=torch.int64, device="cuda"))


def _prepare_compact(c, g):
    _, held, place, _ = _beam_tables(c, g)
    pool = int(_used(c) * (1 + c["spare"])) + 8
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.where(place >= 0, ids[place.clamp(min=0)], -1)
    i32 = lambda *s: torch.full(s, -1, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(op="compact", pool=pool, held=held, table=table, table_out=i32(*table.shape), ring=i32(pool), pairs=i32(pool // 2, 2),
                state_out=torch.zeros(4, dtype=torch.int64, device="cuda"))


def _prepare_copy(c, g):
    size = c["bytes"]
    caches = [torch.randint(-(1 << 15), 1 << 15, (c["blocks"], size // 2), generator=g, device="cuda", dtype=torch.int16) for _ in range(c["caches"])]
    ids = torch.randperm(c["blocks"], generator=g, device="cuda").to(torch.int32)
    pairs = torch.full((c["rows"], 2), -1, dtype=torch.int32, device="cuda")
    at = torch.randperm(c["rows"], generator=g, device="cuda")[: c["pairs"]]
    pairs[at, 0] = ids[_ints(g, (c["pairs"],), 0, (c["blocks"] - c["pairs"] - 1) // 2)]    # one block may go to several
    pairs[at, 1] = ids[c["blocks"] - c["pairs"]:]
    return dict(op="copy", caches=caches, pairs=pairs)


# --------------------------------------------------------------------- runs

def run(s):
    if own:
        return _run_own(s)
    return {"recur": _recur, "back": _back, "beam": _beam, "fork": _fork, "compact": _compact, "copy": _copy}[s["op"]](s)


def _run_own(s):
    import reduction_primitives_amd as rk
    op = s["op"]
    if op == "recur":
        return rk.linear_recurrence(s["gate"], s["x"], state=s["state"], kind=s["kind"], blend=s["blend"], starts=s["starts"],
                                    sources=s["sources"], out=s["out"], state_out=s["state_out"])
    if op == "back":
        return rk.linear_recurrence_backward(s["gate"], s["x"], s["out"], s["dout"], state=s["state"], dstate_out=s["dstate_out"],
                                             kind=s["kind"], blend=s["blend"], starts=s["starts"], dgate=s["dgate"], dx=s["dx"], dstate=s["dstate"])
    if op == "beam":
        return rk.beam_select(s["logits"], s["scores"], s["count"], ended=s["ended"], end_token=s["end"], best=s["best"],
                              tokens=s["tokens"], parents=s["parents"])
    if op == "fork":
        return rk.fork_blocks(s["parents"], s["lens"], s["block"], s["held"], s["table"], s["ring"], s["state"], s["pool"],
                              table_out=s["table_out"], held_out=s["held_out"], lens_out=s["lens_out"], pairs=s["pairs"],
                              state_out=s["state_out"]) + (s["ring"],)
    if op == "compact":
        return rk.compact_blocks(s["held"], s["table"], s["ring"], s["pool"], table_out=s["table_out"], pairs=s["pairs"],
                                 state_out=s["state_out"]) + (s["ring"],)
    return rk.copy_blocks(s["caches"], s["pairs"])


def _gates(s):
    """(a, w) of every token, flat over the batch."""
    gate = s["gate"].float().reshape(-1, s["gate"].shape[-1])
    if s["kind"] == "sigmoid":
        return torch.sigmoid(gate), torch.sigmoid(-gate) if s["blend"] else torch.ones_like(gate)
    if s["kind"] == "log":
        return torch.exp(gate), -torch.expm1(gate) if s["blend"] else torch.ones_like(gate)
    return gate, 1 - gate if s["blend"] else torch.ones_like(gate)


def _bounds(s):
    """The sequences with tokens, their first and last tokens in the flat batch."""
    if s["starts"] is not None:
        lo, hi = s["starts"][:-1].long(), s["starts"][1:].long()
    else:
        b, t = s["x"].shape[:2]
        lo = torch.arange(b, device="cuda") * t
        hi = lo + t
    return hi > lo, lo, hi


def _put(to, rows, value, some):
    """to[rows] = value where some."""
    longer = torch.cat([to, to[:1]])
    longer[torch.where(some, rows, to.shape[0])] = value
    return longer[:-1]


def _first_state(s):
    h0 = s["state"]
    if h0 is None:
        return torch.zeros_like(s["state_out"])
    return h0 if s["sources"] is None else h0[s["sources"].long()]


def _scan(a, b, longest):
    """y_t = a_t y_(t-1) + b_t by doubling: after a step of d every token has its last 2 d ones folded."""
    d = 1
    while d < longest:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([torch.zeros_like(a[:d]), a[d:] * a[:-d]])
        d *= 2
    return b


def _recur(s):
    a, w = _gates(s)
    b = w * s["x"].float().reshape(a.shape)
    some, lo, hi = _bounds(s)
    h0 = _first_state(s)
    at = lo.clamp(max=a.shape[0] - 1)
    b = _put(b, lo, b[at] + a[at] * h0, some)
    h = _scan(_put(a, lo, torch.zeros_like(h0), some), b, s["longest"])
    last = torch.where(some[:, None], h[(hi - 1).clamp(min=0)], h0)
    return h.to(s["x"].dtype).view(s["x"].shape), last


def _back(s):
    a, w = _gates(s)
    x, h, g = (s[k].float().reshape(a.shape) for k in ("x", "out", "dout"))
    some, lo, hi = _bounds(s)
    h0 = _first_state(s)
    d1 = torch.zeros_like(h0) if s["dstate_out"] is None else s["dstate_out"]
    last, first = (hi - 1).clamp(min=0), lo.clamp(max=a.shape[0] - 1)
    g = _put(g, hi - 1, g[last] + d1, some)
    # u_t = a_t g_t, what a token hands to the one before it
    u = _scan(_put(a, hi - 1, torch.zeros_like(h0), some).flip(0), (a * g).flip(0), s["longest"]).flip(0)
    g = g + torch.cat([_put(u, lo, torch.zeros_like(h0), some)[1:], torch.zeros_like(u[:1])])
    before = _put(torch.cat([torch.zeros_like(h[:1]), h[:-1]]), lo, h0, some)
    da = g * (before - x) if s["blend"] else g * before
    if s["kind"] == "sigmoid":
        da = da * a * torch.sigmoid(-s["gate"].float().reshape(a.shape))
    elif s["kind"] == "log":
        da = da * a
    shape = s["x"].shape
    return da.to(s["gate"].dtype).view(shape), (w * g).to(s["x"].dtype).view(shape), torch.where(some[:, None], u[first], d1)


def _beam(s):
    x, scores = s["logits"], s["scores"]
    req, beams = scores.shape
    n, none = x.shape[1], float("-inf")
    x = x.float()
    top = x.amax(1, keepdim=True)
    some = top > none
    total = torch.exp(x - torch.where(some, top, 0.0)).sum(1, keepdim=True, dtype=torch.float64)
    # borders between candidates of two lines are as near as their logarithms: 64 bits
    base = torch.where(some, scores.view(-1, 1).double() - top.double() - torch.log(total), none)
    v = torch.arange(n, device=x.device)
    cand = x.double() + base
    if s["ended"] is not None:
        alone = torch.where(v == s["end"], scores.view(-1, 1).double(), none)
        cand = torch.where(s["ended"].view(-1, 1), alone, cand)
    cand = cand.view(req, beams * n)
    at = torch.arange(beams * n, device=x.device)
    best, place = [], []
    for _ in range(s["count"]):
        b = cand.amax(1, keepdim=True)
        i = torch.where(cand == b, at, beams * n).amin(1, keepdim=True)
        cand.scatter_(1, i, none)
        best.append(b)
        place.append(i)
    best, place = torch.cat(best, 1), torch.cat(place, 1)
    there = best > none
    line = torch.arange(req, device=x.device)[:, None] * beams + place // n
    return best.float(), torch.where(there, place % n, -1).to(s["tokens"].dtype), torch.where(there, line, -1).to(torch.int32)


def _fork(s):
    table, ring, block, pool = s["table"], s["ring"], s["block"], s["pool"]
    (rows, width), size = table.shape, ring.numel()
    held, par = s["held"].long(), s["parents"].long()
    ok = (par >= 0) & (par < rows)
    p = torch.where(ok, par, 0)
    r = torch.arange(rows, device=par.device)
    child = torch.full((rows + 1,), rows, device=par.device).scatter_reduce_(0, torch.where(ok, par, rows), r, "amin")[:rows]
    first = ok & (child[p] == r)
    j = torch.arange(width, device=par.device)
    # blocks that no new row names, where an old row first names them
    there = (j < held[:, None]) & (table >= 0) & (table < pool)
    lost = there & (child == rows)[:, None]
    ids = torch.where(there, table, pool).long()
    kept = torch.zeros(pool + 1, dtype=torch.bool, device=par.device)
    kept[torch.where(lost, pool, ids)] = True
    entry = torch.arange(rows * width, device=par.device).view(rows, width)
    owner = torch.full((pool + 1,), rows * width, device=par.device)
    owner.scatter_reduce_(0, torch.where(lost, ids, pool).view(-1), entry.view(-1), "amin")
    free = lost & ~kept[ids] & (owner[ids] == entry)
    rank = (free.view(-1).cumsum(0) - 1).view(rows, width)
    head, tail = s["state"][0], s["state"][1]
    room = size - (tail - head)
    longer = torch.cat([ring, ring[:1]])
    longer[torch.where(free & (rank < room), (tail + rank) % size, size)] = table
    ring.copy_(longer[:size])
    given = torch.minimum(free.sum(), room)
    # the last, partly filled block of the children after the first
    n = s["lens"].long().clamp(min=0)[p]
    full, part = n // block, n % block > 0
    wants = ok & ~first & part & (full < held[p])
    turn = wants.long().cumsum(0) - 1
    got = wants & (turn < tail + given - head)
    new = ring[(head + turn.clamp(min=0)) % size]
    h = torch.where(ok, torch.where(first, held[p], torch.minimum(held[p], full + got.long())), 0)
    rowp = torch.where((j == full[:, None]) & got[:, None], new[:, None], table[p])
    s["table_out"].copy_(torch.where(j < h[:, None], rowp, s["table_out"]))
    src = table[p, full.clamp(max=width - 1)]
    pairs = torch.where(got[:, None], torch.stack([src, new], 1), -1)
    after = torch.stack([head + got.sum(), tail + given, wants.sum() - got.sum(), free.sum() - given])
    return s["table_out"], h.to(torch.int32), torch.where(ok, n, 0).to(torch.int32), pairs.to(torch.int32), after, ring


def _compact(s):
    table, pool, ring = s["table"], s["pool"], s["ring"]
    j = torch.arange(table.shape[1], device=table.device)
    named = j < s["held"][:, None]
    there = named & (table >= 0) & (table < pool)
    used = torch.zeros(pool + 1, dtype=torch.bool, device=table.device)
    used[torch.where(there, table, pool).long()] = True
    used = used[:pool]
    u = used.sum()
    i = torch.arange(pool, device=table.device)
    src, dst = used & (i >= u), ~used & (i < u)
    moves = src.sum()
    k = torch.where(src, src.cumsum(0) - 1, pool)
    frm, to = torch.full((2, pool + 1), -1, device=table.device)
    frm[k] = i
    to[torch.where(dst, dst.cumsum(0) - 1, pool)] = i
    where = torch.where(src, to[k.clamp(max=pool - 1)], i)
    s["table_out"].copy_(torch.where(there, where[table.clamp(0, pool - 1).long()].to(torch.int32), torch.where(named, table, s["table_out"])))
    m = s["pairs"].shape[0]
    some = torch.arange(m, device=table.device) < moves
    pairs = torch.where(some[:, None], torch.stack([frm[:m], to[:m]], 1), -1).to(torch.int32)
    ring.copy_(torch.where(i < pool - u, u + i, ring))
    zero = torch.zeros_like(u)
    return s["table_out"], pairs, torch.stack([zero, pool - u, moves, zero]), ring


def _copy(s):
    src, dst = s["pairs"].long().unbind(1)
    there = (src >= 0) & (dst >= 0)
    src = torch.where(there, src, 0)
    for c in s["caches"]:
        i = torch.where(there, dst, c.shape[0])
        rows = c[src]
        longer = torch.cat([c, c[:1]])
        longer[i] = rows
        c.copy_(longer[:-1])
    return s["caches"]


# --------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] in ("recur", "back"):
        rows = c["tokens"] * (1 if c["ragged"] else c["batch"])
        e, st, x, g = rows * c["channels"], c["batch"] * c["channels"] * 4, SIZE[c["dtype"]], SIZE[c["gate"]]
        if c["op"] == "recur":
            return dict(bytes=e * (g + 2 * x) + st * (1 + c["state"]), flops=8 * e)
        return dict(bytes=e * (2 * g + (4 if c["blend"] else 3) * x) + st * (1 + 2 * c["state"]), flops=14 * e)
    if c["op"] == "beam":
        e = c["req"] * c["beams"] * c["n"] * (1 - c["ended"])
        return dict(bytes=e * SIZE[c["dtype"]] + c["req"] * (5 * c["beams"] + 16 * c["count"]), flops=4 * e)
    if c["op"] in ("fork", "compact"):
        rows, held = c["req"] * c["beams"], c["beams"] * sum(-(-n // c["block"]) for n, _ in _lengths(c))
        if c["op"] == "fork":
            return dict(bytes=4 * (held * (2 - c["ended"]) + 7 * rows), flops=4 * held)
        pool = _used(c) * (1 + c["spare"])
        return dict(bytes=8 * held + 8 * pool, flops=4 * held + pool)
    return dict(bytes=2 * c["pairs"] * c["caches"] * c["bytes"] + 8 * c["rows"], flops=0)


# -------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"recur": _exact_recur, "back": _exact_back, "beam": _exact_beam, "fork": _exact_fork, "compact": _exact_compact, "copy": _exact_copy}[s["op"]](s)


def _exact_tokens(s):
    """A sequence's tokens as rows of the flat batch, in lists, and the gates' function."""
    if s["starts"] is None:
        b, t = s["x"].shape[:2]
        lo, n = [i * t for i in range(b)], [t] * b
    else:
        st = s["starts"].tolist()
        lo, n = st[:-1], [j - i for i, j in zip(st, st[1:])]
    lo, n = torch.tensor(lo, device="cuda"), torch.tensor(n, device="cuda")

    def gates(rows):
        g = s["gate"].view(-1, s["gate"].shape[-1])[rows].double()
        if s["kind"] == "value":
            return g, 1 - g
        if s["kind"] == "log":
            return g.exp(), -torch.expm1(g)
        return 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))

    return lo, n, gates


def _exact_start(s):
    if s["state"] is None:
        return torch.zeros(s["state_out"].shape, dtype=torch.float64, device="cuda")
    h = s["state"].double()
    return h if s["sources"] is None else torch.stack([h[i] for i in s["sources"].tolist()])


def _exact_recur(s):
    lo, n, gates = _exact_tokens(s)
    x, h = s["x"].view(-1, s["x"].shape[-1]), _exact_start(s)
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for t in range(int(n.max())):
        live = (n > t).nonzero().view(-1)
        rows = lo[live] + t
        a, w = gates(rows)
        h[live] = a * h[live] + (w if s["blend"] else 1.0) * x[rows].double()
        out[rows] = h[live]
    return out.view(s["x"].shape), h


def _exact_back(s):
    lo, n, gates = _exact_tokens(s)
    flat = lambda k: s[k].view(-1, s["x"].shape[-1])  # noqa: E731
    x, h, dout, h0 = flat("x"), flat("out"), flat("dout"), _exact_start(s)
    u = torch.zeros_like(h0) if s["dstate_out"] is None else s["dstate_out"].double()
    dgate, dx = torch.empty((2,) + x.shape, dtype=torch.float64, device="cuda")
    for t in range(int(n.max()) - 1, -1, -1):
        live = (n > t).nonzero().view(-1)
        rows = lo[live] + t
        a, w = gates(rows)
        g = dout[rows].double() + u[live]
        before = h[rows - 1].double() if t else h0[live]
        da = g * (before - x[rows].double()) if s["blend"] else g * before
        dgate[rows] = da * {"value": 1.0, "log": a, "sigmoid": a * w}[s["kind"]]
        dx[rows] = g * (w if s["blend"] else 1.0)
        u[live] = a * g
    return dgate.view(s["x"].shape), dx.view(s["x"].shape), u


def _exact_beam(s):
    req, beams = s["scores"].shape
    n, k = s["logits"].shape[1], s["count"]
    best, tokens, parents = np.full((req, k), -np.inf), np.full((req, k), -1, np.int64), np.full((req, k), -1, np.int64)
    for b in range(req):
        cand = torch.empty(beams, n, dtype=torch.float64, device="cuda")
        for j in range(beams):
            score = s["scores"][b, j].double()
            if s["ended"] is not None and s["ended"][b, j]:
                cand[j] = float("-inf")
                cand[j, s["end"]] = score
            else:
                x = s["logits"][b * beams + j].double()
                cand[j] = x - torch.logsumexp(x, 0) + score
        cand = torch.where(cand.isnan(), float("-inf"), cand).view(-1)
        near = (cand >= torch.topk(cand, min(k, cand.numel())).values[-1]) & (cand > float("-inf"))
        near = near.nonzero().view(-1)
        near, value = near.cpu().numpy(), cand[near].cpu().numpy()
        order = np.lexsort((near, -value))[:k]
        m = order.size
        best[b, :m], tokens[b, :m], parents[b, :m] = value[order], near[order] % n, b * beams + near[order] // n
    return torch.from_numpy(best), torch.from_numpy(tokens).to(s["tokens"].dtype), torch.from_numpy(parents).to(torch.int32)


def _exact_fork(s):
    table, ring, out = (s[k].cpu().numpy().copy() for k in ("table", "ring", "table_out"))
    held, lens, parents, block = s["held"].tolist(), s["lens"].tolist(), s["parents"].tolist(), s["block"]
    head, tail = s["state"].tolist()[:2]
    rows = len(held)
    alive = {p for p in parents if 0 <= p < rows}
    kept = np.zeros(s["pool"], bool)
    for p in alive:
        kept[table[p, : held[p]]] = True
    for p in range(rows):
        if p not in alive:
            for i in table[p, : held[p]]:
                if not kept[i]:
                    kept[i] = True
                    ring[tail % ring.size] = i
                    tail += 1
    after, pairs, missing, seen = np.zeros(rows, np.int64), np.full((rows, 2), -1, np.int64), 0, set()
    for r, p in enumerate(parents):
        if p not in alive:
            continue
        n, full = held[p], lens[p] // block
        row = table[p].copy()
        if p in seen:
            n = min(n, -(-lens[p] // block))
            if full < n:
                if head < tail:
                    pairs[r] = row[full], ring[head % ring.size]
                    row[full] = pairs[r, 1]
                    head += 1
                else:
                    n = full
                    missing += 1
        seen.add(p)
        out[r, :n] = row[:n]
        after[r] = n
    new_lens = [lens[p] if p in alive else 0 for p in parents]
    i32 = lambda v: torch.from_numpy(np.asarray(v).astype(np.int32))  # noqa: E731
    return i32(out), i32(after), i32(new_lens), i32(pairs), torch.tensor([head, tail, missing, 0]), i32(ring)


def _exact_compact(s):
    table, held, pool = s["table"].cpu().numpy(), s["held"].tolist(), s["pool"]
    out, ring = s["table_out"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    used = np.unique(np.concatenate([table[r, :h] for r, h in enumerate(held)]))
    u = used.size
    src = used[used >= u]
    dst = np.setdiff1d(np.arange(u), used)
    to = np.arange(pool)
    to[src] = dst
    for r, h in enumerate(held):
        out[r, :h] = to[table[r, :h]]
    pairs = np.full(s["pairs"].shape, -1, np.int64)
    pairs[: src.size, 0], pairs[: src.size, 1] = src, dst
    ring[: pool - u] = np.arange(u, pool)
    i32 = lambda v: torch.from_numpy(np.asarray(v).astype(np.int32))  # noqa: E731
    return i32(out), i32(pairs), torch.tensor([0, pool - u, src.size, 0]), i32(ring)


def _exact_copy(s):
    pairs = [(i, j) for i, j in s["pairs"].tolist() if i >= 0]
    src, dst = torch.tensor(pairs, device="cuda").unbind(1)
    return [c.index_copy(0, dst, c.index_select(0, src)) for c in s["caches"]]
