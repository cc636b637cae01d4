"""Cases and plain forms of the operators a language-model serving step needs
around its model: softmax of logit lines, verification of drafted tokens,
block tables and slot maps.

`listed()` and `draw()` give cases, `prepare()` their inputs, `run()` one pass
(the plain form below, or with `own` the library's calls), `work()` the bytes
and operations a pass cannot do without, `exact()` the results in 64 bits.

Plain forms:
  softmax       p_i = exp((x_i - max x) / t) / sum_j exp((x_j - max x) / t); t <= 0 puts 1 on
                the first largest entry; a line of -inf alone gives zeros
  draft_verify  request b keeps its drafted tokens x_0, x_1, ... while u_i * q_i(x_i) < p_i(x_i);
                at the first i that fails it draws from max(p_i - q_i, 0), after the last one
                from p_n: the first index whose running sum passes r * (whole sum)
  block_tables  every request holds ceil(len / block) blocks: those it has too many go to the
                back of a ring of free blocks, those it lacks come from its front
  slot_map      token i of a request's new ones sits at position len - new + i, in slot
                table[position / block] * block + position % block
"""
import numpy as np
import torch

own = False

F32, BF16, F16 = "f32", "bf16", "f16"
DT = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}


def listed():
    return [
        # one request's four drafted tokens and the one after them: latency
        dict(name="softmax_5x32768_f32", op="softmax", lines=5, n=32768, pad=0, dtype=F32, out=F32, masked=0.0, greedy=0.0),
        # 64 requests of four drafts, logits as the model's last product leaves them
        dict(name="softmax_320x131072_bf16", op="softmax", lines=320, n=131072, pad=0, dtype=BF16, out=F32, masked=0.0, greedy=0.1),
        # an odd vocabulary in padded lines, grammar masks, some greedy requests
        dict(name="softmax_96x50001_f16", op="softmax", lines=96, n=50001, pad=47, dtype=F16, out=F16, masked=0.6, greedy=0.3),
        # a single request
        dict(name="verify_1x4x32768_f32", op="verify", req=1, k=4, n=32768, dtype=F32, draft=True, ragged=False, ids="i64"),
        # a serving batch
        dict(name="verify_64x4x131072_f32", op="verify", req=64, k=4, n=131072, dtype=F32, draft=True, ragged=True, ids="i64"),
        # drafts found by looking up earlier text: no draft probabilities
        dict(name="verify_96x7x50001_bf16", op="verify", req=96, k=7, n=50001, dtype=BF16, draft=False, ragged=True, ids="i32"),
        # the largest batch
        dict(name="verify_256x7x131072_f32", op="verify", req=256, k=7, n=131072, dtype=F32, draft=True, ragged=True, ids="i64"),
        # a decode step: every request grows by a few tokens
        dict(name="tables_decode_256", op="tables", req=256, block=16, longest=8192, grow=5, turnover=0.0),
        # requests that finish and others that start, prompts of up to 65536 tokens
        dict(name="tables_mixed_2048", op="tables", req=2048, block=16, longest=65536, grow=8, turnover=0.4),
        # a decode step with four drafts each
        dict(name="slots_decode_256", op="slots", req=256, block=16, longest=8192, new=5, spare=64, ids="i64"),
        # prompts packed into one batch
        dict(name="slots_prompts_97", op="slots", req=97, block=32, longest=20000, new=20000, spare=1000, ids="i32"),
        # the largest prompt batch
        dict(name="slots_prompts_1024", op="slots", req=1024, block=16, longest=4096, new=4096, spare=0, ids="i64"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["softmax", "verify", "tables", "slots"])
    if op == "softmax":
        n = _log(rng, 1000, 200000)
        return dict(op=op, lines=_log(rng, 1, max(1, min(512, 320 * 131072 // n))), n=n, pad=rng.choice([0, 0, 1, 24, 64]),
                    dtype=rng.choice([F32, BF16, F16]), out=rng.choice([F32, F32, BF16, F16]),
                    masked=rng.choice([0.0, 0.0, 0.5, 0.95]), greedy=rng.choice([0.0, 0.2]))
    if op == "verify":
        n, k = _log(rng, 1000, 200000), rng.randint(1, 8)
        return dict(op=op, req=_log(rng, 1, max(1, min(256, 256 * 8 * 131072 // (n * (k + 1))))), k=k, n=n,
                    dtype=rng.choice([F32, F32, BF16, F16]), draft=rng.random() < 0.75, ragged=rng.random() < 0.7,
                    ids=rng.choice(["i32", "i64"]))
    block = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "tables":
        return dict(op=op, req=_log(rng, 1, 2048), block=block, longest=_log(rng, 64, 65536), grow=rng.randint(1, 16),
                    turnover=rng.choice([0.0, 0.1, 0.4]))
    longest = _log(rng, 16, 32768)
    return dict(op=op, req=_log(rng, 1, max(1, min(2048, (1 << 22) // longest))), block=block, longest=longest,
                new=rng.choice([1, 1 + rng.randint(1, 8), longest]), spare=rng.choice([0, 7, 300]), ids=rng.choice(["i32", "i64"]))


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _ints(g, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")


def _logits(g, rows, n, spread=3.0):
    return torch.randn(rows, n, generator=g, device="cuda").mul_(spread)


def prepare(case, seed):
    g = _gen(seed)
    return {"softmax": _prepare_softmax, "verify": _prepare_verify, "tables": _prepare_tables, "slots": _prepare_slots}[case["op"]](case, g)


def _prepare_softmax(c, g):
    lines, n = c["lines"], c["n"]
    x = _logits(g, lines, n)
    if c["masked"]:
        x.masked_fill_(torch.rand(lines, n, generator=g, device="cuda") < c["masked"], float("-inf"))
        x[lines - 1, n // 2:] = torch.finfo(DT[c["dtype"]]).min   # another way to mask
    buf = torch.zeros(lines, n + c["pad"], dtype=DT[c["dtype"]], device="cuda")
    buf[:, :n] = x
    t = torch.rand(lines, generator=g, device="cuda") + 0.5
    t[torch.rand(lines, generator=g, device="cuda") < c["greedy"]] = 0.0
    s = dict(op="softmax", x=buf[:, :n], t=t, out=torch.empty(lines, n, dtype=DT[c["out"]], device="cuda"))
    s["workspace"] = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    return s


def _prepare_verify(c, g):
    req, k, n, dt = c["req"], c["k"], c["n"], DT[c["dtype"]]
    counts = _ints(g, (req,), 0, k) if c["ragged"] else torch.full((req,), k, device="cuda")
    counts[0] = k
    starts = torch.zeros(req + 1, dtype=torch.int64, device="cuda")
    starts[1:] = counts.cumsum(0)
    rows = int(starts[-1])
    z = _logits(g, rows + req, n)
    sure = _ints(g, (rows + req, 1), 0, n - 1)   # most lines have one token that stands out
    z.scatter_add_(1, sure, torch.randn(rows + req, 1, generator=g, device="cuda").mul_(4.0).add_(20.0))
    p = torch.softmax(z, 1).to(dt)
    # the draft's distribution at each drafted position: the target's, roughly
    at = torch.arange(rows, device="cuda") + torch.repeat_interleave(torch.arange(req, device="cuda"), counts)
    z = z[at].add_(_logits(g, rows, n, 0.5))
    q = torch.softmax(z, 1, out=z)
    if c["draft"]:
        drafted = torch.multinomial(q, 1, generator=g).view(-1)
    else:
        wrong = torch.rand(rows, generator=g, device="cuda") < 0.2
        drafted = torch.where(wrong, _ints(g, (rows,), 0, n - 1), sure.view(-1)[at])
    q = q.to(dt)
    i = torch.int64 if c["ids"] == "i64" else torch.int32
    return dict(op="verify", k=k, p=p, q=q if c["draft"] else None, starts=starts.to(torch.int32), drafted=drafted.to(i),
                u=torch.rand(rows, generator=g, device="cuda"), r=torch.rand(req, generator=g, device="cuda"),
                tokens=torch.empty(req, k + 1, dtype=i, device="cuda"), accepted=torch.empty(req, dtype=torch.int32, device="cuda"),
                workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


def _prepare_tables(c, g):
    req, block, longest = c["req"], c["block"], c["longest"]
    width = -(-(longest + c["grow"]) // block)
    old = _ints(g, (req,), 1, longest)
    lens = old + _ints(g, (req,), 1, c["grow"])
    if c["turnover"]:
        kind = torch.rand(req, generator=g, device="cuda")
        lens = torch.where(kind < c["turnover"] / 2, 0, lens)          # finished
        old = torch.where(kind > 1 - c["turnover"] / 2, 0, old)        # new
        back = (kind > 0.45) & (kind < 0.55)                           # drafts that were turned down
        lens = torch.where(back, (old - _ints(g, (req,), 0, c["grow"])).clamp(min=1), lens)
    held = (old + block - 1) // block
    base = held.cumsum(0) - held
    used, pool = int(held.sum()), req * width + 100
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(width, device="cuda")
    table = torch.where(j < held[:, None], ids[(base[:, None] + j).clamp(max=pool - 1)], -1)
    head = int(_ints(g, (1,), 0, 10 * pool))
    ring = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(pool - used, device="cuda")) % pool] = ids[used:]
    held = held.to(torch.int32)
    return dict(op="tables", block=block, lens=lens.to(torch.int32), held=held, table=table, ring=ring,
                state=torch.tensor([head, head + pool - used, 0, 0], device="cuda"),
                held_out=torch.empty_like(held), state_out=torch.zeros(4, dtype=torch.int64, device="cuda"),
                workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


def _new_counts(c):
    """The new tokens of each request, shortest first: from half of c["new"] up to all of it."""
    low = max(1, c["new"] // 2)
    return [low + (c["new"] - low) * i // max(1, c["req"] - 1) for i in range(c["req"])]


def _prepare_slots(c, g):
    req, block, longest = c["req"], c["block"], c["longest"]
    counts = _new_counts(c)
    new = torch.tensor(counts, device="cuda")[torch.randperm(req, generator=g, device="cuda")]
    lens = new + ((longest - new + 1) * torch.rand(req, generator=g, device="cuda")).long()
    held = (lens + block - 1) // block
    width = -(-longest // block)
    table = torch.randperm(req * width, generator=g, device="cuda").to(torch.int32).view(req, width)
    cap = sum(counts) + c["spare"]
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(op="slots", block=block, lens=lens.to(torch.int32), new=new.to(torch.int32), table=table, held=held.to(torch.int32),
                n_blocks=req * width, cap=cap, slots=torch.empty(cap, dtype=torch.int64 if c["ids"] == "i64" else torch.int32, device="cuda"),
                positions=i32(cap), requests=i32(cap), starts=i32(req + 1))


# --------------------------------------------------------------------- runs

def run(s):
    if own:
        return _run_own(s)
    return {"softmax": _softmax, "verify": _verify, "tables": _tables, "slots": _slots}[s["op"]](s)


def _run_own(s):
    import reduction_primitives_amd as rk
    op = s["op"]
    if op == "softmax":
        return rk.softmax(s["x"], temperature=s["t"], out=s["out"], workspace=s["workspace"])
    if op == "verify":
        return rk.draft_verify(s["p"], s["q"], s["drafted"], s["u"], s["r"], starts=s["starts"], max_draft=s["k"],
                               tokens=s["tokens"], accepted=s["accepted"], workspace=s["workspace"])
    if op == "tables":
        rk.block_tables(s["lens"], s["block"], s["held"], s["table"], s["ring"], s["state"],
                        held_out=s["held_out"], state_out=s["state_out"], workspace=s["workspace"])
        return s["table"], s["ring"], s["held_out"], s["state_out"]
    return rk.slot_map(s["lens"], s["new"], s["block"], s["table"], s["held"], s["n_blocks"], slots=s["slots"],
                       positions=s["positions"], requests=s["requests"], starts=s["starts"])


def _softmax(s):
    x, t = s["x"].float(), s["t"][:, None]
    top = x.amax(1, keepdim=True)
    some = top > float("-inf")
    e = torch.where(x > float("-inf"), torch.exp((x - top) / torch.where(t > 0, t, 1.0)), 0.0)
    p = e / torch.where(some, e.sum(1, keepdim=True), 1.0)
    j = torch.arange(x.shape[1], device=x.device)
    first = torch.where(x == top, j, x.shape[1]).amin(1, keepdim=True)
    p = torch.where(t > 0, p, ((j == first) & some).float())
    return p.to(s["out"].dtype)


def _verify(s):
    p, q, k = s["p"], s["q"], s["k"]
    req, n = s["r"].numel(), p.shape[1]
    starts = s["starts"].long()
    count = starts[1:] - starts[:-1]
    b = torch.arange(req, device=p.device)
    i = torch.arange(k, device=p.device)
    there = i < count[:, None]
    at = torch.where(there, starts[:-1, None] + i, 0)
    x = s["drafted"].long()[at]
    px = p[at + b[:, None], x].double()
    qx = q[at, x].double() if q is not None else torch.ones_like(px)
    ok = (s["u"][at].double() * qx < px) & there
    kept = ok.long().cumprod(1).sum(1)
    w = p[starts[:-1] + b + kept].double()
    turned = kept < count
    last = torch.where(turned, starts[:-1] + kept, 0)
    if q is not None:
        less = q[last].double()
    else:
        less = (torch.arange(n, device=p.device) == s["drafted"].long()[last][:, None]).double()
    res = (w - torch.where(turned[:, None], less, 0.0)).clamp(min=0)
    res = torch.where(res.sum(1, keepdim=True) > 0, res, w)
    run_sum = res.cumsum(1)
    token = (run_sum <= s["r"].double()[:, None] * run_sum[:, -1:]).sum(1)
    slot = torch.arange(k + 1, device=p.device)
    drafted = torch.cat([x, x[:, :1]], 1)
    out = torch.where(slot < kept[:, None], drafted, torch.where(slot == kept[:, None], token[:, None], -1))
    return out.to(s["drafted"].dtype), kept.to(torch.int32)


def _tables(s):
    table, ring, state, block = s["table"], s["ring"], s["state"], s["block"]
    width, size = table.shape[1], ring.numel()
    held = s["held"].long()
    need = ((s["lens"].long() + block - 1) // block).clamp(max=width)
    give, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    g0, t0 = give.cumsum(0) - give, take.cumsum(0) - take
    head, tail = state[0], state[1]
    j = torch.arange(width, device=table.device)
    # given back, in order, behind the ring's end (an entry more takes what is not given)
    giving = (j >= need[:, None]) & (j < held[:, None])
    place = torch.where(giving, (tail + g0[:, None] + j - need[:, None]) % size, size)
    longer = torch.cat([ring, ring[:1]])
    longer[place] = table
    ring.copy_(longer[:size])
    tail = tail + give.sum()
    got = torch.minimum(take, (tail - head - t0).clamp(min=0))
    taking = (j >= held[:, None]) & (j < (held + got)[:, None])
    table.copy_(torch.where(taking, ring[(head + t0[:, None] + j - held[:, None]) % size], table))
    zero = torch.zeros_like(head)
    after = torch.stack([head + got.sum(), tail, take.sum() - got.sum(), zero])
    return table, ring, (torch.minimum(held, need) + got).to(torch.int32), after


def _slots(s):
    new, cap, block = s["new"].long(), s["cap"], s["block"]
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(cap, device=new.device)
    b = torch.searchsorted(starts, t, right=True) - 1
    there = b < new.numel()
    b = torch.where(there, b, 0)
    pos = s["lens"].long()[b] - new[b] + t - starts[b]
    pos = torch.where(there, pos, 0)
    slot = s["table"][b, pos // block].long() * block + pos % block
    return (torch.where(there, slot, -1).to(s["slots"].dtype), pos.to(torch.int32), torch.where(there, b, -1).to(torch.int32),
            starts.to(torch.int32))


# --------------------------------------------------------------------- work

SIZE = {F32: 4, BF16: 2, F16: 2}


def work(case):
    c = case
    if c["op"] == "softmax":
        e = c["lines"] * c["n"]
        return dict(bytes=e * (SIZE[c["dtype"]] + SIZE[c["out"]]) + 4 * c["lines"], flops=5 * e)
    if c["op"] == "verify":
        # one line of the target's for each request, one of the draft's where a draft is turned down (about
        # seven in ten drafted tokens are kept), and a few words for each draft
        counts = range(c["k"] + 1) if c["ragged"] else [c["k"]]
        turned = sum(1 - 0.7 ** i for i in counts) / len(counts) if c["draft"] else 0.0
        e = c["req"] * c["n"]
        return dict(bytes=e * SIZE[c["dtype"]] * (1 + turned) + 20 * c["req"] * c["k"], flops=3 * e)
    if c["op"] == "tables":
        mean = c["longest"] / 2 / c["block"]
        moved = c["req"] * (c["turnover"] * mean + (1 - c["turnover"]) * c["grow"] / 2 / c["block"])
        return dict(bytes=12 * c["req"] + 8 * moved + 64, flops=4 * c["req"] + 4 * moved)
    tokens = sum(_new_counts(c))
    blocks = c["req"] + tokens / c["block"]
    return dict(bytes=(tokens + c["spare"]) * (16 if c["ids"] == "i64" else 12) + 4 * blocks + 16 * c["req"], flops=6 * tokens)


# -------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "softmax":
        return _exact_softmax(s)
    if s["op"] == "verify":
        return _exact_verify(s)
    if s["op"] == "tables":
        return _exact_tables(s)
    return _exact_slots(s)


def _exact_softmax(s):
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device=s["x"].device)
    for i, t in enumerate(s["t"].tolist()):
        x = s["x"][i].to(torch.float64)
        if t > 0:
            z = x / t
            out[i] = torch.exp(z - torch.logsumexp(z, 0))
        else:
            out[i, int(np.argmax(x.cpu().numpy()))] = 1.0
    return out


def _exact_verify(s):
    starts, drafted = s["starts"].tolist(), s["drafted"].tolist()
    u, r = s["u"].double().cpu().numpy(), s["r"].double().cpu().numpy()
    x = torch.tensor(drafted, dtype=torch.int64, device="cuda")
    req, k = len(starts) - 1, s["k"]
    which = torch.tensor([b for b in range(req) for _ in range(starts[b + 1] - starts[b])], dtype=torch.int64, device="cuda")
    rows = torch.arange(x.numel(), device="cuda")
    px = s["p"][rows + which, x].double().cpu().numpy()
    qx = np.ones_like(px) if s["q"] is None else s["q"][rows, x].double().cpu().numpy()
    tokens, accepted = np.full((req, k + 1), -1, np.int64), np.zeros(req, np.int64)
    for b in range(req):
        lo, hi = starts[b], starts[b + 1]
        i = lo
        while i < hi and u[i] * qx[i] < px[i]:
            tokens[b, i - lo] = drafted[i]
            i += 1
        w = s["p"][i + b].double().cpu().numpy()
        if i < hi:
            less = w.copy()
            if s["q"] is None:
                less[drafted[i]] = max(0.0, w[drafted[i]] - 1.0)
            else:
                less = np.maximum(w - s["q"][i].double().cpu().numpy(), 0.0)
            w = less if less.any() else w
        c = np.cumsum(w)
        tokens[b, i - lo] = np.searchsorted(c, r[b] * c[-1], side="right")
        accepted[b] = i - lo
    return torch.from_numpy(tokens).to(s["drafted"].dtype), torch.from_numpy(accepted).to(torch.int32)


def _exact_tables(s):
    table, ring = s["table"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    lens, held, block = s["lens"].tolist(), s["held"].tolist(), s["block"]
    head, tail = s["state"].tolist()[:2]
    need = [min(-(-n // block), table.shape[1]) for n in lens]
    for b, n in enumerate(need):
        for j in range(n, held[b]):
            ring[tail % ring.size] = table[b, j]
            tail += 1
    after, missing = [min(h, n) for h, n in zip(held, need)], 0
    for b, n in enumerate(need):
        for j in range(held[b], n):
            if head < tail:
                table[b, j] = ring[head % ring.size]
                head += 1
                after[b] += 1
            else:
                missing += 1
    return torch.from_numpy(table), torch.from_numpy(ring), torch.tensor(after, dtype=torch.int32), torch.tensor([head, tail, missing, 0])


def _exact_slots(s):
    lens, new, block = s["lens"].tolist(), s["new"].tolist(), s["block"]
    table = s["table"].cpu().numpy().astype(np.int64)
    slots, positions, requests, starts = [], [], [], [0]
    for b, (n, m) in enumerate(zip(lens, new)):
        pos = np.arange(n - m, n)
        slots.append(table[b][pos // block] * block + pos % block)
        positions.append(pos)
        requests.append(np.full(m, b))
        starts.append(starts[-1] + m)
    rest = s["cap"] - starts[-1]
    slots.append(np.full(rest, -1))
    positions.append(np.zeros(rest, np.int64))
    requests.append(np.full(rest, -1))
    back = lambda parts, t: torch.from_numpy(np.concatenate(parts).astype(np.int64)).to(t)  # noqa: E731
    return back(slots, s["slots"].dtype), back(positions, torch.int32), back(requests, torch.int32), torch.tensor(starts, dtype=torch.int32)
