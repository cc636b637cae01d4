"""GPU tests of the gated linear recurrence and its gradient against the plain
64-bit forms of tests/recur_ref.py."""
import numpy as np
import pytest
import torch

from tests import recur_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")
TYPES = [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)]      # of x and of the gate
KINDS = ["value", "log", "sigmoid"]


def _rk():
    import reduction_primitives_amd as rk
    rk.load()
    return rk


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def np64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def gates(g, shape, kind, dt, sign=False):
    if kind == "sigmoid":
        v = torch.randn(shape, generator=g) * 2 + 1
    elif kind == "log":
        v = -torch.exp(torch.randn(shape, generator=g) * 1.5 - 2)
    else:
        v = 1 - torch.rand(shape, generator=g) ** 2
        if sign:
            v *= torch.where(torch.rand(shape, generator=g) < 0.5, -1.0, 1.0)
    return v.to(dt)


def near(got, want, err):
    """got is want, rounded to its type, within err."""
    f = torch.finfo(got.dtype)
    half, low = (f.eps / 2, f.tiny * f.eps / 2) if got.dtype != F32 else (0.0, 0.0)   # (the float32's own is in err)
    g = np64(got)
    live = ~np.isnan(err)
    ok = np.abs(g - want) <= err + half * (np.abs(want) + err) + low
    bad = live & ~ok
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], want[bad][:4], err[bad][:4])


def check(gate, x, kind, blend, starts=None, state=None, sources=None, dout=None, dlast=None, backward=True):
    rk = _rk()
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    at = [dev(t) for t in (gate, x, starts, state, sources)]
    out, last = rk.linear_recurrence(at[0], at[1], state=at[3], kind=kind, blend=blend, starts=at[2], sources=at[4])
    assert out.dtype == x.dtype and out.shape == x.shape and last.dtype == F32
    st = None if starts is None else starts.numpy()
    so = None if sources is None else sources.numpy()
    want, want_last, err, err_last = ref.forward(np64(gate), np64(x), kind, blend, st, np64(state), so)
    near(out, want, err)
    near(last, want_last, err_last)
    if not backward:
        return
    g = gen(x.numel())
    dout = torch.randn(x.shape, generator=g).to(x.dtype) if dout is None else dout
    got = rk.linear_recurrence_backward(at[0], at[1], out, dev(dout), state=at[3], dstate_out=dev(dlast), kind=kind, blend=blend,
                                        starts=at[2])
    wants, errs = ref.backward(np64(gate), np64(x), np64(out), np64(dout), kind, blend, st, np64(state), np64(dlast))
    for v, w, e in zip(got, wants, errs):
        near(v, w, e)


@pytest.mark.parametrize("channels", [1, 2, 3, 4, 5, 7, 8, 33, 64, 65, 130, 1001])
@pytest.mark.parametrize("batch,tokens", [(1, 1), (3, 2), (2, 17), (1, 300), (5, 64)])
@pytest.mark.parametrize("types", TYPES)
def test_sizes(channels, batch, tokens, types):
    g = gen(channels * 1000 + tokens)
    kind = KINDS[(channels + tokens) % 3]
    blend = (channels + batch) % 2 == 0
    shape = (batch, tokens, channels)
    state = torch.randn(batch, channels, generator=g)
    check(gates(g, shape, kind, types[1], sign=True), torch.randn(shape, generator=g).to(types[0]), kind, blend, state=state,
          dlast=torch.randn(batch, channels, generator=g))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", [(1, 5000, 70), (2, 1025, 260), (1, 4097, 6), (300, 9, 40)])
def test_long(kind, blend, types, shape):
    """Many tiles along the tokens: every state goes through the look-back."""
    g = gen(shape[1])
    check(gates(g, shape, kind, types[1]), torch.randn(shape, generator=g).to(types[0]), kind, blend)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("channels", [3, 64, 201])
@pytest.mark.parametrize("cuts", [
    [0, 1, 2, 3, 3, 3, 20, 700, 1400], [0, 0, 1400], [0, 1400, 1400, 1400], [0, 256, 512, 1400], [0, 255, 257, 1399, 1400],
    [5, 9, 9, 1000], [-3, 40, 5000], [1400, 1400], [0, 0], list(range(0, 1401)), list(range(0, 1401, 7))])
def test_packed(types, channels, cuts):
    g = gen(len(cuts))
    kind = KINDS[len(cuts) % 3]
    shape, n = (1400, channels), len(cuts) - 1
    starts = torch.tensor(cuts, dtype=torch.int32)
    check(gates(g, shape, kind, types[1]), torch.randn(shape, generator=g).to(types[0]), kind, channels != 64, starts=starts,
          state=torch.randn(n, channels, generator=g), dlast=torch.randn(n, channels, generator=g))
    check(gates(g, shape, kind, types[1]), torch.randn(shape, generator=g).to(types[0]), kind, channels == 64, starts=starts)


def test_tokens_of_no_sequence_are_left():
    rk = _rk()
    g = gen(5)
    gate, x = gates(g, (900, 40), "sigmoid", F32).to(DEV), torch.randn(900, 40, generator=g).to(DEV)
    starts = torch.tensor([10, 10, 400, 750], dtype=torch.int32, device=DEV)
    out, dg, dx = (torch.full((900, 40), 7.0, device=DEV) for _ in range(3))
    rk.linear_recurrence(gate, x, kind="sigmoid", starts=starts, out=out)
    rk.linear_recurrence_backward(gate, x, out, x, kind="sigmoid", starts=starts, dgate=dg, dx=dx)
    for t in (out, dg, dx):
        assert (t[:10] == 7.0).all() and (t[750:] == 7.0).all() and (t[10:750] != 7.0).all()
    dg, dx, _ = rk.linear_recurrence_backward(gate, x, out, x, kind="sigmoid", starts=starts)
    assert not dg[:10].any() and not dx[750:].any()


@pytest.mark.parametrize("channels", [2, 64, 300])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_sources(channels, types):
    g = gen(channels)
    state = torch.randn(9, channels, generator=g)
    sources = torch.tensor([3, 3, 8, 0, -1, 9, 5, 2 ** 31 - 1, 0, -2 ** 31, 4], dtype=torch.int32)
    for shape, starts in (((11, 1, channels), None), ((11, 5, channels), None),
                          ((60, channels), torch.tensor([0, 1, 2, 2, 30, 31, 31, 40, 55, 56, 58, 60], dtype=torch.int32))):
        check(gates(g, shape, "sigmoid", types[1]), torch.randn(shape, generator=g).to(types[0]), "sigmoid", True, starts=starts,
              state=state, sources=sources, backward=False)


@pytest.mark.parametrize("tokens,channels", [(1, 40), (700, 40), (3, 6)])
def test_state_in_place(tokens, channels):
    """The last states take the place of the first ones, step after step."""
    rk = _rk()
    g = gen(tokens)
    batch = 5
    state = torch.randn(batch, channels, generator=g)
    gate, x = gates(g, (batch, tokens, channels), "sigmoid", BF16), torch.randn(batch, tokens, channels, generator=g).to(BF16)
    s = state.to(DEV)
    for _ in range(3):
        want, want_last, err, err_last = ref.forward(np64(gate), np64(x), "sigmoid", True, state=np64(s))
        out, last = rk.linear_recurrence(gate.to(DEV), x.to(DEV), state=s, kind="sigmoid", blend=True, state_out=s)
        assert last is s
        near(out, want, err)
        near(s, want_last, err_last)
    starts = torch.tensor([0, 0, 1, 1, tokens], dtype=torch.int32)
    s = state[:4].to(DEV)
    want, want_last, err, err_last = ref.forward(np64(gate[0]), np64(x[0]), "sigmoid", True, starts.numpy(), np64(s))
    out, _ = rk.linear_recurrence(gate[0].to(DEV), x[0].to(DEV), state=s, kind="sigmoid", blend=True, starts=starts.to(DEV), state_out=s)
    near(out, want, err)
    near(s, want_last, err_last)


@pytest.mark.parametrize("tokens", [1, 30, 600])
@pytest.mark.parametrize("layout", ["time_major", "columns", "padded", "odd"])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_strides(tokens, layout, dt):
    rk = _rk()
    g = gen(tokens)
    batch, ch = 3, 37
    x, gate, dout = (torch.randn(batch, tokens, ch, generator=g).to(dt) for _ in range(3))

    def place(t, fill=None):
        if layout == "time_major":
            b = torch.zeros(tokens, batch, ch, dtype=t.dtype, device=DEV).transpose(0, 1)
        elif layout == "columns":
            b = torch.zeros(batch, tokens, 3 * ch, dtype=t.dtype, device=DEV)[:, :, ch:2 * ch]
        elif layout == "padded":
            b = torch.zeros(batch, tokens + 5, ch + 3, dtype=t.dtype, device=DEV)[:, :tokens, :ch]
        else:
            b = torch.zeros(1 + batch * tokens * ch, dtype=t.dtype, device=DEV)[1:].view(batch, tokens, ch)
        return b.copy_(t.to(DEV)) if fill is None else b.fill_(fill)

    out, dg, dx = (place(x, 7.0) for _ in range(3))
    rk.linear_recurrence(place(gate), place(x), kind="sigmoid", blend=True, out=out)
    want, _, err, _ = ref.forward(np64(gate), np64(x), "sigmoid", True)
    near(out, want, err)
    rk.linear_recurrence_backward(place(gate), place(x), out, place(dout), kind="sigmoid", blend=True, dgate=dg, dx=dx)
    wants, errs = ref.backward(np64(gate), np64(x), np64(out), np64(dout), "sigmoid", True)
    near(dg, wants[0], errs[0])
    near(dx, wants[1], errs[1])
    if layout == "columns":
        for t in (out, dg, dx):
            whole = t.as_strided((batch, tokens, 3 * ch), (tokens * 3 * ch, 3 * ch, 1), 0)
            assert not whole[:, :, :ch].any() and not whole[:, :, 2 * ch:].any()


def test_columns_of_one_buffer_and_in_place():
    rk = _rk()
    g = gen(8)
    both = torch.randn(2, 500, 3 * 50, generator=g)
    both[..., :50] = gates(g, (2, 500, 50), "sigmoid", F32)
    want, _, err, _ = ref.forward(np64(both[..., :50]), np64(both[..., 50:100]), "sigmoid", False)
    d = both.to(DEV)
    rk.linear_recurrence(d[..., :50], d[..., 50:100], kind="sigmoid", out=d[..., 100:])
    near(d[..., 100:], want, err)
    assert torch.equal(d[..., :100].cpu(), both[..., :100])
    for place in (0, 1):
        gate, x = both[..., :50].contiguous().to(DEV), both[..., 50:100].contiguous().to(DEV)
        rk.linear_recurrence(gate, x, kind="sigmoid", out=(gate, x)[place])
        near((gate, x)[place], want, err)
    gate, x, dout = (both[..., i:i + 50].contiguous().to(DEV) for i in (0, 50, 100))
    out, _ = rk.linear_recurrence(gate, x, kind="sigmoid", blend=True)
    wants, errs = ref.backward(np64(gate), np64(x), np64(out), np64(dout), "sigmoid", True)
    rk.linear_recurrence_backward(gate, x, out, dout, kind="sigmoid", blend=True, dgate=gate, dx=dout)
    near(gate, wants[0], errs[0])
    near(dout, wants[1], errs[1])


def test_broadcast_gate():
    """One line of gates for every sequence."""
    rk = _rk()
    g = gen(11)
    gate, x = gates(g, (1, 70, 24), "log", F32), torch.randn(4, 70, 24, generator=g)
    out, _ = rk.linear_recurrence(gate.to(DEV).expand(4, 70, 24), x.to(DEV), kind="log")
    want, _, err, _ = ref.forward(np64(gate.expand(4, 70, 24)), np64(x), "log", False)
    near(out, want, err)


def test_sequences_do_not_meet():
    """Infinities and NaN stay in their sequence and channel, and go on to its end."""
    rk = _rk()
    g = gen(2)
    starts = torch.tensor([0, 3, 40, 41, 300, 800, 1500], dtype=torch.int32)
    gate, x = gates(g, (1500, 20), "sigmoid", F32), torch.randn(1500, 20, generator=g)
    bad = x.clone()
    bad[5, 3], bad[40, 4], bad[310, 5], bad[799, 6], bad[1, 7] = INF, NAN, NAN, -INF, NAN
    state = torch.zeros(6, 20)
    state[4, 8] = NAN
    out, last = rk.linear_recurrence(gate.to(DEV), bad.to(DEV), state=state.to(DEV), kind="sigmoid", starts=starts.to(DEV))
    want, want_last, err, _ = ref.forward(np64(gate), np64(bad), "sigmoid", False, starts.numpy(), np64(state))
    got = np64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want))
    assert np.array_equal(np.isnan(np64(last)), np.isnan(want_last))
    fine = np.isfinite(want)
    assert fine.sum() > 25000 and (np.abs(got - want)[fine] <= err[fine] + 1e-30).all()
    dout = torch.randn(1500, 20, generator=g)
    dout[20, 0], dout[300, 1], dout[1499, 2] = NAN, INF, NAN
    out, _ = rk.linear_recurrence(gate.to(DEV), x.to(DEV), kind="sigmoid", starts=starts.to(DEV))
    got = rk.linear_recurrence_backward(gate.to(DEV), x.to(DEV), out, dout.to(DEV), kind="sigmoid", starts=starts.to(DEV))
    wants, errs = ref.backward(np64(gate), np64(x), np64(out), np64(dout), "sigmoid", False, starts.numpy())
    for v, w, e in zip(got, wants, errs):
        v = np64(v)
        assert np.array_equal(np.isnan(v), np.isnan(w))
        fine = np.isfinite(w)
        assert (np.abs(v - w)[fine] <= e[fine] + 1e-30).all()


def test_extreme_gates():
    """Gates that let all or nothing through, and products past float32's range over states that are 0."""
    rk = _rk()
    for kind, values in (("sigmoid", [-200.0, 200.0, -INF, INF, 0.0]), ("log", [-200.0, -INF, 0.0, -1e-8, -0.0]), ("value", [0.0, 1.0, -1.0])):
        g = gen(3)
        gate = torch.tensor(values)[torch.randint(len(values), (2, 600, 16), generator=g)]
        x = torch.randn(2, 600, 16, generator=g)
        for blend in (False, True):
            check(gate, x, kind, blend, state=torch.randn(2, 16, generator=g))
    gate = torch.full((1, 5000, 8), 1.5)
    x = torch.zeros(1, 5000, 8)
    x[0, -3:] = 1.0                            # a product of 1.5^4997 meets a state of 0 only
    out, last = rk.linear_recurrence(gate.to(DEV), x.to(DEV))
    assert not out[0, :-3].any() and (out[0, -3:, 0].cpu() == torch.tensor([1.0, 2.5, 4.75])).all() and (last == 4.75).all()
    gate = torch.full((1, 500, 8), 30.0)
    x = torch.full((1, 500, 8), 0.0)
    out, _ = rk.linear_recurrence(gate.to(DEV), x.to(DEV), kind="log")
    assert not out.any()


def test_of_nothing():
    rk = _rk()
    z = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    state = torch.randn(3, 5, generator=gen(1)).to(DEV)
    out, last = rk.linear_recurrence(z(3, 0, 5), z(3, 0, 5), state=state)
    assert out.shape == (3, 0, 5) and torch.equal(last, state)
    out, last = rk.linear_recurrence(z(3, 0, 5), z(3, 0, 5), state=state, sources=torch.tensor([2, 7, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(last, torch.stack([state[2], state[0] * 0, state[0]]))
    out, last = rk.linear_recurrence(z(0, 4, 5), z(0, 4, 5))
    assert last.shape == (0, 5)
    out, last = rk.linear_recurrence(z(3, 4, 0), z(3, 4, 0))
    assert last.shape == (3, 0)
    out, last = rk.linear_recurrence(z(0, 5), z(0, 5), state=state, starts=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert torch.equal(last, state)
    out, last = rk.linear_recurrence(z(8, 5), z(8, 5), starts=torch.zeros(1, dtype=torch.int32, device=DEV))
    assert last.shape == (0, 5)
    dg, dx, ds = rk.linear_recurrence_backward(z(3, 0, 5), z(3, 0, 5), z(3, 0, 5), z(3, 0, 5), dstate_out=state)
    assert torch.equal(ds, state)
    dg, dx, ds = rk.linear_recurrence_backward(z(3, 0, 5), z(3, 0, 5), z(3, 0, 5), z(3, 0, 5))
    assert not ds.any()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kind,blend", [("sigmoid", True), ("log", False), ("value", True), ("log", True)])
def test_autograd(packed, kind, blend):
    """torch's autograd through the call, against the formula and against differences in 64 bits."""
    rk = _rk()
    g = gen(21)
    shape, n = ((90, 6), 4) if packed else ((2, 45, 6), 2)
    starts = torch.tensor([0, 30, 30, 80, 90], dtype=torch.int32) if packed else None
    gate, x, state = gates(g, shape, kind, F32), torch.randn(shape, generator=g), torch.randn(n, 6, generator=g)
    wo, wl = torch.randn(shape, generator=g), torch.randn(n, 6, generator=g)
    leaves = [t.clone().to(DEV).requires_grad_() for t in (gate, x, state)]
    out, last = rk.linear_recurrence(leaves[0], leaves[1], state=leaves[2], kind=kind, blend=blend,
                                     starts=None if starts is None else starts.to(DEV))
    loss = (out * wo.to(DEV)).sum() + (last * wl.to(DEV)).sum()
    grads = torch.autograd.grad(loss, leaves)
    st = None if starts is None else starts.numpy()
    wants, errs = ref.backward(np64(gate), np64(x), np64(out), np64(wo), kind, blend, st, np64(state), np64(wl))
    for v, w, e in zip(grads, wants, errs):
        near(v, w, e)

    def value(a, b, c):
        o, l, _, _ = ref.forward(a, b, kind, blend, st, c)
        return (o * np64(wo)).sum() + (l * np64(wl)).sum()

    base = [np64(gate), np64(x), np64(state)]
    rng = np.random.default_rng(1)
    for i, grad in enumerate(grads):
        way = rng.standard_normal(base[i].shape)
        step = [[b + s * 1e-6 * way if j == i else b for j, b in enumerate(base)] for s in (1, -1)]
        slope = (value(*step[0]) - value(*step[1])) / 2e-6
        # the difference is off by 1e-12 of third derivatives and by 2^-52 / 1e-6 of the value's terms, the
        # gradient by float32's rounding of h and its own
        size = (np.abs(way) * np.abs(np64(grad))).sum()
        assert abs((np64(grad) * way).sum() - slope) <= 1e-4 * size + 1e-6


def test_autograd_of_parts():
    """Only what requires a gradient gets one; shared and broadcast inputs sum theirs."""
    rk = _rk()
    g = gen(4)
    gate = gates(g, (1, 50, 12), "sigmoid", F32).to(DEV).requires_grad_()
    x = torch.randn(3, 50, 12, generator=g).to(DEV)
    out, last = rk.linear_recurrence(gate.expand(3, 50, 12), x, kind="sigmoid")
    out.sum().backward()
    wants, errs = ref.backward(np64(gate.expand(3, 50, 12)), np64(x), np64(out), np.ones(x.shape), "sigmoid", False)
    near(gate.grad, wants[0].sum(0, keepdims=True), errs[0].sum(0, keepdims=True) + 2.0 ** -22 * np.abs(wants[0]).sum(0, keepdims=True))
    both = torch.randn(3, 50, 12, generator=g).to(DEV).requires_grad_()      # gate and input at once
    out, last = rk.linear_recurrence(both, both, kind="sigmoid", blend=True)
    last.sum().backward()
    wants, errs = ref.backward(np64(both), np64(both), np64(out), np.zeros(x.shape), "sigmoid", True, dlast=np.ones((3, 12)))
    near(both.grad, wants[0] + wants[1], errs[0] + errs[1] + 2.0 ** -22 * np.abs(wants[0] + wants[1]))
    with torch.no_grad():
        out, _ = rk.linear_recurrence(both, both, kind="sigmoid")
    assert not out.requires_grad
    for extra in (dict(out=torch.empty_like(x)), dict(state_out=torch.empty(3, 12, device=DEV)),
                  dict(state=torch.zeros(3, 12, device=DEV), sources=torch.zeros(3, dtype=torch.int32, device=DEV)),
                  dict(stream=torch.cuda.current_stream())):
        with pytest.raises(ValueError, match="no gradient"):
            rk.linear_recurrence(both, both, **extra)
    out, _ = rk.linear_recurrence(both, both, kind="sigmoid")
    with pytest.raises(RuntimeError):
        (first,) = torch.autograd.grad(out.sum(), both, create_graph=True)
        torch.autograd.grad(first.sum(), both)


def test_tangents_are_refused():
    """Forward derivatives: refused, with and without gradients recorded, and where copy_blocks would leave them behind."""
    from torch.autograd import forward_ad
    rk = _rk()
    x, state = torch.rand(2, 30, 8, generator=gen(2)).to(DEV), torch.zeros(2, 8, device=DEV)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for call in (lambda: rk.linear_recurrence(dual, x), lambda: rk.linear_recurrence(x, dual),
                     lambda: rk.linear_recurrence(x, x, state=forward_ad.make_dual(state, state.clone())),
                     lambda: rk.linear_recurrence_backward(x, x, x, dual),
                     lambda: rk.copy_blocks([x, dual], torch.tensor([[0, 1]], dtype=torch.int32, device=DEV))):
            with pytest.raises(ValueError, match="carries a tangent"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="carries a tangent"):
                call()
        with pytest.raises(RuntimeError):                        # torch's own word, of an autograd function
            rk.linear_recurrence(dual, x.clone().requires_grad_())
        out, _ = rk.linear_recurrence(forward_ad.unpack_dual(dual).primal, x)
    assert torch.equal(out, rk.linear_recurrence(x, x)[0])


def test_gradients_are_not_dropped():
    rk = _rk()
    x = torch.rand(2, 30, 8, generator=gen(2)).to(DEV)
    leaf, pairs = x.clone().requires_grad_(), torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    for call in (lambda: rk.linear_recurrence_backward(leaf, x, x, x), lambda: rk.linear_recurrence_backward(x, x, x, leaf),
                 lambda: rk.linear_recurrence(x, x, out=leaf), lambda: rk.linear_recurrence_backward(x, x, x, x, dx=leaf),
                 lambda: rk.copy_blocks([x.clone(), leaf], pairs)):
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad():
            call()
    assert torch.equal(leaf[0], leaf[1])


def test_what_is_written_is_known_to_autograd():
    """A tensor that a graph has saved and a call then overwrites: the graph's backward pass refuses, and what is only
    read stays usable."""
    rk = _rk()
    g = gen(6)
    n = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    w, x = n(4, 6, 8).requires_grad_(), n(4, 6, 8).sigmoid()

    def overwrite(t, call):
        """call(t) writes to t, which a product with a leaf has saved."""
        leaf = torch.randn(t.shape, generator=g).to(DEV).requires_grad_()
        saved = (leaf * t).sum()
        with torch.no_grad():
            call(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.backward()

    overwrite(x.clone(), lambda t: rk.linear_recurrence(t, x, out=t))
    overwrite(n(4, 8), lambda t: rk.linear_recurrence(x, x, state=t, state_out=t))
    for name in ("dgate", "dx", "dstate"):
        overwrite(n(4, 8) if name == "dstate" else x.clone(), lambda t: rk.linear_recurrence_backward(x, x, x, x, **{name: t}))
    overwrite(n(4, 6), lambda t: rk.copy_blocks([t], i32([1, 2])))
    overwrite(n(2, 3), lambda t: rk.beam_select(n(6, 9), n(2, 3), best=t))
    overwrite(n(4, 9), lambda t: rk.softmax(t, out=t))

    table, held, ring, state = i32([3, 1], [2, 0]), i32(2, 2), i32(4, 5, 6, 7, 8, 9, 10, 11), torch.tensor([0, 8, 0, 0], device=DEV)
    outs = dict(table_out=i32([0, 0], [0, 0]), held_out=i32(0, 0), lens_out=i32(0, 0), pairs=i32([0, 0], [0, 0]))
    every = [ring, state, *outs.values()]
    before = [t._version for t in every]
    rk.fork_blocks(i32(0, 0), i32(20, 20), 16, held, table, ring, state, 12, **outs)
    assert all(t._version > b for t, b in zip(every, before)) and table._version == held._version == 0
    moves, after = torch.empty(6, 2, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int64, device=DEV)
    every = [table, moves, after]
    before = [t._version for t in every]
    ring12 = i32(*range(12))
    rk.compact_blocks(held, table, ring12, 12, pairs=moves, state_out=after)
    assert all(t._version > b for t, b in zip(every, before)) and ring12._version > 0 and held._version == 0
    every = [table, held, ring, state]
    before = [t._version for t in every]
    rk.block_tables(i32(20, 20), 16, held, table, ring, state)
    assert all(t._version > b for t, b in zip(every, before))
    outs = rk.slot_map(i32(20, 20), i32(1, 1), 16, table, held, 12, capacity=4)
    before = [t._version for t in outs]
    rk.slot_map(i32(20, 20), i32(1, 1), 16, table, held, 12, slots=outs[0], positions=outs[1], requests=outs[2], starts=outs[3])
    assert all(t._version > b for t, b in zip(outs, before))

    # inputs that are only read, a refused call's buffers, and tensors of inference mode
    out, _ = rk.linear_recurrence(w, x, kind="sigmoid")
    with torch.no_grad():
        rk.linear_recurrence(w, x)
        with pytest.raises(rk.RkError):
            rk.linear_recurrence(x, w, out=out[:, :1].expand(4, 6, 8))
    out.sum().backward()
    with torch.inference_mode():
        t = x.clone()
    with torch.no_grad():
        rk.linear_recurrence(t, x, out=t)


def test_same_bits_every_time():
    rk = _rk()
    g = gen(1)
    gate, x = gates(g, (1, 20000, 128), "sigmoid", BF16).to(DEV), torch.randn(1, 20000, 128, generator=g).to(BF16).to(DEV)
    a, la = rk.linear_recurrence(gate, x, kind="sigmoid", blend=True)
    ga = rk.linear_recurrence_backward(gate, x, a, x, kind="sigmoid", blend=True)
    for _ in range(10):
        b, lb = rk.linear_recurrence(gate, x, kind="sigmoid", blend=True)
        assert torch.equal(a, b) and torch.equal(la, lb)
        for u, v in zip(ga, rk.linear_recurrence_backward(gate, x, a, x, kind="sigmoid", blend=True)):
            assert torch.equal(u, v)


def test_streams_and_captures():
    """Calls on two streams at once, and two captured graphs, each with its own workspace, replayed in turn."""
    rk = _rk()
    g = gen(9)
    ins = [(gates(g, (2, 3000, 64), "sigmoid", F32).to(DEV), torch.randn(2, 3000, 64, generator=g).to(DEV)) for _ in range(2)]
    want = [rk.linear_recurrence(a, x, kind="sigmoid")[0].clone() for a, x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [rk.linear_recurrence(a, x, kind="sigmoid", stream=s)[0] for s, (a, x) in zip(streams, ins)]
        torch.cuda.synchronize()
        for o, w in zip(got, want):
            assert torch.equal(o, w)
    graphs, outs = [], []
    n = rk.rk_linear_recurrence_workspace_size(rk.RK_F32, rk.RK_F32, 2, 3000, 64, 0)
    for a, x in ins:
        out, last, ws = torch.empty_like(x), torch.empty(2, 64, device=DEV), torch.empty(n, dtype=torch.uint8, device=DEV)
        dg, dx, ds = torch.empty_like(x), torch.empty_like(x), torch.empty(2, 64, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rk.linear_recurrence(a, x, kind="sigmoid", out=out, state_out=last, workspace=ws)
            rk.linear_recurrence_backward(a, x, out, x, kind="sigmoid", dgate=dg, dx=dx, dstate=ds, workspace=ws)
        graphs.append(graph)
        outs.append((out, dg, dx, last, ds, ws))       # all that a graph uses lives as long as the graph
    wantg = [rk.linear_recurrence_backward(a, x, w, x, kind="sigmoid")[0] for (a, x), w in zip(ins, want)]
    for _ in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o, w, wg in zip(outs, want, wantg):
            assert torch.equal(o[0], w) and torch.equal(o[1], wg)


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
def test_blocks_help_where_they_would_wait(types):
    """Every block that looks back computes the map of the tile before its own, too: the same bits."""
    rk = _rk()
    g = gen(9)
    for shape, starts in (((1, 9000, 64), None), ((2, 1500, 130), None), ((9000, 70), torch.tensor([0, 5, 3000, 3001, 8999, 9000], dtype=torch.int32, device=DEV))):
        gate, x = gates(g, shape, "sigmoid", types[1]).to(DEV), torch.randn(shape, generator=g).to(types[0]).to(DEV)
        n = shape[0] if starts is None else 5
        state = torch.randn(n, shape[-1], generator=g).to(DEV)
        call = lambda: rk.linear_recurrence(gate, x, state=state, kind="sigmoid", blend=True, starts=starts)  # noqa: E731
        out, last = call()
        back = lambda: rk.linear_recurrence_backward(gate, x, out, x, state=state, dstate_out=state, kind="sigmoid", blend=True, starts=starts)  # noqa: E731
        want = (out, last, *back())
        rk.rk_debug_force_wait_timeout(0)
        try:
            got = (*call(), *back())
            torch.cuda.synchronize()
        finally:
            rk.rk_debug_force_wait_timeout(-1)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert rk.rk_stream_timeouts(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("channels", [6, 64, 130])
@pytest.mark.parametrize("cuts", [None, [0, 5, 3000, 3001, 8999, 9000], [0, 200, 200, 520, 4000, 4000, 4001, 9000], [100, 700, 8500],
                                  list(range(0, 9001, 300))])
def test_blocks_help_in_place(types, channels, cuts):
    """The same with the last states in the first ones' place, and what is written in an input's place: a tile's inputs
    and first states are read again, by its own block and by another one, and are what they were."""
    rk = _rk()
    g = gen(channels)
    shape, n = ((2, 4500, channels), 2) if cuts is None else ((9000, channels), len(cuts) - 1)
    starts = None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device=DEV)
    gate, x = gates(g, shape, "sigmoid", types[1]).to(DEV), torch.randn(shape, generator=g).to(types[0]).to(DEV)
    dout, state = torch.randn(shape, generator=g).to(types[0]).to(DEV), torch.randn(n, channels, generator=g).to(DEV)
    how = dict(kind="sigmoid", blend=True, starts=starts)
    want, want_last = rk.linear_recurrence(gate, x, state=state, out=x.clone(), **how)
    wants = rk.linear_recurrence_backward(gate, x, want, dout, state=state, dstate_out=state, dgate=gate.clone(), dx=dout.clone(), **how)
    for force in (-1, 0, 0, 0):
        rk.rk_debug_force_wait_timeout(force)
        try:
            s, s2, o, other = state.clone(), state.clone(), x.clone(), gate.clone()
            out, last = rk.linear_recurrence(gate, o, state=s, out=o, state_out=s, **how)
            assert out is o and last is s
            rk.linear_recurrence(other, x, state=s2, out=other, state_out=s2, **how)
            dg, dx = gate.clone(), dout.clone()
            got = rk.linear_recurrence_backward(dg, x, want, dx, state=state, dstate_out=state, dgate=dg, dx=dx, **how)
            torch.cuda.synchronize()
        finally:
            rk.rk_debug_force_wait_timeout(-1)
        assert torch.equal(s, want_last) and torch.equal(s2, want_last)
        rows = slice(None) if cuts is None else slice(cuts[0], cuts[-1])
        for a, b in ((out, want), (other, want), *zip(got, wants)):
            assert torch.equal(a[rows] if a.shape == x.shape else a, b[rows] if b.shape == x.shape else b)


def test_states_in_place_in_a_captured_graph():
    """Chunk after chunk through one graph, the last states in the first ones' place: each replay starts from what the one
    before left, and keeps it apart in the workspace again."""
    rk = _rk()
    g = gen(12)
    chunks = [(gates(g, (3, 900, 70), "sigmoid", BF16).to(DEV), torch.randn(3, 900, 70, generator=g).to(BF16).to(DEV)) for _ in range(4)]
    first = torch.randn(3, 70, generator=g).to(DEV)
    want, last = [], first
    for a, v in chunks:
        out, last = rk.linear_recurrence(a, v, state=last, kind="sigmoid", blend=True)
        want.append((out, last))
    gate, x, state = chunks[0][0].clone(), chunks[0][1].clone(), first.clone()
    out = torch.empty_like(x)
    n = rk.rk_linear_recurrence_workspace_size(rk.RK_BF16, rk.RK_BF16, 3, 900, 70, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rk.linear_recurrence(gate, x, state=state, kind="sigmoid", blend=True, out=out, state_out=state, workspace=ws)
    for _ in range(2):
        state.copy_(first)
        for (a, v), (o, s) in zip(chunks, want):
            gate.copy_(a)
            x.copy_(v)
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, o) and torch.equal(state, s)


def test_no_gradients_are_recorded_in_a_capture():
    """An eager graph of the same leaves is alive; the captured backward call gives what autograd gives."""
    rk = _rk()
    g = gen(5)
    gate, x = gates(g, (3, 200, 64), "sigmoid", F32).to(DEV), torch.randn(3, 200, 64, generator=g).to(DEV)
    leaves = [gate.clone().requires_grad_(), x.clone().requires_grad_()]
    eager, _ = rk.linear_recurrence(*leaves, kind="sigmoid", blend=True)
    n = rk.rk_linear_recurrence_workspace_size(rk.RK_F32, rk.RK_F32, 3, 200, 64, 0)
    out, last, ws = torch.empty_like(x), torch.empty(3, 64, device=DEV), torch.empty(max(n, 8), dtype=torch.uint8, device=DEV)
    dg, dx, ds = torch.empty_like(x), torch.empty_like(x), torch.empty(3, 64, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            rk.linear_recurrence(*leaves, kind="sigmoid", blend=True)
        with torch.no_grad():
            rk.linear_recurrence(*leaves, kind="sigmoid", blend=True, out=out, state_out=last, workspace=ws)
            rk.linear_recurrence_backward(*leaves, out, x, kind="sigmoid", blend=True, dgate=dg, dx=dx, dstate=ds, workspace=ws)
    want = torch.autograd.grad(eager, leaves, x)
    for _ in range(3):
        for t in (out, dg, dx):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(dg, want[0]) and torch.equal(dx, want[1])


def test_launch_failures_and_small_workspaces():
    rk = _rk()
    x = torch.randn(1, 9000, 64, generator=gen(1)).to(DEV)
    out, last = torch.full_like(x, 7.0), torch.full((1, 64), 7.0, device=DEV)
    rk.rk_debug_fail_launches(1)
    with pytest.raises(rk.RkError, match="HIP"):
        rk.linear_recurrence(x, x, kind="sigmoid", out=out, state_out=last)
    with pytest.raises(rk.RkError, match="invalid"):
        rk.linear_recurrence(x, x, kind="sigmoid", out=out, state_out=last, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (last == 7.0).all()


def test_tensors_are_checked():
    rk = _rk()
    z = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    x = z(2, 9, 8)
    i32 = z(3, dtype=torch.int32)
    bad = [
        dict(gate=z(2, 9, 7)), dict(gate=z(2, 9, 8, dtype=torch.float64)), dict(x=z(2, 9, 8, dtype=torch.int32)),
        dict(x=z(2, 8, 9).transpose(1, 2)), dict(x=x.cpu()), dict(gate=x.cpu()), dict(state=z(3, 8)), dict(state=z(2, 8, dtype=BF16)),
        dict(state=z(8, 2).t()), dict(kind="exp"), dict(starts=i32), dict(out=z(2, 9, 8, dtype=BF16)), dict(out=z(2, 9, 9)),
        dict(state_out=z(2, 9)), dict(sources=i32, state=z(2, 8)), dict(gate=z(9, 8), x=z(9, 8)),
        dict(gate=z(9, 8), x=z(9, 8), starts=z(3, dtype=torch.int64)), dict(gate=z(9, 8), x=z(9, 8), starts=z(0, dtype=torch.int32)),
        dict(workspace=z(64, 64).t()),
    ]
    for b in bad:
        with pytest.raises(ValueError):
            rk.linear_recurrence(**{**dict(gate=x, x=x), **b})
    with pytest.raises(TypeError):
        rk.linear_recurrence(x, x, state=x, out=3)
    for b, code in ((dict(sources=i32[:2]), "invalid"), (dict(gate=z(2, 9, 8, dtype=BF16)), "unsupported"),
                    (dict(out=x[:, :1].expand(2, 9, 8)), "invalid")):
        with pytest.raises(rk.RkError, match=code):
            rk.linear_recurrence(**{**dict(gate=x, x=x), **b})
    h = z(2, 9, 8)
    for b in (dict(dgate=h), dict(dx=h), dict(dx=x, dgate=x), dict(dstate=h[0, :2])):
        with pytest.raises(rk.RkError, match="invalid"):
            rk.linear_recurrence_backward(x, x, h, z(2, 9, 8), **b)


def test_tokens_past_2_31_elements():
    """Offsets of tokens pass 32 bits: only the last ones are looked at."""
    rk = _rk()
    rows, ch = 70001, 40000                   # 2.8e9 elements of 2 bytes
    gate = torch.zeros(1, rows, ch, dtype=BF16, device=DEV)
    x = torch.zeros(1, rows, ch, dtype=BF16, device=DEV)
    x[0, -600:] = torch.randn(600, ch, generator=gen(2)).to(BF16).to(DEV)
    out, last = rk.linear_recurrence(gate, x, kind="sigmoid", out=x)
    want, _ = rk.linear_recurrence(gate[:, -600:], torch.randn(600, ch, generator=gen(2)).to(BF16).to(DEV)[None], kind="sigmoid")
    assert not out[0, 1000].any() and not out[0, -601].any()
    a, b = out[0, -600:].double(), want[0].double()
    # The tiles lie otherwise, so each side has a rounding of its own: half a step of bfloat16 (2^-8 of it), and in
    # float32, with a = 1/2, at most 2 * 16 * 2^-24 of sum |x| / 2^k <= 2 max |x| < 12.
    assert ((a - b).abs() <= 2 * 2.0 ** -8 * (b.abs() + (a - b).abs()) + 2 * 32 * 2.0 ** -24 * 12).all()


@pytest.mark.parametrize("channels", [1, 3, 4, 5, 1023, 1024, 1025, 2050])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F16, F32)])
def test_single_tokens(channels, types):
    """In place of the inputs, whose last channels no whole vector holds, and beside them; every kind."""
    rk = _rk()
    g = gen(channels)
    for kind, blend in (("sigmoid", True), ("log", False), ("log", True), ("value", False)):
        gate, x = gates(g, (37, 1, channels), kind, types[1]), torch.randn(37, 1, channels, generator=g).to(types[0])
        state = torch.randn(37, channels, generator=g)
        check(gate, x, kind, blend, state=state, backward=False)
        want, want_last, err, err_last = ref.forward(np64(gate), np64(x), kind, blend, state=np64(state))
        there, s = x.to(DEV), state.to(DEV)
        out, last = rk.linear_recurrence(gate.to(DEV), there, state=s, kind=kind, blend=blend, out=there, state_out=s)
        assert out is there and last is s
        near(out, want, err)
        near(last, want_last, err_last)


def test_more_single_tokens_than_a_launch_has_blocks():
    """17 million rows of 1024 channels go through tiles; float16 of one bit, so that a row of each is enough to look at."""
    rk = _rk()
    rows, channels = 0xffffff + 9, 1024
    x = torch.ones(1, 1, channels, dtype=F16, device=DEV).expand(rows, 1, channels)
    gate = torch.full((1, 1, channels), 0.5, dtype=F16, device=DEV).expand(rows, 1, channels)
    out = torch.empty(rows, 1, channels, dtype=F16, device=DEV)
    last = torch.empty(rows, channels, device=DEV)
    sources = torch.arange(rows, dtype=torch.int32, device=DEV) % 2
    rk.linear_recurrence(gate, x, state=torch.tensor([[2.0], [4.0]], device=DEV).expand(2, channels).contiguous(), sources=sources, out=out,
                         state_out=last)
    for at in (0, 1, 2, 0xfffffe, 0xffffff, 0x1000000, rows - 1):
        assert (out[at] == 2 + at % 2).all() and (last[at] == 2 + at % 2).all()
    assert int((out[:, 0, 5] == 2).sum()) == (rows + 1) // 2 and int((last[:, 1023] == 3).sum()) == rows // 2
