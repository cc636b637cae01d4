"""CPU tests of the gated linear recurrence: refusals, workspace sizes, and the
plain forms the GPU tests compare with."""
import numpy as np
import pytest
import torch

from tests import recur_ref as ref

FAKE = 0x1000000        # never dereferenced: every call below fails validation
MB = 1 << 20


def _rk():
    import reduction_primitives_amd as rk
    rk.load()
    return rk


BASE = dict(xd=0, gd=0, kind=2, blend=1, gate=(FAKE, 5000, 50), x=(FAKE + MB, 5000, 50), state=FAKE + 2 * MB, n_states=3,
            sources=None, starts=None, n_seq=3, tokens=100, ch=50, out=(FAKE + 3 * MB, 5000, 50), last=FAKE + 4 * MB,
            ws=FAKE + 8 * MB, ws_bytes=8 * MB)


def forward(**args):
    a = {**BASE, **args}
    return _rk().rk_linear_recurrence(a["xd"], a["gd"], a["kind"], a["blend"], a["gate"], a["x"], a["state"], a["n_states"],
                                      a["sources"], a["starts"], a["n_seq"], a["tokens"], a["ch"], a["out"], a["last"], a["ws"],
                                      a["ws_bytes"], None)


BACK = dict(dout=(FAKE + 5 * MB, 5000, 50), dlast=FAKE + 6 * MB, dgate=(FAKE + 7 * MB, 5000, 50), dx=(FAKE + 16 * MB, 5000, 50),
            dstate=FAKE + 17 * MB)


def backward(**args):
    a = {**BASE, **BACK, **args}
    return _rk().rk_linear_recurrence_backward(a["xd"], a["gd"], a["kind"], a["blend"], a["gate"], a["x"], a["out"], a["dout"],
                                               a["state"], a["dlast"], a["starts"], a["n_seq"], a["tokens"], a["ch"], a["dgate"],
                                               a["dx"], a["dstate"], a["ws"], a["ws_bytes"], None)


SHARED = [
    (dict(xd=9), 1), (dict(gd=-1), 1), (dict(xd=3, gd=3), 2), (dict(gd=1), 2), (dict(xd=1, gd=2), 2), (dict(kind=3), 1), (dict(kind=-1), 1),
    (dict(blend=2), 1), (dict(n_seq=-1), 1), (dict(tokens=-1), 1), (dict(ch=-1), 1), (dict(n_seq=1 << 31), 2), (dict(tokens=1 << 31), 2),
    (dict(ch=1 << 31), 2), (dict(gate=None), 1), (dict(x=None), 1), (dict(gate=(None, 5000, 50)), 1), (dict(x=(None, 5000, 50)), 1),
    (dict(gate=(FAKE + 2, 5000, 50)), 1), (dict(x=(FAKE + 1, 5000, 50)), 1), (dict(gate=(FAKE, -1, 50)), 1), (dict(x=(FAKE, 5000, 1 << 60)), 1),
    (dict(state=FAKE + 2), 1), (dict(starts=FAKE + 2), 1),
]


@pytest.mark.parametrize("args,code", SHARED + [
    (dict(out=None), 1), (dict(out=(None, 5000, 50)), 1), (dict(last=None), 1), (dict(last=FAKE + 2), 1), (dict(sources=FAKE + 2), 1),
    (dict(sources=FAKE + 9 * MB, state=None), 1), (dict(n_states=-1), 1),
    (dict(out=(FAKE + 3 * MB, 5000, 49)), 1), (dict(out=(FAKE + 3 * MB, 4999, 50)), 1), (dict(out=(FAKE + 3 * MB, 0, 50)), 1),   # folded
    (dict(out=(FAKE + 200, 5000, 50)), 1), (dict(out=(FAKE + MB + 4, 5000, 50)), 1),                # neither in place nor beside it
    (dict(out=(FAKE, 5000, 50), xd=1), 1),                                                         # in place of a wider type
    (dict(last=FAKE), 1), (dict(last=FAKE + 2 * MB + 4), 1), (dict(last=FAKE + 3 * MB), 1),
    (dict(last=FAKE + 2 * MB, sources=FAKE + 9 * MB), 1),                                          # in place, but by sources
    (dict(out=(FAKE + 2 * MB, 5000, 50)), 1),
    (dict(tokens=1000, gate=(FAKE, 50000, 50), x=(FAKE + MB, 50000, 50), out=(FAKE + 3 * MB, 50000, 50), ws=None), 1),
])
def test_forward_refusals(args, code):
    assert forward(**args) == code


@pytest.mark.parametrize("args,code", SHARED + [
    (dict(out=None), 1), (dict(dout=None), 1), (dict(dgate=None), 1), (dict(dx=None), 1), (dict(dx=(None, 5000, 50)), 1),
    (dict(dlast=FAKE + 1), 1), (dict(dstate=FAKE + 1), 1), (dict(dgate=(FAKE + 7 * MB, 10, 50)), 1),
    (dict(dgate=(FAKE + 3 * MB, 5000, 50)), 1), (dict(dx=(FAKE + 3 * MB, 5000, 50)), 1),           # the outputs of the forward pass
    (dict(dgate=(FAKE, 5000, 50), dx=(FAKE, 5000, 50)), 1), (dict(dx=(FAKE + 7 * MB + 4, 5000, 50)), 1),
    (dict(dstate=FAKE + 6 * MB), 1), (dict(dstate=FAKE + 2 * MB), 1), (dict(dstate=FAKE + 16 * MB), 1),
])
def test_backward_refusals(args, code):
    assert backward(**args) == code


def long(**args):
    """Extents that need a workspace, tensors apart."""
    rows = lambda i: (FAKE + i * 64 * MB, 50 * 20000, 50)  # noqa: E731
    return dict(tokens=20000, gate=rows(1), x=rows(2), out=rows(3), dout=rows(4), dgate=rows(5), dx=rows(6), ws=FAKE + 1024 * MB,
                ws_bytes=64 * MB, **args)


@pytest.mark.parametrize("args", [dict(ws=None), dict(ws=FAKE + 1024 * MB + 4), dict(ws_bytes=1000), dict(ws=FAKE + 64 * MB),
                                  dict(ws=FAKE + 3 * 64 * MB), dict(ws=FAKE + 2 * MB), dict(ws=FAKE + 4 * MB)])
def test_workspaces(args):
    assert forward(**{**long(), **args}) == 1
    if args != dict(ws=FAKE + 4 * MB):
        assert backward(**{**long(), **args}) == 1


def test_workspace_sizes():
    size = _rk().rk_linear_recurrence_workspace_size
    assert size(0, 0, 64, 1, 2048, 0) == 0 and size(0, 0, 1, 0, 5, 0) == 0 and size(0, 0, 0, 9, 5, 0) == 0
    assert size(9, 0, 1, 100000, 64, 0) == 0 and size(1, 2, 1, 100000, 64, 0) == 0 and size(0, 0, -1, 5, 5, 0) == 0
    assert size(1, 1, 1, 100000, 64, 0) % 256 == 0 and size(1, 1, 1, 100000, 64, 0) >= 782 * 1024
    assert size(0, 0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 0) == 0


def test_first_states_are_kept_where_the_last_ones_take_their_place():
    """A tile may be computed late, or once more by a block that helps, and reads its sequences' first states again then:
    the workspace has room for them beside the records, and a call that needs it asks for it."""
    size = _rk().rk_linear_recurrence_workspace_size
    records = (3 * 157 + 3) * 1024                # 157 tiles of 128 tokens of each sequence
    assert size(1, 1, 3, 20000, 50, 0) >= records + 3 * 50 * 4
    assert size(1, 1, 1000, 20000, 50, 1) >= (157 + 3) * 1024 + 1000 * 50 * 4
    inside = dict(last=BASE["state"], ws_bytes=records)
    assert forward(**{**long(), **inside}) == 1
    assert forward(**{**long(), **inside, "ws_bytes": records + 3 * 50 * 4 - 1}) == 1
    assert size(0, 0, 1 << 30, 20000, 1 << 20, 1) == 0       # (more states than a call takes)


def test_calls_of_nothing():
    assert forward(n_seq=0) == 0 and forward(ch=0) == 0 and backward(n_seq=0) == 0
    assert backward(tokens=0, dstate=None) == 0


def test_tensor_refusals():
    """What the Python calls refuse before the library sees it (CPU tensors
    among it: there is no fallback)."""
    rk = _rk()
    x = torch.zeros(2, 3, 4)
    for call in (lambda: rk.linear_recurrence(x, x), lambda: rk.linear_recurrence_backward(x, x, x, x)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
    with pytest.raises(ValueError, match="kind"):
        rk.linear_recurrence(x, x, kind="tanh")
    with pytest.raises(ValueError, match="no gradient"):
        rk.linear_recurrence(x.requires_grad_(), x, out=x)


def test_tangents_are_not_dropped():
    """No call has a forward derivative: its module says so before it looks at devices, under no_grad, too."""
    from torch.autograd import forward_ad
    rk = _rk()
    calls = rk.linear_recurrence.__globals__["_calls"]
    x, s = torch.zeros(2, 3, 4), torch.zeros(2, 4)
    with forward_ad.dual_level():
        def each(names, run):
            """run(arguments, one of them with a tangent at a time)"""
            base = {n: torch.zeros_like(s) if n in ("state", "dstate_out", "logits", "scores") else torch.zeros_like(x) for n in names}
            for n in names:
                dual = forward_ad.make_dual(base[n], torch.ones_like(base[n]))
                for grad in (True, False):
                    with torch.set_grad_enabled(grad), pytest.raises(ValueError, match=n + " carries a tangent"):
                        run({**base, n: dual})
            with pytest.raises(ValueError, match="not on a GPU"):       # (refused for that alone)
                run(base)

        each(["gate", "x", "state"], lambda a: calls.linear_recurrence(0, a["gate"], a["x"], a["state"], 0, 0, None, None, x, s, None))
        each(["gate", "x", "out", "dout", "state", "dstate_out"],
             lambda a: calls.linear_recurrence_backward(0, a["gate"], a["x"], a["out"], a["dout"], a["state"], a["dstate_out"], 0, 0, None,
                                                        x, x, s, None))
        each(["logits", "scores"], lambda a: calls.beam_select(0, a["logits"], a["scores"], 1, None, 0, s, s, s, None))
        each(["x"], lambda a: calls.softmax(0, a["x"], None, x, None))


def test_gradients_are_not_dropped():
    """What requires grad, read or written, is refused where gradients are recorded and the call would leave it without."""
    rk = _rk()
    calls = rk.linear_recurrence.__globals__["_calls"]
    x = torch.zeros(2, 3, 4)
    inputs = ["gate", "x", "out", "dout", "state", "dstate_out", "dgate", "dx", "dstate"]
    for n in inputs:
        a = {i: torch.zeros(2, 4) if "state" in i else x.clone() for i in inputs}
        a[n].requires_grad_()
        back = lambda: calls.linear_recurrence_backward(  # noqa: E731
            0, a["gate"], a["x"], a["out"], a["dout"], a["state"], a["dstate_out"], 0, 0, None, a["dgate"], a["dx"], a["dstate"], None)
        forward = lambda: calls.linear_recurrence(0, a["gate"], a["x"], a["state"], 0, 0, None, None, a["out"], a["dstate"], None)  # noqa: E731
        for call, name in ((back, n), (forward, {"dstate": "state_out"}.get(n, n) if n in ("gate", "x", "state", "out", "dstate") else None)):
            if name:
                with pytest.raises(ValueError, match=name + " requires grad"):
                    call()
                with torch.no_grad(), pytest.raises(ValueError, match="not on a GPU"):
                    call()
    s = torch.zeros(2, 4)
    with pytest.raises(ValueError, match="best requires grad"):
        calls.beam_select(0, s, s, 1, None, 0, s.clone().requires_grad_(), s, s, None)


@pytest.mark.parametrize("kind", ["value", "log", "sigmoid"])
@pytest.mark.parametrize("blend", [False, True])
def test_plain_gradient_is_the_slope(kind, blend):
    """The plain backward form against differences of the plain forward one."""
    rng = np.random.default_rng(3)
    starts = [0, 4, 4, 9]
    gate, x, state = rng.standard_normal((9, 3)) * 0.5 - 0.2, rng.standard_normal((9, 3)), rng.standard_normal((3, 3))
    wo, wl = rng.standard_normal((9, 3)), rng.standard_normal((3, 3))

    def value(*v):
        out, last, _, _ = ref.forward(v[0], v[1], kind, blend, starts, v[2])
        return (out * wo).sum() + (last * wl).sum()

    base = [gate, x, state]
    out = ref.forward(gate, x, kind, blend, starts, state)[0]
    grads, _ = ref.backward(gate, x, out, wo, kind, blend, starts, state, wl)
    for i, g in enumerate(grads):
        for at in np.ndindex(g.shape):
            step = []
            for s in (1e-6, -1e-6):
                moved = [b.copy() for b in base]
                moved[i][at] += s
                step.append(value(*moved))
            assert abs((step[0] - step[1]) / 2e-6 - g[at]) < 1e-7
