"""CPU tests of the serving operators: refusals, plans, the plain forms the GPU
tests compare with, and the division by a block size."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from tests import serving_ref as ref

FAKE = 0x1000000        # never dereferenced: every call below fails validation
MB = 1 << 20


def _rk():
    import reduction_primitives_amd as rk
    rk.load()
    return rk


@pytest.mark.parametrize("args,code", [
    (dict(in_dtype=9), 1), (dict(out_dtype=-1), 1), (dict(in_dtype=3), 2), (dict(in_dtype=4), 2), (dict(out_dtype=5), 2),
    (dict(n=-1), 1), (dict(lines=-1), 1), (dict(n=1 << 31), 2), (dict(x=None), 1), (dict(x=FAKE + 2), 1),
    (dict(out=None), 1), (dict(out=FAKE + 64 * MB + 1), 1), (dict(xs=-1), 1), (dict(os=99), 1), (dict(xs=1 << 60), 1),
    (dict(temp=FAKE + 2), 1),
    (dict(out=FAKE + 400), 1),                                     # overlaps x, neither in place nor beside it
    (dict(out=FAKE, os=200), 1), (dict(out=FAKE, out_dtype=1), 1),  # in place with another stride or size
    (dict(ws=None), 1), (dict(ws=FAKE + 32 * MB + 4), 1), (dict(ws_bytes=16), 1),
    (dict(ws=FAKE), 1), (dict(ws=FAKE + 64 * MB), 1), (dict(temp=FAKE + 64 * MB), 1),
])
def test_softmax_refusals(args, code):
    a = dict(in_dtype=0, out_dtype=0, x=FAKE, n=100000, lines=4, xs=100000, temp=None, out=FAKE + 64 * MB, os=100000,
             ws=FAKE + 32 * MB, ws_bytes=MB)
    if "os" in args and args["os"] in (99, 200):
        a.update(n=100, xs=100)
    a.update(args)
    rk = _rk()
    assert rk.rk_softmax(a["in_dtype"], a["out_dtype"], a["x"], a["n"], a["lines"], a["xs"], a["temp"], a["out"], a["os"],
                         a["ws"], a["ws_bytes"], None) == code


def test_softmax_of_nothing():
    rk = _rk()
    assert rk.rk_softmax(0, 0, None, 0, 5, 0, None, None, 0, None, 0, None) == 0
    assert rk.rk_softmax(0, 0, None, 5, 0, 5, None, None, 5, None, 0, None) == 0


@pytest.mark.parametrize("args,code", [
    (dict(dtype=7), 1), (dict(dtype=3), 2), (dict(dtype=4), 2), (dict(token=1), 2), (dict(token=9), 1), (dict(vocab=0), 1),
    (dict(vocab=1 << 31), 2), (dict(req=-1), 1), (dict(drafts=-1), 1), (dict(max_draft=-1), 1), (dict(max_draft=1 << 25), 1),
    (dict(starts=None, drafts=7), 1),                              # 2 requests of 4 drafts are 8
    (dict(p=None), 1), (dict(r=None), 1), (dict(u=None), 1), (dict(drafted=None), 1), (dict(tokens=None), 1),
    (dict(accepted=None), 1), (dict(ps=-1), 1), (dict(qs=-1), 1), (dict(p=FAKE + 1), 1), (dict(q=FAKE + 64 * MB + 2), 1),
    (dict(drafted=FAKE + 130 * MB + 4), 1), (dict(tokens=FAKE + 160 * MB + 4), 1), (dict(u=FAKE + 140 * MB + 1), 1),
    (dict(ws=None), 1), (dict(ws=FAKE + 192 * MB + 4), 1), (dict(ws_bytes=8), 1),
    (dict(tokens=FAKE + 130 * MB), 1), (dict(accepted=FAKE + 150 * MB), 1), (dict(accepted=FAKE + 160 * MB + 8), 1),
    (dict(ws=FAKE), 1),
])
def test_draft_verify_refusals(args, code):
    a = dict(dtype=0, token=5, p=FAKE, ps=1000, q=FAKE + 64 * MB, qs=1000, vocab=1000, req=2, drafts=8, max_draft=4,
             starts=FAKE + 120 * MB, drafted=FAKE + 130 * MB, u=FAKE + 140 * MB, r=FAKE + 150 * MB, tokens=FAKE + 160 * MB,
             accepted=FAKE + 170 * MB, ws=FAKE + 192 * MB, ws_bytes=MB)
    a.update(args)
    rk = _rk()
    assert rk.rk_draft_verify(a["dtype"], a["token"], a["p"], a["ps"], a["q"], a["qs"], a["vocab"], a["req"], a["drafts"],
                              a["max_draft"], a["starts"], a["drafted"], a["u"], a["r"], a["tokens"], a["accepted"], a["ws"],
                              a["ws_bytes"], None) == code


@pytest.mark.parametrize("args,code", [
    (dict(req=-1), 1), (dict(block=0), 1), (dict(max_blocks=-1), 1), (dict(size=0), 1), (dict(size=1 << 31), 2),
    (dict(ts=3), 1), (dict(ts=-1), 1), (dict(lens=None), 1), (dict(held=None), 1), (dict(held_out=None), 1),
    (dict(table=None), 1), (dict(ring=None), 1), (dict(state=None), 1), (dict(state_out=None), 1), (dict(ws=None), 1),
    (dict(ws_bytes=40), 1), (dict(lens=FAKE + 2), 1), (dict(ring=FAKE + 4 * MB + 1), 1), (dict(state=FAKE + 5 * MB + 4), 1),
    (dict(ws=FAKE + 7 * MB + 4), 1),
    (dict(held_out=FAKE), 1),                                      # lens
    (dict(held_out=FAKE + MB + 4), 1),                             # held, but not held itself
    (dict(ring=FAKE + 3 * MB + 4), 1),                             # table
    (dict(state_out=FAKE + 5 * MB + 8), 1), (dict(state_out=FAKE + 4 * MB), 1), (dict(ws=FAKE + 3 * MB), 1),
])
def test_block_tables_refusals(args, code):
    a = dict(lens=FAKE, req=5, block=16, held=FAKE + MB, held_out=FAKE + 2 * MB, table=FAKE + 3 * MB, ts=4, max_blocks=4,
             ring=FAKE + 4 * MB, size=100, state=FAKE + 5 * MB, state_out=FAKE + 6 * MB, ws=FAKE + 7 * MB, ws_bytes=MB)
    a.update(args)
    rk = _rk()
    assert rk.rk_block_tables(a["lens"], a["req"], a["block"], a["held"], a["held_out"], a["table"], a["ts"], a["max_blocks"],
                              a["ring"], a["size"], a["state"], a["state_out"], a["ws"], a["ws_bytes"], None) == code


@pytest.mark.parametrize("args,code", [
    (dict(req=-1), 1), (dict(block=0), 1), (dict(max_blocks=-1), 1), (dict(n_blocks=-1), 1), (dict(capacity=-1), 1),
    (dict(dtype=8), 1), (dict(dtype=0), 2), (dict(capacity=1 << 31), 2), (dict(dtype=4, n_blocks=(1 << 27) + 1), 2),
    (dict(ts=3), 1), (dict(lens=None), 1), (dict(fresh=None), 1), (dict(table=None), 1), (dict(held=None), 1),
    (dict(slots=None), 1), (dict(starts=None), 1), (dict(slots=FAKE + 4 * MB + 4), 1), (dict(positions=FAKE + 5 * MB + 2), 1),
    (dict(slots=FAKE), 1), (dict(positions=FAKE + 4 * MB), 1), (dict(requests=FAKE + 5 * MB), 1), (dict(starts=FAKE + 2 * MB), 1),
])
def test_slot_map_refusals(args, code):
    a = dict(lens=FAKE, fresh=FAKE + MB, req=5, block=16, table=FAKE + 2 * MB, ts=4, max_blocks=4, held=FAKE + 3 * MB,
             n_blocks=100, dtype=5, capacity=64, slots=FAKE + 4 * MB, positions=FAKE + 5 * MB, requests=FAKE + 6 * MB,
             starts=FAKE + 7 * MB)
    a.update(args)
    rk = _rk()
    assert rk.rk_slot_map(a["lens"], a["fresh"], a["req"], a["block"], a["table"], a["ts"], a["max_blocks"], a["held"],
                          a["n_blocks"], a["dtype"], a["capacity"], a["slots"], a["positions"], a["requests"], a["starts"],
                          None) == code


def test_tensor_refusals():
    """What the Python calls refuse before the library sees it (CPU tensors
    among it: there is no fallback)."""
    rk = _rk()
    x = torch.zeros(2, 8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64)  # noqa: E731
    for call in (lambda: rk.softmax(x),
                 lambda: rk.draft_verify(torch.zeros(6, 8), None, i32(4), torch.zeros(4), torch.zeros(2)),
                 lambda: rk.block_tables(i32(3), 16, i32(3), i32(3, 4), i32(9), i64(4)),
                 lambda: rk.slot_map(i32(3), i32(3), 16, i32(3, 4), i32(3), 10, capacity=5)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_plans():
    rk = _rk()
    assert rk.rk_plan_softmax(0, 0, 0, 5).kernel == rk.RK_KERNEL_NONE
    for n in (1, 2048, 2049, 8192, 8193, 16384, 16385, 32768, 32769, 131072, 200001):
        p = rk.rk_plan_softmax(1, 0, n, 7)
        assert p.split * p.tile_outputs >= n > (p.split - 1) * p.tile_outputs
        assert p.workspace_bytes % 256 == 0
        line = n <= 32768
        assert p.kernel == (rk.RK_KERNEL_SOFTMAX_LINE if line else rk.RK_KERNEL_SOFTMAX_SPLIT)
        assert p.launches == (1 if line else 2) and (p.workspace_bytes == 0) == line
    p = rk.rk_plan_softmax(0, 0, 10 ** 8, 3)
    assert p.launches == 3 and p.workspace_bytes >= 3 * (p.split + 1) * 12
    for n, lines in ((2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1), (10 ** 9, 10 ** 5)):   # beyond the threads of a launch
        with pytest.raises(rk.RkError, match="unsupported"):
            rk.rk_plan_softmax(0, 0, n, lines)
    assert rk.rk_plan_softmax(0, 0, 2 ** 31 - 1, 3).grid == 3 * -(-(2 ** 31 - 1) // 8192)
    with pytest.raises(rk.RkError, match="unsupported"):
        rk.rk_plan_draft_verify(0, 131072, 2 ** 30, 256)
    p = rk.rk_plan_draft_verify(0, 131072, 64, 256)
    assert p.kernel == rk.RK_KERNEL_DRAFT_VERIFY and p.launches == 1
    assert p.workspace_bytes >= 64 * -(-131072 // p.tile_outputs) * 8
    assert rk.rk_plan_draft_verify(0, 131072, 5000, 256).split == 1         # a block a request fills the chip
    assert rk.rk_plan_draft_verify(0, 131072, 256, 256).launches == 2       # many blocks: finished apart
    assert rk.rk_plan_draft_verify(0, 32000, 257, 256).launches == 2        # many requests
    assert rk.rk_plan_draft_verify(0, 32000, 256, 256).launches == 1
    assert rk.rk_plan_draft_verify(0, 100, 1, 256).split == 1
    prev = rk.rk_debug_set_fused_finish(0)
    try:
        assert rk.rk_plan_draft_verify(0, 131072, 64, 256).launches == 2
    finally:
        rk.rk_debug_set_fused_finish(prev)
    assert rk.rk_block_tables_workspace_size(-1) == 0
    assert rk.rk_block_tables_workspace_size(0) > 0


def test_softmax_plans_name_the_loads():
    """Elements of a load in the first launch: 16 bytes of the wider type where
    it writes too, of the input where it only reads."""
    rk = _rk()
    f32, f16 = rk.RK_F32, rk.RK_F16
    for n, loads in ((1000, {(f32, f32): 4, (f16, f32): 4, (f32, f16): 4, (f16, f16): 8}),
                     (50000, {(f32, f32): 4, (f16, f32): 8, (f32, f16): 4, (f16, f16): 8})):
        for (din, dout), vec in loads.items():
            assert rk.rk_plan_softmax(din, dout, n, 3).vec == vec


def test_plain_forms():
    """The plain forms themselves, on values worked out by hand."""
    p = np.array([[0.5, 0.25, 0.25, 0.0]] * 3)
    q = np.array([[0.25, 0.75, 0.0, 0.0], [0.0, 0.0, 1.0, 0.0]])
    # token 0: 0.9 * 0.25 < 0.5 kept; token 2: 0.5 * 1 < 0.25 no; what is left: (0.5, 0.25, 0, 0)
    t, k = ref.draft_verify(p, q, [0, 2], [0.9, 0.5], [0.7], [0, 2], 2)
    assert t.tolist() == [[0, 1, -1]] and k.tolist() == [1]
    t, k = ref.draft_verify(p, q, [0, 2], [0.9, 0.2], [0.74], [0, 2], 2)    # both kept: p, 0.5 <= 0.74 < 0.75
    assert t.tolist() == [[0, 2, 1]] and k.tolist() == [2]
    held, table, ring, state = ref.block_tables([33, 0], 16, [1, 2], np.array([[7, -1, -1], [8, 9, -1]]),
                                                np.array([-1, 4, -1, -1]), [1, 2])
    assert held.tolist() == [3, 0] and table[0].tolist() == [7, 4, 8] and state.tolist() == [3, 4, 0, 0]
    assert ring.tolist() == [-1, 4, 8, 9]
    s = ref.slot_map([3, 17], [3, 2], 16, np.array([[5, 0], [2, 1]]), [1, 2], 10, 6)
    assert s[0].tolist() == [80, 81, 82, 47, 16, -1] and s[3].tolist() == [0, 3, 5]
    assert ref.softmax(np.array([[0.0, -np.inf, 0.0]]), [1.0]).tolist() == [[0.5, 0.0, 0.5]]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_divider(tmp_path):
    """The multiplication that stands for the division by a block size, at
    every size up to 4096, powers of two and their neighbours, and the
    numerators next to multiples."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "reduction_primitives_amd", "csrc")
    src = tmp_path / "d.cpp"
    src.write_text('''
#include "rk_serve.hpp"
#include <cstdio>
using namespace rk;
static int bad(uint32_t x, uint32_t d) {
    const Divider r = make_divider(d);
    const uint32_t q = r.shift ? uint32_t((uint64_t(x) * r.m) >> r.shift) : x;
    if (q != x / d) { std::printf("%u / %u gave %u\\n", x, d, q); return 1; }
    return 0;
}
int main() {
    const uint32_t top = 0x7fffffffu;
    for (uint64_t i = 1; i < 4096 + 200; ++i) {
        uint32_t d = uint32_t(i);
        if (i >= 4096) { const int k = int(i - 4096); d = (1u << (k / 6 % 31)) + uint32_t(k % 6) - 2u; if (d == 0 || d > top) continue; }
        const uint32_t qs[] = {0, 1, 2, 3, 1000, top / d / 2, top / d - (top / d > 0), top / d};
        for (uint32_t q : qs)
            for (int64_t e = -2; e <= 2; ++e) {
                const int64_t x = int64_t(q) * d + e;
                if (x >= 0 && x <= top && bad(uint32_t(x), d)) return 1;
            }
        if (bad(top, d)) return 1;
    }
    return 0;
}
''')
    exe = str(tmp_path / "d")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I" + csrc, str(src),
                    os.path.join(csrc, "rk_serve_plan.cpp"), os.path.join(csrc, "rk_plan.cpp"), "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0, run.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_slot_map_search_stays_in_range(tmp_path):
    """The search for a token's request among as many requests as rk_slot_map
    takes: only places of the range are looked at, and the last request that
    begins at or before the token is found, empty ones before it passed by."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "reduction_primitives_amd", "csrc")
    src = tmp_path / "s.cpp"
    src.write_text('''
#include "rk_serve.hpp"
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
int main() {
    const int sizes[] = {1, 2, 3, 4097, 1 << 30, (1 << 30) + 1, 0x7ffffffe};
    for (int req : sizes)
        for (int empty : {1, 3})              // of every `empty` requests all but the last have no token
            for (int64_t t = 0; t < req / empty; t = t < 5 || t > req / empty - 9 ? t + 1 : t + (req / empty - 8 - t + 1) / 2) {
                const auto start = [&](int i) {
                    if (i < 0 || i >= req) { std::printf("looked at %d of %d\\n", i, req); std::exit(1); }
                    return int64_t(i) / empty;
                };
                const int b = rk::last_start(start, 0, req, t);
                const int64_t want = (t + 1) * empty - 1;
                if (b != (want < req ? want : req - 1)) { std::printf("%lld of %d: %d\\n", (long long)t, req, b); return 1; }
            }
    return 0;
}
''')
    exe = str(tmp_path / "s")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I" + csrc, str(src),
                    "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0, run.stdout + run.stderr


def _build_in(tmp_path, monkeypatch):
    """The build module with every product under tmp_path, and of the
    library's units the plain C++ ones alone (seconds to compile)."""
    from reduction_primitives_amd import build as b
    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "librk.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_serving.so"))
    monkeypatch.setattr(b, "KERNEL_UNITS", [])
    monkeypatch.setattr(b, "HIP_HOST_UNITS", [])
    return b


def test_library_builds_without_torch(tmp_path, monkeypatch):
    """The C ABI needs no torch: without it librk.so is built all the same,
    and said to stand without the Python module."""
    import sys
    b = _build_in(tmp_path, monkeypatch)
    if not os.path.exists(b.HIPCC):
        pytest.skip("needs hipcc")
    monkeypatch.setitem(sys.modules, "torch", None)        # import torch: ImportError
    with pytest.warns(UserWarning, match="_serving.so"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


def test_python_module_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    """_serving.so holds to torch's C++ ABI and Python's: one that was built
    for others is not taken, however new it is."""
    import sys
    import types
    b = _build_in(tmp_path, monkeypatch)
    os.makedirs(b.OUT_DIR)
    compiled = []

    def run(cmd, **kw):
        compiled.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(b.subprocess, "run", run)
    builds = lambda: (b._build_binding(False), len(compiled))[1]  # noqa: E731
    assert builds() == 1 and builds() == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert builds() == 2 and builds() == 2
    monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-399")
    assert builds() == 3 and builds() == 3
    monkeypatch.setitem(sys.modules, "torch", None)        # (nothing to build it with, and one is there)
    assert builds() == 3


def test_softmax_refuses_to_drop_gradients():
    """The call has no backward pass: its module says so, where gradients are
    recorded, before it looks at devices."""
    call = _rk().softmax.__globals__["_calls"].softmax
    x, t = torch.zeros(2, 8), torch.ones(2)
    leaf = lambda v: v.clone().requires_grad_()  # noqa: E731
    for what, args in (("x", (leaf(x), None, x)), ("temperature", (x, leaf(t), x)), ("out", (x, t, leaf(x))),
                       ("x", (leaf(x) * 2, t, x))):
        with pytest.raises(ValueError, match=what + " requires grad and the call has no gradient"):
            call(0, *args, None)
        with torch.no_grad(), pytest.raises(ValueError, match="not on a GPU"):     # (refused for that alone)
            call(0, *args, None)
