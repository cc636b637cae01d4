"""GPU tests of the serving operators' launch paths: each path that a rule on
sizes picks is run and compared with the plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.test_gpu_serving import BF16, DEV, F32, _rk, drafts, gen, np64, run_verify

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
