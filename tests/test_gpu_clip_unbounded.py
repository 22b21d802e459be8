"""Clipping with an infinite bound measures the norm and changes nothing, an infinite norm among them."""
import math

import pytest
import torch

from combine_router_top_expert_gb300 import mok

INF, NAN = math.inf, math.nan


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bad", [None, INF, -INF, NAN])
@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("max_norm", [INF, 1.0, 0.0])
def test_norms_and_bounds_that_are_not_finite(dt, bad, inplace, max_norm):
    grads = [torch.full((n,), 0.5, device="cuda").to(dt) for n in (1, 33, 20000)]
    if bad is not None:
        grads[1][7] = bad
    before = [g.clone() for g in grads]
    out = None if inplace else [torch.full_like(g, 7.0) for g in grads]
    norm, ws = torch.empty((), device="cuda"), mok.alloc_bytes(mok.grad_workspace_size())
    mok.grad_clip(mok.grad_list(grads, out), max_norm, norm, ws)
    got = grads if inplace else out
    if bad is None:
        assert math.isclose(float(norm), math.sqrt(20034 * 0.25), rel_tol=11 * 2.0 ** -24)
    else:
        assert math.isnan(float(norm)) if bad != bad else float(norm) == INF
    if bad is not None and bad != bad:
        assert all(torch.isnan(g).all() for g in got)
    elif max_norm == INF:
        assert all(torch.equal(a, b) for a, b in zip(got, before))
    elif bad is not None:
        for a, b in zip(got, before):
            assert torch.equal(torch.isnan(a), torch.isinf(b)) and not a[torch.isfinite(b)].any()
    elif max_norm == 0.0:
        assert not any(g.any() for g in got)
