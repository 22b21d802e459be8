"""Rows of ignored tokens reach no gradient, whatever they hold: the norm's backward with labels, and a model's last norm
and loss (VocabHead)."""
import ctypes

import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import build, mok
from combine_router_top_expert_gb300.head import VocabHead

NAN, INF = float("nan"), float("inf")


def _rows(g, T, H, std=1.0):
    return (torch.randn((T, H), generator=g, device="cuda") * std).to(torch.bfloat16)


def _labels(T, V, seed, dtype, drop=0.3):
    g = ref.gen(seed)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    return torch.where(torch.rand(T, generator=g, device="cuda") < drop, -100, y).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 8), (5, 256), (700, 264), (500, 7168), (160, 8200), (160, 20000), (155, 65536)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("dsum", [False, True])
def test_norm_backward_with_labels(T, H, dtype, dsum):
    """The bits of a call without labels on the same rows with zeros for the ignored ones."""
    V, g = 50, ref.gen(T + H)
    y = _labels(T, V, T, dtype)
    if T > 4:
        y[1], y[3], y[4] = V, V - 1, (2 ** 40 if dtype is torch.int64 else 2 ** 31 - 1)
    live = ((y >= 0) & (y < V))[:, None]
    s, dy, extra = _rows(g, T, H), _rows(g, T, H), _rows(g, T, H) if dsum else None
    gain, rstd = torch.randn(H, generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")
    ws = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(T, H))

    def run(s, dy, rstd, **kw):
        dx, dgain = torch.full_like(dy, 7.0), torch.full((H,), 7.0, device="cuda")
        mok.rmsnorm_backward(dy, gain, rstd, dx, dgain, ws, s=s, dsum=extra, **kw)
        return dx, dgain
    want = run(torch.where(live, s, 0), torch.where(live, dy, 0), torch.where(live[:, 0], rstd, 0))
    got = run(torch.where(live, s, NAN), torch.where(live, dy, INF), torch.where(live[:, 0], rstd, NAN), labels=y, V=V)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    every = run(s, dy, rstd, labels=torch.zeros_like(y), V=1)
    assert all(torch.equal(a, b) for a, b in zip(every, run(s, dy, rstd)))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 9, 300])
@pytest.mark.parametrize("bad", [NAN, INF, -INF, 3e38])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_head(T, bad, residual, dtype):
    H, V, g = 256, 1001, ref.gen(T)
    head = VocabHead(_rows(g, V, H, 0.05), 1 + 0.2 * torch.randn(H, generator=g, device="cuda"))
    x, r = _rows(g, T, H), _rows(g, T, H) if residual else None
    y = _labels(T, V, T, dtype)
    live = (y >= 0)[:, None]

    def run(fill):
        rows = [None if t is None else torch.where(live, t, fill) for t in (x, r)]
        loss, grads = head.train(rows[0], y, residual=rows[1], scale=1 / 300)
        assert head.status() == (mok.OK, 0)
        return [loss, *head.score(rows[0], y, residual=rows[1]), *(grads[n] for n in ("dx", "dgain", "dW"))]
    want, got = run(0.0), run(bad)
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not got[3][~live[:, 0]].any()


def test_labels_that_are_refused():
    build.build()
    L, ptr = mok.lib(), 1 << 20
    good = dict(dy=ptr, sum=ptr, rstd=ptr, gain=ptr, dx=ptr, dgain=ptr, workspace=ptr, ws_bytes=0, labels=ptr, V=5)
    call = lambda **kw: L.mok_rmsnorm_backward(4, 64, ctypes.byref(mok.RmsNormBwdArgs(**{**good, **kw})), None)
    if not torch.cuda.is_available():
        assert call() == call(labels_i64=1) == call(labels=None, V=0) == mok.ERR_CUDA
    for bad in (dict(V=0), dict(V=-1), dict(labels=ptr + 2), dict(labels=ptr + 4, labels_i64=1),
                dict(sum=None, sum_q=ptr, sum_sf=ptr)):
        assert call(**bad) == mok.ERR_INVALID, bad
    x, f = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(AssertionError):
        mok.rmsnorm_backward(x, f, f[:4], x, f, f, s=x, labels=torch.zeros(4, dtype=torch.long), V=3)
