"""The common factor of the vocabulary loss's gradient: dl is rounded to BF16 without it.

Inputs whose logits are all exactly 0 (x and W have no column in common where both are not zero), V = 2^12: the softmax
is 2^-12 everywhere, which BF16 holds, and the label's entry 1 - 2^-12 becomes 1, an error of 2^-12 of the coefficient.
So with a coefficient c that all tokens share the gradients differ from the formula by

    dx: c (2^-12 |W_y| + V 2^-23 sum_v |dl_v W_v|) and the result's rounding
    dW: c (2^-12 sum_{t: y_t = v} |x_t| + T 2^-23 sum_t |dl_t x_t|), and in BF16 the result's rounding

where the second terms are the products' sums (each addition at no worse than 2^-23 of the magnitudes) and 2^-21 of all
magnitudes covers the fp32 factor, its product and the softmax's own rounding before BF16. A coefficient that is rounded
with dl is off by up to 2^-8 for all tokens alike: 1/4080 by 0.0038, 1/300 by 0.0018.
"""
import math

import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import mok

V = 4096


def _inputs(T, H, seed):
    g = ref.gen(seed)
    x, W = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((T, H), (V, H)))
    x[:, H // 2:] = 0
    W[:, :H // 2] = 0
    W[:, -1] = 1            # dx's last column is the sum of a token's dl
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    return x, W, torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, -100, y)


def _grad(x, W, y, call, dloss, scale, piece=0, dW_type=torch.bfloat16, start=None):
    T, H = x.shape
    ws = mok.alloc_bytes(mok.head_workspace_size(T, H, V, True, piece)).fill_(0xA5)
    dx = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dW = torch.full((V, H), float("nan"), dtype=dW_type, device="cuda") if start is None else start.clone()
    kw = dict(dloss=dloss, scale=scale, piece=piece, accumulate=start is not None)
    if call == "train":
        mok.head_loss_train(x, W, y, torch.empty(T, device="cuda"), dx, dW, ws, **kw)
    else:
        lse = torch.full((T,), 12 * math.log(2), device="cuda")
        mok.head_loss_backward(x, W, y, lse, dx, dW, ws, **kw)
    assert mok.device_status(ws) == (mok.OK, 0)
    return dx, dW


def _check(x, W, y, c, dx, dW, start=None):
    T = x.shape[0]
    live = (y >= 0).double()[:, None]
    xd, Wd, yc = x.double() * live, W.double(), y.clamp(min=0)
    p = 2.0 ** -12
    at, mags = Wd[yc] * live, live * (p * Wd.abs().sum(0) + Wd[yc].abs())
    want = c * (live * p * Wd.sum(0) - at)
    tol = c * (p * at.abs() + (V * 2.0 ** -23 + 2.0 ** -21) * mags) + 2.0 ** -8 * want.abs()
    assert ((dx.double() - want).abs() <= tol).all()
    own = torch.zeros_like(Wd).index_add_(0, yc, xd)
    own_mag = torch.zeros_like(Wd).index_add_(0, yc, xd.abs())
    want = c * (p * xd.sum(0) - own)
    mags = p * xd.abs().sum(0) + own_mag
    tol = c * (p * own_mag + (T * 2.0 ** -23 + 2.0 ** -21) * mags)
    if start is not None:
        want = want + start.double()
        tol = tol + (1 + -(-T // 128)) * 2.0 ** -23 * (start.double().abs() + c * mags)
    elif dW.dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    assert ((dW.double() - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 256), (100, 256), (300, 256), (300, 5120)])
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("scale,weight", [(1 / 4080, None), (1 / 300, None), (1 / 2560, None), (1.0, 1 / 4080), (0.3, 1 / 300),
                                          (0.25, None)])
def test_shared_coefficient(T, H, call, scale, weight):
    """Given as the scale, or as the same weight of every token (the gradient of a mean)."""
    x, W, y = _inputs(T, H, T + H)
    dloss = None if weight is None else torch.where(y >= 0, weight, 77.0).float()
    c = float(torch.tensor(scale).double()) * (1 if weight is None else float(torch.tensor(weight)))
    for dt in (torch.bfloat16, torch.float32):
        dx, dW = _grad(x, W, y, call, dloss, scale, dW_type=dt)
        _check(x, W, y, c, dx, dW)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("T,piece", [(300, 0), (300, 128), (100, 40)])
def test_in_pieces_and_added(call, T, piece):
    x, W, y = _inputs(T, 256, 5)
    start = torch.randn((V, 256), generator=ref.gen(6), device="cuda") * 2.0 ** -12
    c = float(torch.tensor(1 / 4080).double())
    _check(x, W, y, c, *_grad(x, W, y, call, None, 1 / 4080, piece, torch.float32, start), start=start)
    _check(x, W, y, c, *_grad(x, W, y, call, None, 1 / 4080, piece))


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_an_infinite_weight_stays_its_tokens(call, T, bad):
    x, W, y = _inputs(T, 256, 7)
    y[3] = 9
    dloss = torch.rand(T, generator=ref.gen(8), device="cuda") + 0.5
    dloss[3] = 0.0
    want = _grad(x, W, y, call, dloss, 0.3)
    dloss[3] = bad
    dx, dW = _grad(x, W, y, call, dloss, 0.3)
    keep = torch.arange(T, device="cuda") != 3
    assert torch.equal(dx[keep], want[0][keep]) and not torch.isfinite(dx[3, -1]) and not torch.isfinite(dW[9, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("T", [40, 300])
def test_factors_out_of_range_and_of_nothing(call, T):
    """Weights below fp32's normal numbers with a scale that brings them back; weights of 0; a scale of infinity or NaN
    (1 / 0) where no token has a label."""
    x, W, y = _inputs(T, 256, 9)
    want = _grad(x, W, y, call, None, 2.0 ** -10)
    got = _grad(x, W, y, call, torch.full((T,), 2.0 ** -140, dtype=torch.float64).float().cuda(), 2.0 ** 127)
    again = _grad(x, W, y, call, None, 2.0 ** -13)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert all(torch.equal(a, b * 2.0 ** -3) for a, b in zip(again, want))
    dx, dW = _grad(x, W, y, call, torch.zeros(T, device="cuda"), 0.3)
    assert not dx.any() and not dW.any()
    for scale in (float("inf"), float("nan")):
        dx, dW = _grad(x, W, torch.full_like(y, -100), call, None, scale)
        assert not dx.any() and not dW.any()
