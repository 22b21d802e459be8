"""Softmax cross entropy over a vocabulary and its gradient against the formulas in 64 bits.

Tolerances. Most inputs have logits that are exact in fp32 (trainref.exact_head). What remains of a log-sum: the
exponentials' arguments are rounded (2 * 2^-24 of |l| log2 e each), ex2 errs by 2^-22, a tile's 128 terms go into four
chains of 32 that are joined in two steps, the tiles of a row into 256 threads, then 5 + 3 steps: below
2^-22 + 2^-22 |l| + (34 + tiles / 256 + 10) 2^-24 relative, then the logarithm. A loss l_rest - l_label has the same
error in its argument. REL = 2^-17 covers all of it for |l| <= 20.
Random inputs add the products' error: H products, each added at no worse than 2^-23 of the sum of magnitudes.
Gradients: dl is rounded to BF16 (2^-8 relative) from values of at most 2^-11 + REL relative error, the products add
K 2^-23 of the sum of magnitudes, and a BF16 result is rounded once more.
"""
import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import mok

REL = 2.0 ** -17
SHAPES = [(1, 8, 1), (1, 64, 5), (2, 16, 64), (3, 72, 257), (130, 264, 1000), (256, 128, 512), (257, 520, 129),
          (300, 1024, 8191), (600, 64, 300), (1000, 2048, 4099)]


def _labels(T, V, seed, dtype=torch.int64, drop=0.2):
    g = ref.gen(seed + 1000)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    return torch.where(torch.rand(T, generator=g, device="cuda") < drop, -100, y).to(dtype)


def _ws(T, H, V, grad=False, piece=0):
    return mok.alloc_bytes(mok.head_workspace_size(T, H, V, grad, piece)).fill_(0xA5)


def _nan(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _score(x, W, y, **kw):
    (T, H), V = x.shape, W.shape[0]
    loss, lse, ws = _nan(T), _nan(T), _ws(T, H, V)
    mok.head_loss(x, W, y, loss, ws, lse=lse, **kw)
    assert mok.device_status(ws) == (mok.OK, 0)
    return loss, lse


def _train(x, W, y, call="train", dloss=None, scale=1.0, dW=None, piece=0, lse=None, **kw):
    (T, H), V = x.shape, W.shape[0]
    ws = _ws(T, H, V, True, piece)
    dx = _nan(T, H, dtype=torch.bfloat16)
    dW = _nan(V, H, dtype=torch.bfloat16) if dW is None else dW
    if call == "train":
        loss, lse = _nan(T), _nan(T)
        mok.head_loss_train(x, W, y, loss, dx, dW, ws, dloss=dloss, scale=scale, lse=lse, piece=piece, **kw)
    else:
        loss, lse0 = _score(x, W, y)
        lse = lse0 if lse is None else lse
        mok.head_loss_backward(x, W, y, lse, dx, dW, ws, dloss=dloss, scale=scale, piece=piece, **kw)
    assert mok.device_status(ws) == (mok.OK, 0)
    return loss, lse, dx, dW


def _check_loss(loss, lse, x, W, y, slack=0.0):
    want, want_lse, _ = ref.head_loss(x, W, y)
    assert ((lse.double() - want_lse).abs() <= REL + REL * want_lse.abs() + slack).all()
    assert ((loss.double() - want).abs() <= (REL + slack) * (1 + want.abs())).all()


def _check_grad(got, want, mags, K, f32=False):
    tol = (2.0 ** -8 + 2.0 ** -10 + K * 2.0 ** -23) * mags + (0 if f32 else 2.0 ** -8 * want.abs()) + 1e-30
    bad = (got.double() - want).abs() - tol
    assert (bad <= 0).all(), float(bad.max())


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_loss(T, H, V, dtype):
    x, W = ref.exact_head(T, H, V, T + H + V)
    y = _labels(T, V, T, dtype)
    loss, lse = _score(x, W, y)
    _check_loss(loss, lse, x, W, y)
    only, again = _nan(T), _score(x, W, y)
    mok.head_loss(x, W, y, only, _ws(T, H, V))
    assert torch.equal(only, loss) and torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(1, 7168, 4096), (64, 7168, 5000), (700, 1024, 3001)])
def test_loss_of_random_rows(T, H, V):
    g = ref.gen(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, H), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    y = _labels(T, V, T)
    loss, lse = _score(x, W, y)
    mags = float((x.double().abs() @ W.double().abs().t()).max())
    _check_loss(loss, lse, x, W, y, slack=H * 2.0 ** -23 * mags)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", SHAPES)
@pytest.mark.parametrize("call", ["train", "backward"])
def test_gradient(T, H, V, call):
    x, W = ref.exact_head(T, H, V, T + H + V)
    y = _labels(T, V, T)
    dloss = torch.rand(T, generator=ref.gen(3), device="cuda") + 0.5
    loss, lse, dx, dW = _train(x, W, y, call, dloss, 0.25)
    _check_loss(loss, lse, x, W, y)
    want_dx, want_dW, mx, mW = ref.head_grad(x, W, y, 0.25 * dloss.double())
    _check_grad(dx, want_dx, mx, V)
    _check_grad(dW, want_dW, mW, T)
    again = _train(x, W, y, call, dloss, 0.25)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, lse, dx, dW)))


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("which", ["dx", "dW"])
def test_one_gradient_alone(call, which):
    T, H, V = 130, 264, 1000
    x, W = ref.exact_head(T, H, V, 7)
    y = _labels(T, V, 7)
    loss, lse, dx, dW = _train(x, W, y, call)
    out = dict(dx=_nan(T, H, dtype=torch.bfloat16), dW=None) if which == "dx" else \
        dict(dx=None, dW=_nan(V, H, dtype=torch.bfloat16))
    if call == "train":
        mok.head_loss_train(x, W, y, _nan(T), out["dx"], out["dW"], _ws(T, H, V, True))
    else:
        mok.head_loss_backward(x, W, y, lse, out["dx"], out["dW"], _ws(T, H, V, True))
    assert torch.equal(out[which], dx if which == "dx" else dW)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_ignored_tokens_do_not_matter(call, bad):
    """Whatever ignored rows hold; labels past the vocabulary and far outside 32 bits are ignored, too."""
    T, H, V = 400, 136, 700
    x, W = ref.exact_head(T, H, V, 5)
    y = _labels(T, V, 5)
    y[3], y[77], y[399] = V, 2 ** 40 + 5, -2 ** 40
    live = (y >= 0) & (y < V)
    dirty = torch.where(live[:, None], x, bad)
    dloss = torch.where(live, torch.rand(T, generator=ref.gen(4), device="cuda"), bad)
    clean = _train(x, W, y, call, torch.where(live, dloss, 1.0))
    got = _train(dirty, W, y, call, dloss)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    assert not got[0][~live].any() and not got[1][~live].any() and not got[2][~live].any()
    loss, lse = _score(dirty, W, y)
    assert torch.equal(loss, got[0]) and torch.equal(lse, got[1])
    few = dirty[:9].contiguous()
    loss, lse = _score(few, W, y[:9].contiguous())
    _check_loss(loss, lse, x[:9], W, y[:9])


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("T", [0, 1, 300])
def test_no_live_tokens(call, T):
    H, V = 72, 300
    x, W = ref.exact_head(max(T, 1), H, V, 1)
    x = x[:T]
    y = torch.full((T,), -1, device="cuda")
    loss, lse, dx, dW = _train(x, W, y, call)
    assert not loss.any() and not lse.any() and not dx.any() and not dW.any()
    acc = torch.ones((V, H), device="cuda")
    _train(x, W, y, call, dW=acc, accumulate=True)
    assert (acc == 1).all()


@pytest.mark.gpu
def test_a_row_with_nan_is_nan_and_stays_apart():
    T, H, V = 40, 64, 300
    x, W = ref.exact_head(T, H, V, 2)
    y = _labels(T, V, 2, drop=0.0)
    clean = _score(x, W, y)
    x[7, 3], x[9, 5] = float("nan"), float("inf")
    loss, lse = _score(x, W, y)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[7] = keep[9] = False
    assert torch.isnan(loss[7]) and torch.isnan(lse[7]) and torch.isnan(loss[9])
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.gpu
def test_small_losses_keep_their_digits():
    """The label takes all but 1e-3 to 1e-9 of the probability: the loss and the label's entry of dl are the others'
    share, relative. One other token, so that the logits are exact and the share is one exponential."""
    T, H, V = 8, 16, 2
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.arange(7, 7 + 2 * T, 2, device="cuda")
    W = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    W[1, 0] = 1.0
    y = torch.ones(T, dtype=torch.long, device="cuda")
    for call in ("train", "backward"):
        loss, lse, dx, dW = _train(x, W, y, call)
        want = torch.log1p(torch.exp(-x[:, 0].double()))
        assert ((loss.double() - want).abs() <= REL * want).all()
        if call == "train":
            # dx = dl[:, 1] = -(1 - p), rounded to BF16 twice
            share = torch.exp(-x[:, 0].double()) / (1 + torch.exp(-x[:, 0].double()))
            assert ((dx[:, 0].double() + share).abs() <= (2.0 ** -7 + 2.0 ** -11 + REL) * share).all()


@pytest.mark.gpu
def test_extreme_logits():
    """Logits of +-1000: the largest is subtracted, so nothing overflows; a label at -1000 loses 2000."""
    T, H, V = 5, 8, 1000
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([1000.0, -1000.0, 1000.0, 0.0, 500.0])
    W = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    W[:, 0] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 1.0, -1.0)
    y = torch.tensor([0, 0, 1, 5, 998], device="cuda")
    loss, lse, dx, dW = _train(x, W, y)
    # arguments of 1000 are rounded at 2^-24 * 1000 * log2 e * 2
    _check_loss(loss, lse, x, W, y, slack=2.0 ** -12)
    want = ref.head_grad(x, W, y, torch.ones(T, dtype=torch.float64, device="cuda"))
    _check_grad(dx, want[0], want[2] * 1.1, V)
    _check_grad(dW, want[1], want[3] * 1.1, T)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["train", "backward"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("piece", [1, 100, 256, 301])
def test_pieces(call, f32, piece):
    """A gradient formed from pieces of the tokens: the loss and dx do not depend on the cut, dW only in the order of
    its fp32 sums."""
    T, H, V = 700, 200, 1000
    x, W = ref.exact_head(T, H, V, 9)
    y = _labels(T, V, 9)
    if piece == 1:
        T = 5
        x, y = x[:T].contiguous(), y[:T].contiguous()
    dt = torch.float32 if f32 else torch.bfloat16
    whole = _train(x, W, y, call)
    got = _train(x, W, y, call, dW=_nan(V, H, dtype=dt), piece=piece)
    assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])
    dx, dW, mx, mW = ref.head_grad(x, W, y, torch.ones(T, dtype=torch.float64, device="cuda"))
    _check_grad(got[2], dx, mx, V)
    _check_grad(got[3], dW, mW, 2 * T, f32)


@pytest.mark.gpu
@pytest.mark.parametrize("piece", [0, 128])
def test_accumulated_weight_gradient(piece):
    T, H, V = 300, 136, 500
    x, W = ref.exact_head(T, H, V, 11)
    y = _labels(T, V, 11)
    start = torch.randn((V, H), generator=ref.gen(1), device="cuda")
    acc = start.clone()
    _train(x, W, y, dW=acc, accumulate=True, piece=piece)
    _, dW, _, mW = ref.head_grad(x, W, y, torch.ones(T, dtype=torch.float64, device="cuda"))
    tol = (2.0 ** -8 + 2.0 ** -10) * mW + T * 2.0 ** -23 * (mW + start.abs())
    assert ((acc.double() - start - dW).abs() <= tol).all()


@pytest.mark.gpu
def test_gradient_against_differences():
    """dx and dW against central differences of the loss in 64 bits along random directions: error e^2 |d|^3 / 6 of the
    third derivative (below 1 in magnitude per unit of the logits' change)."""
    T, H, V = 17, 64, 130
    x, W = ref.exact_head(T, H, V, 13)
    y = _labels(T, V, 13)
    _, _, dx, dW = _train(x, W, y)
    g = ref.gen(2)
    e = 1e-5
    for wrt, grad in ((x, dx), (W, dW)):
        d = torch.randn(wrt.shape, generator=g, device="cuda", dtype=torch.float64)
        total = [float(ref.head_loss(wrt.double() + s * e * d if wrt is x else x, W if wrt is x else W.double() + s * e * d, y)[0].sum())
                 for s in (1, -1)]
        want = (total[0] - total[1]) / (2 * e)
        _, _, mx, mW = ref.head_grad(x, W, y, torch.ones(T, dtype=torch.float64, device="cuda"))
        tol = float(((2.0 ** -7 + 2.0 ** -10) * (mx if wrt is x else mW) * d.abs()).sum()) + 1e-5
        assert abs(float((grad.double() * d).sum()) - want) <= tol


@pytest.mark.gpu
def test_strides_and_streams():
    T, H, V = 300, 128, 1000
    x, W = ref.exact_head(T, H, V, 17)
    y = _labels(T, V, 17)
    want = _train(x, W, y)
    wide = torch.full((T, H + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + H] = x
    view = wide[:, 8:8 + H]
    got = _train(view, W, y)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws, loss, dx, dW = _ws(T, H, V, True), _nan(T), _nan(T, H, dtype=torch.bfloat16), _nan(V, H, dtype=torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    mok.head_loss_train(view, W, y, loss, dx, dW, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(loss, want[0]) and torch.equal(dx, want[2]) and torch.equal(dW, want[3])


@pytest.mark.gpu
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_captured_and_replayed(drop):
    T, H, V = 300, 136, 1000
    x, W = ref.exact_head(T, H, V, 19)
    y = _labels(T, V, 19, drop=drop)
    ws, loss, dx, dW = _ws(T, H, V, True), _nan(T), _nan(T, H, dtype=torch.bfloat16), _nan(V, H, dtype=torch.bfloat16)
    _train(x, W, y)   # kernels loaded before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mok.head_loss_train(x, W, y, loss, dx, dW, ws)
    for seed in (20, 21):
        x.copy_(ref.exact_head(T, H, V, seed)[0])
        y.copy_(_labels(T, V, seed, drop=0.5 if drop else 0.0))
        graph.replay()
        want = _train(x, W, y)
        assert torch.equal(loss, want[0]) and torch.equal(dx, want[2]) and torch.equal(dW, want[3])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("num_sms", [1, 2, 20])
def test_fewer_sms(T, num_sms):
    """The loss does not depend on the SMs that may be used, the gradients only in the order of their sums."""
    H, V = 136, 1000
    x, W = ref.exact_head(T, H, V, 23)
    y = _labels(T, V, 23)
    cfg = mok.make_config(num_sms=num_sms)
    loss, lse = _score(x, W, y)
    ws = mok.alloc_bytes(mok.head_workspace_size(T, H, V, True, 0, cfg))
    got, dx, dW = _nan(T), _nan(T, H, dtype=torch.bfloat16), _nan(V, H, dtype=torch.bfloat16)
    mok.head_loss_train(x, W, y, got, dx, dW, ws, cfg=cfg)
    assert mok.device_status(ws) == (mok.OK, 0)
    _check_loss(got, lse, x, W, y)
    want_dx, want_dW, mx, mW = ref.head_grad(x, W, y, torch.ones(T, dtype=torch.float64, device="cuda"))
    _check_grad(dx, want_dx, mx, V)
    _check_grad(dW, want_dW, mW, T)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(3, 256, 1000), (400, 512, 3000)])
@pytest.mark.parametrize("call", ["score", "train", "backward"])
def test_waits_that_run_out(T, H, V, call):
    """A block that never comes: the call reports it after its limit, every CTA ends, and the next call is right."""
    x, W = ref.exact_head(T, H, V, 29)
    y = _labels(T, V, 29)
    want = _train(x, W, y, "backward" if call == "backward" else "train")
    ws = _ws(T, H, V, True)
    loss, lse, dx, dW = _nan(T), want[1].clone(), _nan(T, H, dtype=torch.bfloat16), _nan(V, H, dtype=torch.bfloat16)

    def run(cfg=None):
        if call == "score":
            mok.head_loss(x, W, y, loss, ws, cfg=cfg)
        elif call == "train":
            mok.head_loss_train(x, W, y, loss, dx, dW, ws, cfg=cfg)
        else:
            mok.head_loss_backward(x, W, y, lse, dx, dW, ws, cfg=cfg)
        return mok.device_status(ws)[0]

    assert run() == mok.OK
    assert run(mok.make_config(timeout_ms=50, flags=mok.FLAG_TEST_WITHHOLD_PUBLISH)) == mok.ERR_TIMEOUT
    for _ in range(2):
        assert run() == mok.OK
        if call != "backward":
            assert torch.equal(loss, want[0])
        if call != "score":
            assert torch.equal(dx, want[2]) and torch.equal(dW, want[3])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 129, 256, 257, 300])
@pytest.mark.parametrize("H,V", [(72, 1003), (512, 2500)])
@pytest.mark.parametrize("call,f32,piece", [("score", False, 0), ("train", False, 0), ("train", True, 128),
                                            ("backward", False, 100)])
def test_nothing_else_is_written(T, H, V, call, f32, piece):
    """Outputs and a workspace of exactly its size lie between bytes that stay as they were, and so do the inputs."""
    grad = call != "score"
    kinds = dict(loss=(torch.float32, (T,)), lse=(torch.float32, (T,)), dx=(torch.bfloat16, (T, H)),
                 dW=(torch.float32 if f32 else torch.bfloat16, (V, H)),
                 ws=(torch.uint8, (mok.head_workspace_size(T, H, V, grad, piece if grad else 0),)))
    gap, spans, at = 8192, {}, 8192
    for name, (dt, shape) in kinds.items():
        n = torch.empty(shape, dtype=dt, device="meta").nbytes
        spans[name] = (at, n)
        at += n + gap
        at = (at + 1023) // 1024 * 1024
    room = torch.full((at + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
    room = room[-room.data_ptr() % 1024:]
    t = {name: room[a:a + n].view(kinds[name][0]).view(kinds[name][1]) for name, (a, n) in spans.items()}
    g = ref.gen(T + V)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, H), generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    y = _labels(T, V, T)
    kept = [v.clone() for v in (x, W, y)]
    if call == "score":
        mok.head_loss(x, W, y, t["loss"], t["ws"], lse=t["lse"])
    elif call == "train":
        mok.head_loss_train(x, W, y, t["loss"], t["dx"], t["dW"], t["ws"], lse=t["lse"], piece=piece)
    else:
        t["lse"].copy_(_score(x, W, y)[1])
        mok.head_loss_backward(x, W, y, t["lse"], t["dx"], t["dW"], t["ws"], piece=piece)
    assert mok.device_status(t["ws"]) == (mok.OK, 0)
    outside = torch.ones(room.numel(), dtype=torch.bool, device="cuda")
    for a, n in spans.values():
        outside[a:a + n] = False
    assert (room[outside] == 0x5A).all()
    assert all(torch.equal(a, b) for a, b in zip(kept, (x, W, y)))
