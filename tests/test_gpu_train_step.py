"""The operators of a training step together: blocks, the vocabulary's head, clipping; and rows sorted for a caller's
own experts, there and back with gradients. Tolerances count the roundings of each step, beside it."""
import math

import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import mok, synth
from combine_router_top_expert_gb300.block import MoEBlock
from combine_router_top_expert_gb300.head import VocabHead
from helpers import dtype_of, layer_for


def _rows(g, T, H, std=1.0):
    return (torch.randn((T, H), generator=g, device="cuda") * std).to(torch.bfloat16)


def _head(V, H, seed, **kw):
    g = ref.gen(seed)
    return VocabHead(_rows(g, V, H, 0.05), 1 + 0.2 * torch.randn(H, generator=g, device="cuda"), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 200, 300])
@pytest.mark.parametrize("residual", [True, False])
def test_head(T, residual):
    """score and train against the formulas in 64 bits on the normed rows as they are (BF16)."""
    H, V = 256, 1001
    g = ref.gen(T)
    head = _head(V, H, 1)
    x, r = _rows(g, T, H), _rows(g, T, H, 2.0) if residual else None
    labels = torch.randint(-1, V, (T,), generator=g, device="cuda")
    loss, lse = head.score(x, labels, residual=r)
    got, grads = head.train(x, labels, residual=r, scale=0.5)
    assert head.status() == (mok.OK, 0)
    y = torch.empty_like(x)
    total, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    mok.rmsnorm(x, head.gain, residual=r, y=y, sum=total, rstd=rstd)
    want, want_lse, _ = ref.head_loss(y, head.W, labels)
    # logits: H products at 2^-23 of the sum of magnitudes (below 60); the rest as in the loss's own tests
    tol = 2.0 ** -17 + H * 2.0 ** -23 * 60
    assert ((loss.double() - want).abs() <= tol * (1 + want.abs())).all()
    assert ((lse.double() - want_lse).abs() <= tol * (1 + want_lse.abs())).all()
    assert torch.equal(got, loss)
    dy, dW, my, mW = ref.head_grad(y, head.W, labels, torch.full((T,), 0.5, dtype=torch.float64, device="cuda"))
    # dl to BF16 from values with 2^-10 and the logits' error, products, rounded to BF16
    rel = 2.0 ** -8 + 2.0 ** -10 + 2 * tol
    assert ((grads["dW"].double() - dW).abs() <= (rel + T * 2.0 ** -23) * mW + 2.0 ** -8 * dW.abs() + 1e-30).all()
    # the norm's backward from that dy: every operation on it is linear, so its error passes through the same sums
    R, gain, s = rstd.double()[:, None], head.gain.double(), total.double()
    xh, a = s * R, gain * dy
    dx = R * (a - xh * (a * xh).mean(1, keepdim=True))
    err = gain.abs() * ((rel + V * 2.0 ** -23) * my + 2.0 ** -8 * dy.abs())
    mag = R * (err + xh.abs() * (err * xh.abs()).mean(1, keepdim=True))
    size = R * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    assert ((grads["dx"].double() - dx).abs() <= 1.01 * mag + 2.0 ** -8 * dx.abs() + 2.0 ** -15 * size + 1e-30).all()
    dg = (dy * xh).sum(0)
    assert ((grads["dgain"].double() - dg).abs() <= 1.01 * ((err / gain.abs() + 2.0 ** -16 * dy.abs()) * xh.abs()).sum(0) + 1e-30).all()


@pytest.mark.gpu
def test_head_of_no_tokens():
    head = _head(1001, 256, 2)
    x, labels = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.long, device="cuda")
    loss, lse = head.score(x, labels)
    assert loss.shape == lse.shape == (0,)
    loss, grads = head.train(x, labels)
    assert loss.shape == (0,) and grads["dx"].shape == (0, 256) and not grads["dW"].any() and not grads["dgain"].any()
    dW = torch.full((1001, 256), 3.0, device="cuda")
    head.train(x, labels, dW=dW)
    assert (dW == 3).all() and head.status() == (mok.OK, 0)


@pytest.mark.gpu
def test_heads_graphs_in_turn_with_eager_calls():
    """Two captured calls of the same workspace, replayed in turn with eager ones of other sizes between them."""
    H, V = 256, 3001
    g = ref.gen(12)
    head = _head(V, H, 3)
    xs = [_rows(g, T, H) for T in (5, 6, 300)]
    ys = [torch.randint(0, V, (x.shape[0],), generator=g, device="cuda") for x in xs]
    want = [head.train(x, y) for x, y in zip(xs, ys)]
    graphs, outs = [], []
    for x, y in zip(xs[:2], ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(head.train(x, y))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
            again = head.train(xs[2], ys[2])
        for (loss, grads), (loss0, grads0) in zip(outs + [again], want):
            assert torch.equal(loss, loss0) and all(torch.equal(grads[n], grads0[n]) for n in grads0)


@pytest.mark.gpu
def test_head_adds_to_a_gradient_and_goes_in_pieces():
    T, H, V = 600, 128, 700
    g = ref.gen(3)
    x, labels = _rows(g, T, H), torch.randint(0, V, (T,), generator=g, device="cuda")
    whole, cut = _head(V, H, 2), _head(V, H, 2, piece=256)
    acc = torch.zeros((V, H), device="cuda")
    loss, a = whole.train(x, labels)
    cut_loss, b = cut.train(x, labels, dW=acc)
    cut.train(x, labels, dW=acc)
    assert b["dW"] is acc and torch.equal(loss, cut_loss)
    _, dW, _, mW = ref.head_grad(*_normed(whole, x), labels, torch.ones(T, dtype=torch.float64, device="cuda"))
    tol = (2.0 ** -8 + 2.0 ** -9 + H * 2.0 ** -22 * 60) * mW + T * 2.0 ** -22 * mW
    assert ((acc.double() - 2 * dW).abs() <= 2 * tol + 1e-30).all()
    assert ((a["dW"].double() - dW).abs() <= tol + 2.0 ** -8 * dW.abs() + 1e-30).all()


def _normed(head, x):
    y = torch.empty_like(x)
    mok.rmsnorm(x, head.gain, y=y)
    return y, head.W


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_step(dtype):
    """Two blocks, the head and clipping: the head's and the blocks' calls by hand give the same bits, the norm is that
    of all gradients, and the clipped ones are them times one factor. The same step captured and replayed on new rows
    gives the bits of a plain one."""
    T, H, V = 300, 512, 1000
    wls = [synth.small("step", T=T, H=H, I=256, E=8, k=2, dtype=dtype) for _ in range(2)]
    blocks = [MoEBlock(layer_for(synth.make_inputs(w, seed=n, with_x=False), dtype_of(w)), torch.ones(H, device="cuda"))
              for n, w in enumerate(wls)]
    head = _head(V, H, 4)
    norm, ws = torch.empty((), device="cuda"), mok.alloc_bytes(mok.grad_workspace_size())
    g = ref.gen(5)
    x, labels = _rows(g, T, H), torch.randint(-1, V, (T,), generator=g, device="cuda")

    def step(clip):
        h, res, ctxs = x, None, []
        for b in blocks:
            h, res, ctx = b.train_forward(h, res)
            ctxs.append(ctx)
        loss, grads = head.train(h, labels, residual=res, scale=1.0 / T)
        d = grads.pop("dx")
        every = list(grads.values())
        for b, ctx in zip(reversed(blocks), reversed(ctxs)):
            grads = b.train_backward(ctx, d, d)
            d = grads.pop("dx")
            every += grads.values()
        mok.grad_clip(every, clip, norm, ws) if clip else mok.grad_norm(every, norm, ws)
        return loss, every

    loss, plain = step(None)
    want = math.sqrt(math.fsum(float(t.double().square().sum()) for t in plain))
    assert math.isfinite(want) and want > 0 and abs(float(norm) - want) <= 11 * 2.0 ** -24 * want
    _, clipped = step(want / 4)
    factor = want / 4 / (want + 1e-6)
    for a, b in zip(plain, clipped):
        half = 2.0 ** -8 if a.dtype is torch.bfloat16 else 2.0 ** -24
        assert ((b.double() - factor * a.double()).abs() <= (half + 2.0 ** -19) * factor * a.double().abs() + 2.0 ** -133).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(want / 4)
    for seed in (6, 7):
        x.copy_(_rows(ref.gen(seed), T, H))
        graph.replay()
        got = [out[0].clone()] + [t.clone() for t in out[1]]
        fresh = step(want / 4)
        assert torch.equal(got[0], fresh[0]) and all(torch.equal(a, b) for a, b in zip(got[1:], fresh[1]))


@pytest.mark.gpu
@pytest.mark.parametrize("drop", [0.0, 0.25])
def test_own_experts(drop):
    """A caller's router (indices and weights of their own) and experts (matrices here) around the sorted rows, against
    automatic differentiation in 64 bits. fp32 rows: the sums' errors are far below 1e-4 of the largest values."""
    T, H, E, k = 120, 64, 6, 3
    g = ref.gen(8)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, W, dout = rnd(T, H), rnd(E, H, H) / 8, rnd(T, H)
    w = torch.rand((T, k), generator=g, device="cuda")
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda")
    idx = torch.where(torch.rand((T, k), generator=g, device="cuda") < drop, -1, idx).int()
    lay = mok.sort_layout(idx, E)
    off = lay["offsets"].tolist()
    xs, ys = (torch.zeros((T * k, H), device="cuda") for _ in range(2))
    mok.sort_rows(x, lay, xs)
    for e in range(E):
        ys[off[e]:off[e + 1]] = xs[off[e]:off[e + 1]].double().matmul(W[e].double()).float()
    out = mok.unsort_rows(ys, lay, torch.empty_like(x), w=w)
    dys, dw, dxs = torch.zeros_like(ys), torch.empty_like(w), torch.zeros_like(xs)
    mok.unsort_rows_backward(dout, ys, lay, w, dys, dw)
    for e in range(E):
        dxs[off[e]:off[e + 1]] = dys[off[e]:off[e + 1]].double().matmul(W[e].double().t()).float()
    dx = mok.unsort_rows(dxs, lay, torch.empty_like(x))
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    each = torch.einsum("th,ehi->tei", xd, W.double())
    picked = each[torch.arange(T, device="cuda")[:, None], idx.long().clamp(min=0)]
    want = ((idx >= 0)[..., None] * wd[..., None] * picked).sum(1)
    want.backward(dout.double())
    for a, b in ((out, want.detach()), (dx, xd.grad), (dw, wd.grad)):
        assert float((a.double() - b).abs().max()) <= 1e-4 * float(b.abs().max())


@pytest.mark.gpu
def test_two_streams_at_once():
    """Training calls, clipping and sorted rows on two streams side by side, each with its own buffers, give the bits
    that they give one after the other."""
    H, V, E, k = 512, 5003, 8, 2
    g = ref.gen(31)
    sets = []
    for T in (300, 64):
        x, labels = _rows(g, T, H), torch.randint(-1, V, (T,), generator=g, device="cuda")
        idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        sets.append((_head(V, H, T), x, labels, idx, torch.rand((T, k), generator=g, device="cuda")))

    def step(head, x, labels, idx, w, stream=None):
        T = x.shape[0]
        loss, grads = head.train(x, labels, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            norm, ws = torch.empty((), device="cuda"), mok.alloc_bytes(mok.grad_workspace_size())
            mok.grad_clip(list(grads.values()), 0.01, norm, ws)
            layout = mok.sort_layout(idx, E)
            xs, out = torch.zeros((T * k, H), dtype=x.dtype, device="cuda"), torch.empty_like(x)
            mok.sort_rows(x, layout, xs)
            mok.unsort_rows(xs, layout, out, w=w)
        return [loss, norm, xs, out, *grads.values()]

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(20):
        for i, s in enumerate(sets):
            got[i].append(step(*s, stream=streams[i]))
    torch.cuda.synchronize()
    for i, s in enumerate(sets):
        assert s[0].status() == (mok.OK, 0)
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))
