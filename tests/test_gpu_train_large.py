"""Offsets of more than 32 bits in the vocabulary loss, the sorted rows and the clipping."""
import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import mok


@pytest.mark.gpu
def test_vocabulary_of_more_than_2_31_weights():
    """Inputs with logits that are exact in fp32, as the loss's own tests have them, in a vocabulary of 2.9e9 weights;
    tolerances as there, with V / 128 / 256 = 13 sums of a thread."""
    T, H, V = 3, 7168, 400009
    g = ref.gen(1)
    W = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    W[:, :64] = (torch.randint(-4, 5, (V, 64), generator=g, device="cuda") / 16).to(torch.bfloat16)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, :64] = (torch.randint(-8, 9, (T, 64), generator=g, device="cuda") / 8).to(torch.bfloat16)
    x[:, -1] = 1.0
    W[-5:, -1] = 2.0                                      # the last rows count by their last column
    y = torch.tensor([V - 1, 7, V - 3], device="cuda")
    loss, dx = torch.empty(T, device="cuda"), torch.empty_like(x)
    lse, dW = torch.empty_like(loss), torch.full_like(W, float("nan"))
    ws = mok.alloc_bytes(mok.head_workspace_size(T, H, V, True))
    mok.head_loss_train(x, W, y, loss, dx, dW, ws, lse=lse)
    assert mok.device_status(ws) == (mok.OK, 0)
    keep = list(range(64)) + [H - 1]
    Wd, xd = W[:, keep].double(), x[:, keep].double()
    logits = xd @ Wd.t()
    want_lse = torch.logsumexp(logits, 1)
    rows = torch.arange(T, device="cuda")
    rel = 2.0 ** -17
    assert ((lse.double() - want_lse).abs() <= rel * (1 + want_lse.abs())).all()
    assert ((loss.double() - (want_lse - logits[rows, y])).abs() <= rel * (1 + want_lse.abs())).all()
    dl = torch.exp(logits - want_lse[:, None])
    dl[rows, y] -= 1
    tol = 2.0 ** -8 + 2.0 ** -10 + T * 2.0 ** -23
    want, mags = dl.t() @ xd, dl.abs().t() @ xd.abs()
    assert ((dW[:, keep].double() - want).abs() <= tol * mags + 2.0 ** -8 * want.abs() + 1e-30).all()
    assert not dW[:, 64:H - 1].any()
    want, mags = dl @ Wd, dl.abs() @ Wd.abs()
    assert ((dx[:, keep].double() - want).abs() <= (tol + V * 2.0 ** -23) * mags + 2.0 ** -8 * want.abs() + 1e-30).all()


@pytest.mark.gpu
def test_pieces_of_more_than_2_31_exponentials():
    """dl of 17000 x 131072 values in one piece: the bits of the losses and of dx do not depend on the pieces."""
    T, H, V = 17000, 64, 131072
    g = ref.gen(2)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, H), generator=g, device="cuda") * 0.2).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    got = []
    for piece in (T, 4096):
        loss, dx, dW = torch.empty(T, device="cuda"), torch.empty_like(x), torch.empty((V, H), device="cuda")
        ws = mok.alloc_bytes(mok.head_workspace_size(T, H, V, True, piece))
        mok.head_loss_train(x, W, y, loss, dx, dW, ws, piece=piece, scale=1.0 / T)
        assert mok.device_status(ws) == (mok.OK, 0)
        got.append((loss, dx, dW))
    (l0, x0, w0), (l1, x1, w1) = got
    assert torch.equal(l0, l1)
    want, _, _ = ref.head_loss(x[-300:], W, y[-300:])
    # H random products at 2^-23 of the sum of magnitudes, below 64 * 4 * 0.9
    assert ((l0[-300:].double() - want).abs() <= (2.0 ** -17 + 64 * 2.0 ** -23 * 230) * (1 + want.abs())).all()
    # the same BF16 dl, summed in other parts: V (dx) and T (dW) steps of 2^-23 of the sum of magnitudes at most, for which
    # a token's dl sum up to 2 / T and a vocabulary row's to the sums of a softmax's column
    big = float(W.abs().max()) * 2 / T
    assert ((x0.float() - x1.float()).abs() <= V * 2.0 ** -23 * big + 2.0 ** -7 * x0.float().abs() + 1e-30).all()
    column = (torch.bincount(y, minlength=V) + 40.0)[:, None] / T * float(x.abs().max())
    assert ((w0 - w1).abs() <= T * 2.0 ** -23 * column).all()


@pytest.mark.gpu
def test_rows_of_more_than_2_31_values():
    T, H, k, E = 38000, 7168, 8, 32
    g = ref.gen(3)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    layout = mok.sort_layout(idx, E)
    xs, out = torch.empty((T * k, H), dtype=x.dtype, device="cuda"), torch.empty_like(x)
    mok.sort_rows(x, layout, xs)
    src = layout["row_src"].long()
    for a in range(0, T * k, 40000):
        assert torch.equal(xs[a:a + 40000], x[src[a:a + 40000] // k])
    w = torch.full((T, k), 0.125, device="cuda")
    mok.unsort_rows(xs, layout, out, w=w)
    assert torch.equal(out, x)                       # eighths of eight equal values
    dy, dw = torch.empty_like(xs), torch.empty_like(w)
    mok.unsort_rows_backward(x, xs, layout, w, dy, dw)
    for a in range(0, T * k, 40000):
        assert torch.equal(dy[a:a + 40000], xs[a:a + 40000] * 0.125)
    square = x.double().square().sum(1, keepdim=True)
    assert ((dw.double() - square).abs() <= H * 2.0 ** -24 * square).all()


@pytest.mark.gpu
def test_a_gradient_of_more_than_2_31_values():
    n = (1 << 31) + 12345
    t = torch.full((n + 3,), 0.5, dtype=torch.bfloat16, device="cuda")
    norm, ws = torch.empty((), device="cuda"), mok.alloc_bytes(mok.grad_workspace_size())
    for first in (0, 3):
        g = t[first:first + n]
        g.fill_(0.5)
        g[-1] = 16384.0
        want = (0.25 * (n - 1) + 16384.0 ** 2) ** 0.5
        mok.grad_clip([g], want / 4, norm, ws)
        assert abs(float(norm) - want) <= 2.0 ** -20 * want
        # the factor is a quarter less 1e-6 / norm, so the values round to an eighth and to 4096
        assert float(g[-1]) == 4096.0 and bool((g[:-1] == 0.125).all())
