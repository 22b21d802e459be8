"""The layer on a routing that the caller chose (mok_sort_layout's layout with the caller's indices and weights), and
what entries that were dropped do where they reach it against its contract."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_top_expert_gb300 import mok, synth
from helpers import TOL, assert_close, dev_f32, dtype_of, host_bf16_f64, layer_for, to_dev_bf16

CASES = [synth.small("given_bf16", T=300, H=256, I=128, E=8, k=3, backward=True),
         synth.small("given_one", T=1, H=128, I=64, E=4, k=4, backward=True),
         synth.small("given_mx", T=300, H=256, I=128, E=8, k=3, dtype="mxfp8", backward=True)]


def _choice(wl, seed):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((wl.T, wl.E)), 1)[:, :wl.k].astype(np.int32)      # distinct, in no order
    w = rng.random((wl.T, wl.k)) + 0.1
    return idx, (w / w.sum(1, keepdims=True)).astype(np.float32)


def _routing(idx, w, E):
    i = torch.from_numpy(idx).cuda()
    return dict(mok.sort_layout(i, E), topk_idx=i, topk_w=dev_f32(w))


def _train(layer, wl, x, dY, rt, saved, ws):
    p = layer.problem(wl.T)
    out = torch.empty_like(x)
    mok.moe_forward(p, x, layer.packed, rt, out, ws, saved=saved)
    g = dict(dX=torch.empty_like(x), dW_gate=torch.empty_like(layer.Wg), dW_up=torch.empty_like(layer.Wu),
             dW_down=torch.empty_like(layer.Wd), dW_r=torch.empty((wl.H, wl.E), device="cuda"))
    assert mok.device_status(ws) == (mok.OK, 0)
    mok.moe_backward(p, x, layer.W_r, layer.Wg, layer.Wu, layer.Wd, layer.packed, dY, rt, saved, g, ws,
                     packed_bwd=layer.packed_bwd)
    assert mok.device_status(ws) == (mok.OK, 0)
    return out, g


@pytest.mark.gpu
@pytest.mark.parametrize("wl", CASES, ids=[w.name for w in CASES])
def test_layer_on_a_given_routing(wl):
    """Forward and backward against the oracle on the same routing, at the tolerances of the layer's own."""
    inp = synth.make_inputs(wl, seed=4)
    layer, x, dY = layer_for(inp, dtype_of(wl)), to_dev_bf16(inp.x), to_dev_bf16(inp.dY)
    idx, w = _choice(wl, 5)
    rt = _routing(idx, w, wl.E)
    p = layer.problem(wl.T)
    ws, saved = mok.alloc_bytes(mok.workspace_size(p)), mok.alloc_bytes(mok.saved_size(p))
    served = torch.empty_like(x)
    mok.moe_forward(p, x, layer.packed, rt, served, ws)
    out, g = _train(layer, wl, x, dY, rt, saved, ws)
    ref = dict(idx=idx, w=w.astype(np.float64), offsets=rt["offsets"].cpu().numpy(), row_src=rt["row_src"].cpu().numpy())
    mode = oracle.MODE_MXFP8 if wl.dtype == "mxfp8" else oracle.MODE_BF16
    c = TOL[dtype_of(wl)]
    want = oracle.moe_forward(inp.x, inp.Wg, inp.Wu, inp.Wd, ref, mode)
    assert_close(host_bf16_f64(served), want, c, "out")
    assert_close(host_bf16_f64(out), want, c, "out of the training forward")
    dX, dWg, dWu, dWd, dWr = oracle.moe_backward(inp.x, inp.W_r, inp.Wg, inp.Wu, inp.Wd, inp.dY, ref, mode)
    for n, r in (("dX", dX), ("dW_gate", dWg), ("dW_up", dWu), ("dW_down", dWd)):
        assert_close(host_bf16_f64(g[n]), r, c, n)
    assert_close(g["dW_r"].cpu().numpy().astype(np.float64), dWr, c, "dW_r", bf16_out=False)


@pytest.mark.gpu
@pytest.mark.parametrize("k,E", [(3, 8), (40, 64)])
def test_dispatch_passes_over_dropped_entries(k, E):
    """The rows of kept entries are mok_dispatch's, and nothing else is written, in the buffers or around them."""
    wl = synth.small("drop", T=70, H=256, I=128, E=E, k=k, dtype="mxfp8")
    inp = synth.make_inputs(wl, seed=3)
    p, x = mok.make_problem(wl.T, wl.H, wl.I, E, k, mok.MXFP8), to_dev_bf16(inp.x)
    idx, w = _choice(wl, 6)
    idx[np.random.default_rng(7).random(idx.shape) < 0.3] = -1
    idx[0, 0], idx[-1, -1] = E, 2 ** 31 - 1
    rt = _routing(idx, w, E)
    rows = mok.padded_rows_max(wl.T, E, k)
    gap, n, m = 1 << 20, rows * wl.H, rows * wl.H // 32
    room = torch.full((3 * gap + n + m,), 0xA5, dtype=torch.uint8, device="cuda")
    A, S = room[gap:gap + n], room[2 * gap + n:2 * gap + n + m]
    A1, S1 = mok.alloc_bytes(n), mok.alloc_bytes(m)
    mok.dispatch(p, x, rt, A1, S1)
    mok.dispatch_tokens(p, x, rt, A, S)
    counts = rt["counts"].tolist()
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    at = 0
    for c in counts:
        live[at:at + c] = True
        at += -(-c // 128) * 128
    A, A1 = A.view(rows, wl.H), A1.view(rows, wl.H)
    assert torch.equal(A[live], A1[live]) and (A[~live] == 0xA5).all()
    outside = torch.ones_like(room, dtype=torch.bool)
    outside[gap:gap + n] = outside[2 * gap + n:2 * gap + n + m] = False
    assert (room[outside] == 0xA5).all()


@pytest.mark.gpu
def test_router_gradient_passes_over_dropped_entries():
    """Dropped entries with weight 0, over buffers that held zeros: their results count as zeros, and the router's
    gradient is that of the entries kept. (What the layer gives for them in general is not specified.)"""
    wl = CASES[0]
    inp = synth.make_inputs(wl, seed=8)
    layer, x, dY = layer_for(inp, mok.BF16), to_dev_bf16(inp.x), to_dev_bf16(inp.dY)
    idx, w = _choice(wl, 9)
    full = _routing(idx, w, wl.E)
    ref = dict(idx=idx, w=w.astype(np.float64), offsets=full["offsets"].cpu().numpy(),
               row_src=full["row_src"].cpu().numpy())
    _, y = oracle.moe_forward(inp.x, inp.Wg, inp.Wu, inp.Wd, ref, oracle.MODE_BF16, return_y=True)
    drop = np.random.default_rng(10).random(idx.shape) < 0.3
    kept, w = np.where(drop, -1, idx).astype(np.int32), np.where(drop, 0, w).astype(np.float32)
    p = layer.problem(wl.T)
    ws, saved = (mok.alloc_bytes(n).zero_() for n in (mok.workspace_size(p), mok.saved_size(p)))
    out, g = _train(layer, wl, x, dY, _routing(kept, w, wl.E), saved, ws)
    want = (w.astype(np.float64)[..., None] * y).sum(1)
    assert_close(host_bf16_f64(out), want, TOL[mok.BF16], "out")
    gw = np.where(drop, 0, (host_bf16_f64(dY)[:, None] * y).sum(2))
    dl = w * (gw - (w * gw).sum(1, keepdims=True))
    dWr = np.zeros((wl.H, wl.E))
    xh = host_bf16_f64(x)
    for j in range(wl.k):
        for t in range(wl.T):
            if kept[t, j] >= 0:
                dWr[:, kept[t, j]] += xh[t] * dl[t, j]
    assert_close(g["dW_r"].cpu().numpy().astype(np.float64), dWr, TOL[mok.BF16], "dW_r", bf16_out=False)
