"""The MXFP8 layer's backward from the 8-bit context: against the gradient
formulas in 64 bits with the backward's own operand rounding, whatever bytes
the context's buffer held before."""
import pytest
import torch

import mxref
from combine_router_top_expert_gb300 import mok, synth
from helpers import TOL, assert_close, dtype_of, host_bf16_f64, layer_for, to_dev_bf16

CASES = [
    synth.small("mx", T=300, H=512, I=256, E=8, k=2, dtype="mxfp8", zipf_s=1.2, backward=True),
    synth.small("mx_idle_experts", T=9, H=256, I=128, E=16, k=1, dtype="mxfp8", backward=True),
    synth.small("mx_h384", T=200, H=384, I=128, E=4, k=3, dtype="mxfp8", backward=True),
    synth.small("bf16", T=300, H=512, I=256, E=8, k=2, zipf_s=1.2, backward=True),
]


def _views(saved, wl):
    R = -(-mok.padded_rows_max(wl.T, wl.E, wl.k) // 128) * 128
    out, at = {}, 0
    for n, r, w, dt, b in (("A", R, wl.H, torch.bfloat16, 2), ("gu", R, 2 * wl.I, torch.float32, 4),
                           ("h", R, wl.I, torch.bfloat16, 2), ("partials", wl.T * wl.k, wl.H, torch.bfloat16, 2)):
        out[n] = saved[at:at + r * w * b].view(dt).view(r, w)
        at += -(-r * w * b // 1024) * 1024
    return out


def _from_checkpoint(wl, seed=4):
    """(inputs, layer, restored x, routing, restored context, gradients per byte that the buffer held before)."""
    inp = synth.make_inputs(wl, seed=seed)
    layer = layer_for(inp, dtype_of(wl))
    x, dY = to_dev_bf16(inp.x), to_dev_bf16(inp.dY)
    layer.forward(x, training=True)
    b, p = layer.buffers(wl.T, True), layer.problem(wl.T)
    ckpt = mok.alloc_bytes(mok.checkpoint_size(p))
    mok.checkpoint_save(p, x, b["routing"], b["saved"], ckpt)
    grads = {}
    for fill in (0, 0xFF, 0x7F):                              # zeros, NaN in every type, NaN in E4M3
        b["saved"].fill_(fill)
        b["ws"].fill_(fill)
        x2 = torch.empty_like(x)
        mok.checkpoint_load(p, ckpt, b["routing"], x2, b["saved"])
        grads[fill] = {n: t.clone() for n, t in layer.backward(x2, dY).items()}
        torch.cuda.synchronize()
        assert layer.status(wl.T, training=True) == (mok.OK, 0)
    return layer, x2, dY, b["routing"], b["saved"], grads


@pytest.mark.gpu
@pytest.mark.parametrize("wl", CASES, ids=[w.name for w in CASES])
def test_earlier_bytes_of_the_context_do_not_matter(wl):
    *_, grads = _from_checkpoint(wl)
    for fill in (0xFF, 0x7F):
        for n, t in grads[0].items():
            assert torch.isfinite(t).all(), n
            assert torch.equal(grads[fill][n].view(torch.uint8), t.view(torch.uint8)), (fill, n)


@pytest.mark.gpu
@pytest.mark.parametrize("wl", [w for w in CASES if w.dtype == "mxfp8"], ids=[w.name for w in CASES if w.dtype == "mxfp8"])
def test_backward_from_the_checkpoint(wl):
    """Every GEMM operand as MXFP8 blocked along that GEMM's reduction: dy and W_down along H, dG|dU and W_gate, W_up
    along I, and for the weight gradients the expert's rows, padded to 128 with zeros, along the tokens. dy, dG and
    dU are BF16 before. The tolerance is that of MXFP8 operands in all of the layer's tests."""
    layer, x2, dY, routing, saved, grads = _from_checkpoint(wl)
    got, v = grads[0xFF], _views(saved, wl)
    T, H, I, E, k = wl.T, wl.H, wl.I, wl.E, wl.k
    counts, off = routing["counts"].long(), routing["offsets"].long()
    seg = (counts + 127) // 128 * 128
    poff = torch.cat([seg.new_zeros(1), seg.cumsum(0)]).tolist()
    e = routing["topk_idx"].long().reshape(-1)
    rows = torch.tensor(poff, device="cuda")[e] + routing["slot_row"].long()[:T * k] - off[e]
    w = routing["topk_w"].double()
    bf16 = lambda t: t.to(torch.bfloat16).double()
    dyk = dY.double().repeat_interleave(k, 0)
    tok = torch.arange(T, device="cuda").repeat_interleave(k)
    d = torch.zeros((poff[-1], H), dtype=torch.float64, device="cuda")
    d[rows] = bf16(w.reshape(-1, 1) * dyk)
    token_of = torch.full((poff[-1],), -1, device="cuda")
    token_of[rows] = tok
    c, dX = TOL[mok.MXFP8], torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for ee in range(E):
        lo, hi = poff[ee], poff[ee + 1]
        if lo == hi:
            for n in ("dW_gate", "dW_up", "dW_down"):
                assert (got[n][ee] == 0).all(), n
            continue
        G, U = v["gu"][lo:hi, :I].double(), v["gu"][lo:hi, I:].double()
        sg = torch.sigmoid(G)
        dh = mxref.values(d[lo:hi]) @ mxref.values(layer.Wd[ee]).t()
        dG, dU = bf16(dh * U * sg * (1 + G * (1 - sg))), bf16(dh * G * sg)
        da = mxref.values(dG) @ mxref.values(layer.Wg[ee]).t() + mxref.values(dU) @ mxref.values(layer.Wu[ee]).t()
        m = token_of[lo:hi] >= 0
        dX.index_add_(0, token_of[lo:hi][m], da[m])
        cols = lambda t: mxref.values(t.t().contiguous())
        a, h = cols(v["A"][lo:hi]), cols(v["h"][lo:hi])
        for n, ref in (("dW_gate", a @ cols(dG).t()), ("dW_up", a @ cols(dU).t()), ("dW_down", h @ cols(d[lo:hi]).t())):
            assert_close(host_bf16_f64(got[n][ee]), ref.cpu().numpy(), c, f"{wl.name} {n}[{ee}]")
    gw = (dyk * v["partials"].double()).sum(1).reshape(T, k)
    dl = w * (gw - (w * gw).sum(1, keepdim=True))
    full = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, e.reshape(T, k), dl)
    dX += full @ layer.W_r.double().t()
    assert_close(host_bf16_f64(got["dX"]), dX.cpu().numpy(), c, f"{wl.name} dX")
    dWr = (x2.double().t() @ full).cpu().numpy()
    if k > 1:                                                 # with one expert a token the weights are 1
        assert_close(got["dW_r"].double().cpu().numpy(), dWr, c, f"{wl.name} dW_r", bf16_out=False)
