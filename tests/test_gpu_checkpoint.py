"""The training context in 8 bits: saved bytes stand for the MXFP8 values of
the context (exactly), the restored context is that of a layer with those
activations, and the backward runs on it."""
import ctypes

import numpy as np
import pytest
import torch

import mxref
from combine_router_top_expert_gb300 import mok, synth
from helpers import TOL, assert_close, dtype_of, host_bf16_f64, layer_for, to_dev_bf16

CASES = [
    synth.small("tiny", T=64, H=128, I=64, E=8, k=2, backward=True),
    synth.small("one_token", T=1, H=256, I=128, E=16, k=4, backward=True),
    synth.small("one_expert", T=130, H=256, I=128, E=1, k=1, backward=True),
    synth.small("sparse", T=8, H=256, I=128, E=64, k=1, backward=True),
    synth.small("ragged", T=700, H=512, I=256, E=8, k=2, zipf_s=1.2, backward=True),
    synth.small("mx", T=300, H=512, I=256, E=8, k=2, dtype="mxfp8", zipf_s=1.2, backward=True),
    synth.small("e256", T=300, H=256, I=128, E=256, k=8, zipf_s=1.2, backward=True),
]
IDS = [w.name for w in CASES]


def saved_views(saved, wl):
    """A, G|U, h and the partials in the saved context (mok_saved_size)."""
    R = -(-mok.padded_rows_max(wl.T, wl.E, wl.k) // 128) * 128
    out, at = {}, 0
    for n, r, w, dt, b in (("A", R, wl.H, torch.bfloat16, 2), ("gu", R, 2 * wl.I, torch.float32, 4),
                           ("h", R, wl.I, torch.bfloat16, 2), ("partials", wl.T * wl.k, wl.H, torch.bfloat16, 2)):
        out[n] = saved[at:at + r * w * b].view(dt).view(r, w)
        at += -(-r * w * b // 1024) * 1024
    return out


def padded_rows(routing, wl):
    """Padded row of every slot t*k + j, and the rows of all segments."""
    counts, off = routing["counts"].long(), routing["offsets"].long()
    seg = (counts + 127) // 128 * 128
    poff = torch.cat([seg.new_zeros(1), seg.cumsum(0)])
    e = routing["topk_idx"].long().reshape(-1)
    return poff[e] + routing["slot_row"].long()[:wl.T * wl.k] - off[e], int(poff[-1])


def trained(wl, seed=0):
    inp = synth.make_inputs(wl, seed=seed)
    layer = layer_for(inp, dtype_of(wl))
    x = to_dev_bf16(inp.x)
    layer.forward(x, training=True)
    b = layer.buffers(wl.T, True)
    return inp, layer, x, b["routing"], b["saved"]


@pytest.mark.gpu
@pytest.mark.parametrize("wl", CASES, ids=IDS)
def test_restored_context_is_the_mxfp8_values_of_the_saved_one(wl):
    inp, layer, x, routing, saved = trained(wl)
    p = layer.problem(wl.T)
    v = {n: t.clone() for n, t in saved_views(saved, wl).items()}
    ckpt = mok.alloc_bytes(mok.checkpoint_size(p))
    ckpt.fill_(0xFF)
    mok.checkpoint_save(p, x, routing, saved, ckpt)
    back = mok.alloc_bytes(mok.saved_size(p))
    back.fill_(0xFF)                                          # NaN wherever nothing is written
    x2 = torch.full_like(x, float("nan"))
    mok.checkpoint_load(p, ckpt, routing, x2, back)
    torch.cuda.synchronize()
    rows, total = padded_rows(routing, wl)
    w = saved_views(back, wl)
    assert torch.equal(x2.double(), mxref.values(x))
    assert torch.equal(w["partials"].double(), mxref.values(v["partials"]))
    want_gu = torch.zeros((total, 2 * wl.I), dtype=torch.float64, device="cuda")
    want_gu[rows] = mxref.values(v["gu"][rows])
    assert torch.equal(w["gu"][:total].double(), want_gu)     # pad rows zero
    want_A = torch.zeros((total, wl.H), dtype=torch.bfloat16, device="cuda")
    want_A[rows] = x2.repeat_interleave(wl.k, 0)
    assert torch.equal(w["A"][:total], want_A)
    g, u = want_gu[:, :wl.I], want_gu[:, wl.I:]
    h = g / (1 + torch.exp(-g)) * u
    # silu and one product in fp32 (a few units of 2^-24), then one BF16 rounding
    assert ((w["h"][:total].double() - h).abs() <= mxref.half_ulp_bf16(h, w["h"][:total]) + 2.0 ** -20 * h.abs()).all()
    assert bool((back.view(torch.uint8) == 0xFF).any()) or total == w["A"].shape[0]
    # a second round changes nothing: the values are those of their own bytes
    ckpt2 = mok.alloc_bytes(mok.checkpoint_size(p))
    ckpt2.fill_(0xFF)
    mok.checkpoint_save(p, x2, routing, back, ckpt2)
    x3 = torch.empty_like(x)
    again = mok.alloc_bytes(mok.saved_size(p))
    mok.checkpoint_load(p, ckpt2, routing, x3, again)
    assert torch.equal(x3, x2)
    for n in ("gu", "h", "A"):
        assert torch.equal(saved_views(again, wl)[n][:total], w[n][:total]), n


@pytest.mark.gpu
@pytest.mark.parametrize("wl", [w for w in CASES if w.dtype == "bf16"], ids=[w.name for w in CASES if w.dtype == "bf16"])
def test_backward_from_the_checkpoint(wl):
    """mok_moe_backward on the restored context against the gradient formulas
    in 64 bits on the same context, at the backward's own tolerance. As in the
    backward's other tests, the reference rounds what the GEMMs take as BF16
    operands (dy = w dY, dG, dU) and nothing else."""
    inp, layer, x, routing, saved = trained(wl, seed=2)
    p = layer.problem(wl.T)
    dY = to_dev_bf16(inp.dY)
    ckpt = mok.alloc_bytes(mok.checkpoint_size(p))
    mok.checkpoint_save(p, x, routing, saved, ckpt)
    saved.fill_(0)                                            # the buffer served another layer meanwhile
    x2 = torch.empty_like(x)
    mok.checkpoint_load(p, ckpt, routing, x2, saved)
    got = layer.backward(x2, dY)
    torch.cuda.synchronize()
    assert layer.status(wl.T, training=True) == (mok.OK, 0)

    v = saved_views(saved, wl)
    rows, _ = padded_rows(routing, wl)
    T, k, I = wl.T, wl.k, wl.I
    e = routing["topk_idx"].long().reshape(-1)
    w = routing["topk_w"].double().reshape(-1)
    bf16 = lambda t: t.to(torch.bfloat16).double()
    dy = dY.double().repeat_interleave(k, 0)
    G, U = v["gu"][rows, :I].double(), v["gu"][rows, I:].double()
    y, h = v["partials"].double(), v["h"][rows].double()
    sg = torch.sigmoid(G)
    dX = torch.zeros((T, wl.H), dtype=torch.float64, device="cuda")
    tok = torch.arange(T, device="cuda").repeat_interleave(k)
    for ee in range(wl.E):
        m = (e == ee).nonzero()[:, 0]
        d = bf16(w[m, None] * dy[m])
        dh = d @ layer.Wd[ee].double().t()
        dG, dU = bf16(dh * U[m] * sg[m] * (1 + G[m] * (1 - sg[m]))), bf16(dh * G[m] * sg[m])
        dX.index_add_(0, tok[m], dG @ layer.Wg[ee].double().t() + dU @ layer.Wu[ee].double().t())
        if len(m):
            a = x2[tok[m]].double()
            for name, ref in (("dW_gate", a.t() @ dG), ("dW_up", a.t() @ dU), ("dW_down", h[m].t() @ d)):
                assert_close(host_bf16_f64(got[name][ee]), ref.cpu().numpy(), TOL[mok.BF16], f"{wl.name} {name}[{ee}]")
    gw = (dy * y).sum(1).reshape(T, k)
    wk = w.reshape(T, k)
    dl = wk * (gw - (wk * gw).sum(1, keepdim=True))
    full = torch.zeros((T, wl.E), dtype=torch.float64, device="cuda").scatter_(1, e.reshape(T, k), dl)
    dX += full @ layer.W_r.double().t()
    assert_close(host_bf16_f64(got["dX"]), dX.cpu().numpy(), TOL[mok.BF16], f"{wl.name} dX")
    dWr = (x2.double().t() @ full).cpu().numpy()
    if np.abs(dWr).max() > 0:
        assert_close(got["dW_r"].double().cpu().numpy(), dWr, TOL[mok.BF16], f"{wl.name} dW_r", bf16_out=False)


@pytest.mark.gpu
def test_checkpoint_keeps_gradients_near():
    """Gradients from the checkpoint differ from those of the full context by
    the rounding of x, G|U and y to four significant bits: each value moves by
    at most 2^-4 of itself (uniformly spread: about 2^-4 / sqrt(3) in the mean),
    and dX and the weight gradients are sums of products of at most four such
    values, so 4 * 2^-4 bounds the relative 2-norm with room."""
    wl = synth.small("near", T=600, H=512, I=256, E=8, k=2, backward=True)
    inp, layer, x, routing, saved = trained(wl, seed=5)
    p, dY = layer.problem(wl.T), to_dev_bf16(inp.dY)
    full = {n: t.clone() for n, t in layer.backward(x, dY).items()}
    ckpt = mok.alloc_bytes(mok.checkpoint_size(p))
    mok.checkpoint_save(p, x, routing, saved, ckpt)
    x2 = torch.empty_like(x)
    mok.checkpoint_load(p, ckpt, routing, x2, saved)
    near = layer.backward(x2, dY)
    for n in full:
        d = (near[n].double() - full[n].double()).norm() / full[n].double().norm()
        print(f"[checkpoint] {n}: relative difference {float(d):.3e}")
        assert float(d) <= 4 * 2.0 ** -4, n


@pytest.mark.gpu
def test_size_is_a_quarter():
    wl = synth.WORKLOADS["bf16_bwd_T4096"]
    p = mok.make_problem(wl.T, wl.H, wl.I, wl.E, wl.k)
    assert 4 * mok.checkpoint_size(p) < mok.saved_size(p)


def test_refusals():
    L = mok.lib()
    p = mok.make_problem(64, 128, 64, 8, 2)
    n = mok.checkpoint_size(p)
    assert n >= 64 * 128 + 128 * 128 + 128 * 128
    assert mok.checkpoint_size(mok.make_problem(64, 100, 64, 8, 2)) == 0
    r = mok.Routing(4096, 4096, 4096, 4096, 4096, 4096)
    ok = dict(p=p, x=4096, r=r, saved=8192, ckpt=16384, n=n)
    for bad in (dict(p=mok.make_problem(64, 100, 64, 8, 2)), dict(x=None), dict(r=mok.Routing()), dict(saved=None),
                dict(ckpt=None), dict(n=n - 1), dict(saved=8448), dict(ckpt=16385), dict(x=4100)):
        a = {**ok, **bad}
        assert L.mok_checkpoint_save(ctypes.byref(a["p"]), a["x"], ctypes.byref(a["r"]), a["saved"], a["ckpt"], a["n"],
                                     None) == mok.ERR_INVALID, bad
        assert L.mok_checkpoint_load(ctypes.byref(a["p"]), a["ckpt"], a["n"], ctypes.byref(a["r"]), a["x"], a["saved"],
                                     None) == mok.ERR_INVALID, bad
