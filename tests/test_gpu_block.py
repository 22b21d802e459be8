"""The block (pre-norm, layer, 8-bit checkpoints): its outputs against the
oracle's layer on the normed rows, its gradients against the formulas."""
import os
import subprocess
import sys

import pytest
import torch

import mxref
import oracle
from combine_router_top_expert_gb300 import mok, synth
from combine_router_top_expert_gb300.block import MoEBlock
from helpers import TOL, assert_close, dtype_of, host_bf16_f64, layer_for

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _block(wl, seed=0):
    inp = synth.make_inputs(wl, seed=seed, with_x=False)
    layer = layer_for(inp, dtype_of(wl))
    g = torch.Generator(device="cuda").manual_seed(seed)
    gain = 1 + 0.2 * torch.randn(wl.H, generator=g, device="cuda")
    x, r = ((torch.randn((wl.T, wl.H), generator=g, device="cuda") * s).to(torch.bfloat16) for s in (1.0, 2.0))
    return inp, MoEBlock(layer, gain), x, r, g


def _normed(block, x, r):
    s = x.double() + r.double()
    y = s * (s.square().mean(1, keepdim=True) + block.eps).rsqrt() * block.gain.double()
    total, out = torch.empty_like(x), torch.empty_like(x)
    mok.rmsnorm(x, block.gain, residual=r, eps=block.eps, sum=total, y=out)
    assert ((out.double() - y).abs() <= mxref.half_ulp_bf16(y, out) + 2.0 ** -16 * y.abs()).all()
    return total, out


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 128, 129, 300])      # few-token kernels up to 128, the stages beyond
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_forward(T, dtype):
    wl = synth.small("block", T=T, H=512, I=256, E=8, k=2, dtype=dtype, shared_I=256)
    inp, block, x, r, _ = _block(wl)
    out, stream = block.forward(x, r)
    total, y = _normed(block, x, r)
    assert torch.equal(stream, total)
    bits = y.view(torch.int16).cpu().numpy().view("uint16")
    rt = oracle.route(bits, inp.W_r, wl.k, inp.bias)
    mode = oracle.MODE_MXFP8 if dtype == "mxfp8" else oracle.MODE_BF16
    ref = oracle.moe_forward(bits, inp.Wg, inp.Wu, inp.Wd, rt, mode=mode, shared=inp.shared)
    assert_close(host_bf16_f64(out), ref, TOL[dtype_of(wl)], f"block T={T}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_training_step(dtype):
    """The layer's gradients are those of mok_moe_backward on the restored
    context, bit for bit; the norm's follow from its dX by the formula on the
    8-bit stream (tolerances as in the norm's own tests). Two forwards before the
    backwards: a context outlives the buffers it was made in."""
    wl = synth.small("block", T=300, H=512, I=256, E=8, k=2, dtype=dtype)
    _, block, x, r, g = _block(wl, seed=3)
    layer = block.layer
    out1, s1, c1 = block.train_forward(x, r)
    _, _, c2 = block.train_forward(x)                         # another input
    again, _ = block.forward(x, r)
    total, y = _normed(block, x, r)
    assert torch.equal(s1, total) and torch.equal(out1, again)
    dout, dstream = ((torch.randn((wl.T, wl.H), generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    g2 = block.train_backward(c2, dout, dstream)
    g1 = block.train_backward(c1, dout, dstream)
    torch.cuda.synchronize()
    assert layer.status(wl.T, training=True) == (mok.OK, 0)
    # by hand
    p, b = layer.problem(wl.T), layer.buffers(wl.T, True)
    y2 = torch.empty_like(y)
    mok.checkpoint_load(p, c1["ckpt"], c1["routing"], y2, b["saved"])
    assert torch.equal(y2.double(), mxref.values(y))
    ref = dict(dX=torch.empty_like(y), dW_gate=torch.empty_like(layer.Wg), dW_up=torch.empty_like(layer.Wu),
               dW_down=torch.empty_like(layer.Wd), dW_r=torch.empty((wl.H, wl.E), device="cuda"))
    mok.moe_backward(p, y2, layer.W_r, layer.Wg, layer.Wu, layer.Wd, layer.packed, dout, c1["routing"], b["saved"],
                     ref, b["ws"], packed_bwd=layer.packed_bwd)
    for n in ("dW_gate", "dW_up", "dW_down", "dW_r"):
        assert torch.equal(g1[n], ref[n]), n
        assert not torch.equal(g2[n], ref[n]), n
    s = mxref.values(total)
    R = c1["rstd"].double()[:, None]
    xh, a, dy = s * R, ref["dX"].double() * block.gain.double(), ref["dX"].double()
    dx = dstream.double() + R * (a - xh * (a * xh).mean(1, keepdim=True))
    size = dstream.double().abs() + R * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    assert ((g1["dx"].double() - dx).abs() <= mxref.half_ulp_bf16(dx, g1["dx"]) + 2.0 ** -16 * size).all()
    dg, mag = (dy * xh).sum(0), (dy * xh).abs().sum(0)
    assert ((g1["dgain"].double() - dg).abs() <= (1 + 64) * 2.0 ** -24 * mag).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 300])
def test_side_stream_keeps_its_temporaries(T):
    """What a call on another stream allocates and drops is not reused by the
    current stream while its kernels wait: memory of the same sizes, taken and
    filled on the current stream right after the call, changes nothing."""
    wl = synth.small("block", T=T, H=512, I=256, E=8, k=2)
    _, block, x, r, _ = _block(wl)
    want, ctx0 = block.train_forward(x, r)[::2]
    gwant = block.train_backward(ctx0, want)
    served = block.forward(x, r)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = block.forward(x, r, stream=side)[0]
    out, _, ctx = block.train_forward(x, r, stream=side)
    g = block.train_backward(ctx, want, stream=side)
    trash = [torch.full((T, 512), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert torch.equal(got, served) and torch.equal(out, want) and len(trash) == 16
    for n, v in gwant.items():
        assert torch.equal(g[n], v), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_no_tokens(dtype):
    wl = synth.small("block", T=4, H=512, I=256, E=8, k=2, dtype=dtype)
    _, block, x, r, _ = _block(wl)
    out, stream = block.forward(x[:0], r[:0])
    assert out.shape == stream.shape == (0, 512)


@pytest.mark.gpu
def test_example_runs():
    for extra in ([], ["--mxfp8"]):
        r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_block.py"), "--layers", "2", "--tokens",
                            "300", "--batch", "3", *extra], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        assert "decoding step" in r.stdout
