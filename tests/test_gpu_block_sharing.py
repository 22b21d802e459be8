"""Blocks that share one full training context: the gradients of blocks with
their own, in the memory of one context and a checkpoint per block."""
import pytest
import torch

from combine_router_top_expert_gb300 import mok, synth
from combine_router_top_expert_gb300.block import BlockBuffers, MoEBlock
from helpers import dtype_of, layer_for

T, H = 700, 512


def _layers(*shapes):
    out = []
    for n, (I, E, k, dtype) in enumerate(shapes):
        wl = synth.small("shared", T=T, H=H, I=I, E=E, k=k, dtype=dtype)
        out.append(layer_for(synth.make_inputs(wl, seed=n, with_x=False), dtype_of(wl)))
    return out


def _step(blocks):
    """Forward through all blocks, then backward: (last output, gradients of every block)."""
    g = torch.Generator(device="cuda").manual_seed(9)
    h, res, ctxs = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16), None, []
    for b in blocks:
        h, res, ctx = b.train_forward(h, res)
        ctxs.append(ctx)
    dout = dstream = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    grads = []
    for b, ctx in zip(reversed(blocks), reversed(ctxs)):
        grads.append(b.train_backward(ctx, dout, dstream))
        dout = dstream = grads[-1]["dx"]
    torch.cuda.synchronize()
    assert all(b.status(c) == (mok.OK, 0) for b, c in zip(blocks, ctxs))
    return h, grads


@pytest.mark.gpu
@pytest.mark.parametrize("shapes", [[(256, 8, 2, "bf16")] * 3,
                                    [(256, 8, 2, "bf16"), (384, 4, 3, "bf16"), (256, 8, 2, "mxfp8")]],
                         ids=["alike", "different"])
def test_gradients_of_blocks_that_share(shapes):
    gain = torch.linspace(0.5, 1.5, H, device="cuda")
    layers, shared = _layers(*shapes), BlockBuffers()
    want, gwant = _step([MoEBlock(l, gain) for l in layers])
    got, ggot = _step([MoEBlock(l, gain, buffers=shared) for l in layers])
    assert torch.equal(got, want)
    for a, b in zip(ggot, gwant):
        for n in b:
            assert torch.equal(a[n], b[n]), n


@pytest.mark.gpu
def test_memory_of_a_stack():
    """One context and the workspaces once, whatever the number of blocks; per block what its ctx holds."""
    n = 6
    layers, gain, shared = _layers(*[(256, 8, 2, "bf16")] * n), torch.ones(H, device="cuda"), BlockBuffers()
    p = layers[0].problem(T)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    blocks = [MoEBlock(l, gain, buffers=shared) for l in layers]
    # bytes asked for: the allocator's blocks are larger where it keeps a remainder of under 1 MB
    asked = lambda: torch.cuda.memory_stats()["requested_bytes.all.current"]
    before = asked()
    ctxs = [b.train_forward(x)[2] for b in blocks]
    held = asked() - before
    once = mok.saved_size(p) + mok.workspace_size(p) + mok.route_workspace_size(T, H, 8, 2)
    per_block = mok.checkpoint_size(p) + T * (H + H // 32 + 4) + T * 2 * 4 * 4
    assert len(ctxs) == n and held <= once + n * (per_block + 16 * 1024) + (1 << 20)
    assert not any(l._bufs for l in layers)
