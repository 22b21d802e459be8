"""Memory that a block keeps between calls: bounded, however many batch sizes it
has seen."""
import pytest
import torch

from combine_router_top_expert_gb300 import mok, synth
from combine_router_top_expert_gb300.block import MoEBlock
from helpers import dtype_of, layer_for


def _block(k=2, E=8, dtype="bf16", T=128):
    wl = synth.small("memory", T=T, H=512, I=256, E=E, k=k, dtype=dtype)
    layer = layer_for(synth.make_inputs(wl, with_x=False), dtype_of(wl))
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, wl.H), generator=g, device="cuda").to(torch.bfloat16)
    return layer, MoEBlock(layer, torch.ones(wl.H, device="cuda")), x


def _held(f):
    """Bytes that are allocated after f() beyond those before it."""
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    f()
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before


@pytest.mark.gpu
@pytest.mark.parametrize("k,E,dtype", [(2, 8, "bf16"), (2, 8, "mxfp8"), (24, 32, "bf16")])   # k=24: 85 tokens at most
def test_decode_batches_of_every_size(k, E, dtype):
    layer, block, x = _block(k, E, dtype)
    most = max(T for T in range(129) if mok.few_tokens_ok(T, k))

    def serve():
        for T in range(most + 1):
            block.forward(x[:T])

    held = _held(serve)
    assert held <= 2.1 * mok.few_workspace_size(layer.problem(most)) + 6 * 4096
    assert _held(serve) == 0
    # a larger workspace than a call needs gives the same bits
    for T in (1, 9, 33, most):
        out, total = block.forward(x[:T])
        y, want = torch.empty_like(total), torch.empty_like(total)
        mok.rmsnorm(x[:T], block.gain, eps=block.eps, y=y)
        p = layer.problem(T)
        mok.moe_few(p, y, layer.W_r, layer.packed, want, mok.alloc_bytes(mok.few_workspace_size(p)))
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), T


@pytest.mark.gpu
def test_training_batches_share_the_norms_workspace():
    layer, block, x = _block(T=2048)
    sizes = (1, 5, 64, 300, 1000, 2048)
    for T in sizes:
        layer.buffers(T, True)

    def train():
        for T in sizes:
            out, _, ctx = block.train_forward(x[:T])
            block.train_backward(ctx, out)

    assert _held(train) <= 1.1 * mok.rmsnorm_bwd_workspace_size(1 << 20, layer.H) + 4096
