"""The block's operators captured in a CUDA graph and replayed on new inputs, as
a decode server runs them: the bits of plain calls."""
import pytest
import torch

from combine_router_top_expert_gb300 import mok, synth
from combine_router_top_expert_gb300.block import MoEBlock
from helpers import dtype_of, layer_for

S = synth.small
FEW = [S("bf16", T=7, H=512, I=256, E=8, k=2),
       S("cut", T=40, H=2048, I=128, E=4, k=2),               # tiles cut over many CTAs
       S("e64_shared", T=33, H=512, I=256, E=64, k=4, shared_I=256),
       S("mx_shared", T=100, H=896, I=128, E=40, k=3, dtype="mxfp8", shared_I=128)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _captured(f):
    """f() recorded after a plain call: (graph, what f returned)."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


@pytest.mark.gpu
@pytest.mark.parametrize("wl", FEW, ids=[w.name for w in FEW])
def test_few_tokens(wl):
    """Three calls back to back in the graph, on one workspace: each waits for the one before."""
    layer = layer_for(synth.make_inputs(wl, with_x=False), dtype_of(wl))
    p, g = layer.problem(wl.T), _gen(5)
    ws = mok.alloc_bytes(mok.few_workspace_size(p))
    xs = [torch.empty((wl.T, wl.H), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    outs = [torch.empty_like(x) for x in xs]

    def call(x, out):
        mok.moe_few(p, x, layer.W_r, layer.packed, out, ws, bias=layer.bias, packed_shared=layer.packed_shared)

    graph, _ = _captured(lambda: [call(x, o) for x, o in zip(xs, outs)])
    for _ in range(3):
        for x in xs:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        graph.replay()
        got = [o.clone() for o in outs]
        torch.cuda.synchronize()
        assert mok.device_status(ws) == (mok.OK, 0)
        for x, a in zip(xs, got):
            want = torch.empty_like(x)
            call(x, want)
            assert torch.equal(a.view(torch.int16), want.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 128, 200])
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_block_forward(T, dtype):
    """Two blocks one after the other. A larger batch in between, outside the graph, leaves it good."""
    wls = [S("graph", T=128, H=512, I=256, E=8, k=2, dtype=dtype) for _ in range(2)]
    blocks = [MoEBlock(layer_for(synth.make_inputs(w, seed=n, with_x=False), dtype_of(w)), torch.ones(512, device="cuda"))
              for n, w in enumerate(wls)]
    g = _gen(6)
    x = torch.randn((T, 512), generator=g, device="cuda").to(torch.bfloat16)

    def forward(x):
        h, res = x, None
        for b in blocks:
            h, res = b.forward(h, res)
        return h, res

    graph, (h, res) = _captured(lambda: forward(x))
    forward(torch.randn((128, 512), generator=g, device="cuda").to(torch.bfloat16))
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        got = h.clone(), res.clone()
        torch.cuda.synchronize()
        assert all(b.status() == (mok.OK, 0) for b in blocks)
        for a, want in zip(got, forward(x)):
            assert torch.equal(a.view(torch.int16), want.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_training_step(dtype):
    wl = S("graph", T=300, H=512, I=256, E=8, k=2, dtype=dtype)
    block = MoEBlock(layer_for(synth.make_inputs(wl, with_x=False), dtype_of(wl)), torch.ones(512, device="cuda"))
    g = _gen(7)
    x, d = (torch.randn((300, 512), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))

    def step():
        out, total, ctx = block.train_forward(x, d)
        return dict(block.train_backward(ctx, d, total), out=out, total=total)

    graph, got = _captured(step)
    for _ in range(2):
        for t in (x, d):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        first = {n: t.clone() for n, t in got.items()}
        torch.cuda.synchronize()
        for n, want in step().items():
            assert torch.equal(first[n].view(torch.uint8), want.view(torch.uint8)), n
