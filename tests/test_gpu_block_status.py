"""Waits that give up inside a block's calls reach its status."""
import pytest
import torch

from combine_router_top_expert_gb300 import mok, synth
from combine_router_top_expert_gb300.block import MoEBlock
from helpers import dtype_of, layer_for

OK = (mok.OK, 0)


def _block(T, k=2, dtype="bf16", H=512):
    wl = synth.small("status", T=T, H=H, I=256, E=32, k=k, dtype=dtype)
    layer = layer_for(synth.make_inputs(wl, with_x=False), dtype_of(wl))
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, wl.H), generator=g, device="cuda").to(torch.bfloat16)
    return layer, MoEBlock(layer, torch.ones(wl.H, device="cuda")), x


def _marks(monkeypatch, name):
    """From here on, `name` leaves a failure in its workspace's status (the layer's own calls have no test hook
    for that)."""
    f = getattr(mok, name)

    def marked(*a, **kw):
        r = f(*a, **kw)
        ws = a[5] if name == "moe_forward" else a[11]
        ws[:8].view(torch.int32).copy_(torch.tensor([mok.ERR_TIMEOUT, 2], dtype=torch.int32))
        return r

    monkeypatch.setattr(mok, name, marked)


@pytest.mark.gpu
def test_few_tokens(monkeypatch):
    layer, block, x = _block(20)
    assert block.status() == OK                               # nothing was called
    want = block.forward(x)[0]
    assert block.status() == OK
    few = mok.moe_few
    cfg = mok.make_config(timeout_ms=50, flags=mok.FLAG_TEST_WITHHOLD_PUBLISH)
    monkeypatch.setattr(mok, "moe_few", lambda *a, **kw: few(*a, cfg=cfg, **kw))
    block.forward(x)
    assert block.status()[0] == mok.ERR_TIMEOUT
    assert block.status(stream=torch.cuda.Stream())[0] == mok.ERR_TIMEOUT
    monkeypatch.undo()
    assert torch.equal(block.forward(x)[0], want) and block.status() == OK


@pytest.mark.gpu
def test_stages(monkeypatch):
    layer, block, x = _block(700, k=8, H=2048)
    mok.route_test_hook(1, timeout_ms=50)                     # a router copy that never comes
    try:
        block.forward(x)
        assert block.status() == (mok.ERR_TIMEOUT, 7)
    finally:
        mok.route_test_hook(0, 0)
    block.forward(x)
    assert block.status() == OK
    with monkeypatch.context() as m:
        _marks(m, "moe_forward")
        block.forward(x)
    assert block.status() == (mok.ERR_TIMEOUT, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["routing", "forward", "backward"])
def test_training_context_keeps_it(what, monkeypatch):
    """Another step on the same buffers comes between: the context's own failure is still there."""
    layer, block, x = _block(700, k=8, H=2048)
    detail = 7 if what == "routing" else 2
    with monkeypatch.context() as m:
        if what == "forward":
            _marks(m, "moe_forward")
        if what == "routing":
            mok.route_test_hook(1, timeout_ms=50)
        try:
            out, _, ctx = block.train_forward(x)
            torch.cuda.synchronize()
        finally:
            mok.route_test_hook(0, 0)
    assert block.status() == block.status(ctx) == (OK if what == "backward" else (mok.ERR_TIMEOUT, detail))
    _, _, good = block.train_forward(x)
    assert block.status() == OK
    with monkeypatch.context() as m:
        if what == "backward":
            _marks(m, "moe_backward")
        block.train_backward(ctx, out)
    block.train_backward(good, out)
    assert block.status(ctx) == (mok.ERR_TIMEOUT, detail)
    assert block.status() == block.status(good) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("training", [False, True])
def test_fresh_buffers_have_a_good_status(training):
    layer, _, x = _block(200)
    trash = [torch.full((1 << 22,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del trash                                                 # what the buffers are then made of
    assert layer.status(200, training) == OK
