"""Layouts on a stream that is not the current one, without a workspace: scratch and outputs are that stream's memory."""
import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import mok


def _owner(t):
    """The stream whose memory holds t, by the allocator's own record."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment")


def _calls():
    T, k, E, H = 3000, 2, 64, 256          # 6000 entries: their places come from the scratch
    idx = torch.randint(-1, E, (T, k), generator=torch.Generator().manual_seed(1)).int()
    x = torch.randn((T, H), generator=ref.gen(2), device="cuda").to(torch.bfloat16)
    W_r = torch.randn((H, E), generator=ref.gen(3), device="cuda")
    dev = idx.cuda()
    torch.cuda.synchronize()
    return {"sort_layout": (lambda s: mok.sort_layout(dev, E, stream=s), idx, E),
            "route_layout": (lambda s: mok.route_layout(x, W_r, k, stream=s), None, E)}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["sort_layout", "route_layout"])
def test_scratch_and_outputs_belong_to_the_given_stream(name, monkeypatch):
    call, _, _ = _calls()[name]
    kept, real = [], mok.alloc_bytes       # kept alive, so that nothing else is put there
    monkeypatch.setattr(mok, "alloc_bytes", lambda *a: kept.append(real(*a)) or kept[-1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = call(side)
    side.synchronize()
    assert len(kept) == 1
    assert all(_owner(t) == side.cuda_stream for t in kept + list(out.values()))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["sort_layout", "route_layout"])
def test_two_streams_with_work_between(name):
    """Calls on two streams in turn, each behind other work, while the current stream allocates and writes blocks of the
    scratch's size: every layout is right."""
    call, idx, E = _calls()[name]
    want = call(None)
    if idx is not None:
        for n, w in zip(("counts", "offsets", "row_src", "slot_row"), ref.layout(idx.tolist(), E)):
            assert want[n].tolist() == list(w), n
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    busy = torch.zeros(1 << 26, device="cuda")
    for i in range(8):
        s = streams[i % 2]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            busy.add_(1) if i % 2 == 0 else torch.zeros(1 << 24, device="cuda")
        got.append(call(s))
        for size in (1 << 10, 1 << 13, 1 << 14, 1 << 16):
            mok.alloc_bytes(size).fill_(0x7F)
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(out[n], want[n]) for n in want)
