"""Rows sorted by given experts and summed back, with their gradients.

Tolerances: unsort adds k products in fp32, each fma rounded at 2^-24 of the sum of magnitudes, and rounds once; dw adds
H products in chains of at most ceil(H / 256) * 8 terms in a thread, 5 shuffle steps and 8 warps; dy is one product,
rounded to fp32 (where the type is smaller) and once more.
"""
import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import mok

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11), "f32": (torch.float32, 0.0)}


def _idx(T, k, E, seed, drop=0.0, distinct=False):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand((T, max(E, k)), generator=g).argsort(1)[:, :k] % E if distinct else \
        torch.randint(0, E, (T, k), generator=g)
    return torch.where(torch.rand((T, k), generator=g) < drop, -1, idx).int()


def _same(lay, want, T, k):
    for n, w in zip(("counts", "offsets", "row_src", "slot_row"), want):
        assert lay[n].tolist() == list(w), n


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 3), (7, 8, 32), (33, 3, 1024), (255, 1, 2), (256, 8, 256),
                                   (257, 8, 256), (1000, 2, 8), (4096, 8, 32), (5000, 7, 129), (40000, 1, 5)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_layout(T, k, E, drop):
    """Duplicates among a token's experts and dropped entries included."""
    idx = _idx(T, k, E, T + k + E, drop)
    if drop:
        idx[T // 2, 0] = E          # just outside, and far outside
        idx[-1, -1] = 2 ** 31 - 1
    lay = mok.sort_layout(idx.cuda(), E)
    _same(lay, ref.layout(idx.tolist(), E), T, k)


@pytest.mark.gpu
def test_layout_of_nothing_and_of_one_expert():
    lay = mok.sort_layout(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6)
    assert lay["counts"].tolist() == [0] * 6 and lay["offsets"].tolist() == [0] * 7
    idx = torch.full((3000, 2), -1, dtype=torch.int32)
    lay = mok.sort_layout(idx.cuda(), 6)
    _same(lay, ref.layout(idx.tolist(), 6), 3000, 2)
    idx[:] = 5
    lay = mok.sort_layout(idx.cuda(), 6)
    _same(lay, ref.layout(idx.tolist(), 6), 3000, 2)


@pytest.mark.gpu
def test_layout_is_the_routers():
    """On the router's own choice: the layout of mok_route_layout."""
    T, H, E, k = 1000, 256, 16, 4
    x = torch.randn((T, H), generator=ref.gen(1), device="cuda").to(torch.bfloat16)
    W_r = torch.randn((H, E), generator=ref.gen(2), device="cuda")
    r = mok.route_layout(x, W_r, k)
    lay = mok.sort_layout(r["topk_idx"], E)
    for n in lay:
        assert torch.equal(lay[n], r[n]), n


ROWS = [(1, 8, 1, 1), (3, 40, 8, 5), (7, 7168, 8, 32), (300, 1024, 2, 8), (33, 2056, 9, 16), (130, 8200, 17, 4),
        (2000, 64, 3, 7)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,k,E", ROWS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_rows(T, H, k, E, kind, drop):
    dt, half = TYPES[kind]
    g = ref.gen(T + H)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    lay = mok.sort_layout(_idx(T, k, E, T, drop).cuda(), E)
    R = int(lay["offsets"][-1])
    src, slot = lay["row_src"][:R].long(), lay["slot_row"].view(T, k).long()
    x, y, dout = rnd(T, H), rnd(T * k, H), rnd(T, H)
    w = torch.rand((T, k), generator=g, device="cuda")
    y[R:] = float("nan")                                    # rows behind the last one are not read
    xs = torch.full((T * k, H), 7.0, dtype=dt, device="cuda")
    mok.sort_rows(x, lay, xs)
    assert torch.equal(xs[:R], x[src // k]) and (xs[R:] == 7).all()
    live = (slot >= 0)[..., None]
    yd = torch.where(live, y[slot.clamp(min=0)].double(), 0.0)
    for weights in (w, None):
        out = torch.full_like(x, float("nan"))
        mok.unsort_rows(y, lay, out, w=weights)
        terms = yd if weights is None else w.double()[..., None] * yd
        want, mag = terms.sum(1), terms.abs().sum(1)
        assert ((out.double() - want).abs() <= half * want.abs() + (k + 1) * 2.0 ** -24 * mag + 2.0 ** -24).all()
    dy = torch.full_like(y, 7.0)
    dw = torch.full_like(w, float("nan"))
    mok.unsort_rows_backward(dout, y, lay, w, dy, dw)
    want = w.view(-1)[src][:, None].double() * dout[src // k].double()
    assert ((dy[:R].double() - want).abs() <= (half * (1 + 2.0 ** -20) + 2.0 ** -24) * want.abs() + 2.0 ** -24).all()
    assert (dy[R:] == 7).all()
    terms = dout.double()[:, None] * yd
    steps = -(-H // 2048) * 8 + 5 + 8 + 2
    assert ((dw.double() - terms.sum(2)).abs() <= steps * 2.0 ** -24 * terms.abs().sum(2)).all()
    assert not dw[slot < 0].any()


@pytest.mark.gpu
def test_unsort_is_the_gradient_of_sort():
    """<sort(x), v> = <x, unsort(v)> with whole numbers, where both sides are exact."""
    T, H, k, E = 50, 64, 4, 6
    lay = mok.sort_layout(_idx(T, k, E, 1, 0.2).cuda(), E)
    g = ref.gen(3)
    whole = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()
    x, v, xs, dx = whole(T, H), whole(T * k, H), torch.zeros((T * k, H), device="cuda"), torch.empty((T, H), device="cuda")
    mok.sort_rows(x, lay, xs)
    mok.unsort_rows(v, lay, dx)
    assert float((xs * v).sum()) == float((x * dx).sum())


@pytest.mark.gpu
def test_weighted_sum_against_differences():
    """dy and dw against central differences of <unsort(y, w), dout>: linear in each, so exact up to fp32."""
    T, H, k, E = 20, 128, 3, 5
    lay = mok.sort_layout(_idx(T, k, E, 2, 0.2).cuda(), E)
    R = int(lay["offsets"][-1])
    g = ref.gen(4)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    y, w, dout, d, c = rnd(T * k, H), rnd(T, k), rnd(T, H), rnd(T * k, H), rnd(T, k)
    dy, dw, a, b = torch.zeros_like(y), torch.empty_like(w), torch.empty_like(dout), torch.empty_like(dout)
    mok.unsort_rows_backward(dout, y, lay, w, dy, dw)
    def value(y, w):
        out = torch.empty_like(dout)
        mok.unsort_rows(y, lay, out, w=w)
        return float((out.double() * dout.double()).sum())
    mag = float(y.abs().max() * dout.abs().max() * w.abs().max()) * T * k * H
    assert abs((value(y + d, w) - value(y - d, w)) / 2 - float((dy.double() * d.double())[:R].sum())) <= 2.0 ** -20 * mag
    assert abs((value(y, w + c) - value(y, w - c)) / 2 - float((dw.double() * c.double()).sum())) <= 2.0 ** -20 * mag


@pytest.mark.gpu
def test_strides_streams_and_graphs():
    T, H, k, E = 100, 264, 4, 8
    wide = torch.randn((T, H + 8), generator=ref.gen(5), device="cuda").to(torch.bfloat16)
    x = wide[:, 8:]
    idx = _idx(T, k, E, 3, 0.1).cuda()
    lay = mok.sort_layout(idx, E)
    want, got = (torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mok.sort_rows(x.contiguous(), lay, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mok.sort_rows(x, lay, got, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    ws = mok.alloc_bytes(mok.sort_workspace_size(T, E, k))
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mok.sort_layout(idx, E, out=lay, workspace=ws)
        mok.sort_rows(x, lay, got)
        mok.unsort_rows(got, lay, out)
    idx.copy_(_idx(T, k, E, 4, 0.3).cuda())
    graph.replay()
    fresh = mok.sort_layout(idx, E)
    assert all(torch.equal(lay[n], fresh[n]) for n in fresh)
    n = (idx >= 0).sum(1, keepdim=True)
    assert torch.equal(out, (x.float() * n).to(torch.bfloat16))   # n equal terms of few bits: exact in fp32
