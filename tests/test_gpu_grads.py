"""The global norm of many gradients, and clipping by it.

Tolerances. A thread adds 16 to 32 squares in fp32 (a chain of at most 17 steps of 2^-24), everything beyond in fp64, so
the sum of squares errs by at most 18 * 2^-24 relative and the norm by half of that and its rounding: 11 * 2^-24.
Clipped values: the factor has the norm's error and its own rounding, the product one, and the type's.
"""
import math

import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import mok

REL = 11 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}   # the least step


def _ws():
    return mok.alloc_bytes(mok.grad_workspace_size()).fill_(0xA5)


def _norm64(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def _grads(shapes, seed, std=1.0):
    g = ref.gen(seed)
    return [(torch.randn(s, generator=g, device="cuda") * std).to(t) for s, t in shapes]


B, F, D = torch.bfloat16, torch.float16, torch.float32
SETS = {
    "one": [((1,), D)],
    "odd": [((7,), B), ((9,), F), ((3,), D), ((0,), B), ((), D), ((5, 11), B)],
    "block": [((8, 128, 64), B), ((8, 128, 64), B), ((8, 64, 128), B), ((128, 8), D), ((128,), D)],
    "chunks": [((16384,), B), ((16385,), B), ((8192,), D), ((8191,), D), ((100003,), F)],
    "many": [((17 + i,), (B, F, D)[i % 3]) for i in range(500)],
    "large": [((3, 1 << 22), B), ((5000001,), D)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("ratio", [0.5, 4.0])
@pytest.mark.parametrize("inplace", [True, False])
def test_norm_and_clip(name, ratio, inplace):
    grads = _grads(SETS[name], 1)
    before = [g.clone() for g in grads]
    want, norm, ws = _norm64(grads), torch.empty((), device="cuda"), _ws()
    mok.grad_norm(grads, norm, ws)
    assert abs(float(norm) - want) <= REL * want
    out = None if inplace else [torch.full_like(g, float("nan")) for g in grads]
    norm.fill_(float("nan"))
    mok.grad_clip(mok.grad_list(grads, out), want / ratio, norm, ws)
    assert abs(float(norm) - want) <= REL * want
    factor = min(1.0, want / ratio / (want + 1e-6))
    for b, g, o in zip(before, grads, grads if inplace else out):
        if not inplace:
            assert torch.equal(b, g)
        if factor == 1.0:
            assert torch.equal(o, b)
            continue
        exact = b.double() * factor
        tol = (HALF[b.dtype] + REL + 3 * 2.0 ** -24) * exact.abs() + TINY[b.dtype]
        assert ((o.double() - exact).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [B, F, D])
@pytest.mark.parametrize("shift", [1, 3])
def test_views_at_any_element(dt, shift):
    flat = torch.randn(100000, generator=ref.gen(2), device="cuda").to(dt)
    keep = flat.clone()
    view = flat[shift:99000]
    want, norm, ws = _norm64([view]), torch.empty((), device="cuda"), _ws()
    mok.grad_clip([view], want / 2, norm, ws)
    assert abs(float(norm) - want) <= REL * want
    exact = keep[shift:99000].double() * (want / 2 / (want + 1e-6))
    assert ((view.double() - exact).abs() <= (HALF[dt] + REL + 3 * 2.0 ** -24) * exact.abs() + TINY[dt]).all()
    assert torch.equal(flat[:shift], keep[:shift]) and torch.equal(flat[99000:], keep[99000:])


@pytest.mark.gpu
@pytest.mark.parametrize("dt,like", [(B, True), (B, False), (D, True), (D, False)])
def test_many_long_views(dt, like):
    """Views of more than a chunk at any element, more of them than one launch lists; outputs that lie the same way
    and others."""
    n, count = 9001, 150
    flat = torch.randn(n * count + 8, generator=ref.gen(5), device="cuda").to(dt)
    keep = flat.clone()
    grads = [flat[1 + i * n:1 + (i + 1) * n] for i in range(count)]
    room = torch.zeros(n * count + 8, dtype=dt, device="cuda")
    shift = 1 if like else 2
    out = [room[shift + i * n:shift + (i + 1) * n] for i in range(count)]
    want, norm = _norm64(grads), torch.empty((), device="cuda")
    mok.grad_clip(mok.grad_list(grads, out), want / 3, norm, _ws())
    assert abs(float(norm) - want) <= REL * want
    exact = keep[1:1 + n * count].double() * (want / 3 / (want + 1e-6))
    got = room[shift:shift + n * count].double()
    assert ((got - exact).abs() <= (HALF[dt] + REL + 3 * 2.0 ** -24) * exact.abs() + TINY[dt]).all()
    assert torch.equal(flat, keep) and not room[:shift].any() and not room[shift + n * count:].any()


@pytest.mark.gpu
def test_a_list_of_another_device_is_refused(monkeypatch):
    plan = mok.grad_list(_grads(SETS["odd"], 6))
    norm, ws = torch.zeros((), device="cuda"), _ws()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (lambda: mok.grad_norm(plan, norm, ws), lambda: mok.grad_clip(plan, 1.0, norm, ws)):
        with pytest.raises(AssertionError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e18, 1e30])
@pytest.mark.parametrize("dt", [B, D])
def test_values_whose_squares_leave_fp32(std, dt):
    grads = _grads([((1000,), dt), ((65537,), dt)], 3, std)
    want, norm = _norm64(grads), torch.empty((), device="cuda")
    mok.grad_norm(grads, norm, _ws())
    assert abs(float(norm) - want) <= REL * want


@pytest.mark.gpu
def test_zeros_nothing_and_non_finite_values():
    norm, ws = torch.empty((), device="cuda"), _ws()
    mok.grad_norm([], norm, ws)
    assert float(norm) == 0
    mok.grad_clip([], 1.0, norm, ws)
    assert float(norm) == 0
    z = torch.zeros(1000, device="cuda")
    mok.grad_clip([z], 0.0, norm, ws)
    assert float(norm) == 0 and not z.any()
    g = torch.ones(1000, dtype=B, device="cuda")
    mok.grad_clip([g], 0.0, norm, ws)
    assert not g.any()
    g.fill_(2.0)
    mok.grad_clip([g], math.inf, norm, ws)
    assert (g == 2).all()
    g[5] = math.inf
    mok.grad_clip([g], 1.0, norm, ws)
    assert math.isinf(float(norm)) and torch.isnan(g[5]) and int(torch.isnan(g).sum()) == 1 and float(g[6]) == 0
    g.fill_(2.0)
    g[999] = math.nan
    mok.grad_clip([g], 1.0, norm, ws)
    assert math.isnan(float(norm)) and torch.isnan(g).all()


@pytest.mark.gpu
def test_same_bits_streams_and_graphs():
    grads = _grads(SETS["chunks"], 4)
    ws, norm = _ws(), torch.empty((), device="cuda")
    out = [torch.empty_like(g) for g in grads]
    plan = mok.grad_list(grads, out)
    mok.grad_clip(plan, 1.0, norm, ws)
    want, first = float(norm), [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mok.grad_clip(plan, 1.0, norm, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert float(norm) == want and all(torch.equal(a, b) for a, b in zip(first, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mok.grad_clip(plan, 1.0, norm, ws)
    for g in grads:
        g.mul_(2)
    graph.replay()
    assert abs(float(norm) - 2 * want) <= 2 * REL * want
