"""Refusals of the vocabulary loss, the sorted rows and the clipping (CPU: before any launch)."""
import ctypes

import pytest
import torch

from combine_router_top_expert_gb300 import build, mok
from combine_router_top_expert_gb300.head import VocabHead

PTR = 1 << 20   # an aligned address that is not read


@pytest.fixture(scope="module")
def L():
    build.build()
    return mok.lib()


def _head(**kw):
    a = mok.HeadArgs(PTR, 64, PTR, PTR, 0, 0, PTR, PTR, None, 1.0, 0, 0, PTR, PTR, PTR, 1 << 62)
    for n, v in kw.items():
        setattr(a, n, v)
    return ctypes.byref(a)


HEAD_BAD = [dict(x=None), dict(W=None), dict(labels=None), dict(workspace=None), dict(x=PTR + 8), dict(W=PTR + 8),
            dict(ldx=56), dict(ldx=68), dict(workspace=PTR + 512), dict(piece=-1), dict(dloss=PTR + 2)]
GRAD_BAD = [dict(dx=None, dW=None), dict(accumulate=1), dict(dx=PTR + 8), dict(dW=PTR + 8),
            dict(labels=PTR + 4, labels_i64=1)]


@pytest.mark.parametrize("call", ["mok_head_loss", "mok_head_loss_backward", "mok_head_loss_train"])
def test_head_arguments(L, call):
    f = getattr(L, call)
    # one that is good (but for the workspace's size, so that nothing is launched)
    good = dict(dx=PTR << 1, W=PTR << 2, dW=PTR << 3)
    if not torch.cuda.is_available():
        assert f(4, 64, 100, _head(**good, ws_bytes=0), None, None) == mok.ERR_CUDA
        assert f(4, 64, 100, _head(**{**good, "dx": PTR, "dW": None}, ws_bytes=0), None, None) == mok.ERR_CUDA
    for bad in HEAD_BAD + ([] if call == "mok_head_loss" else GRAD_BAD):
        assert f(4, 64, 100, _head(**{**good, **bad}), None, None) == mok.ERR_INVALID, bad
    for T, H, V in ((-1, 64, 100), (4, 60, 100), (4, 0, 100), (4, 65544, 100), (4, 64, 0), (4, 64, (1 << 24) + 1),
                    ((1 << 24) + 1, 64, 100)):
        assert f(T, H, V, _head(**good, ldx=1 << 20), None, None) == mok.ERR_INVALID
        assert mok.head_workspace_size(T, H, V, True) == 0
    assert f(4, 64, 100, None, None, None) == mok.ERR_INVALID
    if call != "mok_head_loss":
        overlaps = [dict(dx=PTR), dict(dx=PTR, dW=None, ldx=72)]              # x's place: with dW, of wider rows
        for at in (PTR + 128, PTR - 128, PTR + 4 * 128 - 16, PTR - 4 * 128 + 16):     # some of x's rows
            overlaps += [dict(dx=at, dW=None), dict(dW=at)]
        overlaps += [dict(dx=PTR << 2), dict(dW=PTR << 2), dict(dW=(PTR << 2) + 99 * 128), dict(dx=(PTR << 3) + 128),
                     dict(dW=(PTR << 2) - 128 * 128, dW_f32=1)]
        for kw in overlaps:
            assert f(4, 64, 100, _head(**{**good, **kw}), None, None) == mok.ERR_INVALID, kw
    missing = dict(lse=None) if call == "mok_head_loss_backward" else dict(loss=None)
    assert f(4, 64, 100, _head(**good, **missing), None, None) == mok.ERR_INVALID


def test_sort_arguments(L):
    p = ctypes.c_void_p(PTR)
    odd = ctypes.c_void_p(PTR + 8)
    lay = lambda T, E, k, i=p, c=p, w=p, n=1 << 40: L.mok_sort_layout(i, T, E, k, c, p, p, p, w, n, None)
    for T, E, k in ((-1, 8, 2), (4, 0, 2), (4, 1025, 2), (4, 8, 0), (1 << 29, 8, 2)):
        assert lay(T, E, k) == mok.ERR_INVALID and mok.sort_workspace_size(T, E, k) == 0
    assert lay(4, 8, 2, i=None) == lay(4, 8, 2, c=None) == lay(4, 8, 2, w=None) == lay(4, 8, 2, n=0) == mok.ERR_INVALID
    rows = lambda x=p, ldx=64, s=p, T=4, H=64, k=2, e=0, o=p: L.mok_sort_rows(x, ldx, s, T, H, k, e, o, None)
    assert {rows(x=None), rows(s=None), rows(o=None), rows(x=odd), rows(o=odd), rows(ldx=56), rows(ldx=68), rows(T=-1),
            rows(H=60, ldx=60), rows(H=0), rows(k=0), rows(e=3), rows(e=-1)} == {mok.ERR_INVALID}
    back = lambda y=p, s=p, w=p, T=4, H=64, k=2, e=0, o=p: L.mok_unsort_rows(y, s, w, T, H, k, e, o, None)
    assert {back(y=None), back(s=None), back(o=None), back(y=odd), back(w=ctypes.c_void_p(PTR + 2)), back(H=12),
            back(e=7)} == {mok.ERR_INVALID}
    grad = lambda d=p, y=p, s=p, w=p, T=4, H=64, k=2, e=0, dy=p, dw=p: L.mok_unsort_rows_backward(
        d, y, s, w, T, H, k, e, dy, dw, None)
    assert {grad(d=None), grad(y=None), grad(s=None), grad(w=None), grad(dy=None), grad(dw=None), grad(dy=odd),
            grad(H=4), grad(T=1 << 30)} == {mok.ERR_INVALID}


def test_clip_arguments(L):
    def call(g=PTR, out=None, n=10, elem=2, norm=PTR, ws=PTR, size=1 << 20, max_norm=1.0, count=1):
        t = (mok.GradTensor * 1)(mok.GradTensor(g, out, n, elem))
        return {L.mok_grad_clip(count, t, max_norm, norm, ws, size, None)} | (
            {L.mok_grad_norm(count, t, norm, ws, size, None)} if max_norm == 1.0 else set())
    for kw in (dict(g=None), dict(g=PTR + 2), dict(out=PTR + 2), dict(n=-1), dict(n=1 << 38), dict(elem=3),
               dict(elem=-1), dict(norm=None), dict(norm=PTR + 2), dict(ws=None), dict(ws=PTR + 8), dict(size=8),
               dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(count=-1)):
        assert call(**kw) == {mok.ERR_INVALID}, kw


def test_host_tensors_are_refused():
    x, W = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((9, 64), dtype=torch.bfloat16)
    y, f, u8 = torch.zeros(4, dtype=torch.long), torch.zeros(4), torch.zeros(1 << 12, dtype=torch.uint8)
    lay = dict(slot_row=torch.zeros(8, dtype=torch.int32))
    rows, w, norm = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((4, 2)), torch.zeros(())
    for call in (lambda: mok.head_loss(x, W, y, f, u8), lambda: mok.head_loss_backward(x, W, y, f, x, W, u8),
                 lambda: mok.head_loss_train(x, W, y, f, x, W, u8),
                 lambda: mok.sort_layout(torch.zeros((4, 2), dtype=torch.int32), 8), lambda: mok.sort_rows(x, lay, rows),
                 lambda: mok.unsort_rows(rows, lay, x), lambda: mok.unsort_rows_backward(x, rows, lay, w, rows, w),
                 lambda: mok.grad_norm([f], norm, u8), lambda: mok.grad_clip([f], 1.0, norm, u8)):
        with pytest.raises(AssertionError):
            call()


def test_a_head_of_other_types_or_sizes_is_refused():
    W, gain = torch.zeros((9, 64), dtype=torch.bfloat16), torch.zeros(64)
    for w, g in ((W.float(), gain), (W, gain[:8]), (W[0], gain), (W, gain[None])):
        with pytest.raises(AssertionError):
            VocabHead(w, g)
    head, x = VocabHead(W, gain), torch.zeros((4, 64), dtype=torch.bfloat16)
    assert head.status() == (mok.OK, 0)
    for labels in (torch.zeros(4, dtype=torch.long), torch.zeros(4)):
        with pytest.raises(AssertionError):
            head.score(x, labels)
        with pytest.raises(AssertionError):
            head.train(x, labels, dW=torch.zeros((9, 64), dtype=torch.float64))
