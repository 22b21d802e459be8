"""A layout goes with the tokens that it was made of (CPU: host tensors that say they are on a device, and a library that
only counts its calls)."""
import pytest
import torch

from combine_router_top_expert_gb300 import mok
from test_train_devices import Lib, _on

H, I, F = 64, torch.int32, torch.float32


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(mok, "lib", Lib)
    monkeypatch.setattr(mok, "_stream", lambda s=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def _layout(T, k, E=8, out=None):
    i32 = lambda *n: _on(0, *n, dtype=I)
    out = dict(counts=i32(E), offsets=i32(E + 1), row_src=i32(T * k), slot_row=i32(T * k)) if out is None else out
    return mok.sort_layout(i32(T, k), E, out=out, workspace=_on(0, 4096, dtype=torch.uint8))


def _calls(T, k):
    x, rows, w = _on(0, T, H), _on(0, T * k, H), _on(0, T, k, dtype=F)
    return (lambda lay: mok.sort_rows(x, lay, rows), lambda lay: mok.unsort_rows(rows, lay, x),
            lambda lay: mok.unsort_rows(rows, lay, x, w=w),
            lambda lay: mok.unsort_rows_backward(x, rows, lay, w, rows, w))


def test_layouts_of_other_tokens_are_refused():
    """Of as many entries, so that the count alone does not tell: 8 tokens x 2 as 4 x 4 and the other way, and the
    router's own layout (its indices say which tokens they are of)."""
    for (T, k), (T2, k2) in (((8, 2), (4, 4)), ((4, 4), (8, 2)), ((16, 1), (2, 8))):
        lay = _layout(T, k)
        routed = dict(lay, topk_idx=_on(0, T, k, dtype=I))
        assert isinstance(lay, mok.SortLayout) and (lay.tokens, lay.k) == (T, k)
        for call in _calls(T, k):
            call(lay), call(routed), call(dict(lay))
        before = Lib.calls
        for call in _calls(T2, k2):
            for wrong in (lay, routed):
                with pytest.raises(AssertionError):
                    call(wrong)
        assert Lib.calls == before
        # the same arrays for new tokens
        again = _layout(T2, k2, out=lay)
        assert again is lay
        for call in _calls(T2, k2):
            call(lay)
        with pytest.raises(AssertionError):
            _calls(T, k)[0](lay)


def test_a_layout_of_no_tokens():
    """Whatever the entries per token; the weights [0, k] of an empty batch included."""
    lay = _layout(0, 4)
    for call in _calls(0, 4):
        call(lay), call(dict(lay))
    with pytest.raises(AssertionError):
        _calls(0, 3)[2](lay)
    with pytest.raises(AssertionError):
        _calls(4, 4)[0](lay)
