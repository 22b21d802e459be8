"""Every tensor of the vocabulary loss, the sorted rows and the clipping is held to the current device (CPU: host tensors
that say they are on a device, and a library that only counts its calls)."""
import pytest
import torch

from combine_router_top_expert_gb300 import mok


class On(torch.Tensor):
    """A host tensor that says that it is on a CUDA device (-1: on the host)."""
    device_index = 0
    is_cuda = property(lambda self: self.device_index >= 0)

    def get_device(self):
        return self.device_index


def _on(index, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.device_index = index
    return t


class Lib:
    calls = 0

    def __getattr__(self, name):
        def call(*a):
            Lib.calls += 0 if name.endswith("_size") else 1
            return 0
        return call


T, H, V, k, E = 4, 64, 9, 2, 8
F, I = torch.float32, torch.int32
HEAD = dict(x=(T, H), W=(V, H), labels=(T, I), loss=(T, F), dx=(T, H), dW=(V, H), workspace=(4096, torch.uint8),
            lse=(T, F), dloss=(T, F))
LAYOUT = dict(counts=(E, I), offsets=(E + 1, I), row_src=(T * k, I), slot_row=(T * k, I))
CALLS = {
    "head_loss": ({n: HEAD[n] for n in ("x", "W", "labels", "loss", "workspace", "lse")}, lambda **a: mok.head_loss(**a)),
    "head_loss_backward": ({n: HEAD[n] for n in HEAD if n != "loss"}, lambda **a: mok.head_loss_backward(**a)),
    "head_loss_train": (HEAD, lambda **a: mok.head_loss_train(**a)),
    "sort_layout": (dict(topk_idx=(T, k, I), workspace=(4096, torch.uint8), **LAYOUT),
                    lambda topk_idx, workspace, **out: mok.sort_layout(topk_idx, E, out=out, workspace=workspace)),
    "sort_rows": (dict(x=(T, H), out=(T * k, H), slot_row=(T * k, I)),
                  lambda x, out, **lay: mok.sort_rows(x, lay, out)),
    "unsort_rows": (dict(y=(T * k, H), out=(T, H), w=(T, k, F), slot_row=(T * k, I)),
                    lambda y, out, w, **lay: mok.unsort_rows(y, lay, out, w=w)),
    "unsort_rows_backward": (dict(dout=(T, H), y=(T * k, H), w=(T, k, F), dy=(T * k, H), dw=(T, k, F), slot_row=(T * k, I)),
                             lambda dout, y, w, dy, dw, **lay: mok.unsort_rows_backward(dout, y, lay, w, dy, dw)),
    "grad_norm": (dict(g=(5,), norm=(F,), workspace=(4096, torch.uint8)),
                  lambda g, norm, workspace: mok.grad_norm([g], norm, workspace)),
    "grad_clip": (dict(g=(5,), out=(5,), norm=(F,), workspace=(4096, torch.uint8)),
                  lambda g, out, norm, workspace: mok.grad_clip(mok.grad_list([g], [out]), 1.0, norm, workspace)),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("elsewhere", [1, -1])
def test_tensors_of_another_device_are_refused(name, elsewhere, monkeypatch):
    monkeypatch.setattr(mok, "lib", Lib)
    monkeypatch.setattr(mok, "_stream", lambda s=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    specs, call = CALLS[name]

    def run(moved=None):
        args = {}
        for n, spec in specs.items():
            dt = spec[-1] if spec and isinstance(spec[-1], torch.dtype) else torch.bfloat16
            shape = [v for v in spec if not isinstance(v, torch.dtype)]
            args[n] = _on(elsewhere if n == moved else 0, *shape, dtype=dt)
        before = Lib.calls
        call(**args)
        assert Lib.calls == before + 1
    run()
    for n in specs:
        before = Lib.calls
        with pytest.raises(AssertionError):
            run(n)
        assert Lib.calls == before, n
