"""Calls that a block refuses before anything runs (CPU: the layer is a stand-in
that fails where it would be used)."""
import types

import pytest
import torch

from combine_router_top_expert_gb300 import mok
from combine_router_top_expert_gb300.block import MoEBlock

H = 128


def _block(**layer):
    kw = dict(H=H, I_shared=0, Wg=torch.zeros(1), k=2)
    kw.update(layer)
    return MoEBlock(types.SimpleNamespace(**kw), torch.ones(H))


@pytest.mark.parametrize("layer,why", [(dict(I_shared=256), "shared expert"), (dict(Wg=None), "unpacked weights")])
def test_training_forward_of_a_layer_without_backward(layer, why):
    with pytest.raises(mok.MokError, match=why) as e:
        _block(**layer).train_forward(torch.zeros((4, H), dtype=torch.bfloat16))
    assert e.value.code == mok.ERR_UNSUPPORTED


def test_gain_of_another_width():
    with pytest.raises(AssertionError, match="gain"):
        MoEBlock(types.SimpleNamespace(H=H), torch.ones(2 * H))


@pytest.mark.parametrize("d", [torch.zeros((4, H)), torch.zeros((3, H), dtype=torch.bfloat16),
                               torch.zeros((1, H), dtype=torch.bfloat16).expand(4, H),
                               torch.zeros((H, 4), dtype=torch.bfloat16).t(), torch.zeros((4, H), dtype=torch.bfloat16)],
                         ids=["type", "rows", "expanded", "transposed", "host"])
@pytest.mark.parametrize("which", ["dout", "dstream"])
def test_backward_of_other_gradients(d, which):
    """The layer's backward reads dout's memory as it lies."""
    good = types.SimpleNamespace(dtype=torch.bfloat16, shape=(4, H), is_cuda=True, is_contiguous=lambda: True)
    with pytest.raises(AssertionError, match=which):
        _block().train_backward(dict(T=4), **{"dout": good, which: d})
