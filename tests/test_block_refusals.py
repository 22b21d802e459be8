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
