"""The few-token layer's waits that run out: the call reports MOK_ERR_TIMEOUT
after timeout_ms, every CTA ends, and the next call on the same workspace is
right. The first CTA withholds its counts, so that the others give up while
weights are on their way and MMAs are queued."""
import time

import pytest
import torch

from combine_router_top_expert_gb300 import mok, synth
from helpers import dtype_of, layer_for, to_dev_bf16

S = synth.small
CASES = [
    # two gate/up tiles for all SMs: cut, so CTAs wait for each other's partial sums
    (S("cut", T=12, H=2048, I=128, E=2, k=2), 0),
    (S("cut_T128", T=128, H=2048, I=128, E=2, k=1), 0),
    (S("cut_mx", T=40, H=2048, I=128, E=2, k=2, dtype="mxfp8"), 0),
    (S("cut_mx_T100", T=100, H=2048, I=128, E=2, k=2, dtype="mxfp8", shared_I=128), 0),
    # one CTA, and few: whole tiles, whose h the down phase waits for
    (S("whole", T=12, H=512, I=256, E=8, k=2), 1),
    (S("whole_T128", T=128, H=512, I=256, E=8, k=2, shared_I=256), 1),
    (S("whole_mx", T=40, H=512, I=256, E=8, k=2, dtype="mxfp8"), 3),
    (S("whole_mx_T128", T=128, H=512, I=256, E=8, k=2, dtype="mxfp8"), 3),
]


@pytest.mark.gpu
@pytest.mark.parametrize("wl,num_sms", CASES, ids=[w.name for w, _ in CASES])
def test_withheld_counts_time_out_cleanly(wl, num_sms):
    inp = synth.make_inputs(wl, seed=2)
    layer = layer_for(inp, dtype_of(wl))
    x = to_dev_bf16(inp.x)
    p = layer.problem(wl.T)
    good = mok.make_config(num_sms=num_sms)
    ws = mok.alloc_bytes(mok.few_workspace_size(p, good))

    def call(cfg):
        out = torch.empty_like(x)
        mok.moe_few(p, x, layer.W_r, layer.packed, out, ws, bias=layer.bias, packed_shared=layer.packed_shared, cfg=cfg)
        torch.cuda.synchronize()
        return out

    want = call(good)
    assert mok.device_status(ws) == (mok.OK, 0)
    t = time.perf_counter()
    call(mok.make_config(num_sms=num_sms, timeout_ms=50, flags=mok.FLAG_TEST_WITHHOLD_PUBLISH))
    assert mok.device_status(ws)[0] == mok.ERR_TIMEOUT
    assert 0.04 < time.perf_counter() - t < 2.0
    for _ in range(2):
        out = call(good)
        assert mok.device_status(ws) == (mok.OK, 0)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
