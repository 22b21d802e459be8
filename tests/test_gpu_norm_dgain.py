"""The gain's gradient against 64 bits, at a bound that follows from the launch.

The workspace holds one partial row for each of the P CTAs that run. A column's sum
goes over the rows of a CTA (at most ceil(T / P), in up to 8 groups of them), over
the groups, over every eighth of the P partial rows, and over 8 warps; every product
is rounded once before it is added. Each of these steps errs by at most 2^-24 of the
sum of magnitudes so far.
"""
import pytest
import torch

import mxref
from combine_router_top_expert_gb300 import mok


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 256), (7, 64), (300, 1024), (1000, 7168), (4097, 1024), (5000, 160), (900, 12288)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_dgain(T, H, ckpt):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    s, dy = ((torch.randn((T, H), generator=g, device="cuda") * c).to(torch.bfloat16) for c in (3.0, 1.0))
    gain, rstd = torch.randn(H, generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda") + 0.5
    kw, value = dict(s=s), s.double()
    if ckpt:
        q, sf = (torch.empty((T, n), dtype=torch.uint8, device="cuda") for n in (H, H // 32))
        mok.rmsnorm(s, gain, sum_q=q, sum_sf=sf)
        kw, value = dict(s_q=q, s_sf=sf), mxref.decode(q, sf)
    size = mok.rmsnorm_bwd_workspace_size(T, H)
    dx, dgain, ws = torch.empty_like(s), torch.empty(H, device="cuda"), mok.alloc_bytes(size)
    mok.rmsnorm_backward(dy, gain, rstd, dx, dgain, ws, **kw)
    P = size // (4 * H)
    steps = 1 + -(-T // P) + 8 + -(-P // 8) + 8
    term = dy.double() * value * rstd.double()[:, None]
    assert ((dgain.double() - term.sum(0)).abs() <= steps * 2.0 ** -24 * term.abs().sum(0)).all()
