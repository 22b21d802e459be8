"""The pre-norm's single rows: a row cut out of any wider buffer, whose pitch
says nothing."""
import pytest
import torch

from combine_router_top_expert_gb300 import mok


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 3, 8, 36])
def test_single_row_of_a_wider_buffer(pad):
    H = 512
    g = torch.Generator(device="cuda").manual_seed(pad)
    wide_x, wide_r = (torch.randn((3, H + pad), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    gain = torch.randn(H, generator=g, device="cuda")
    x, r = wide_x[:1, :H], wide_r[:1, :H]                     # the buffer's first row: aligned, any pitch
    want_s, want_y, s, y = (torch.empty((1, H), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    mok.rmsnorm(x.contiguous(), gain, residual=r.contiguous(), sum=want_s, y=want_y)
    mok.rmsnorm(x, gain, residual=r, sum=s, y=y)
    assert torch.equal(s, want_s) and torch.equal(y, want_y)
    rest = wide_x.flatten()[H:].clone(), wide_r.flatten()[H:].clone()
    mok.rmsnorm(x, gain, residual=r, sum=r, y=x)              # in place, and nothing past the row is written
    assert torch.equal(r, want_s) and torch.equal(x, want_y)
    assert torch.equal(wide_x.flatten()[H:], rest[0]) and torch.equal(wide_r.flatten()[H:], rest[1])
