"""The binding's checks of tensors hold with Python's assertions off, too (CPU:
host tensors are refused before the library is called)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PRELUDE = """
import torch
from combine_router_top_expert_gb300 import mok
def no_call(*a):
    raise SystemExit("the library was called")
class Lib:
    def __getattr__(self, name):
        return (lambda *a: 0) if name.endswith("_size") else no_call
mok.lib = lambda: Lib()
x = torch.zeros((4, 128), dtype=torch.bfloat16)
gain, rstd, u8 = torch.ones(128), torch.ones(4), torch.zeros(1 << 16, dtype=torch.uint8)
p = mok.make_problem(4, 128, 128, 8, 2)
routing = dict.fromkeys(("topk_idx", "topk_w", "counts", "offsets", "row_src", "slot_row"), u8)
try:
    {call}
except AssertionError:
    print("refused")
"""
CALLS = {
    "rmsnorm": "mok.rmsnorm(x, gain, y=torch.empty_like(x))",
    "rmsnorm_backward": "mok.rmsnorm_backward(x, gain, rstd, x, gain, u8, s=x)",
    "dequantize_rows": "mok.dequantize_rows(u8[:512].view(4, 128), u8[:16].view(4, 4), x)",
    "moe_few": "mok.moe_few(p, x, torch.zeros(128, 8), u8, x, u8)",
    "checkpoint_save": "mok.checkpoint_save(p, x, routing, u8, u8)",
    "checkpoint_load": "mok.checkpoint_load(p, u8, routing, x, u8)",
}


@pytest.mark.parametrize("flags", [[], ["-O"]], ids=["assertions", "optimised"])
@pytest.mark.parametrize("name", CALLS)
def test_host_tensors_are_refused(name, flags):
    r = subprocess.run([sys.executable, *flags, "-c", PRELUDE.replace("{call}", CALLS[name])], cwd=ROOT,
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stdout + r.stderr
