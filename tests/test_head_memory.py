"""VocabHead keeps one workspace that serves every call it is large enough for (CPU: sizes from the library, memory on
the host)."""
import pytest
import torch

from combine_router_top_expert_gb300 import build, mok
from combine_router_top_expert_gb300.head import VocabHead

TRAIN = mok.HEAD_DX | mok.HEAD_DW


@pytest.fixture
def held(monkeypatch):
    build.build()
    blocks = []
    monkeypatch.setattr(mok, "alloc_bytes", lambda n, device: blocks.append(torch.empty(n, dtype=torch.uint8, device="meta"))
                        or blocks[-1])
    return blocks


def _head(piece=0):
    return VocabHead(torch.zeros((131072, 64), dtype=torch.bfloat16), torch.zeros(64), piece=piece)


def test_smaller_calls_take_the_largest_ones_workspace(held):
    head = _head()
    first = head._workspace(4097, TRAIN)
    assert first.numel() == mok.head_workspace_size(4097, 64, 131072, TRAIN)
    for T, grad in ((4097, 0), (1, 0), (4096, TRAIN), (100, TRAIN), (300, TRAIN), (0, 0)):
        assert head._workspace(T, grad) is first and head._last is first
    assert len(held) == 1


def test_growing_calls_hold_three_times_the_largest_at_most(held):
    head, largest = _head(), 0
    for T in range(1, 6000, 7):
        for grad in (0, TRAIN):
            need = mok.head_workspace_size(T, 64, 131072, grad)
            largest = max(largest, need)
            assert head._workspace(T, grad).numel() >= need
            assert sum(b.numel() for b in held) <= 3 * head._ws.numel() and head._ws.numel() <= 1.5 * largest + 1
    assert all(any(b is kept for kept in head._all_ws) for b in held)      # captured calls stay good


def test_the_sum_of_an_fp32_gradient_is_not_held_twice(held):
    head = _head(piece=256)
    with_sum = mok.head_workspace_size(4096, 64, 131072, TRAIN, 256)
    assert head._workspace(4096, mok.HEAD_DX | mok.HEAD_DW_F32).numel() == with_sum - 131072 * 64 * 4
