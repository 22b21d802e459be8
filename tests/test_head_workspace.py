"""What the vocabulary loss's workspace holds: nothing that the gradients at hand do not need."""
import pytest
import torch

import trainref as ref
from combine_router_top_expert_gb300 import build, mok

KINDS = {"dx": mok.HEAD_DX, "dW": mok.HEAD_DW, "dW_f32": mok.HEAD_DW_F32, "dx,dW": mok.HEAD_DX | mok.HEAD_DW,
         "dx,dW_f32": mok.HEAD_DX | mok.HEAD_DW_F32}


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


@pytest.mark.parametrize("T,H,V,piece", [(300, 512, 8000, 128), (5000, 64, 1 << 20, 0), (300, 512, 8000, 0), (1, 64, 5, 0)])
def test_the_running_sum_is_held_for_a_bf16_gradient_in_pieces_alone(T, H, V, piece):
    pieces = piece or T > 2048
    size = lambda g: mok.head_workspace_size(T, H, V, g, piece)
    most, sum_bytes = size(True), V * H * 4 if pieces else 0
    assert size(KINDS["dx,dW"]) == most
    assert size(KINDS["dx,dW_f32"]) + sum_bytes <= most < size(KINDS["dx,dW_f32"]) + sum_bytes + 1024
    assert size(KINDS["dx"]) == size(KINDS["dx,dW_f32"])
    assert 0 < size(False) < size(KINDS["dW_f32"]) <= size(KINDS["dW"]) <= most


@pytest.mark.parametrize("T,V,piece,rows", [(10000, 1 << 24, 0, 256), (10000, 1 << 23, 0, 256), (10000, 1 << 22, 0, 512),
                                            (200000, 8, 0, 65536), (200000, 8, 1 << 20, 65536), (5000, 8000, 1, 256),
                                            (5000, 8000, 300, 512), (256, 8000, 1, 1), (256, 8000, 100, 100),
                                            (5000, 131072, 0, 5120)])
def test_tokens_of_a_piece(T, V, piece, rows):
    """dl is the only part that grows with V's columns by rows x 2 bytes (beside 16 bytes a row and 256 columns)."""
    size = lambda V: mok.head_workspace_size(T, 8, V, KINDS["dx,dW_f32"], piece)
    tiles = -(-V // 256)
    dl, stats = rows * -(-V // 64) * 64 * 2, rows * 2 * tiles * 8
    rest = size(V) - dl
    parts = -(-V // 64) // 8 * rows * 8 * 4          # dX's, at most
    assert 0 <= rest <= stats + parts + rows * 64 + (1 << 14)


@pytest.mark.gpu
@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("T,piece", [(5, 0), (100, 40), (300, 0), (300, 128)])
@pytest.mark.parametrize("call", ["train", "backward"])
def test_that_much_is_enough_and_less_is_refused(kinds, T, piece, call):
    """The gradients of a call whose workspace is of the smallest size, between bytes that stay as they were, are those
    of a call with the largest."""
    H, V = 264, 1003
    x, W = ref.exact_head(T, H, V, 3)
    y = torch.randint(-1, V, (T,), generator=ref.gen(4), device="cuda")
    f32 = "f32" in kinds
    loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
    mok.head_loss(x, W, y, loss, mok.alloc_bytes(mok.head_workspace_size(T, H, V)), lse=lse)

    def run(ws):
        dx = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda") if "dx" in kinds else None
        dW = torch.full((V, H), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda") if "dW" in kinds else None
        if call == "train":
            mok.head_loss_train(x, W, y, loss, dx, dW, ws, scale=0.5, piece=piece)
        else:
            mok.head_loss_backward(x, W, y, lse, dx, dW, ws, scale=0.5, piece=piece)
        assert mok.device_status(ws) == (mok.OK, 0)
        return [t for t in (dx, dW) if t is not None]

    need, gap = mok.head_workspace_size(T, H, V, KINDS[kinds], piece), 1 << 16
    room = mok.alloc_bytes(need + 2 * gap).fill_(0x5A)
    got = run(room[gap:gap + need])
    assert (room[:gap] == 0x5A).all() and (room[gap + need:] == 0x5A).all()
    want = run(mok.alloc_bytes(mok.head_workspace_size(T, H, V, True, piece)).fill_(0xA5))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(mok.MokError):
        run(room[gap:gap + need - 1024])
