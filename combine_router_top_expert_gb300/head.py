"""A model's end on one GPU: the norm with the residual's addition, and the loss of the next token over the vocabulary.

    stream = x + residual
    loss   = cross entropy of rmsnorm(stream) * gain against the vocabulary's rows W

x and residual are the last block's `out` and `stream` (block.py). `score` gives the losses, `train` the losses and all
gradients in one call; neither holds the logits. Tokens whose label is outside the vocabulary (-100, say) are ignored,
whatever their rows hold.

The workspaces belong to the head: calls that use them go to one stream at a time. With `stream` given, the new
tensors are that stream's in the allocator, and the inputs have to be ready on it.
"""
from __future__ import annotations

import torch

from . import mok
from .block import _on_stream


class VocabHead:
    def __init__(self, W: torch.Tensor, gain: torch.Tensor, eps: float = 1e-6, piece: int = 0):
        """W: [V, H] bf16, gain: [H] fp32. piece: tokens of which the training call's [piece, V] bf16 buffer is held at
        once, in whole tiles of 256 above 256 tokens (0: as many as 4 GB hold, but 256 at least)."""
        if W.dim() != 2 or W.dtype is not torch.bfloat16 or gain.shape != (W.shape[1],):
            raise AssertionError("W: [V, H] bf16 and gain: [H] expected")
        self.W, self.gain, self.eps, self.piece = W, gain, eps, piece
        self.V, self.H = W.shape
        self._ws = None        # of the largest call so far; smaller ones take part of it
        self._all_ws = []      # none is given back, so that captured calls stay good
        self._norm_ws = None
        self._last = None

    def _workspace(self, T, grad):
        need = mok.head_workspace_size(T, self.H, self.V, grad, self.piece if grad else 0)
        if self._ws is None or self._ws.numel() < need:
            # half as much again as the last one at least, so that all of them are three times the largest at most
            room = need if self._ws is None else max(need, self._ws.numel() * 3 // 2)
            self._ws = mok.alloc_bytes(room, self.W.device)
            self._all_ws.append(self._ws)
        self._last = self._ws
        return self._ws

    def _normed(self, x, residual, keep_sum):
        T, H = x.shape
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        total = torch.empty_like(y) if keep_sum else None
        rstd = torch.empty(T, dtype=torch.float32, device=x.device) if keep_sum else None
        mok.rmsnorm(x, self.gain, residual=residual, eps=self.eps, sum=total, y=y, rstd=rstd)
        return y, total, rstd

    @_on_stream
    def score(self, x, labels, residual=None):
        """(loss, log-sum) of each token, [T] fp32."""
        T = x.shape[0]
        y, _, _ = self._normed(x, residual, False)
        loss, lse = (torch.empty(T, dtype=torch.float32, device=x.device) for _ in range(2))
        mok.head_loss(y, self.W, labels, loss, self._workspace(T, 0), lse=lse)
        return loss, lse

    @_on_stream
    def train(self, x, labels, residual=None, dloss=None, scale=1.0, dW=None):
        """(loss [T], gradients): dx (of x and of the residual alike), dgain and dW of the sum of scale * dloss * loss
        (dloss: [T] fp32 or None for 1). dW: an fp32 [V, H] tensor that the gradient is added to; without it a new
        bf16 one."""
        T = x.shape[0]
        y, total, rstd = self._normed(x, residual, True)
        loss = torch.empty(T, dtype=torch.float32, device=x.device)
        dy = torch.empty_like(y)
        added = dW is not None
        if added and dW.dtype is not torch.float32:
            raise AssertionError("dW: fp32 expected")
        if not added:
            dW = torch.empty_like(self.W)
        ws = self._workspace(T, mok.HEAD_DX | (mok.HEAD_DW_F32 if added else mok.HEAD_DW))
        mok.head_loss_train(y, self.W, labels, loss, dy, dW, ws, dloss=dloss, scale=scale, accumulate=added,
                            piece=self.piece)
        dgain = torch.empty(self.H, dtype=torch.float32, device=x.device)
        if self._norm_ws is None:   # a partial row per SM at most, so one for any T
            self._norm_ws = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(1 << 24, self.H), x.device)
        # dx takes dy's place: the norm's output gradient is read before it is overwritten
        mok.rmsnorm_backward(dy, self.gain, rstd, dy, dgain, self._norm_ws, s=total, labels=labels, V=self.V)
        return loss, dict(dx=dy, dgain=dgain, dW=dW)

    @_on_stream
    def status(self):
        """(code, detail) of the first device-side wait that gave up in the last call; (mok.OK, 0) if none did. Waits
        for the stream's work."""
        return (mok.OK, 0) if self._last is None else mok.device_status(self._last)
