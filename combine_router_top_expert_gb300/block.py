"""The mixture-of-experts half of a transformer block on one GPU: pre-norm with
the residual's addition, then the layer, for serving and for training.

    stream = x + residual              (the residual stream, BF16)
    out    = moe(rmsnorm(stream) * gain)

`out` and `stream` go on as the next block's x and residual, whose pre-norm adds
them. Decode-sized batches take the few-token kernels, others the layer's
stages. Training keeps 8-bit checkpoints: the stream as MXFP8 rows for the norm's
backward, and the layer's context (mok_checkpoint_save) in a quarter of the
memory, so that one full context serves every block of a model.
"""
from __future__ import annotations

import torch

from . import mok
from .layer import MoELayer


class MoEBlock:
    def __init__(self, layer: MoELayer, gain: torch.Tensor, eps: float = 1e-6):
        """gain: [H] fp32 on the layer's device."""
        self.layer, self.gain, self.eps = layer, gain, eps
        self._few = {}
        self._norm_ws = {}

    # ------------------------------------------------------------------ serving

    def forward(self, x, residual=None, stream=None):
        """(out, residual stream), both [T, H] bf16 (new tensors). x and residual may be row-strided."""
        T, H = x.shape
        total, y = (torch.empty((T, H), dtype=torch.bfloat16, device=x.device) for _ in range(2))
        mok.rmsnorm(x, self.gain, residual=residual, eps=self.eps, sum=total, y=y, stream=stream)
        out = torch.empty_like(y)
        if mok.few_tokens_ok(T, self.layer.k):
            self._forward_few(y, out, stream)
        else:
            self.layer.forward(y, stream=stream, out=out)
        return out, total

    def _forward_few(self, y, out, stream):
        T, layer = y.shape[0], self.layer
        p = layer.problem(T)
        if T not in self._few:
            self._few[T] = mok.alloc_bytes(mok.few_workspace_size(p), layer.device)
        mok.moe_few(p, y, layer.W_r, layer.packed, out, self._few[T], bias=layer.bias,
                    packed_shared=layer.packed_shared, stream=stream)

    # ------------------------------------------------------------------ training

    def train_forward(self, x, residual=None, stream=None):
        """(out, residual stream, ctx): ctx holds what train_backward needs."""
        T, H = x.shape
        layer, dev = self.layer, x.device
        total, y = (torch.empty((T, H), dtype=torch.bfloat16, device=dev) for _ in range(2))
        ctx = dict(T=T, rstd=torch.empty(T, dtype=torch.float32, device=dev),
                   sum_q=torch.empty((T, H), dtype=torch.uint8, device=dev),
                   sum_sf=torch.empty((T, H // 32), dtype=torch.uint8, device=dev))
        mok.rmsnorm(x, self.gain, residual=residual, eps=self.eps, sum=total, y=y, sum_q=ctx["sum_q"],
                    sum_sf=ctx["sum_sf"], rstd=ctx["rstd"], stream=stream)
        p, b = layer.problem(T), layer.buffers(T, True)
        # the checkpoint refers to this routing until the backward, so it is its own
        ctx["routing"] = mok.route_layout(y, layer.W_r, layer.k, layer.bias, workspace=b["route_ws"], stream=stream)
        out = torch.empty_like(y)
        mok.moe_forward(p, y, layer.packed, ctx["routing"], out, b["ws"], saved=b["saved"],
                        packed_shared=layer.packed_shared, stream=stream)
        ctx["ckpt"] = mok.alloc_bytes(mok.checkpoint_size(p), dev)
        mok.checkpoint_save(p, y, ctx["routing"], b["saved"], ctx["ckpt"], stream=stream)
        return out, total, ctx

    def train_backward(self, ctx, dout, dstream=None, stream=None):
        """Gradients of a train_forward: dict with dx (of x and of the residual alike), dgain, and the layer's
        dW_gate, dW_up, dW_down, dW_r. dout, dstream: gradients of out and of the residual stream."""
        T, layer = ctx["T"], self.layer
        p, b, H = layer.problem(T), layer.buffers(T, True), layer.H
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dout.device)
        mok.checkpoint_load(p, ctx["ckpt"], ctx["routing"], y, b["saved"], stream=stream)
        g = dict(dX=torch.empty_like(y), dW_gate=torch.empty_like(layer.Wg), dW_up=torch.empty_like(layer.Wu),
                 dW_down=torch.empty_like(layer.Wd),
                 dW_r=torch.empty((H, layer.E), dtype=torch.float32, device=dout.device))
        mok.moe_backward(p, y, layer.W_r, layer.Wg, layer.Wu, layer.Wd, layer.packed, dout, ctx["routing"],
                         b["saved"], g, b["ws"], stream=stream, packed_bwd=layer.packed_bwd)
        if T not in self._norm_ws:
            self._norm_ws[T] = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(T, H), dout.device)
        g["dx"] = g.pop("dX")
        g["dgain"] = torch.empty(H, dtype=torch.float32, device=dout.device)
        # dx takes dy's place: the layer's input gradient is read before it is overwritten
        mok.rmsnorm_backward(g["dx"], self.gain, ctx["rstd"], g["dx"], g["dgain"], self._norm_ws[T],
                             s_q=ctx["sum_q"], s_sf=ctx["sum_sf"], dsum=dstream, stream=stream)
        return g
