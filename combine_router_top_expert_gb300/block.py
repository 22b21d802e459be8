"""The mixture-of-experts half of a transformer block on one GPU: pre-norm with
the residual's addition, then the layer, for serving and for training.

    stream = x + residual              (the residual stream, BF16)
    out    = moe(rmsnorm(stream) * gain)

`out` and `stream` go on as the next block's x and residual, whose pre-norm adds
them. Decode-sized batches take the few-token kernels, others the layer's
stages. Training keeps 8-bit checkpoints: the stream as MXFP8 rows for the norm's
backward, and the layer's context (mok_checkpoint_save) in a quarter of the
memory. The full context is needed inside a call only: blocks that are given the
same BlockBuffers hold one between them, others use their layer's own.

The workspaces belong to the block (and the full context to its layer or its
BlockBuffers): calls that use them go to one stream at a time. With `stream` given,
the new tensors are that stream's in the allocator, and the inputs have to be ready
on it.
"""
from __future__ import annotations

import functools

import torch

from . import mok
from .layer import MoELayer


def _on_stream(f):
    """Runs a method with its `stream` as the current one, so that what it allocates and drops again is not
    handed to another stream's work while its kernels still use it."""
    @functools.wraps(f)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return wrapped


class BlockBuffers:
    """The full training context and the layer's workspaces for the blocks of a model, which train on one stream one
    after the other. One set for each problem (sizes, experts, type and tokens), so the layers need not be alike."""

    def __init__(self):
        self._sets = {}

    def training(self, layer: MoELayer, T):
        p = layer.problem(T)
        key = bytes(p)
        if key not in self._sets:
            self._sets[key] = dict(
                route_ws=mok.alloc_bytes(mok.route_workspace_size(T, layer.H, layer.E, layer.k), layer.device),
                ws=mok.alloc_bytes(mok.workspace_size(p), layer.device),
                saved=mok.alloc_bytes(mok.saved_size(p), layer.device))
        return self._sets[key]


class MoEBlock:
    def __init__(self, layer: MoELayer, gain: torch.Tensor, eps: float = 1e-6, buffers: BlockBuffers | None = None):
        """gain: [H] fp32 on the layer's device. buffers: shared with other blocks (training)."""
        if gain.shape != (layer.H,):   # the pre-norm holds x to it
            raise AssertionError(f"gain: [{layer.H}] expected")
        self.layer, self.gain, self.eps, self.buffers = layer, gain, eps, buffers
        self._few = {}         # few-token workspaces by the most tokens that they hold
        self._norm_ws = None
        self._last = ()        # status blocks of the last call

    # ------------------------------------------------------------------ serving

    @_on_stream
    def forward(self, x, residual=None):
        """(out, residual stream), both [T, H] bf16 (new tensors). x and residual may be row-strided."""
        T, H = x.shape
        total, y = (torch.empty((T, H), dtype=torch.bfloat16, device=x.device) for _ in range(2))
        mok.rmsnorm(x, self.gain, residual=residual, eps=self.eps, sum=total, y=y)
        out = torch.empty_like(y)
        if mok.few_tokens_ok(T, self.layer.k):
            self._forward_few(y, out)
        else:
            self.layer.forward(y, out=out)
            b = self.layer.buffers(T)
            self._last = (b["route_ws"], b["ws"])
        return out, total

    def _forward_few(self, y, out):
        T, layer = y.shape[0], self.layer
        # workspaces for the most tokens, half as many, a quarter and so on (0.8 MB a token at H=7168, I=2048, E=32):
        # together about twice the largest, and none is given back, so that captured calls stay good
        most = min(mok.FEW_MAX_TOKENS, mok.FEW_MAX_PAIRS // layer.k)
        while most > 8 and (most + 1) // 2 >= T:
            most = (most + 1) // 2
        if most not in self._few:
            self._few[most] = mok.alloc_bytes(mok.few_workspace_size(layer.problem(most)), layer.device)
        mok.moe_few(layer.problem(T), y, layer.W_r, layer.packed, out, self._few[most], bias=layer.bias,
                    packed_shared=layer.packed_shared)
        self._last = (self._few[most],)

    @_on_stream
    def status(self, ctx=None):
        """(code, detail) of the first device-side wait that gave up in this block's last call, or in the calls on a
        training context so far; (mok.OK, 0) if none did. Waits for the stream's work, as MoELayer.status does."""
        for t in self._last if ctx is None else ctx["status"]:
            code, detail = mok.device_status(t)
            if code != mok.OK:
                return code, detail
        return mok.OK, 0

    # ------------------------------------------------------------------ training

    @_on_stream
    def train_forward(self, x, residual=None):
        """(out, residual stream, ctx): ctx holds what train_backward needs. Refuses layers without a backward: with
        a shared expert, or made with keep_unpacked=False."""
        T, H = x.shape
        layer, dev = self.layer, x.device
        if layer.I_shared or layer.Wg is None:
            raise mok.MokError(mok.ERR_UNSUPPORTED, "MoEBlock.train_forward: " + (
                "no backward of a shared expert" if layer.I_shared else "the layer keeps no unpacked weights"))
        total, y = (torch.empty((T, H), dtype=torch.bfloat16, device=dev) for _ in range(2))
        ctx = dict(T=T, rstd=torch.empty(T, dtype=torch.float32, device=dev),
                   sum_q=torch.empty((T, H), dtype=torch.uint8, device=dev),
                   sum_sf=torch.empty((T, H // 32), dtype=torch.uint8, device=dev),
                   # of the routing, the forward and the backward: later calls on their workspaces clear these
                   status=torch.zeros((3, mok.STATUS_BYTES), dtype=torch.uint8, device=dev))
        mok.rmsnorm(x, self.gain, residual=residual, eps=self.eps, sum=total, y=y, sum_q=ctx["sum_q"],
                    sum_sf=ctx["sum_sf"], rstd=ctx["rstd"])
        p, b = layer.problem(T), self._training_buffers(T)
        # the checkpoint refers to this routing until the backward, so it is its own
        ctx["routing"] = mok.route_layout(y, layer.W_r, layer.k, layer.bias, workspace=b["route_ws"])
        self._keep_status(ctx, 0, b["route_ws"])
        out = torch.empty_like(y)
        mok.moe_forward(p, y, layer.packed, ctx["routing"], out, b["ws"], saved=b["saved"],
                        packed_shared=layer.packed_shared)
        self._keep_status(ctx, 1, b["ws"])
        ctx["ckpt"] = mok.alloc_bytes(mok.checkpoint_size(p), dev)
        mok.checkpoint_save(p, y, ctx["routing"], b["saved"], ctx["ckpt"])
        return out, total, ctx

    def _training_buffers(self, T):
        return self.layer.buffers(T, True) if self.buffers is None else self.buffers.training(self.layer, T)

    def _keep_status(self, ctx, i, ws):
        ctx["status"][i].copy_(ws[:mok.STATUS_BYTES])
        self._last = ctx["status"]

    @_on_stream
    def train_backward(self, ctx, dout, dstream=None):
        """Gradients of a train_forward: dict with dx (of x and of the residual alike), dgain, and the layer's
        dW_gate, dW_up, dW_down, dW_r. dout, dstream: gradients of out and of the residual stream, contiguous."""
        T, layer = ctx["T"], self.layer
        mok._dense("dout", dout, torch.bfloat16, T, layer.H)
        mok._dense("dstream", dstream, torch.bfloat16, T, layer.H)
        p, b, H = layer.problem(T), self._training_buffers(T), layer.H
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dout.device)
        mok.checkpoint_load(p, ctx["ckpt"], ctx["routing"], y, b["saved"])
        g = dict(dX=torch.empty_like(y), dW_gate=torch.empty_like(layer.Wg), dW_up=torch.empty_like(layer.Wu),
                 dW_down=torch.empty_like(layer.Wd),
                 dW_r=torch.empty((H, layer.E), dtype=torch.float32, device=dout.device))
        mok.moe_backward(p, y, layer.W_r, layer.Wg, layer.Wu, layer.Wd, layer.packed, dout, ctx["routing"],
                         b["saved"], g, b["ws"], packed_bwd=layer.packed_bwd)
        self._keep_status(ctx, 2, b["ws"])
        if self._norm_ws is None:   # a partial row per SM at most, so one for any T
            self._norm_ws = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(1 << 24, H), dout.device)
        g["dx"] = g.pop("dX")
        g["dgain"] = torch.empty(H, dtype=torch.float32, device=dout.device)
        # dx takes dy's place: the layer's input gradient is read before it is overwritten
        mok.rmsnorm_backward(g["dx"], self.gain, ctx["rstd"], g["dx"], g["dgain"], self._norm_ws,
                             s_q=ctx["sum_q"], s_sf=ctx["sum_sf"], dsum=dstream)
        return g
