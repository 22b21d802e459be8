"""A stack of mixture-of-experts blocks with a vocabulary's head on one GB300: training
steps with 8-bit checkpoints and clipped gradients, then a few decoding steps, with the
memory and the times of both.

    python examples/moe_block.py [--layers 4] [--tokens 2048] [--batch 8] [--mxfp8]
"""
import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_router_top_expert_gb300 import mok, synth  # noqa: E402
from combine_router_top_expert_gb300.block import BlockBuffers, MoEBlock  # noqa: E402
from combine_router_top_expert_gb300.head import VocabHead  # noqa: E402
from combine_router_top_expert_gb300.layer import MoELayer  # noqa: E402


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--mxfp8", action="store_true")
    a = ap.parse_args()
    H, I, E, k = 1024, 512, 16, 4
    wl = synth.small("block", T=1, H=H, I=I, E=E, k=k, dtype="mxfp8" if a.mxfp8 else "bf16")
    shared = BlockBuffers()   # one full training context for every block: the checkpoints hold the rest
    blocks = []
    for n in range(a.layers):
        inp = synth.make_inputs(wl, seed=n, with_x=False)
        layer = MoELayer(inp.W_r, inp.Wg, inp.Wu, inp.Wd, k, dtype=mok.MXFP8 if a.mxfp8 else mok.BF16)
        blocks.append(MoEBlock(layer, torch.ones(H, device="cuda"), buffers=shared))

    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((a.tokens, H), generator=g, device="cuda").to(torch.bfloat16)
    V = 32003
    W = (torch.randn((V, H), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    head = VocabHead(W, torch.ones(H, device="cuda"))
    labels = torch.randint(0, V, (a.tokens,), generator=g, device="cuda")
    norm, clip_ws = torch.empty((), device="cuda"), mok.alloc_bytes(mok.grad_workspace_size())
    p = blocks[0].layer.problem(a.tokens)
    for step in range(3):
        torch.cuda.synchronize()
        t = time.perf_counter()
        h, res, ctxs = x, None, []
        for b in blocks:
            h, res, ctx = b.train_forward(h, res)
            ctxs.append(ctx)
        loss, grads = head.train(h, labels, residual=res, scale=1.0 / a.tokens)
        dout = dstream = grads.pop("dx")
        every = list(grads.values())
        for b, ctx in zip(reversed(blocks), reversed(ctxs)):
            grads = b.train_backward(ctx, dout, dstream)
            dout = dstream = grads.pop("dx")
            every += grads.values()
        mok.grad_clip(every, 1.0, norm, clip_ws)
        torch.cuda.synchronize()
        print(f"training step {step}: loss {float(loss.mean()):.4f}, gradient norm {float(norm):.3e}, "
              f"{(time.perf_counter() - t) * 1e3:.2f} ms for {a.layers} blocks x {a.tokens} tokens")
    full, small = mok.saved_size(p), mok.checkpoint_size(p)
    print(f"training context of a block: {full / 2**20:.0f} MiB in full (one for all blocks), "
          f"{small / 2**20:.0f} MiB checkpointed (one per block)")

    x = torch.randn((a.batch, H), generator=g, device="cuda").to(torch.bfloat16)
    times = []
    for _ in range(20):
        torch.cuda.synchronize()
        t = time.perf_counter()
        h, res = x, None
        for b in blocks:
            h, res = b.forward(h, res)
        loss, _ = head.score(h, labels[:a.batch], residual=res)
        torch.cuda.synchronize()
        times.append(time.perf_counter() - t)
    assert bool(torch.isfinite(loss).all())
    print(f"decoding step: {np.median(times) * 1e6:.0f} us for {a.layers} blocks x {a.batch} tokens, scored")


if __name__ == "__main__":
    main()
