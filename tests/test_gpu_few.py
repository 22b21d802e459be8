"""The whole layer for a few tokens against the fp64 oracle, at the layer's own
tolerance (2e-2 BF16, 5e-2 MXFP8 operands, of the output's rms, beyond the
output's rounding), and its routing against the routing kernels, bit for bit."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from combine_router_top_expert_gb300 import mok, synth
from helpers import TOL, assert_close, dev_f32, dtype_of, host_bf16_f64, layer_for, to_dev_bf16

S = synth.small
CASES = [
    S("one_token", T=1, H=256, I=128, E=16, k=4),
    S("tiny", T=64, H=128, I=64, E=8, k=2),                       # 128-row weight tiles
    S("tiny_T1", T=1, H=128, I=64, E=8, k=1),
    S("dense", T=33, H=256, I=128, E=1, k=1),
    S("sparse", T=8, H=256, I=128, E=64, k=1),
    S("all_experts", T=100, H=256, I=128, E=4, k=4),
    S("k_eq_E", T=13, H=384, I=192 * 2, E=37, k=37),              # odd expert count, many slots
    S("odd_E", T=17, H=640, I=256, E=5, k=3, zipf_s=1.2),
    S("e256", T=30, H=256, I=128, E=256, k=8, zipf_s=1.2),
    S("e256_full", T=128, H=512, I=128, E=256, k=16),
    S("two_passes", T=9, H=8448, I=128, E=33, k=2),               # router: more h than one pass holds
    S("wide", T=32, H=1024, I=2048, E=8, k=2, zipf_s=1.2),
    S("T16", T=16, H=1024, I=512, E=32, k=8),
    S("T31", T=31, H=1024, I=512, E=32, k=8),
    S("T65", T=65, H=1024, I=512, E=32, k=8),
    S("T128", T=128, H=1024, I=512, E=32, k=8, zipf_s=1.2),
    S("shared", T=21, H=512, I=256, E=8, k=2, shared_I=512),
    S("shared64", T=5, H=384, I=64, E=8, k=2, shared_I=64),
    S("mx_T1", T=1, H=256, I=128, E=16, k=4, dtype="mxfp8"),
    S("mx_T20", T=20, H=1024, I=512, E=32, k=8, dtype="mxfp8"),
    S("mx_T50", T=50, H=512, I=256, E=8, k=2, dtype="mxfp8", zipf_s=1.2),
    S("mx_T128", T=128, H=512, I=256, E=8, k=2, dtype="mxfp8", zipf_s=1.2),
    S("mx_h896", T=40, H=896, I=256, E=8, k=2, dtype="mxfp8"),    # down scales per 224-row tile
    S("mx_h384", T=7, H=384, I=128, E=8, k=2, dtype="mxfp8"),     # 128-row down tiles
    S("mx_shared", T=33, H=512, I=256, E=8, k=2, dtype="mxfp8", zipf_s=1.2, shared_I=256),
    S("mx_shared_h896", T=100, H=896, I=128, E=8, k=2, dtype="mxfp8", shared_I=384),
    S("mx_e256", T=60, H=512, I=128, E=256, k=4, dtype="mxfp8"),
]


def run(wl, inp, layer, x, cfg=None, stream=None):
    """(out, topk_idx, topk_w) on a workspace of NaN bytes; the output's guard rows stay untouched."""
    T = x.shape[0]
    p = layer.problem(T)
    ws = mok.alloc_bytes(mok.few_workspace_size(p, cfg))
    ws.fill_(0xFF)
    buf = torch.full((T + 2, layer.H), 7.0, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((T, layer.k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, layer.k), float("nan"), device="cuda")
    torch.cuda.synchronize()
    mok.moe_few(p, x, layer.W_r, layer.packed, buf[1:T + 1], ws, bias=layer.bias, packed_shared=layer.packed_shared,
                topk_idx=idx, topk_w=w, cfg=cfg, stream=stream)
    torch.cuda.synchronize()
    assert mok.device_status(ws) == (mok.OK, 0)
    assert (buf[0] == 7).all() and (buf[T + 1] == 7).all()
    return buf[1:T + 1], idx, w


def reference(wl, inp):
    r = oracle.route(inp.x, inp.W_r, wl.k, inp.bias)
    mode = oracle.MODE_MXFP8 if wl.dtype == "mxfp8" else oracle.MODE_BF16
    return r, oracle.moe_forward(inp.x, inp.Wg, inp.Wu, inp.Wd, r, mode=mode, shared=inp.shared)


@pytest.mark.gpu
@pytest.mark.parametrize("wl", CASES, ids=[w.name for w in CASES])
def test_matches_the_oracle(wl):
    inp = synth.make_inputs(wl, seed=1)
    layer = layer_for(inp, dtype_of(wl))
    x = to_dev_bf16(inp.x)
    out, idx, w = run(wl, inp, layer, x)
    r, ref = reference(wl, inp)
    assert np.array_equal(idx.cpu().numpy(), r["idx"])
    assert_close(host_bf16_f64(out), ref, TOL[dtype_of(wl)], wl.name)
    routed = mok.route_layout(x, layer.W_r, wl.k, layer.bias)
    assert torch.equal(idx, routed["topk_idx"])
    assert torch.equal(w.view(torch.int32), routed["topk_w"].view(torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_every_token_count(dtype):
    """1 .. 128 tokens of one batch: each prefix is the same layer."""
    wl = S("prefix", T=128, H=256, I=128, E=8, k=2, dtype=dtype, shared_I=128)
    inp = synth.make_inputs(wl, seed=4)
    layer = layer_for(inp, dtype_of(wl))
    x = to_dev_bf16(inp.x)
    _, ref = reference(wl, inp)
    for T in list(range(1, 20)) + [31, 32, 33, 47, 63, 64, 65, 96, 127, 128]:
        out, _, _ = run(wl, inp, layer, x[:T])
        assert_close(host_bf16_f64(out), ref[:T], TOL[dtype_of(wl)], f"T={T}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_any_number_of_sms(dtype):
    """Ranges cut over 1 .. all SMs: whole tiles, tiles over several CTAs, CTAs without work."""
    wl = S("sms", T=10, H=1024, I=384, E=8, k=2, dtype=dtype, shared_I=256)
    inp = synth.make_inputs(wl, seed=5)
    layer = layer_for(inp, dtype_of(wl))
    x = to_dev_bf16(inp.x)
    _, ref = reference(wl, inp)
    for n in (1, 2, 3, 7, 31, 100, 0):
        out, _, _ = run(wl, inp, layer, x, cfg=mok.make_config(num_sms=n))
        assert_close(host_bf16_f64(out), ref, TOL[dtype_of(wl)], f"num_sms={n}")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 40, 100])
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_cut_tiles_before_whole_ones(T, dtype):
    """CTAs with cut gate/up tiles at both ends of their range and whole ones between: few SMs, many tiles."""
    wl = S("cuts", T=T, H=2048, I=512, E=8, k=2, dtype=dtype, shared_I=512)
    inp = synth.make_inputs(wl, seed=6)
    layer = layer_for(inp, dtype_of(wl))
    x = to_dev_bf16(inp.x)
    _, ref = reference(wl, inp)
    for n in (5, 6, 7, 10, 20, 24, 28):
        cfg = mok.make_config(num_sms=n)
        out, _, _ = run(wl, inp, layer, x, cfg=cfg)
        assert_close(host_bf16_f64(out), ref, TOL[dtype_of(wl)], f"num_sms={n}")
        again, _, _ = run(wl, inp, layer, x, cfg=cfg)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)), n


@pytest.mark.gpu
def test_bitwise_deterministic_and_stream_ordered():
    """Many calls back to back on one workspace and on a side stream give the same bits."""
    for wl in (S("det", T=40, H=1024, I=512, E=16, k=4, zipf_s=1.2),
               S("det_mx", T=40, H=1024, I=512, E=16, k=4, dtype="mxfp8", zipf_s=1.2, shared_I=256)):
        inp = synth.make_inputs(wl, seed=3)
        layer = layer_for(inp, dtype_of(wl))
        x = to_dev_bf16(inp.x)
        first, _, _ = run(wl, inp, layer, x)
        p = layer.problem(wl.T)
        ws = mok.alloc_bytes(mok.few_workspace_size(p))
        outs = [torch.empty_like(first) for _ in range(20)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for o in outs:
            mok.moe_few(p, x, layer.W_r, layer.packed, o, ws, bias=layer.bias, packed_shared=layer.packed_shared,
                        stream=side)
        torch.cuda.synchronize()
        assert mok.device_status(ws) == (mok.OK, 0)
        for o in outs:
            assert torch.equal(o.view(torch.int16), first.view(torch.int16))


@pytest.mark.gpu
def test_ties_and_signed_zeros_take_the_lowest_expert():
    T, H, E, k = 3, 256, 40, 5
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    W_r = torch.zeros((H, E), device="cuda")
    W_r[:, 7] = W_r[:, 35] = 1.0
    W_r[0, 3] = -0.0
    Wg = torch.zeros((E, H, 128), dtype=torch.bfloat16, device="cuda")
    Wd = torch.zeros((E, 128, H), dtype=torch.bfloat16, device="cuda")
    p = mok.make_problem(T, H, 128, E, k)
    ws = mok.alloc_bytes(mok.few_workspace_size(p))
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    mok.moe_few(p, x, W_r, mok.pack_weights(Wg, Wg, Wd, mok.BF16), out, ws, topk_idx=idx)
    assert idx.tolist() == [[7, 35, 0, 1, 2]] * T
    assert (out == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_a_token_without_numbers_stays_apart(dtype):
    """A row of NaN or infinities (its own routing is unspecified, its result is no
    number) leaves the other tokens' results as they are, up to the order of the
    partial sums."""
    wl = S("nan", T=6, H=512, I=256, E=8, k=2, dtype=dtype)
    inp = synth.make_inputs(wl, seed=6)
    layer = layer_for(inp, dtype_of(wl))
    x = to_dev_bf16(inp.x)
    _, ref = reference(wl, inp)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[2] = bad
        out, _, _ = run(wl, inp, layer, y)
        assert not torch.isfinite(out[2]).any()
        keep = [0, 1, 3, 4, 5]
        assert_close(host_bf16_f64(out)[keep], ref[keep], TOL[dtype_of(wl)], f"{bad}")


@pytest.mark.gpu
def test_optional_outputs_and_no_tokens():
    wl = S("opt", T=5, H=256, I=128, E=8, k=2)
    inp = synth.make_inputs(wl)
    layer = layer_for(inp, mok.BF16)
    x = to_dev_bf16(inp.x)
    want, _, _ = run(wl, inp, layer, x)
    p = layer.problem(wl.T)
    ws = mok.alloc_bytes(mok.few_workspace_size(p))
    out = torch.empty_like(x)
    mok.moe_few(p, x, layer.W_r, layer.packed, out, ws)
    assert torch.equal(out, want)
    p0 = layer.problem(0)
    ws0 = mok.alloc_bytes(mok.few_workspace_size(p0))
    ws0.fill_(0xFF)
    mok.moe_few(p0, x[:0], layer.W_r, layer.packed, out[:0], ws0)
    assert mok.device_status(ws0) == (mok.OK, 0)


@pytest.mark.gpu
def test_agrees_with_the_staged_layer():
    """At the layer's full size (H = 7168, I = 2048, 32 experts): the few-token
    path against mok_moe_forward, which differs by the BF16 rounding of each
    expert output (at most 2^-9 of it) and the order of fp32 sums."""
    wl = synth.WORKLOADS["bf16_fwd_T2560"]
    T, H, I, E, k = 24, wl.H, wl.I, wl.E, wl.k
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    Wg, Wu, Wd = rnd(E, H, I), rnd(E, H, I), rnd(E, I, H)
    W_r = torch.randn((H, E), generator=g, device="cuda") * 0.02
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    for dt in (mok.BF16, mok.MXFP8):
        p = mok.make_problem(T, H, I, E, k, dt)
        packed = mok.pack_weights(Wg, Wu, Wd, dt)
        routing = mok.route_layout(x, W_r, k)
        a, b = torch.empty_like(x), torch.empty_like(x)
        mok.moe_forward(p, x, packed, routing, a, mok.alloc_bytes(mok.workspace_size(p)))
        ws = mok.alloc_bytes(mok.few_workspace_size(p))
        mok.moe_few(p, x, W_r, packed, b, ws)
        torch.cuda.synchronize()
        assert mok.device_status(ws) == (mok.OK, 0)
        assert_close(host_bf16_f64(b), host_bf16_f64(a), TOL[dt], f"staged, dtype {dt}")


def test_limits_and_refusals():
    L = mok.lib()
    ok = mok.make_problem(4, 256, 128, 8, 2)
    assert mok.few_workspace_size(ok) > 0
    for T, k, E in ((129, 2, 8), (128, 17, 32), (9, 256, 256)):
        assert mok.few_workspace_size(mok.make_problem(T, 256, 128, E, k)) == 0
    assert mok.few_workspace_size(mok.make_problem(8, 256, 128, 256, 256)) > 0
    assert mok.few_workspace_size(mok.make_problem(4, 200, 128, 8, 2)) == 0

    def call(p=ok, **kw):
        a = mok.FewArgs(x=4096, W_r=8192, packed=16384, out=32768, workspace=65536, ws_bytes=1 << 40)
        for n, v in kw.items():
            setattr(a, n, v)
        return L.mok_moe_few(ctypes.byref(p), ctypes.byref(a), None, None)

    for bad in (dict(x=None), dict(W_r=None), dict(packed=None), dict(out=None), dict(workspace=None), dict(x=4104),
                dict(packed=16400), dict(out=32776), dict(workspace=65600), dict(topk_idx=2), dict(topk_w=6),
                dict(packed_shared=4096), dict(bias=3), dict(p=mok.make_problem(129, 256, 128, 8, 2)),
                dict(p=mok.make_problem(4, 256, 128, 8, 9)), dict(p=mok.make_problem(4, 256, 128, 8, 2, 0, 128))):
        assert call(**bad) == mok.ERR_INVALID, bad
    assert L.mok_moe_few(ctypes.byref(ok), None, None, None) == mok.ERR_INVALID
