"""Pre-norm with the residual's addition, its backward pass and the read-back
of MXFP8 rows, against the formulas in 64 bits.

Tolerances. A row's sum runs over at most 64 terms in a thread, 5 shuffle steps
and 32 warps, all in fp32, so its relative error is below 101 * 2^-24 of the
sum of magnitudes; 2^-16 covers that with the few roundings around it. A BF16
output adds half a BF16 spacing. dgain adds at most ceil(T / 300) rows in a
CTA and then at most 64 terms over the CTAs.
"""
import numpy as np
import pytest
import torch

import mxref
from combine_router_top_expert_gb300 import mok

REL = 2.0 ** -16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _bf16(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _outs(T, H, mx=True):
    b = lambda: torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    u = lambda n: torch.full((T, n), 0xAA, dtype=torch.uint8, device="cuda")
    o = dict(sum=b(), y=b(), rstd=torch.full((T,), float("nan"), device="cuda"))
    if mx:
        o.update(y_q=u(H), y_sf=u(H // 32), sum_q=u(H), sum_sf=u(H // 32))
    return o


def _ref(x, r, gain, eps):
    s = x.double() + (0 if r is None else r.double())
    rstd = (s.square().mean(1) + eps).rsqrt()
    return s, rstd, s * rstd[:, None] * gain.double()


SHAPES = [(1, 8), (3, 40), (1, 128), (5, 1000), (7, 4096), (2, 4104), (4, 7168), (300, 1024), (3, 8200), (2, 33000),
          (1, 65536), (1000, 7168)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(T, H, residual):
    g = _gen(T * 7 + H)
    x, r = _bf16(g, (T, H)), _bf16(g, (T, H), 3.0) if residual else None
    gain = torch.randn(H, generator=g, device="cuda")
    mx = H % 32 == 0
    o = _outs(T, H, mx)
    mok.rmsnorm(x, gain, residual=r, eps=1e-5, **o)
    s, rstd, y = _ref(x, r, gain, 1e-5)
    assert ((o["rstd"].double() - rstd).abs() <= REL * rstd).all()
    assert ((o["sum"].double() - s).abs() <= mxref.half_ulp_bf16(s, o["sum"]) + 2.0 ** -23 * s.abs()).all()
    assert ((o["y"].double() - y).abs() <= mxref.half_ulp_bf16(y, o["y"]) + REL * y.abs()).all()
    if mx:
        for n in ("y", "sum"):
            assert torch.equal(mxref.decode(o[n + "_q"], o[n + "_sf"]), mxref.values(o[n])), n
            assert torch.equal(o[n + "_sf"].long(), mxref.scale_codes(o[n])), n


@pytest.mark.gpu
def test_mxfp8_outputs_are_the_bytes_of_quantize_rows():
    T, H = 130, 7168
    g = _gen(1)
    x, gain = _bf16(g, (T, H), 2.0), torch.randn(H, generator=g, device="cuda")
    x[3] = 0                       # blocks without a value
    x[4, :64] *= 1e-30
    o = _outs(T, H)
    mok.rmsnorm(x, gain, **o)
    for n in ("y", "sum"):
        q, sf = torch.empty_like(o["y_q"]), torch.empty_like(o["y_sf"])
        mok.quantize_rows(o[n], q, sf)
        assert torch.equal(q, o[n + "_q"]) and torch.equal(sf, o[n + "_sf"]), n


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["sum", "y", "rstd", "y_q", "sum_q"])
def test_each_output_alone(which):
    T, H = 33, 1024
    g = _gen(2)
    x, r, gain = _bf16(g, (T, H)), _bf16(g, (T, H)), torch.randn(H, generator=g, device="cuda")
    full, one = _outs(T, H), _outs(T, H)
    mok.rmsnorm(x, gain, residual=r, **full)
    names = [which] + ([which[:-1] + "sf"] if which.endswith("_q") else [])
    mok.rmsnorm(x, gain, residual=r, **{n: one[n] for n in names})
    for n in names:
        assert torch.equal(one[n].view(torch.uint8), full[n].view(torch.uint8)), n


@pytest.mark.gpu
def test_row_strides_in_place_and_streams():
    T, H = 65, 1024
    g = _gen(3)
    wide_x, wide_r = _bf16(g, (T, H + 72)), _bf16(g, (T, 2 * H))
    x, r = wide_x[:, 8:8 + H], wide_r[:, H:]
    gain = torch.randn(H, generator=g, device="cuda")
    want = _outs(T, H)
    mok.rmsnorm(x.contiguous(), gain, residual=r.contiguous(), **want)
    got = _outs(T, H)
    mok.rmsnorm(x, gain, residual=r, **got)
    for n in want:
        assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), n
    # the sum in the residual's own buffer and y in x's, on another stream
    xc, rc = x.contiguous(), r.contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mok.rmsnorm(xc, gain, residual=rc, sum=rc, y=xc, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(rc, want["sum"]) and torch.equal(xc, want["y"])


@pytest.mark.gpu
def test_rows_of_zeros_infinities_and_nan_stay_apart():
    T, H = 5, 512
    g = _gen(4)
    x, gain = _bf16(g, (T, H)), torch.ones(H, device="cuda")
    clean = torch.empty_like(x)
    mok.rmsnorm(x, gain, y=clean)
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    mok.rmsnorm(x, gain, eps=1e-6, y=y, rstd=rstd)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[4], clean[4])
    assert (y[1] == 0).all() and abs(float(rstd[1]) - 1e3) < 0.1
    assert torch.isnan(y[2, 7]) and torch.isnan(y[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", SHAPES + [(4097, 1024), (5, 160), (700, 96), (300, 4128), (170, 12288)])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("with_dsum", [False, True])
def test_backward(T, H, ckpt, with_dsum):
    if ckpt and H % 32:
        pytest.skip("MXFP8 rows need H % 32 == 0")
    g = _gen(T + H)
    s, dy = _bf16(g, (T, H), 3.0), _bf16(g, (T, H))
    dsum = _bf16(g, (T, H)) if with_dsum else None
    gain = torch.randn(H, generator=g, device="cuda")
    kw = dict(s=s)
    if ckpt:
        q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        sf = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
        mok.rmsnorm(s, gain, sum_q=q, sum_sf=sf)
        s = mxref.decode(q, sf)
        kw = dict(s_q=q, s_sf=sf)
    rstd = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    dx = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgain = torch.full((H,), float("nan"), device="cuda")
    ws = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(T, H))
    ws.fill_(0xFF)
    mok.rmsnorm_backward(dy, gain, rstd, dx, dgain, ws, dsum=dsum, **kw)
    R = rstd.double()[:, None]
    xh, a = s.double() * R, dy.double() * gain.double()
    ref = R * (a - xh * (a * xh).mean(1, keepdim=True))
    size = R * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    if with_dsum:
        ref, size = ref + dsum.double(), size + dsum.double().abs()
    assert ((dx.double() - ref).abs() <= mxref.half_ulp_bf16(ref, dx) + REL * size).all()
    dg, mag = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    n = -(-T // 300) + 64
    assert ((dgain.double() - dg).abs() <= n * 2.0 ** -24 * mag).all()
    # the same bits again, dx in dy's own buffer
    dx2, dg2 = dy, torch.empty_like(dgain)
    mok.rmsnorm_backward(dy, gain, rstd, dx2, dg2, ws, dsum=dsum, **kw)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dgain)


@pytest.mark.gpu
def test_backward_from_scale_codes_at_any_address():
    T, H = 40, 1024
    g = _gen(8)
    s, dy, gain = _bf16(g, (T, H), 3.0), _bf16(g, (T, H)), torch.randn(H, generator=g, device="cuda")
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    raw = torch.empty(T * H // 32 + 8, dtype=torch.uint8, device="cuda")
    sf = raw[:T * H // 32].view(T, H // 32)
    mok.rmsnorm(s, gain, sum_q=q, sum_sf=sf)
    rstd = torch.rand(T, generator=g, device="cuda")
    ws = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(T, H))
    outs = []
    for off in (0, 1, 2):
        odd = raw[off:off + T * H // 32].view(T, H // 32)
        odd.copy_(sf.clone()) if off == 0 else odd.copy_(keep)
        keep = odd.clone()
        dx, dg = torch.empty_like(dy), torch.empty(H, device="cuda")
        mok.rmsnorm_backward(dy, gain, rstd, dx, dg, ws, s_q=q, s_sf=odd)
        outs.append((dx, dg))
    for dx, dg in outs[1:]:
        assert torch.equal(dx, outs[0][0]) and torch.equal(dg, outs[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(37, 64), (300, 1024)])
def test_dgain_at_any_float_address(T, H):
    """dgain needs four-byte alignment only: the same bits one float further on."""
    g = _gen(21)
    x, dy = _bf16(g, (T, H)), _bf16(g, (T, H))
    gain = torch.randn(H, device="cuda", generator=g)
    rstd = torch.rand(T, device="cuda", generator=g) + 0.5
    ws = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(T, H))
    got = []
    for shift in (0, 1, 3):
        dx = torch.empty_like(x)
        d = torch.full((H + 8,), -1.0, device="cuda")
        mok.rmsnorm_backward(dy, gain, rstd, dx, d[shift:shift + H], ws, s=x)
        got.append(d[shift:shift + H].clone())
        assert (d[:shift] == -1).all() and (d[shift + H:] == -1).all()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of the 64-bit forward, loss = <dy, y> + <dsum, s>,
    step 1e-5 (error about 1e-9); the BF16 dx adds half a spacing."""
    T, H = 3, 64
    g = _gen(9)
    x, dy, dsum = _bf16(g, (T, H), 2.0), _bf16(g, (T, H)), _bf16(g, (T, H))
    gain = torch.randn(H, generator=g, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    mok.rmsnorm(x, gain, y=y, rstd=rstd)
    dx, dgain = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(T, H))
    mok.rmsnorm_backward(dy, gain, rstd, dx, dgain, ws, s=x, dsum=dsum)

    def loss(xd, gd):
        s, _, yy = _ref(xd, None, gd, 1e-6)
        return float((dy.double() * yy).sum() + (dsum.double() * s).sum())

    xd, gd, d = x.double(), gain.double(), 1e-5
    for t, h in [(0, 0), (1, 17), (2, 63)]:
        p, m = xd.clone(), xd.clone()
        p[t, h] += d
        m[t, h] -= d
        num = (loss(p, gd) - loss(m, gd)) / (2 * d)
        assert abs(num - float(dx[t, h])) <= 2.0 ** -8 * abs(num) + 1e-4
    for h in (0, 31, 63):
        p, m = gd.clone(), gd.clone()
        p[h] += d
        m[h] -= d
        num = (loss(xd, p) - loss(xd, m)) / (2 * d)
        assert abs(num - float(dgain[h])) <= 1e-4 * (1 + abs(num))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 32), (5, 160), (257, 7168)])
def test_dequantize_rows(T, H):
    g = _gen(T)
    x = _bf16(g, (T, H), 4.0)
    x[0, :32] = 0
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sf = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    mok.rmsnorm(x, torch.ones(H, device="cuda"), sum_q=q, sum_sf=sf)
    out = torch.empty_like(x)
    mok.dequantize_rows(q, sf, out)
    assert torch.equal(out.double(), mxref.values(x))


@pytest.mark.gpu
def test_every_e4m3_code_and_scale_reads_back():
    q = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(255, 1)
    q[(q & 127) == 127] = 0                                   # NaN codes are never written
    sf = torch.arange(255, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 8).contiguous()
    out = torch.empty((255, 256), dtype=torch.bfloat16, device="cuda")
    mok.dequantize_rows(q, sf, out)
    want = mxref.decode(q, sf)
    # values of the lowest scales fall below BF16's smallest spacing and round;
    # those of the highest pass its range
    assert torch.equal(out, want.to(torch.float32).to(torch.bfloat16))


@pytest.mark.gpu
def test_no_rows():
    H = 256
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(H, device="cuda")
    mok.rmsnorm(e, gain, y=e.clone())
    dg = torch.full((H,), 7.0, device="cuda")
    mok.rmsnorm_backward(e, gain, torch.empty(0, device="cuda"), e.clone(), dg,
                         mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(0, H)), s=e.clone())
    assert (dg == 0).all()


def test_refusals():
    """Bad arguments are refused on the host before anything runs."""
    import ctypes
    L = mok.lib()

    def fwd(T=4, H=64, **kw):
        a = mok.RmsNormArgs(x=4096, ldx=H, gain=8192, eps=1e-6, y=16384)
        for n, v in kw.items():
            setattr(a, n, v)
        return L.mok_rmsnorm(T, H, ctypes.byref(a), None)

    bad = [dict(H=60), dict(H=0), dict(T=-1), dict(H=65544), dict(x=None), dict(gain=None), dict(y=None), dict(eps=-1.0),
           dict(eps=float("nan")), dict(ldx=56), dict(ldx=68), dict(x=4098), dict(y=16386), dict(y_q=32768),
           dict(y_sf=32768), dict(sum_q=32768), dict(residual=4096, ldr=8), dict(residual=4100, ldr=64),
           dict(H=40, y_q=32768, y_sf=65536), dict(y=4096, ldx=72), dict(sum=512, residual=512, ldr=72)]
    for kw in bad:
        assert fwd(**kw) == mok.ERR_INVALID, kw
    assert L.mok_rmsnorm(4, 64, None, None) == mok.ERR_INVALID

    def bwd(T=4, H=64, **kw):
        a = mok.RmsNormBwdArgs(dy=4096, sum=8192, rstd=256, gain=512, dx=16384, dgain=1024, workspace=2048,
                               ws_bytes=1 << 40)
        for n, v in kw.items():
            setattr(a, n, v)
        return L.mok_rmsnorm_backward(T, H, ctypes.byref(a), None)

    bad = [dict(H=60), dict(T=-1), dict(dy=None), dict(sum=None), dict(rstd=None), dict(gain=None), dict(dx=None),
           dict(dgain=None), dict(workspace=None), dict(sum_q=4096), dict(sum_q=4096, sum_sf=512),
           dict(sum=None, sum_q=4096), dict(dsum=4100), dict(H=40, sum=None, sum_q=4096, sum_sf=512)]
    for kw in bad:
        assert bwd(**kw) == mok.ERR_INVALID, kw
    assert mok.rmsnorm_bwd_workspace_size(4, 60) == 0
    assert L.mok_dequantize_rows(None, None, 4, 64, None, None) == mok.ERR_INVALID
    assert L.mok_dequantize_rows(4096, 64, 4, 48, 4096, None) == mok.ERR_INVALID
    assert L.mok_dequantize_rows(4104, 64, 4, 64, 4096, None) == mok.ERR_INVALID


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)            # not on a GPU
    with pytest.raises(AssertionError):
        mok.rmsnorm(x, torch.ones(64), y=torch.empty_like(x))
    assert np.isfinite(mok.rmsnorm_bwd_workspace_size(4, 64))
