"""Cases of the operators around one mixture-of-experts layer: the pre-norm with the residual's addition and its
backward pass, the layer for a few tokens, and the 8-bit checkpoint of the layer's training context.

The plain forms are elementary torch operations in 32 bits. The layer's shapes are those of the workloads in
combine_router_top_expert_gb300/synth.py (H = 7168, I = 2048, E = 32, k = 8) and of the GPU tests.
MXFP8 is E4M3 elements with one power-of-two scale per 32 elements: scale = 2^(floor(log2 amax) - 8), elements
rounded to nearest even and saturated at 448.
"""
import math

import torch

own = False

EPS = 1e-6
FEW_MAX = 128     # most tokens of the few-token layer


# ----------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's pre-norm: latency, rows inside a wider buffer
        dict(name="norm_T8", op="norm", T=8, H=7168, mx=False, residual=True, strided=True),
        # a prompt's pre-norm with the 8-bit output that the MXFP8 layer takes, read back
        dict(name="norm_mx_T4096", op="norm", T=4096, H=7168, mx=True, residual=True, strided=False),
        # a training step's pre-norm backward: short ragged batch, input kept in BF16
        dict(name="norm_bwd_T300", op="norm_bwd", T=300, H=1024, ckpt=False, dsum=True),
        # the same at the training benchmark's size, input kept in the 8-bit checkpoint
        dict(name="norm_bwd_ck_T4096", op="norm_bwd", T=4096, H=7168, ckpt=True, dsum=True),
        # the layer for single tokens and decode batches: a small layer (latency), one token, a batch, the largest
        dict(name="few_small_T3", op="few", T=3, H=512, I=256, E=8, k=2, mx=False, zipf=0.0, I_shared=0),
        dict(name="few_bf16_T1", op="few", T=1, H=7168, I=2048, E=32, k=8, mx=False, zipf=0.0, I_shared=0),
        dict(name="few_mx_T4_shared", op="few", T=4, H=7168, I=2048, E=32, k=8, mx=True, zipf=1.2, I_shared=2048),
        dict(name="few_bf16_T16", op="few", T=16, H=7168, I=2048, E=32, k=8, mx=False, zipf=0.0, I_shared=0),
        dict(name="few_mx_T64", op="few", T=64, H=7168, I=2048, E=32, k=8, mx=True, zipf=1.2, I_shared=0),
        dict(name="few_bf16_T125", op="few", T=125, H=7168, I=2048, E=32, k=8, mx=False, zipf=0.0, I_shared=0),
        # the training context in 8 bits and back: a ragged small layer, the training benchmark's size
        dict(name="ckpt_T300", op="ckpt", T=300, H=1024, I=512, E=8, k=2),
        dict(name="ckpt_T4096", op="ckpt", T=4096, H=7168, I=2048, E=32, k=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log128(rng, lo, hi):
    """A multiple of 128 between lo and hi; 24 blocks of 128 is no size of this repository."""
    while True:
        v = 128 * _log(rng, lo // 128, hi // 128)
        if v != 24 * 128:
            return v


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "few", "few", "few", "ckpt"])
    if op == "norm":
        mx = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 4096), H=_log128(rng, 256, 7168), mx=mx, residual=rng.random() < 0.75,
                    strided=rng.random() < 0.3)
    if op == "norm_bwd":
        return dict(op=op, T=_log(rng, 1, 4096), H=_log128(rng, 256, 7168), ckpt=rng.random() < 0.5,
                    dsum=rng.random() < 0.75)
    if op == "ckpt":
        E = rng.choice([4, 8, 16, 32])
        return dict(op=op, T=_log(rng, 16, 4096), H=_log128(rng, 256, 7168), I=_log128(rng, 128, 2048), E=E,
                    k=rng.randint(1, min(8, E)))
    while True:
        H, I, E = _log128(rng, 256, 7168), _log128(rng, 128, 2048), _log(rng, 4, 128)
        if E * H * I <= 32 * 7168 * 2048:
            break
    return dict(op=op, T=_log(rng, 1, FEW_MAX), H=H, I=I, E=E, k=rng.randint(1, min(8, E)), mx=rng.random() < 0.5,
                zipf=rng.choice([0.0, 1.2]), I_shared=rng.choice([0, 0, I]))


# ----------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _weights(g, E, K, N, mx):
    """[E, K, N] BF16 weights ~ N(0, 0.02). MXFP8 layers: values that their 8-bit form, blocked along K, stands for."""
    W = torch.empty((E, K, N), device="cuda", dtype=torch.bfloat16)
    for e in range(E):
        w = torch.randn((K, N), generator=g, device="cuda", dtype=torch.float32).mul_(0.02).to(torch.bfloat16)
        W[e] = _mx_values(w.float().t().contiguous()).t() if mx else w
    return W


def _zipf_bias(E, s):
    z = torch.arange(1, E + 1, dtype=torch.float64) ** (-s)
    return torch.log(z / z.sum()).float()


def _aligned_bytes(n):
    """n zeroed bytes on a 1024-byte boundary."""
    raw = torch.zeros(n + 1024, dtype=torch.uint8, device="cuda")
    off = (-raw.data_ptr()) % 1024
    return raw[off:off + n]


def _up(v, a):
    return (v + a - 1) // a * a


def _saved_views(c, buf=None):
    """The training context of one layer (include/mok.h, mok_saved_size): gathered rows A [R, H] bf16, G|U [R, 2I]
    f32, h [R, I] bf16, partials [T*k, H] bf16, each on a 1024-byte boundary, R = T*k + 128*E rounded up to 128."""
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    R = _up(T * k + 128 * E, 128)
    parts = [("A", R, H, torch.bfloat16, 2), ("gu", R, 2 * I, torch.float32, 4), ("h", R, I, torch.bfloat16, 2),
             ("partials", T * k, H, torch.bfloat16, 2)]
    total = sum(_up(r * w * b, 1024) for _, r, w, _, b in parts)
    if buf is None:
        buf = _aligned_bytes(total)
    views, at = {}, 0
    for name, r, w, dt, b in parts:
        views[name] = buf[at:at + r * w * b].view(dt).view(r, w)
        at += _up(r * w * b, 1024)
    return buf, views


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    T, H = c["T"], c["H"]
    s = {"c": c}
    if c["op"] == "norm":
        wide = H + 256 if c["strided"] else H
        s["x"] = _normal(g, (T, wide))[:, :H]
        s["r"] = _normal(g, (T, H), 3.0) if c["residual"] else None
        s["gain"] = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")
        if own:
            s["sum"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            s["y"] = torch.empty_like(s["sum"])
            s["rstd"] = torch.empty(T, dtype=torch.float32, device="cuda")
            if c["mx"]:
                s["q"] = torch.empty((T, H), dtype=torch.uint8, device="cuda")
                s["sf"] = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    elif c["op"] == "norm_bwd":
        rows = _normal(g, (T, H), 3.0)
        s["rstd"] = torch.rsqrt(rows.float().square().mean(1) + EPS)
        if c["ckpt"]:
            s["q"], s["sf"] = _mx_codes(rows.float())
        else:
            s["s"] = rows
        s["dy"] = _normal(g, (T, H))
        s["dsum"] = _normal(g, (T, H)) if c["dsum"] else None
        s["gain"] = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")
        if own:
            from combine_router_top_expert_gb300 import mok
            s["dx"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            s["dgain"] = torch.empty(H, dtype=torch.float32, device="cuda")
            s["ws"] = mok.alloc_bytes(mok.rmsnorm_bwd_workspace_size(T, H))
    elif c["op"] == "few":
        I, E, k, Is = c["I"], c["E"], c["k"], c["I_shared"]
        s["x"] = _normal(g, (T, H))
        s["W_r"] = torch.randn((H, E), generator=g, device="cuda") * 0.02
        s["bias"] = _zipf_bias(E, c["zipf"]).cuda() if c["zipf"] else None
        s["Wg"], s["Wu"] = _weights(g, E, H, I, c["mx"]), _weights(g, E, H, I, c["mx"])
        s["Wd"] = _weights(g, E, I, H, c["mx"])
        if Is:   # the shared expert is BF16 in every mode
            s["Sg"], s["Su"], s["Sd"] = (_weights(g, 1, *d, False) for d in ((H, Is), (H, Is), (Is, H)))
        if own:
            # the packed weights, buffers and problem that a serving program keeps
            from combine_router_top_expert_gb300 import mok
            dt = mok.MXFP8 if c["mx"] else mok.BF16
            s["p"] = mok.make_problem(T, H, I, E, k, dt, Is)
            s["packed"] = mok.pack_weights(s.pop("Wg"), s.pop("Wu"), s.pop("Wd"), dt)
            s["packed_shared"] = mok.pack_weights(s.pop("Sg"), s.pop("Su"), s.pop("Sd"), mok.BF16) if Is else None
            s["ws"] = mok.alloc_bytes(mok.few_workspace_size(s["p"]))
            s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            s["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    else:
        I, E, k = c["I"], c["E"], c["k"]
        s["x"] = _normal(g, (T, H))
        # k distinct experts per token, skewed; rows in (expert, token) order, segments padded to 128 rows
        noise = torch.rand((T, E), generator=g, device="cuda") + 0.02 * torch.arange(E, 0, -1, device="cuda")
        idx = noise.topk(k, dim=1).indices
        w = torch.rand((T, k), generator=g, device="cuda")
        flat = idx.reshape(-1)
        row_src = torch.sort(flat, stable=True).indices
        counts = torch.bincount(flat, minlength=E)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        poff = torch.cat([counts.new_zeros(1), ((counts + 127) // 128 * 128).cumsum(0)])
        slot_row = torch.empty_like(row_src)
        slot_row[row_src] = torch.arange(T * k, device="cuda")
        s["rows"] = (poff[flat] + slot_row - offsets[flat])       # padded row of slot t*k + j
        s["routing"] = dict(topk_idx=idx.int().contiguous(), topk_w=w, counts=counts.int(), offsets=offsets.int(),
                            row_src=row_src.int(), slot_row=slot_row.int())
        s["saved"], v = _saved_views(c)
        v["A"][s["rows"]] = s["x"].repeat_interleave(k, 0)
        gu = torch.randn((T * k, 2 * I), generator=g, device="cuda") * (0.02 * math.sqrt(H))
        v["gu"][s["rows"]] = gu
        v["h"][s["rows"]] = (gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]).to(torch.bfloat16)
        v["partials"].copy_(_normal(g, (T * k, H), 0.02 * math.sqrt(I)))
        s["views"] = v
        if own:
            from combine_router_top_expert_gb300 import mok
            s["p"] = mok.make_problem(T, H, I, E, k)
            s["ckpt"] = mok.alloc_bytes(mok.checkpoint_size(s["p"]))
            s["restored"], s["restored_views"] = _saved_views(c)
            s["x_restored"] = torch.empty_like(s["x"])
    return s


# ----------------------------------------------------------------------------------------------- plain forms

def _mx_scale_exp(v):
    """Exponent of the scale of each block of 32 along the last axis of v (blocks on the axis before the last)."""
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax).exponent - 1 - 8
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)


def _mx_round(v, e):
    return torch.ldexp(v, -e).clamp(-448, 448).to(torch.float8_e4m3fn)


def _mx_values(v):
    """The values that the MXFP8 form of v (32 bits, blocks along the last axis) stands for."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    e = _mx_scale_exp(b)
    return torch.ldexp(_mx_round(b, e).float(), e).reshape(v.shape)


def _mx_codes(v):
    b = v.reshape(*v.shape[:-1], -1, 32)
    e = _mx_scale_exp(b)
    return _mx_round(b, e).view(torch.uint8).reshape(v.shape), (e + 127).to(torch.uint8).squeeze(-1)


def _swiglu(g, u):
    return g / (1 + torch.exp(-g)) * u


def _norm_plain(s):
    c = s["c"]
    t = s["x"].float()
    if s["r"] is not None:
        t = t + s["r"].float()
    rstd = 1 / torch.sqrt((t * t).mean(1) + EPS)
    y = (t * rstd[:, None] * s["gain"]).to(torch.bfloat16)
    if c["mx"]:
        y = _mx_values(y.float()).to(torch.bfloat16)   # every 8-bit value with its scale is a BF16 value
    return {"sum": t.to(torch.bfloat16), "y": y, "rstd": rstd}


def _norm_bwd_plain(s):
    if "q" in s:
        q = s["q"].view(torch.float8_e4m3fn).float()
        rows = torch.ldexp(q.reshape(q.shape[0], -1, 32), s["sf"].int()[..., None] - 127).reshape(q.shape)
    else:
        rows = s["s"].float()
    xh = rows * s["rstd"][:, None]
    dy = s["dy"].float()
    a = dy * s["gain"]
    dx = s["rstd"][:, None] * (a - xh * (a * xh).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(torch.bfloat16), "dgain": (dy * xh).sum(0)}


def _few_plain(s):
    c = s["c"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["x"].float()
    logits = x @ s["W_r"]
    if s["bias"] is not None:
        logits = logits + s["bias"]
    l, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    l, idx = l[:, :k], idx[:, :k]
    w = torch.exp(l - l[:, :1])
    w = w / w.sum(1, keepdim=True)
    xq = _mx_values(x) if c["mx"] else x
    if T * k <= E:      # fewer pairs than experts: each pair's own weights
        f = idx.reshape(-1)
        xx = xq.repeat_interleave(k, 0)[:, None]
        h = _swiglu(xx @ s["Wg"][f].float(), xx @ s["Wu"][f].float())
        y = ((_mx_values(h) if c["mx"] else h) @ s["Wd"][f].float()).reshape(T, k, -1)
    else:               # every token through every expert, the selected results kept
        h = _swiglu(xq @ s["Wg"].float(), xq @ s["Wu"].float())
        y = (_mx_values(h) if c["mx"] else h) @ s["Wd"].float()
        y = y[idx, torch.arange(T, device=idx.device)[:, None]]
    out = (w[..., None] * y).sum(1)
    if c["I_shared"]:
        out = out + _swiglu(x @ s["Sg"][0].float(), x @ s["Su"][0].float()) @ s["Sd"][0].float()
    return {"out": out.to(torch.bfloat16), "idx": idx.int(), "w": w}


def _ckpt_plain(s):
    c, v, rows = s["c"], s["views"], s["rows"]
    I, k = c["I"], c["k"]
    x = _mx_values(s["x"].float()).to(torch.bfloat16)
    gu = _mx_values(v["gu"][rows])
    out = {"x": x, "partials": _mx_values(v["partials"].float()).to(torch.bfloat16)}
    out["A"] = torch.zeros_like(v["A"])
    out["A"][rows] = x.repeat_interleave(k, 0)
    out["gu"] = torch.zeros_like(v["gu"])
    out["gu"][rows] = gu
    out["h"] = torch.zeros_like(v["h"])
    out["h"][rows] = _swiglu(gu[:, :I], gu[:, I:]).to(torch.bfloat16)
    return out


# ----------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["c"]["op"]
    if not own:
        return {"norm": _norm_plain, "norm_bwd": _norm_bwd_plain, "few": _few_plain, "ckpt": _ckpt_plain}[op](s)
    from combine_router_top_expert_gb300 import mok
    if op == "norm":
        if s["c"]["mx"]:
            mok.rmsnorm(s["x"], s["gain"], residual=s["r"], eps=EPS, sum=s["sum"], y_q=s["q"], y_sf=s["sf"],
                        rstd=s["rstd"])
            mok.dequantize_rows(s["q"], s["sf"], s["y"])
        else:
            mok.rmsnorm(s["x"], s["gain"], residual=s["r"], eps=EPS, sum=s["sum"], y=s["y"], rstd=s["rstd"])
        return {"sum": s["sum"], "y": s["y"], "rstd": s["rstd"]}
    if op == "norm_bwd":
        mok.rmsnorm_backward(s["dy"], s["gain"], s["rstd"], s["dx"], s["dgain"], s["ws"], s=s.get("s"),
                             s_q=s.get("q"), s_sf=s.get("sf"), dsum=s["dsum"])
        return {"dx": s["dx"], "dgain": s["dgain"]}
    if op == "few":
        mok.moe_few(s["p"], s["x"], s["W_r"], s["packed"], s["out"], s["ws"], bias=s["bias"],
                    packed_shared=s["packed_shared"], topk_idx=s["idx"], topk_w=s["w"])
        return {"out": s["out"], "idx": s["idx"], "w": s["w"]}
    mok.checkpoint_save(s["p"], s["x"], s["routing"], s["saved"], s["ckpt"])
    mok.checkpoint_load(s["p"], s["ckpt"], s["routing"], s["x_restored"], s["restored"])
    v = s["restored_views"]
    return {"x": s["x_restored"], "partials": v["partials"], "A": v["A"], "gu": v["gu"], "h": v["h"]}


# ----------------------------------------------------------------------------------------------- work

def _active_experts(c):
    """Distinct experts that T tokens select, by simulation of the router's logits (they decide what is read)."""
    g = torch.Generator().manual_seed(1)
    n = 8
    l = torch.randn((n, c["T"], c["E"]), generator=g) * (0.02 * math.sqrt(c["H"]))
    if c["zipf"]:
        l = l + _zipf_bias(c["E"], c["zipf"])
    hit = torch.zeros((n, c["E"])).scatter_(1, l.topk(c["k"], dim=2).indices.reshape(n, -1), 1.0)
    return float(hit.sum()) / n


def work(case):
    c = case
    T, H = c["T"], c["H"]
    mx8 = 1 + 1 / 32                # bytes of an MXFP8 element with its share of the scale
    if c["op"] == "norm":
        n = T * H * (2 + (2 if c["residual"] else 0) + 2) + H * 4 + T * 4
        # 8-bit output: written, read back and written as the BF16 values it stands for
        return {"bytes": n + (T * H * (2 * mx8 + 2) if c["mx"] else T * H * 2), "flops": 6 * T * H}
    if c["op"] == "norm_bwd":
        n = T * H * ((mx8 if c["ckpt"] else 2) + 2 + (2 if c["dsum"] else 0) + 2) + H * 8 + T * 4
        return {"bytes": n, "flops": 12 * T * H}
    I, E, k = c["I"], c["E"], c["k"]
    if c["op"] == "few":
        n = _active_experts(c) * 3 * H * I * (mx8 if c["mx"] else 2) + 3 * H * c["I_shared"] * 2
        n += H * E * 4 + T * H * 4 + T * k * 8
        return {"bytes": n, "flops": 6 * H * T * (I * k + c["I_shared"]) + 2 * T * H * E}
    r = T * k
    small = (T * H + r * 2 * I + r * H) * mx8          # the checkpoint
    save = T * H * 2 + r * 2 * I * 4 + r * H * 2       # x, G|U, partials
    load = save + r * H * 2 + r * I * 2                # and the gathered rows and h
    return {"bytes": save + 2 * small + load, "flops": 10 * r * I}


# ----------------------------------------------------------------------------------------------- 64 bits

def _mx64(v):
    """MXFP8 values of v (64 bits) by the definition: the scale from floor(log2 amax), then the nearest number with
    three fraction bits (steps of 2^-9 below 2^-6), ties to even, at most 448."""
    b = v.double().reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    tiny = 2.0 ** -126
    scale = torch.exp2((torch.floor(torch.log2(amax.clamp(min=tiny))) - 8).clamp(min=-127))
    z = b / scale
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return ((torch.round(z / step) * step).clamp(-448, 448) * scale).reshape(v.shape)


def _silu64(z):
    return z * torch.sigmoid(z)


def _exact_few(s):
    c = s["c"]
    x = s["x"].double()
    l = x @ s["W_r"].double()
    if s["bias"] is not None:
        l += s["bias"].double()
    idx = torch.argsort(l, dim=1, descending=True, stable=True)[:, :c["k"]]
    w = torch.softmax(torch.gather(l, 1, idx), 1)
    xq = _mx64(x) if c["mx"] else x
    out = torch.zeros_like(x)
    for e in range(c["E"]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            h = _silu64(xq[t] @ s["Wg"][e].double()) * (xq[t] @ s["Wu"][e].double())
            out[t] += w[t, j][:, None] * ((_mx64(h) if c["mx"] else h) @ s["Wd"][e].double())
    if c["I_shared"]:
        out += (_silu64(x @ s["Sg"][0].double()) * (x @ s["Su"][0].double())) @ s["Sd"][0].double()
    return {"out": out, "idx": None, "w": w}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "norm":
        t = s["x"].double() + (s["r"].double() if s["r"] is not None else 0)
        rstd = (t.pow(2).sum(1) / c["H"] + EPS).pow(-0.5)
        y = t * rstd[:, None] * s["gain"].double()
        return {"sum": t, "y": _mx64(y.to(torch.bfloat16)) if c["mx"] else y, "rstd": rstd}
    if c["op"] == "norm_bwd":
        if c["ckpt"]:
            v = s["q"].view(torch.float8_e4m3fn).double().reshape(c["T"], -1, 32)
            rows = (v * torch.exp2(s["sf"].double() - 127)[..., None]).reshape(c["T"], -1)
        else:
            rows = s["s"].double()
        r, gain, dy = s["rstd"].double()[:, None], s["gain"].double(), s["dy"].double()
        dot = (gain * dy * rows).sum(1, keepdim=True)
        dx = r * gain * dy - rows * r.pow(3) * dot / c["H"]
        if c["dsum"]:
            dx = dx + s["dsum"].double()
        return {"dx": dx, "dgain": (dy * rows * r).sum(0)}
    if c["op"] == "few":
        return _exact_few(s)
    if c["T"] * c["k"] * (c["H"] + 2 * c["I"]) > 5e7:
        return None                    # gigabytes of 64-bit values: the smaller cases give them
    v, rows, I = s["views"], s["rows"], c["I"]
    x, gu = _mx64(s["x"]), _mx64(v["gu"][rows])
    whole = {n: torch.zeros(v[n].shape, dtype=torch.float64, device="cuda") for n in ("A", "gu", "h")}
    whole["A"][rows] = x.repeat_interleave(c["k"], 0)
    whole["gu"][rows] = gu
    whole["h"][rows] = _silu64(gu[:, :I]) * gu[:, I:]
    return {"x": x, "partials": _mx64(v["partials"]), **whole}
