"""Plain MXFP8 arithmetic for the tests, in 64 bits: E4M3 elements (three
fraction bits, steps of 2^-9 below 2^-6, ties to even, at most 448) with one
scale 2^(floor(log2 amax) - 8) per 32 elements along the last axis. Exponents
come from frexp and powers of two from their bit patterns, so every operation
here is exact."""
import torch


def pow2(e):
    """2^e in float64 for whole e in -1022 .. 1023."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _floor_log2(v):
    return torch.frexp(v).exponent - 1


def scale_codes(v):
    """E8M0 codes [..., n/32] of v [..., n]."""
    amax = v.double().reshape(*v.shape[:-1], -1, 32).abs().amax(-1)
    code = _floor_log2(torch.where(amax > 0, amax, torch.ones_like(amax))) - 8 + 127
    return torch.where(amax > 0, code.clamp(0, 254), torch.zeros_like(code))


def values(v):
    """The values that the MXFP8 form of v stands for, as float64."""
    b = v.double().reshape(*v.shape[:-1], -1, 32)
    scale = pow2(scale_codes(v) - 127)[..., None]
    z = b / scale
    e = _floor_log2(z.abs().clamp(min=2.0 ** -6))
    step = pow2(e - 3)
    return ((torch.round(z / step) * step).clamp(-448, 448) * scale).reshape(v.shape)


def decode(q, sf):
    """Values of E4M3 bytes q [..., n] with codes sf [..., n/32], as float64."""
    c = q.to(torch.int64)
    sign = torch.where(c >= 128, -1.0, 1.0).double()
    ex, m = (c >> 3) & 15, c & 7
    mag = torch.where(ex > 0, (8 + m).double() * pow2(ex - 10),
                      m.double() * 2.0 ** -9)
    s = pow2(sf.to(torch.int64) - 127)
    return (sign * mag).reshape(*q.shape[:-1], -1, 32).mul(s[..., None]).reshape(q.shape)


def half_ulp_bf16(*vs):
    """Half the BF16 spacing at the largest of the magnitudes."""
    a = torch.stack([v.double().abs() for v in vs]).amax(0).clamp(min=2.0 ** -126)
    return pow2(_floor_log2(a) - 8)
