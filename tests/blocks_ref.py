"""The 8-bit block format and its products in 64 bits, from the definitions.

Shares no code with the library: exponents are found by comparing with
448 * 2^e, e4m3 numbers by enumerating their 256 bytes, and products are
float64 matrix products (on the device where they would take long on a CPU)."""
import math

import torch

EMIN, EMAX = -117, 119


def e4m3_table():
    """The 256 values of e4m3 bytes (float64; NaN for 0x7f and 0xff)."""
    t = []
    for b in range(256):
        ex, fr = (b >> 3) & 15, b & 7
        v = math.ldexp(fr, -9) if ex == 0 else math.ldexp(8 + fr, ex - 10)
        if b & 127 == 127:
            v = math.nan
        t.append(-v if b & 128 else v)
    return torch.tensor(t, dtype=torch.float64)


def exponent(a):
    """The block exponent of the largest finite magnitude a (a Python float)."""
    if a == 0:
        return 0
    e = EMIN
    while e < EMAX and a > math.ldexp(448.0, e):
        e += 1
    return e


_POW = torch.tensor([2.0 ** j for j in range(-300, 301)], dtype=torch.float64)


def pow2(e):
    """2^e in float64 for whole e, exactly."""
    return _POW.to(e.device)[e.long() + 300]


def quant(x):
    """x [R, C] -> (code bytes [R, Cp], scale bytes [R, Sp]) as uint8 CPU tensors.
    -0 and values that round to it keep their sign; infinities and NaNs are 0x7f."""
    x = x.detach().cpu().double()
    R, C = x.shape
    nb = -(-C // 128)
    sp = -(-nb // 4) * 4
    codes = torch.zeros(R, nb * 128, dtype=torch.uint8)
    scales = torch.full((R, sp), 127, dtype=torch.uint8)
    mags = e4m3_table()[:127]                      # 0 .. 448, ascending
    for b in range(nb):
        v = x[:, b * 128:(b + 1) * 128]
        fin = torch.isfinite(v)
        top = torch.where(fin, v.abs(), 0.0).amax(1)
        e = torch.tensor([exponent(float(a)) for a in top], dtype=torch.float64)
        scales[:, b] = (e + 127).to(torch.uint8)
        s = v.abs() * pow2(-e).unsqueeze(1)
        s = torch.where(fin, s, 0.0).clamp_max(448.0)
        hi = torch.searchsorted(mags, s.contiguous()).clamp_max(126)   # mags[hi] >= s
        lo = (hi - 1).clamp_min(0)
        up, down = mags[hi] - s, s - mags[lo]
        pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        pick = torch.where(mags[hi] == s, hi, pick)
        byte = pick + 128 * torch.signbit(v).long()
        codes[:, b * 128:b * 128 + v.shape[1]] = \
            torch.where(fin, byte, torch.full_like(byte, 0x7f)).to(torch.uint8)
    return codes, scales


def values(codes, scales, cols):
    """The float64 values [R, cols] of code and scale bytes, on their device."""
    codes, scales = codes.view(torch.uint8), scales.view(torch.uint8)
    v = e4m3_table().to(codes.device)[codes.long()[:, :cols]]
    e = scales.long().repeat_interleave(128, dim=1)[:, :cols] - 127
    return v * pow2(e)


def product(a, b):
    """(a b^T, |a| |b|^T) in float64."""
    return a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()


def off(got, want, mass, terms, fast=False):
    """The largest |got - want| as a share of what rounding may cause.

    terms products are exact and summed in fp32 in some order: each of the at
    most `terms` additions is off by half a unit, 2^-24 of a partial sum of at
    most `mass` = sum |product|; matrix instructions may cut instead of round,
    so a whole unit, 2^-23, is counted.  The result is rounded once to its type.
    fast: the 8-bit matrix instruction; it lines 128 products up with the
    largest and cuts what falls below its adder, 2^-13.3 of the 128 products'
    mass at worst over random codes of the whole range; 2^-12 is counted."""
    info = torch.finfo(got.dtype)
    half = info.eps / 2
    tol = mass * (terms * 2.0 ** -23 + (2.0 ** -12 if fast else 0.0))
    # below its smallest normal number a type's spacing is tiny * eps
    tol = tol + half * (want.abs() + tol) + info.tiny * half
    return float(((got.double() - want).abs() / tol).max()) if got.numel() else 0.0
