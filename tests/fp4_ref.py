"""The 4-bit block format in 64 bits, from the definition.

Shares no code with the library: exponents are found by comparing with 6 * 2^e, e2m1
numbers by enumerating the 8 magnitudes, products are float64 matrix products."""
import math

import torch

EMIN, EMAX = -125, 125
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TABLE = torch.tensor(MAGNITUDES + [-v for v in MAGNITUDES], dtype=torch.float64)
_POW = torch.tensor([2.0 ** j for j in range(-400, 401)], dtype=torch.float64)


def pow2(e):
    """2^e in float64 for whole e, exactly."""
    return _POW.to(e.device)[e.long() + 400]


def exponent(a):
    """The block exponent of the largest magnitude a (a Python float)."""
    if a == 0:
        return 0
    e = EMIN
    while e < EMAX and a > math.ldexp(6.0, e):
        e += 1
    return e


def quant(x):
    """x [R, C] -> (code bytes [R, Cp / 2], scale bytes [R, Cp / 32]) as uint8 CPU tensors."""
    x = x.detach().cpu().double()
    R, C = x.shape
    cp = -(-C // 128) * 128
    codes = torch.zeros(R, cp, dtype=torch.uint8)
    scales = torch.full((R, cp // 32), 127, dtype=torch.uint8)
    for b in range(-(-C // 32)):
        v = x[:, b * 32:(b + 1) * 32]
        for r in range(R):
            if not bool(torch.isfinite(v[r]).all()):
                scales[r, b] = 255
                continue
            e = exponent(float(v[r].abs().max()))
            scales[r, b] = e + 127
            s = v[r].abs() * 2.0 ** -e
            dist = (s.clamp_max(6.0).unsqueeze(1) - TABLE[:8].unsqueeze(0)).abs()
            near = dist.min(1).values
            for c in range(v.shape[1]):
                ties = [k for k in range(8) if dist[c, k] == near[c]]
                k = ties[0] if len(ties) == 1 else next(t for t in ties if t % 2 == 0)
                codes[r, b * 32 + c] = k + 8 * int(torch.signbit(v[r, c]))
    return codes[:, 0::2] + 16 * codes[:, 1::2], scales


def values(codes, scales, cols):
    """The float64 values [R, cols] of code and scale bytes, on their device."""
    codes, scales = codes.view(torch.uint8), scales.view(torch.uint8)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :cols].long()
    s = scales.long().repeat_interleave(32, dim=1)[:, :cols]
    v = TABLE.to(codes.device)[c] * pow2(s - 127)
    return torch.where(s == 255, torch.full_like(v, math.nan), v)
