"""Newton-Schulz orthogonalisation in 64 bits, and an emulation of the roundings that
a kernel with fp16 factors makes.  Shares no code with the library."""
import math

import torch

QUINTIC = (3.4445, -4.7750, 2.0315)


def triples(coefficients, steps):
    return [coefficients] * steps if not isinstance(coefficients[0], (tuple, list)) else coefficients


def exact(g, steps=5, coefficients=QUINTIC):
    """One matrix, from the definition."""
    x = g.double()
    if x.shape[0] > x.shape[1]:
        return exact(x.t().contiguous(), steps, coefficients).t().contiguous()
    norm = torch.sqrt((x * x).sum())
    if float(norm) == 0:
        return torch.zeros_like(x)
    x = x / norm
    for a, b, c in triples(coefficients, steps):
        p = x @ x.t().contiguous()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x


def _half(t, scale):
    return (t * scale).to(torch.float16).double() / scale


def emulated(g, steps=5, coefficients=QUINTIC, both=256):
    """`exact` with X as two fp16 numbers, its products' factors without diagonals in
    one (X X^T, P) or, up to `both` rows, two (the X of P X)."""
    x = g.double()
    if x.shape[0] > x.shape[1]:
        return emulated(x.t().contiguous(), steps, coefficients, both).t().contiguous()
    r, c = x.shape
    if r <= 32:
        return exact(g, steps, coefficients)
    norm = float(torch.sqrt((x * x).sum()))
    if norm == 0:
        return torch.zeros_like(x)
    sx = 2.0 ** min(14, int(math.log2(r * c) / 2))
    x = x * 2.0 ** -math.frexp(norm)[1]
    first = 1 / math.frexp(norm)[0]
    for s, (a, b, cc) in enumerate(triples(coefficients, steps)):
        f = first if s == 0 else 1.0
        hi = _half(x, sx)
        lo = _half(x - hi, sx)
        p = (hi @ hi.t().contiguous()) * f * f
        d = p.diagonal().clone()
        o = _half(p - torch.diag(d), 4096.0)
        oo = o @ o
        q = a + b * d + cc * (d * d + oo.diagonal())
        rest = b * o + cc * ((d[:, None] + d[None, :]) * o + oo)
        rest = _half(rest - torch.diag(rest.diagonal()), 1024.0)
        factor = hi + lo if r <= both else hi
        x = (rest @ factor + q[:, None] * (hi + lo)) * f
    return x


def off(got, want):
    """The norm of the difference over the norm of `want`."""
    n = float(want.double().norm())
    d = float((got.double() - want.double()).norm())
    return d / n if n else (0.0 if d == 0 else math.inf)


def gradient(r, c, seed, kind="heavy", dtype=torch.float32, device="cpu"):
    """full: every direction alike.  heavy: a few directions far above a floor whose
    rows and columns differ in size.  low: of rank r / 8."""
    gen = torch.Generator().manual_seed(seed)
    def n(*s):
        return torch.randn(*s, generator=gen)
    g = n(r, c)
    if kind == "heavy":
        few = max(1, min(r, c) // 64)
        g = g * torch.exp(0.5 * n(r, 1)) * torch.exp(0.5 * n(1, c))
        g = g + n(r, few) @ n(few, c) * 2
    elif kind == "low":
        k = max(1, min(r, c) // 8)
        g = n(r, k) @ n(k, c)
    return (g * 1e-3).to(dtype).to(device)
