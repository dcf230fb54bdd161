"""How far the roundings of tide_ortho reach in more than 5 steps, and for matrices that
average none of them out: the emulation in 64 bits (ortho_ref.py), no GPU."""
import pytest
import torch

import ortho_ref as ref

# The steps' a multiplied exceed 512 from 6 steps on: R X takes X's lo for every size.
RAISING = [(8.2, -22.0, 16.0), (4.1, -2.95, 0.55), (3.95, -2.9, 0.55), (3.3, -2.5, 0.51),
           (2.3, -1.7, 0.42)]
# steps, coefficients, off by in the emulation, and with sums in fp32 alone
CASES = [(6, ref.QUINTIC, 1.66e-3, 1e-4), (8, ref.QUINTIC, 1.66e-3, 1e-3),
         (10, ref.QUINTIC, 4e-3, 8e-3), (5, RAISING, 2e-3, 1e-4)]
SHAPES = [(300, 420), (420, 300), (512, 700)]


def in_fp32(g, steps, coefficients):
    x = g.float()
    if x.shape[0] > x.shape[1]:
        return in_fp32(x.t().contiguous(), steps, coefficients).t().contiguous()
    x = x / torch.sqrt((x * x).sum())
    for a, b, c in ref.triples(coefficients, steps):
        p = x @ x.t().contiguous()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["full", "low"])
def test_more_steps(shape, kind):
    for dtype in (torch.float32, torch.bfloat16):
        g = ref.gradient(*shape, 7, kind, dtype)
        for steps, coefficients, factors, sums in CASES:
            want = ref.exact(g, steps, coefficients)
            assert ref.off(ref.emulated(g, steps, coefficients, both=1 << 20), want) < factors
            assert ref.off(in_fp32(g, steps, coefficients), want) < sums


def test_hi_alone_would_not_do():
    """Why: a low rank in 8 steps."""
    g = ref.gradient(300, 420, 7, "low")
    assert ref.off(ref.emulated(g, 8), ref.exact(g, 8)) > 3e-2


# Of rank one, all entries of one magnitude: every rounding is the same, none averages out.
ONE_MAGNITUDE = [(71, 99), (39, 370), (64, 64), (315, 1504), (512, 1024), (325, 600)]
ONE_MAGNITUDE_OFF = 1.05e-2


def signs(r, c, seed=1):
    gen = torch.Generator().manual_seed(seed)
    rows, cols = (torch.sign(torch.randn(n, generator=gen)) for n in (r, c))
    return rows[:, None] * cols[None, :] * 0.25


@pytest.mark.parametrize("shape", ONE_MAGNITUDE)
def test_entries_of_one_magnitude(shape):
    g = signs(*shape)
    assert ref.off(ref.emulated(g), ref.exact(g)) < ONE_MAGNITUDE_OFF


def test_entries_of_one_magnitude_are_the_worst_known():
    assert ref.off(ref.emulated(signs(315, 1504)), ref.exact(signs(315, 1504))) > 9e-3
