"""tide_ortho of matrices with more than 256 rows and columns in more than 5 steps, or in
steps that raise small singular values further, on the GPU, against the steps in 64 bits.

Tolerance of a result's norm: rounding to bf16, 2^-8; what the fp16 factors cost in the
emulation; and what sums in fp32 cost, taken from the same steps in fp32 throughout.
test_ortho_steps_host.py pins the last two."""
import pytest
import torch

import ortho_ref as ref
import parameter_layout_collectives_amd as tide
from gpu_helpers import note
from test_ortho_steps_host import CASES, ONE_MAGNITUDE, ONE_MAGNITUDE_OFF, SHAPES, signs

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", SHAPES + [(700, 512), (2050, 300)])
@pytest.mark.parametrize("kind", ["full", "low"])
def test_more_steps(shape, dtype, kind):
    note(f"ortho, more steps, {shape} {dtype} {kind}")
    g = ref.gradient(*shape, 7, kind, dtype, "cuda")
    for steps, coefficients, factors, sums in CASES:
        out = tide.ortho(g, steps=steps, coefficients=coefficients)
        err = ref.off(out, ref.exact(g, steps, coefficients))
        assert err <= 2.0 ** -8 + factors + sums, (steps, err)


def test_large_tiles():
    note("ortho, more steps, large tiles")
    for shape in ((2050, 4100), (4100, 2050)):
        g = ref.gradient(*shape, 5, "low", BF, "cuda")
        steps, coefficients, factors, sums = CASES[1]
        out = tide.ortho(g, steps=steps, coefficients=coefficients)
        err = ref.off(out, ref.exact(g, steps, coefficients))
        assert err <= 2.0 ** -8 + factors + sums, (shape, err)


def test_many_steps_stay_bounded():
    note("ortho, 64 steps")
    for shape in ((300, 420), (420, 300), (40, 500)):
        for kind in ("full", "low"):
            out = tide.ortho(ref.gradient(*shape, 3, kind, FP, "cuda"), steps=64)
            assert bool(torch.isfinite(out).all()) and float(out.abs().max()) <= 1.3


@pytest.mark.parametrize("shape", ONE_MAGNITUDE + [(99, 71), (1504, 315)])
def test_entries_of_one_magnitude(shape):
    note(f"ortho, entries of one magnitude {shape}")
    for dtype in (BF, FP):
        g = signs(*shape).to(dtype).cuda()
        err = ref.off(tide.ortho(g), ref.exact(g))
        assert err <= 2.0 ** -8 + ONE_MAGNITUDE_OFF, (dtype, err)
