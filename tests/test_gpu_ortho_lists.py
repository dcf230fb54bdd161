"""A matrix gets the same bits from tide_ortho whatever else is in the list: the others
decide how large the products' tiles are."""
import pytest
import torch

import ortho_ref as ref
import parameter_layout_collectives_amd as tide
from gpu_helpers import note

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
SHAPES = [(33, 40), (128, 300), (300, 128), (256, 640), (333, 1000), (500, 1030), (1030, 500), (37, 129)]
# beside 1 [2048, 2048] the products take tiles of 128 rows and columns, beside 7 of 256;
# alone these matrices take 64
BESIDE = [(1, 2048), (7, 2048)]


@pytest.mark.parametrize("steps", [5, 7])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind", ["full", "heavy", "low"])
def test_alone_and_beside_others(kind, dtype, steps):
    note(f"ortho alone and in lists, {kind} {dtype} {steps} steps")
    gs = [ref.gradient(*s, i, kind, dtype, "cuda") for i, s in enumerate(SHAPES)]
    alone = [tide.ortho(g, steps=steps) for g in gs]
    together = tide.ortho(gs, steps=steps)
    for s, a, b in zip(SHAPES, alone, together):
        assert torch.equal(a, b), s
    for count, side in BESIDE:
        big = [ref.gradient(side, side, 50, "full", dtype, "cuda")] * count
        for s, g, a in zip(SHAPES, gs, alone):
            got = tide.ortho(big + [g], steps=steps)[-1]
            assert torch.equal(a, got), (s, count, int((a != got).sum()))


def test_many_shapes():
    note("ortho of 300 matrices of 70 shapes, each as alone")
    shapes = [(1 + 7 * (i % 10), 1 + 11 * (i // 10)) for i in range(70)]
    gs = [ref.gradient(*shapes[i % 70], i, "heavy", FP, "cuda") for i in range(300)]
    outs = tide.ortho(gs)
    for i in range(0, 300, 7):
        assert torch.equal(tide.ortho(gs[i]), outs[i]), i
