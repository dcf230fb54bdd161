"""TideUnit.muon_step of units with empty matrices, on the GPU."""
import pytest
import torch

import ortho_ref as ref
from gpu_helpers import note
from parameter_layout_collectives_amd.fsdp import TideUnit

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("world", [1, 3])
def test_unit_with_empty_matrices(world):
    """[0, C] and [R, 0] stand beside others, which are updated as without them; the
    tolerance is that of two bf16 results of test_gpu_ortho.py."""
    note(f"muon_step, empty matrices, world {world}")
    shapes = [(0, 7), (40, 70), (5, 0), (70, 40), (0, 0)]
    unit, plain = TideUnit(shapes, world), TideUnit([shapes[1], shapes[3]], world)
    full = [ref.gradient(*s, 3, "full").cuda() if s[0] * s[1] else torch.zeros(s, device="cuda")
            for s in shapes]
    unit.load(full)
    plain.load([full[1], full[3]])
    for step in range(2):
        grads = [[(ref.gradient(*s, 10 * step + r, "heavy") if s[0] * s[1] else torch.zeros(s)).to(BF).cuda()
                  for s in shapes] for r in range(world)]
        unit.reduce_scatter(grads)
        plain.reduce_scatter([[g[1], g[3]] for g in grads])
        unit.muon_step(0.1)
        plain.muon_step(0.1)
    unit.all_gather()
    plain.all_gather()
    for a, b, f in zip((unit.params[1], unit.params[3]), plain.params, (full[1], full[3])):
        assert torch.equal(a, b)
        assert not torch.equal(a, f.to(BF))


def test_unit_of_empty_matrices_only():
    note("muon_step, empty matrices only")
    unit = TideUnit([(0, 7), (3, 0), (4,)], 2)
    unit.load([torch.zeros(0, 7, device="cuda"), torch.zeros(3, 0, device="cuda"),
               torch.ones(4, device="cuda")])
    before = unit.master.clone()
    unit.muon_step(0.1)
    assert torch.equal(unit.master, before)
