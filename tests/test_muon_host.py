"""What TideUnit.muon_step refuses, it refuses before the momentum moves: no GPU."""
import pytest
import torch

import parameter_layout_collectives_amd as tide
from parameter_layout_collectives_amd.fsdp import TideUnit

SHAPES = [(4, 64), (6, 32), (5,)]


def refused_scale(rows, cols):
    raise ZeroDivisionError("scale")


@pytest.mark.parametrize("kw,error,needle", [
    (dict(steps=0), tide.TideError, "steps"),
    (dict(steps=65), tide.TideError, "steps"),
    (dict(coefficients=(1.0, 2.0)), ValueError, "triples"),
    (dict(coefficients=[(3.0, -3.0, 1.0)] * 2), ValueError, "triples"),
    (dict(coefficients=(3.0, float("nan"), 1.0)), tide.TideError, "finite"),
    (dict(scale=refused_scale), ZeroDivisionError, "scale"),
    (dict(select=[0, 0]), ValueError, "twice"),
    (dict(select=[-1]), ValueError, "out of range"),
    (dict(select=[3]), ValueError, "out of range"),
    (dict(momentum="much"), ValueError, "much"),
    (dict(weight_decay=None), TypeError, "float"),
])
def test_refusals_leave_the_unit_as_it_was(kw, error, needle):
    unit = TideUnit(SHAPES, 2, device="cpu")
    unit.grad.fill_(1.0)
    with pytest.raises(error, match=needle):
        unit.muon_step(0.1, **kw)
    assert unit.momentum is None or not bool(unit.momentum.any())
    assert unit._muon is None                    # another selection may follow
    assert not bool(unit.master.any())
