"""Blocks whose memory is released, restored and replaced between calls, as an FSDP
unit does with its gathered weights."""
import pytest
import torch

import parameter_layout_collectives_amd as tide
from gpu_helpers import note
from test_gpu_blocks import FP, bytes_of, rand, unit_with_weights

pytestmark = pytest.mark.gpu


def release(q):
    for t in (q.codes, q.scales):
        t.untyped_storage().resize_(0)


def restore(q):
    """New memory, elsewhere: what is allocated meanwhile stays until after."""
    hold = [torch.empty(t.shape, dtype=torch.uint8, device=t.device) for t in (q.codes, q.scales)]
    for t in (q.codes, q.scales):
        t.untyped_storage().resize_(t.numel())
    return hold


@pytest.mark.parametrize("m", [3, 70])
def test_weights_released_and_restored(m):
    note(f"block products of released and restored weights {m}")
    x, wr = rand((m, 264), 1), rand((40, 264), 2, FP, 0.02)
    w, same = tide.block_quant(wr), tide.block_quant(wr)
    dy = rand((m, 40), 3)
    release(w)
    for call in (lambda: tide.block_linear(x, w), lambda: tide.block_mm(tide.block_quant(x), w),
                 lambda: tide.block_mm_dx(dy, w), lambda: tide.block_dequant(w)):
        with pytest.raises(tide.TideError, match="NULL"):
            call()
    hold = restore(w)
    tide.block_quant(wr, out=w)
    assert torch.equal(tide.block_linear(x, w), tide.block_linear(x, same))
    assert torch.equal(tide.block_mm_dx(dy, w), tide.block_mm_dx(dy, same))
    assert torch.equal(tide.block_dequant(w), tide.block_dequant(same))
    other = tide.block_quant(2 * wr)
    w.codes, w.scales = other.codes, other.scales
    assert torch.equal(tide.block_linear(x, w), tide.block_linear(x, other))
    del hold


def test_unit_whose_weights_move():
    note("TideUnit blocks released, restored and replaced")
    unit, full = unit_with_weights(3, [0, 2])
    x = rand((5, 200), 4)
    unit.all_gather()
    want = unit.linear(0, x)
    release(unit.params[0])
    hold = restore(unit.params[0])
    unit.params[2] = tide.Blocks.empty(200, 96)
    unit.all_gather()
    assert torch.equal(unit.linear(0, x), want)
    unit.params[0].codes = torch.zeros_like(unit.params[0].codes)
    unit.all_gather()
    assert torch.equal(unit.linear(0, x), want)
    for i in (0, 2):
        got, q = bytes_of(unit.params[i]), bytes_of(tide.block_quant(full[i]))
        assert torch.equal(got[0], q[0]) and torch.equal(got[1], q[1])
    del hold
