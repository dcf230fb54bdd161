"""No derivative is dropped in silence: host-side checks that need no GPU."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import parameter_layout_collectives_amd as tide
from test_blocks_host import _Stub, stub_blocks


def test_dual_tensors_are_refused():
    """A dual tensor requires no gradient, so nothing else would notice it."""
    bf = torch.bfloat16
    x, w = stub_blocks(4, 200), stub_blocks(8, 200)
    plan = tide.BlockPlan(tide.Plan([(8, 200)], 2))
    gathered = _Stub((2, plan.S), torch.int32)
    with fwd.dual_level():
        def dual(*shape):
            return fwd.make_dual(torch.zeros(shape, dtype=bf), torch.ones(shape, dtype=bf))
        for call in (lambda: tide.block_linear(dual(4, 200), w),
                     lambda: tide.block_quant(dual(4, 200)),
                     lambda: tide.block_mm_dx(dual(4, 8), w),
                     lambda: tide.block_mm_dw(dual(4, 8), x),
                     lambda: tide.block_mm(x, w, out=dual(4, 8)),
                     lambda: tide.block_dequant(x, out=dual(4, 200)),
                     lambda: tide.block_shard(plan, 0, dual(4, 200).float(), None),
                     lambda: tide.block_unshard(plan, gathered, [dual(8, 200)])):
            with pytest.raises(NotImplementedError, match="dual"):
                call()
