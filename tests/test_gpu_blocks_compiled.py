"""The 8-bit block operators in a compiled step."""
import pytest
import torch

import parameter_layout_collectives_amd as tide
import parameter_layout_collectives_amd.torch_ops as tops
from gpu_helpers import note
from test_gpu_blocks import BF, rand, shards

pytestmark = pytest.mark.gpu


def test_block_ops_under_torch_compile():
    """A step that gathers a unit in blocks, quantises an activation and multiplies
    forward and backward gives the eager bits when compiled."""
    plan, full, master = shards([(72, 264), (9, 130)], 3, 80)
    pid = tops.register_plan(tide.BlockPlan(plan))
    ops = torch.ops.tide
    try:
        bp = tops._PLANS[pid]
        m, n, k = 70, 72, 264
        w = tide.block_quant(full[0])
        x, dy = rand((m, k), 81), rand((m, n), 82, BF, 1e-3)

        def step(master, gathered, params, x, dy, codes, scales, y, back, dx, dw):
            for r in range(3):
                ops.block_shard(pid, r, master[r], gathered[r])
            ops.block_unshard(pid, gathered, params)
            ops.block_quant(x, codes, scales)
            ops.block_dequant(codes, scales, back)
            ops.block_mm(codes, scales, w.codes, w.scales, k, y)
            ops.block_mm_dx(dy, w.codes, w.scales, dx)
            ops.block_mm_dw(dy, codes, scales, dw, True)
            return y.float() * 2.0

        res = []
        for name, fn in (("eager", step),
                         ("compiled", torch.compile(step, backend="aot_eager", fullgraph=True))):
            note(f"block operators, {name}")
            q = tide.Blocks.empty(m, k)
            out = [bp.empty().zero_(), [torch.zeros(s, dtype=BF, device="cuda") for s in bp.matrices],
                   x, dy, q.codes, q.scales, torch.zeros(m, n, dtype=BF, device="cuda"),
                   torch.zeros(m, k, dtype=BF, device="cuda"),
                   torch.zeros(m, k, dtype=BF, device="cuda"), torch.ones(n, k, device="cuda")]
            res.append((fn(master, *out), out))
        (y1, o1), (y2, o2) = res
        assert torch.equal(y1, y2)
        for a, b in zip(o1, o2):
            for s, t in zip(a, b) if isinstance(a, list) else [(a, b)]:
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
        assert torch.equal(y1, 2 * tide.block_mm(tide.block_quant(x), w).float())
        assert torch.equal(o1[1][0], tide.block_dequant(w))
    finally:
        tops.unregister_plan(pid)
