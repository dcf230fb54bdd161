"""TIDE collectives as PyTorch custom operators (torch.library).

    import parameter_layout_collectives_amd.torch_ops as tops
    pid = tops.register_plan(plan)
    torch.ops.tide.rs(pid, rank, grads_flat, out, small, avg)
    torch.ops.tide.ag(pid, gathered, params, small, copy_engine)
    torch.ops.tide.pack(pid, tensors, slot, small)
    torch.ops.tide.rs_slots(pid, rank, slots, out, small, avg)
    torch.ops.tide.block_shard(block_pid, rank, master, block)
    torch.ops.tide.block_unshard(block_pid, gathered, params)
    torch.ops.tide.block_quant(x, codes, scales)
    torch.ops.tide.block_dequant(codes, scales, out)
    torch.ops.tide.block_mm(x_codes, x_scales, w_codes, w_scales, cols, out, short_sums)
    torch.ops.tide.block_mm_dx(dy, w_codes, w_scales, out)
    torch.ops.tide.block_mm_dw(dy, x_codes, x_scales, out, accumulate)
    torch.ops.tide.fp4_shard(fp4_pid, rank, master, block)
    torch.ops.tide.fp4_unshard(fp4_pid, gathered, params)
    torch.ops.tide.fp4_quant(x, codes, scales)
    torch.ops.tide.fp4_dequant(codes, scales, out)
    torch.ops.tide.fp4_mm(x_codes, x_scales, w_codes, w_scales, cols, out)
    torch.ops.tide.fp4_linear(x, w_codes, w_scales, out_dtype, quant_x)
    torch.ops.tide.fp4_mm_dx(dy, w_codes, w_scales, out)
    torch.ops.tide.ortho(g, out, steps, coefficients)

(block_pid, fp4_pid: the id of a registered BlockPlan or Fp4Plan.)
They are how a training framework calls the collectives in place of
FSDP2's gradient pack and all-gather copy-out ("FSDP通信终局：TIDE零拷贝集合
通信优化", §"TIDE的设计思路": TIDE sits under FSDP2 and keeps its
per-parameter storage).  Each operator declares the tensors it writes, so
autograd and torch.compile see the mutation; the work itself runs in the
library's kernels on the current stream.  grads_flat is rank-major: entry
r*P + i is rank r's gradient of parameter i.  Marshalling walks the tensor
lists on every call; hot loops that reuse the same tensors call the plain
binding with a PointerTable instead.
"""
import itertools
import threading
from typing import List

import torch

from . import (Blocks, Fp4Blocks, Plan, ag, block_dequant, block_mm, block_mm_dw, block_mm_dx,
               block_quant, block_shard, block_unshard, fp4_dequant, fp4_linear, fp4_mm, fp4_mm_dx,
               fp4_quant, fp4_shard, fp4_unshard, ortho, pack, rs, rs_slots)

_PLANS = {}
_LOCK = threading.Lock()
_IDS = itertools.count(1)


def register_plan(plan: Plan) -> int:
    """An integer id for `plan` that the operators accept (kept until
    unregister_plan)."""
    with _LOCK:
        pid = next(_IDS)
        _PLANS[pid] = plan
    return pid


def unregister_plan(pid: int) -> None:
    with _LOCK:
        _PLANS.pop(pid, None)


def _plan(pid):
    try:
        return _PLANS[pid]
    except KeyError:
        raise ValueError(f"no plan registered under id {pid}") from None


def _by_rank(flat, plan):
    if len(flat) != plan.world * plan.P:
        raise ValueError(f"expected N*P = {plan.world * plan.P} gradients, got {len(flat)}")
    P = plan.P
    return [list(flat[r * P:(r + 1) * P]) for r in range(plan.world)]


@torch.library.custom_op("tide::rs", mutates_args=("out",))
def rs_op(pid: int, rank: int, grads: List[torch.Tensor], out: torch.Tensor,
          small: bool = False, avg: bool = False) -> None:
    plan = _plan(pid)
    rs(plan, rank, _by_rank(grads, plan), out, small=small, avg=avg)


@rs_op.register_fake
def _(pid, rank, grads, out, small=False, avg=False):
    return None


@torch.library.custom_op("tide::ag", mutates_args=("params",))
def ag_op(pid: int, gathered: torch.Tensor, params: List[torch.Tensor], small: bool = False,
          copy_engine: bool = False) -> None:
    ag(_plan(pid), gathered, list(params), small=small, copy_engine=copy_engine)


@ag_op.register_fake
def _(pid, gathered, params, small=False, copy_engine=False):
    return None


@torch.library.custom_op("tide::pack", mutates_args=("slot",))
def pack_op(pid: int, tensors: List[torch.Tensor], slot: torch.Tensor,
            small: bool = False) -> None:
    pack(_plan(pid), list(tensors), slot, small=small)


@pack_op.register_fake
def _(pid, tensors, slot, small=False):
    return None


@torch.library.custom_op("tide::rs_slots", mutates_args=("out",))
def rs_slots_op(pid: int, rank: int, slots: torch.Tensor, out: torch.Tensor,
                small: bool = False, avg: bool = False) -> None:
    rs_slots(_plan(pid), rank, slots, out, small=small, avg=avg)


@rs_slots_op.register_fake
def _(pid, rank, slots, out, small=False, avg=False):
    return None


# Matrices in 8-bit blocks (blocks.py): codes and scales are passed as tensors.

@torch.library.custom_op("tide::block_shard", mutates_args=("block",))
def block_shard_op(pid: int, rank: int, master: torch.Tensor, block: torch.Tensor) -> None:
    block_shard(_plan(pid), rank, master, block)


@block_shard_op.register_fake
def _(pid, rank, master, block):
    return None


@torch.library.custom_op("tide::block_unshard", mutates_args=("params",))
def block_unshard_op(pid: int, gathered: torch.Tensor, params: List[torch.Tensor]) -> None:
    block_unshard(_plan(pid), gathered, list(params))


@block_unshard_op.register_fake
def _(pid, gathered, params):
    return None


@torch.library.custom_op("tide::block_quant", mutates_args=("codes", "scales"))
def block_quant_op(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor) -> None:
    block_quant(x, out=Blocks(codes, scales, x.shape[1]))


@block_quant_op.register_fake
def _(x, codes, scales):
    return None


@torch.library.custom_op("tide::block_dequant", mutates_args=("out",))
def block_dequant_op(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor) -> None:
    block_dequant(Blocks(codes, scales, out.shape[1]), out=out)


@block_dequant_op.register_fake
def _(codes, scales, out):
    return None


@torch.library.custom_op("tide::block_mm", mutates_args=("out",))
def block_mm_op(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor,
                w_scales: torch.Tensor, cols: int, out: torch.Tensor,
                short_sums: bool = False) -> None:
    block_mm(Blocks(x_codes, x_scales, cols), Blocks(w_codes, w_scales, cols), out=out,
             short_sums=short_sums)


@block_mm_op.register_fake
def _(x_codes, x_scales, w_codes, w_scales, cols, out, short_sums=False):
    return None


@torch.library.custom_op("tide::block_mm_dx", mutates_args=("out",))
def block_mm_dx_op(dy: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                   out: torch.Tensor) -> None:
    block_mm_dx(dy, Blocks(w_codes, w_scales, out.shape[1]), out=out)


@block_mm_dx_op.register_fake
def _(dy, w_codes, w_scales, out):
    return None


@torch.library.custom_op("tide::block_mm_dw", mutates_args=("out",))
def block_mm_dw_op(dy: torch.Tensor, x_codes: torch.Tensor, x_scales: torch.Tensor,
                   out: torch.Tensor, accumulate: bool = False) -> None:
    block_mm_dw(dy, Blocks(x_codes, x_scales, out.shape[1]), out=out, accumulate=accumulate)


@block_mm_dw_op.register_fake
def _(dy, x_codes, x_scales, out, accumulate=False):
    return None


# Matrices in 4-bit blocks (fp4.py), likewise.

@torch.library.custom_op("tide::fp4_shard", mutates_args=("block",))
def fp4_shard_op(pid: int, rank: int, master: torch.Tensor, block: torch.Tensor) -> None:
    fp4_shard(_plan(pid), rank, master, block)


@fp4_shard_op.register_fake
def _(pid, rank, master, block):
    return None


@torch.library.custom_op("tide::fp4_unshard", mutates_args=("params",))
def fp4_unshard_op(pid: int, gathered: torch.Tensor, params: List[torch.Tensor]) -> None:
    fp4_unshard(_plan(pid), gathered, list(params))


@fp4_unshard_op.register_fake
def _(pid, gathered, params):
    return None


@torch.library.custom_op("tide::fp4_quant", mutates_args=("codes", "scales"))
def fp4_quant_op(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor) -> None:
    fp4_quant(x, out=Fp4Blocks(codes, scales, x.shape[1]))


@fp4_quant_op.register_fake
def _(x, codes, scales):
    return None


@torch.library.custom_op("tide::fp4_dequant", mutates_args=("out",))
def fp4_dequant_op(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor) -> None:
    fp4_dequant(Fp4Blocks(codes, scales, out.shape[1]), out=out)


@fp4_dequant_op.register_fake
def _(codes, scales, out):
    return None


@torch.library.custom_op("tide::fp4_mm", mutates_args=("out",))
def fp4_mm_op(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor,
              w_scales: torch.Tensor, cols: int, out: torch.Tensor) -> None:
    fp4_mm(Fp4Blocks(x_codes, x_scales, cols), Fp4Blocks(w_codes, w_scales, cols), out=out)


@fp4_mm_op.register_fake
def _(x_codes, x_scales, w_codes, w_scales, cols, out):
    return None


@torch.library.custom_op("tide::fp4_linear", mutates_args=())
def fp4_linear_op(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                  out_dtype: torch.dtype, quant_x: bool = False) -> torch.Tensor:
    return fp4_linear(x, Fp4Blocks(w_codes, w_scales, x.shape[-1]), dtype=out_dtype,
                      quant_x=quant_x)


@fp4_linear_op.register_fake
def _(x, w_codes, w_scales, out_dtype, quant_x=False):
    return x.new_empty(*x.shape[:-1], w_codes.shape[0], dtype=out_dtype)


@torch.library.custom_op("tide::fp4_mm_dx", mutates_args=("out",))
def fp4_mm_dx_op(dy: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                 out: torch.Tensor) -> None:
    fp4_mm_dx(dy, Fp4Blocks(w_codes, w_scales, out.shape[1]), out=out)


@fp4_mm_dx_op.register_fake
def _(dy, w_codes, w_scales, out):
    return None


@torch.library.custom_op("tide::ortho", mutates_args=("out",))
def ortho_op(g: List[torch.Tensor], out: List[torch.Tensor], steps: int,
             coefficients: List[float]) -> None:
    ortho(list(g), out=list(out), steps=steps, coefficients=coefficients)


@ortho_op.register_fake
def _(g, out, steps, coefficients):
    return None
