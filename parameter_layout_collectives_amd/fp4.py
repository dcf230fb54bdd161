"""Matrices in microscaled 4-bit blocks: the 4-bit gather of an FSDP unit's weights
and the products of a layer whose weights are frozen or serve.

    q = fp4_quant(x)                         # x [m, k] -> Fp4Blocks
    x = fp4_dequant(q)                       # ... and back
    y = fp4_mm(q, w)                         # y [m, n] = x w^T, both in 4-bit blocks
    y = fp4_linear(x, w)                     # ... x as it is, and through autograd
    y = fp4_linear(x, w, quant_x=True)       # ... x rounded to 4-bit blocks on the way
    dx = fp4_mm_dx(dy, w)                    # dx [m, k] = dy w

    plan = Fp4Plan(Plan(shapes, world))      # gather matrices in 4 bits
    fp4_shard(plan, rank, master, gathered[rank])
    ag(plan, gathered, plan.views(weights))  # -> Fp4Blocks for the products, or
    fp4_unshard(plan, gathered, params)      # -> full tensors

The format (e2m1 codes, one power of two per 32 columns of a row), the arguments
and the errors are documented in include/tide.h (tide_mx_*).  A 4-bit gather moves about a
quarter of the bytes of a bf16 all-gather ("FSDP通信终局：TIDE零拷贝集合通信优化",
§"FSDP2通信开销的根源": the all-gather's bytes are part of every step).

As with the 8-bit blocks, the linear call is the differentiable one, in reverse
mode; the others' results carry no gradient, and dual tensors are refused.
Streams, graphs and allocation are as there, too.
"""
import torch

from . import _numel
from ._lib import lib
from .blocks import (_IN_FLAG, _IN_TYPES, _OUT_FLAG, _OUT_TYPES, _PRODUCT_TYPES, Blocks, _call,
                     _code_cols, _Codes, _CodesPlan, _matrix, _no_dual, _out, _same_device, _shard,
                     _unshard, _values, block_mm_dw, block_quant)

FP4_BLOCK = 32         # columns of a block
QUANT_X = 0x200

_MM, _DX, _LINEAR = 0, 1, 2


class Fp4Blocks(_Codes):
    """A matrix [rows, cols] in microscaled 4-bit blocks.

    codes: [rows, cols rounded up to 128, halved], uint8 or float4_e2m1fn_x2, the
    even column of a pair in the low half of its byte.
    scales: [rows, cols rounded up to 128, / 32], uint8 or float8_e8m0fnu, 2 to 252,
    or 255 for a block of NaNs.  Codes past the last column are 0 and scales past the
    last block 127, as fp4_quant, fp4_shard and ag() write them.  The calls do not
    look for other scales or for codes behind the last column, which blocks made
    elsewhere might hold: they would enter the sums.  Either tensor may be replaced,
    or its storage released and restored, as those of Blocks."""

    __slots__ = ()
    _code_types = (torch.uint8, torch.float4_e2m1fn_x2)

    @staticmethod
    def _code_cols(cols):
        return _code_cols(cols) // 2

    @staticmethod
    def _scale_cols(cols):
        return _code_cols(cols) // FP4_BLOCK

    @property
    def _ptrs(self):
        raise TypeError("4-bit blocks where 8-bit ones are expected")

    @property
    def _ptrs4(self):
        return self._codes.data_ptr(), self._scales.data_ptr()


def fp4_quant(x, out=None):
    """x [rows, cols] (bf16, fp16 or fp32) in 4-bit blocks: `out` or new Fp4Blocks.
    They carry no gradient to x."""
    _values(x, "x", _IN_TYPES)
    rows, cols = x.shape
    if out is None:
        out = Fp4Blocks.empty(rows, cols, x.device)
    elif out.shape != (rows, cols):
        raise ValueError(f"out holds {out.shape}, x is {(rows, cols)}")
    _same_device(x.device, out)
    _call(x.device, lib().tide_mx_quant, x.data_ptr(), rows, cols, *out._ptrs4,
          _IN_FLAG[x.dtype])
    return out


def fp4_dequant(q, out=None, dtype=torch.bfloat16):
    """The values of 4-bit blocks: in `out`, or in a new tensor of `dtype`."""
    ptrs = q._ptrs4
    out = _out(out, q.shape, dtype, _OUT_TYPES, q.device, "out")
    _call(q.device, lib().tide_mx_dequant, *ptrs, q.rows, q.cols, out.data_ptr(),
          _OUT_FLAG[out.dtype])
    return out


def _workspace(op, m, n, k, flags, device):
    size = lib().tide_mx_workspace(op, m, n, k, flags)
    if size <= 0:
        return None, None, 0
    buf = torch.empty(size, dtype=torch.uint8, device=device)
    return buf, buf.data_ptr(), size


def fp4_mm(x, w, out=None, dtype=torch.bfloat16):
    """x w^T for x [m, k] and w [n, k] in 4-bit blocks: [m, n] in bf16 or fp32.
    Sums are held in fp32."""
    xp, wp = x._ptrs4, w._ptrs4
    if x.cols != w.cols:
        raise ValueError(f"x has {x.cols} columns, w has {w.cols}")
    _same_device(x.device, w)
    out = _out(out, (x.rows, w.rows), dtype, _PRODUCT_TYPES, x.device, "out")
    flags = _OUT_FLAG[out.dtype]
    keep, ptr, size = _workspace(_MM, x.rows, w.rows, x.cols, flags, x.device)
    _call(x.device, lib().tide_mx_mm, *xp, x.rows, *wp, w.rows, w.cols, out.data_ptr(), flags,
          ptr, size)
    return out


def fp4_mm_dx(dy, w, out=None, dtype=torch.bfloat16):
    """dy w for dy [m, n] in bf16 and w [n, k] in 4-bit blocks: [m, k] in bf16 or fp32."""
    wp = w._ptrs4
    _values(dy, "dy", (torch.bfloat16,))
    if dy.shape[1] != w.rows:
        raise ValueError(f"dy has {dy.shape[1]} columns, w has {w.rows} rows")
    _same_device(dy.device, w)
    m, n = dy.shape
    out = _out(out, (m, w.cols), dtype, _PRODUCT_TYPES, dy.device, "out")
    flags = _OUT_FLAG[out.dtype]
    keep, ptr, size = _workspace(_DX, m, n, w.cols, flags, dy.device)
    _call(dy.device, lib().tide_mx_mm_dx, dy.data_ptr(), m, n, *wp, w.cols, out.data_ptr(),
          flags, ptr, size)
    return out


def _linear(x, w, dtype, quant_x):
    wp = w._ptrs4
    m, k = x.shape
    _same_device(x.device, w)
    out = _out(None, (m, w.rows), dtype, _PRODUCT_TYPES, x.device, "out")
    flags = _OUT_FLAG[dtype] | (_IN_FLAG[x.dtype] | QUANT_X if quant_x else 0)
    keep, ptr, size = _workspace(_LINEAR, m, w.rows, k, flags, x.device)
    _call(x.device, lib().tide_mx_linear, x.data_ptr(), m, k, *wp, w.rows, out.data_ptr(), flags,
          ptr, size)
    return out


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, anchor, w, dtype, quant_x, grad, accumulate):
        ctx.cols, ctx.x_dtype, ctx.grad, ctx.accumulate = w.cols, x.dtype, grad, accumulate
        if grad is None:         # frozen weights: nothing of x is needed again
            ctx.save_for_backward(w.codes, w.scales)
        else:
            q = block_quant(x)   # 8 bits, whatever the product reads of x
            ctx.save_for_backward(w.codes, w.scales, q.codes, q.scales)
        return _linear(x, w, dtype, quant_x)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        wc, ws, *q = ctx.saved_tensors
        # dy enters the bf16 matrix instruction: an fp32 dy is rounded to 8
        # significant bits here, where w holds 2.
        dy = dy.to(torch.bfloat16).contiguous()
        dx = None
        if ctx.needs_input_grad[0]:
            half = ctx.x_dtype == torch.float16
            dx = fp4_mm_dx(dy, Fp4Blocks(wc, ws, ctx.cols),
                           dtype=torch.float32 if half else ctx.x_dtype)
            dx = dx.to(ctx.x_dtype) if half else dx
        if ctx.grad is not None:
            block_mm_dw(dy, Blocks(*q, ctx.cols), out=ctx.grad, accumulate=ctx.accumulate)
        # the anchor's gradient: an empty tensor of this stream
        da = dy.new_empty(0, dtype=torch.float32) if ctx.needs_input_grad[1] else None
        return dx, da, None, None, None, None, None


def fp4_linear(x, w, dtype=None, quant_x=False, grad=None, accumulate=False):
    """A linear layer: x [..., k] times w [n, k] (4-bit blocks) -> [..., n].

    x is contiguous, in bf16; with quant_x in bf16, fp16 or fp32, and rounded to
    4-bit blocks on its way into the product, which then runs on the 4-bit matrix
    instruction (up to 4 times as fast as bf16's for many rows).
    dtype: the output's, bf16 or fp32 (default: fp32 for an fp32 x, else bf16).
    The backward pass takes the output's gradient in bf16 and returns x's gradient in
    x's dtype, treating the rounding of x as the identity.  Without `grad` the
    weights are frozen and nothing of x is kept.  With it (as for block_linear, and
    in the same way) an 8-bit checkpoint of x is, and the gradient of the weights
    that the 4-bit ones were made from is written there, or added with accumulate."""
    if x.shape[-1] != w.cols:
        raise ValueError(f"x has {x.shape[-1]} columns, w has {w.cols}")
    _no_dual(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if dtype is None:
        dtype = torch.float32 if x.dtype == torch.float32 else torch.bfloat16
    if grad is not None:
        _out(grad, w.shape, None, _PRODUCT_TYPES, w.device, "grad")
    elif accumulate:
        raise ValueError("accumulate needs a grad to add to")
    lead = x.shape[:-1]
    if x.dim() != 2:
        x = x.reshape(_numel(lead), w.cols)
    _matrix(x, "x", _IN_TYPES if quant_x else (torch.bfloat16,))
    if torch.is_grad_enabled() and (x.requires_grad or grad is not None):
        # an empty leaf of x's device makes autograd run the backward pass, and join
        # its stream, where x needs no gradient (see block_linear)
        anchor = None if grad is None else \
            torch.empty(0, dtype=torch.float32, device=x.device, requires_grad=True)
        y = _Linear.apply(x, anchor, w, dtype, quant_x, grad, accumulate)
    else:
        y = _linear(x, w, dtype, quant_x)
    return y if len(lead) == 1 else y.view(*lead, w.rows)


class Fp4Plan(_CodesPlan):
    """The plan of a 4-bit gather of `plan`'s matrices (tide_plan_create_mx), to be
    used as a BlockPlan is: ag(plan, gathered, plan.views(blocks)) places them."""

    _create, _kind = "tide_plan_create_mx", Fp4Blocks


def fp4_shard(plan, rank, master, block):
    """Rank `rank`'s fp32 master shard (source_S elements) -> its 4-bit rank
    block (plan.S int32 words, e.g. a row of plan.empty())."""
    _shard(lib().tide_mx_shard, plan, rank, master, block)


def fp4_unshard(plan, gathered, params):
    """Gathered 4-bit rank blocks (plan.empty()) -> full tensors, as block_unshard."""
    _unshard(lib().tide_mx_unshard, "fp4_unshard", plan, gathered, params)


__all__ = ["Fp4Blocks", "Fp4Plan", "fp4_quant", "fp4_dequant", "fp4_mm", "fp4_mm_dx", "fp4_linear",
           "fp4_shard", "fp4_unshard"]
