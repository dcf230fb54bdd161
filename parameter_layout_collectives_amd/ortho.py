"""Orthogonalised updates: what a Muon optimizer makes of a gradient matrix between
the reduce-scatter that sums it and the all-gather of the new weights.

    u = ortho(g)                             # a matrix, or a stack [b, rows, cols]
    us = ortho([g0, g1, ...])                # a unit's matrices in one call

Newton-Schulz products bring all singular values of g near 1 and leave its
singular vectors; the arithmetic, its exactness and the limits are documented in
include/tide.h (tide_ortho).  TideUnit.muon_step (fsdp.py) is the whole update of
an FSDP unit.  The result carries no gradient; streams, graphs and allocation as
for the blocked products.
"""
import ctypes

import torch

from . import _check
from ._lib import lib
from .blocks import _IN_FLAG, _IN_TYPES, _call, _no_dual, _same_device

# Quintic steps that raise small singular values fast; 5 of them bring those above
# 2e-3 of the norm to between 0.68 and 1.21.
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _check_stack(t, what, dtypes):
    if t.dtype not in dtypes:
        raise TypeError(f"{what} is {t.dtype}, expected one of "
                        f"{', '.join(str(d).replace('torch.', '') for d in dtypes)}")
    if not t.is_cuda or t.dim() not in (2, 3) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 2-D or 3-D device tensor")


def _steps(steps, coefficients):
    """The steps' number and coefficients as the library takes them."""
    flat = [float(v) for step in coefficients for v in step] \
        if len(coefficients) and isinstance(coefficients[0], (tuple, list)) \
        else [float(v) for v in coefficients] * int(steps)
    steps = int(steps)
    if len(flat) != 3 * steps:
        raise ValueError(f"coefficients: need (a, b, c), or {steps} triples of them")
    return steps, (ctypes.c_float * max(1, len(flat)))(*flat)


def check_steps(steps, coefficients):
    """Refuses the steps that ortho() would refuse for any matrices."""
    steps, flat = _steps(steps, coefficients)
    _check(lib().tide_ortho(0, None, None, None, None, steps, flat, 0, None, 0, None))


def ortho(g, out=None, steps=5, coefficients=COEFFICIENTS):
    """g orthogonalised, in bf16.

    g: a tensor [rows, cols] or [b, rows, cols], bf16, fp16 or fp32, or a list of
    such tensors of one dtype and device.  out: bf16 tensors of their shapes (a
    bf16 g itself may be one), by default new ones.  coefficients: (a, b, c) of
    every step, or one such triple per step.  Returns `out`, a list for a list."""
    one = isinstance(g, torch.Tensor)
    gs = [g] if one else list(g)
    steps, flat = _steps(steps, coefficients)
    if not gs:
        return []
    dtype, device = gs[0].dtype, gs[0].device
    for i, t in enumerate(gs):
        _no_dual(t, f"g[{i}]")
        _check_stack(t, f"g[{i}]", _IN_TYPES)
        if t.dtype != dtype:
            raise TypeError(f"g[{i}] is {t.dtype}, the others are {dtype}")
    _same_device(device, *gs)
    if out is None:
        outs = [torch.empty(t.shape, dtype=torch.bfloat16, device=device) for t in gs]
    else:
        outs = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(outs) != len(gs):
            raise ValueError(f"{len(outs)} outs for {len(gs)} matrices")
        for i, (o, t) in enumerate(zip(outs, gs)):
            _no_dual(o, f"out[{i}]")
            _check_stack(o, f"out[{i}]", (torch.bfloat16,))
            if o.shape != t.shape:
                raise ValueError(f"out[{i}] has shape {tuple(o.shape)}, expected {tuple(t.shape)}")
        _same_device(device, *outs)
    src, dst, rows, cols = [], [], [], []
    for t, o in zip(gs, outs):
        r, c = t.shape[-2:]
        s, d = t.data_ptr(), o.data_ptr()
        if t.dim() == 2:
            src.append(s), dst.append(d), rows.append(r), cols.append(c)
            continue
        b, es = t.shape[0], t.element_size()
        src += [s + i * r * c * es for i in range(b)]
        dst += [d + i * r * c * 2 for i in range(b)]
        rows += [r] * b
        cols += [c] * b
    n = len(src)
    if n:
        sizes = ctypes.c_int64 * n
        rows, cols = sizes(*rows), sizes(*cols)
        size = lib().tide_ortho_workspace(n, rows, cols)
        # the allocator's blocks start at multiples of 512 bytes
        keep = torch.empty(size, dtype=torch.uint8, device=device) if size > 0 else None
        _call(device, lib().tide_ortho, n, (ctypes.c_void_p * n)(*src), (ctypes.c_void_p * n)(*dst),
              rows, cols, steps, flat, _IN_FLAG[dtype],
              keep.data_ptr() if keep is not None else None, max(size, 0))
    return outs[0] if one else outs


__all__ = ["ortho"]
