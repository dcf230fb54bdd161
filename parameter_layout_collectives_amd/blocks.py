"""Matrices in 8-bit blocks: the 8-bit gather of an FSDP unit's weights, 8-bit
activation checkpoints, and the products of a linear layer over both.

    q = block_quant(x)                       # x [m, k] -> Blocks (the checkpoint)
    x = block_dequant(q)                     # ... and back
    y = block_mm(q, w)                       # y [m, n] = x w^T, both in blocks
    dx = block_mm_dx(dy, w)                  # dx [m, k] = dy w
    dw = block_mm_dw(dy, q)                  # dw [n, k] = dy^T x
    y = block_linear(x, w, grad=dw)          # all of it through autograd

    plan = BlockPlan(Plan(shapes, world))    # gather matrices in 8 bits
    block_shard(plan, rank, master, gathered[rank])
    ag(plan, gathered, plan.views(weights))  # -> Blocks for the products, or
    block_unshard(plan, gathered, params)    # -> full tensors

The format (e4m3 codes, one power of two per 128 columns of a row), the
arguments and the errors are documented in include/tide.h.  An FSDP unit that
gathers its weights this way moves half the bytes of a bf16 all-gather
("FSDP通信终局：TIDE零拷贝集合通信优化", §"FSDP2通信开销的根源": the all-gather's
bytes are part of every step).

block_linear is the differentiable call, in reverse mode.  The others are what it
is made of: their results carry no gradient, whatever their inputs require.  A
forward-mode dual tensor is refused by all of them.

The calls run on PyTorch's current stream of the tensors' device; outputs and
workspaces that they make come from PyTorch's allocator, so they may be
captured into a graph.
"""
import ctypes

import torch
from torch.autograd.forward_ad import unpack_dual

from . import GRAD_F16, GRAD_F32, OUT_BF16, Plan, PointerTable, _check, _numel
from ._lib import lib

BLOCK = 128            # columns of a block
ACCUMULATE = 0x40
OUT_F16 = 0x80
SHORT_SUMS = 0x100

_IN_FLAG = {torch.bfloat16: 0, torch.float16: GRAD_F16, torch.float32: GRAD_F32}
_OUT_FLAG = {torch.float32: 0, torch.bfloat16: OUT_BF16, torch.float16: OUT_F16}
_IN_TYPES, _OUT_TYPES = tuple(_IN_FLAG), tuple(_OUT_FLAG)
_MM, _DX, _DW, _LINEAR = 0, 1, 2, 3


def _code_cols(cols):
    return -(-cols // BLOCK) * BLOCK


def _scale_cols(cols):
    return -(-cols // (4 * BLOCK)) * 4


# The handle of a device's current stream (a public call makes a Stream object
# for it, which costs as much as the rest of a small call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, fn, *args):
    """fn(*args, stream) with `device` current, on its current stream."""
    index = device.index
    if index == torch.cuda.current_device():
        _check(fn(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, _raw_stream(index)))


def _no_dual(t, what):
    if unpack_dual(t).tangent is not None:
        raise NotImplementedError(f"{what} is a dual tensor: no forward-mode derivative")


def _matrix(t, what, dtypes):
    if t.dtype not in dtypes:
        raise TypeError(f"{what} is {t.dtype}, expected one of "
                        f"{', '.join(str(d).replace('torch.', '') for d in dtypes)}")
    if not t.is_cuda or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 2-D device tensor")


def _same_device(device, *tensors):
    for t in tensors:
        if t.device != device:
            raise ValueError(f"tensors on {device} and {t.device}")


def _values(t, what, dtypes):
    """_matrix for numbers that a derivative could go through."""
    _no_dual(t, what)
    _matrix(t, what, dtypes)


class _Codes:
    """What matrices in 8-bit and 4-bit blocks have in common: two tensors and a
    number of columns."""

    __slots__ = ("_codes", "_scales", "_rows", "_cols", "_device", "_word_views")

    def __init__(self, codes, scales, cols):
        self._set(codes, scales, int(cols))

    def _set(self, codes, scales, cols):
        _matrix(codes, "codes", self._code_types)
        _matrix(scales, "scales", (torch.uint8, torch.float8_e8m0fnu))
        _same_device(codes.device, scales)
        rows = codes.shape[0]
        if cols < 0 or codes.shape[1] != self._code_cols(cols) \
                or tuple(scales.shape) != (rows, self._scale_cols(cols)):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not "
                             f"hold {rows} rows of {cols} columns")
        self._codes, self._scales, self._word_views = codes, scales, None
        self._rows, self._cols, self._device = rows, cols, codes.device

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        self = object.__new__(cls)          # right by construction: no checks
        self._codes = torch.empty((rows, cls._code_cols(cols)), dtype=cls._code_types[0],
                                  device=device)
        self._scales = torch.empty((rows, cls._scale_cols(cols)), dtype=torch.uint8,
                                   device=device)
        self._rows, self._cols, self._device = rows, cols, self._codes.device
        self._word_views = None
        return self

    @property
    def codes(self):
        return self._codes

    @codes.setter
    def codes(self, t):
        self._replace(t, self._scales)

    @property
    def scales(self):
        return self._scales

    @scales.setter
    def scales(self, t):
        self._replace(self._codes, t)

    def _replace(self, codes, scales):
        _matrix(codes, "codes", self._code_types)
        if codes.shape[0] != self._rows:
            raise ValueError(f"codes of {codes.shape[0]} rows in place of {self._rows}")
        self._set(codes, scales, self._cols)

    @property
    def rows(self):
        return self._rows

    @property
    def cols(self):
        return self._cols

    @property
    def device(self):
        return self._device

    @property
    def shape(self):
        return self._rows, self._cols

    def words(self):
        """(codes, scales) as int32 views."""
        if self._word_views is None:
            self._word_views = _words(self._codes), _words(self._scales)
        return self._word_views


class Blocks(_Codes):
    """A matrix [rows, cols] in 8-bit blocks.

    codes: [rows, cols rounded up to 128], float8_e4m3fn or uint8.
    scales: [rows, blocks of a row rounded up to 4], uint8 or float8_e8m0fnu,
    10 to 246.  Codes past the last column are 0 and scales past the last block 127,
    as block_quant, block_shard and ag() write them: the products count on it.
    Either may be replaced by another tensor of its shape, and its storage may be
    released and restored in between, as an FSDP unit does with gathered weights:
    every call asks the tensors where they are, and refuses one without memory."""

    __slots__ = ()
    _code_types = (torch.float8_e4m3fn, torch.uint8)
    _code_cols, _scale_cols = staticmethod(_code_cols), staticmethod(_scale_cols)

    @property
    def _ptrs(self):
        return self._codes.data_ptr(), self._scales.data_ptr()

    @property
    def _ptrs4(self):
        raise TypeError("8-bit blocks where 4-bit ones are expected")


def _out(out, shape, dtype, dtypes, device, what):
    """`out` checked, or a new tensor."""
    if out is None:
        if dtype not in dtypes:
            raise TypeError(f"{what} cannot be {dtype}")
        return torch.empty(shape, dtype=dtype, device=device)
    _values(out, what, dtypes)
    _same_device(device, out)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(out.shape)}, expected {tuple(shape)}")
    return out


def block_quant(x, out=None):
    """x [rows, cols] (bf16, fp16 or fp32) in 8-bit blocks: `out` or new Blocks.
    They carry no gradient to x."""
    _values(x, "x", _IN_TYPES)
    rows, cols = x.shape
    if out is None:
        out = Blocks.empty(rows, cols, x.device)
    elif out.shape != (rows, cols):
        raise ValueError(f"out holds {out.shape}, x is {(rows, cols)}")
    _same_device(x.device, out)
    _call(x.device, lib().tide_block_quant, x.data_ptr(), rows, cols, *out._ptrs,
          _IN_FLAG[x.dtype])
    return out


def block_dequant(q, out=None, dtype=torch.bfloat16):
    """The values of 8-bit blocks: in `out`, or in a new tensor of `dtype`."""
    out = _out(out, q.shape, dtype, _OUT_TYPES, q.device, "out")
    _call(q.device, lib().tide_block_dequant, *q._ptrs, q.rows, q.cols, out.data_ptr(),
          _OUT_FLAG[out.dtype])
    return out


def _workspace(op, m, n, k, flags, device):
    size = lib().tide_block_workspace(op, m, n, k, flags)
    if size <= 0:
        return None, None, 0
    buf = torch.empty(size, dtype=torch.uint8, device=device)
    return buf, buf.data_ptr(), size


_PRODUCT_TYPES = (torch.bfloat16, torch.float32)


def _mm_flags(dtype, short_sums):
    if short_sums and dtype != torch.bfloat16:
        raise ValueError("short_sums needs a bfloat16 output")
    return _OUT_FLAG[dtype] | (SHORT_SUMS if short_sums else 0)


def block_mm(x, w, out=None, dtype=torch.bfloat16, short_sums=False):
    """x w^T for x [m, k] and w [n, k] in 8-bit blocks: [m, n] in bf16 or fp32.

    Sums are held in fp32.  With short_sums (bf16 only) the 8-bit matrix
    instruction adds the products of more than 16 rows: up to twice as fast, off by
    up to about 2^-10 of the sum of the products' magnitudes, which matters where
    large products cancel (TIDE_F_SHORT_SUMS in include/tide.h)."""
    if x.cols != w.cols:
        raise ValueError(f"x has {x.cols} columns, w has {w.cols}")
    _same_device(x.device, w)
    out = _out(out, (x.rows, w.rows), dtype, _PRODUCT_TYPES, x.device, "out")
    flags = _mm_flags(out.dtype, short_sums)
    keep, ptr, size = _workspace(_MM, x.rows, w.rows, x.cols, flags, x.device)
    _call(x.device, lib().tide_block_mm, *x._ptrs, x.rows, *w._ptrs, w.rows, w.cols,
          out.data_ptr(), flags, ptr, size)
    return out


def block_mm_dx(dy, w, out=None, dtype=torch.bfloat16):
    """dy w for dy [m, n] in bf16 and w [n, k] in 8-bit blocks: [m, k] in bf16 or fp32."""
    _values(dy, "dy", (torch.bfloat16,))
    if dy.shape[1] != w.rows:
        raise ValueError(f"dy has {dy.shape[1]} columns, w has {w.rows} rows")
    _same_device(dy.device, w)
    m, n = dy.shape
    out = _out(out, (m, w.cols), dtype, _PRODUCT_TYPES, dy.device, "out")
    flags = _OUT_FLAG[out.dtype]
    keep, ptr, size = _workspace(_DX, m, n, w.cols, flags, dy.device)
    _call(dy.device, lib().tide_block_mm_dx, dy.data_ptr(), m, n, *w._ptrs, w.cols,
          out.data_ptr(), flags, ptr, size)
    return out


def block_mm_dw(dy, x, out=None, dtype=torch.bfloat16, accumulate=False):
    """dy^T x for dy [m, n] in bf16 and the checkpoint x [m, k] in 8-bit blocks:
    [n, k] in bf16 or fp32; with accumulate, added to what `out` holds."""
    _values(dy, "dy", (torch.bfloat16,))
    if dy.shape[0] != x.rows:
        raise ValueError(f"dy has {dy.shape[0]} rows, x has {x.rows}")
    if accumulate and out is None:
        raise ValueError("accumulate needs an out to add to")
    _same_device(dy.device, x)
    m, n = dy.shape
    out = _out(out, (n, x.cols), dtype, _PRODUCT_TYPES, dy.device, "out")
    flags = _OUT_FLAG[out.dtype] | (ACCUMULATE if accumulate else 0)
    keep, ptr, size = _workspace(_DW, m, n, x.cols, flags, dy.device)
    _call(dy.device, lib().tide_block_mm_dw, dy.data_ptr(), m, n, *x._ptrs, x.cols,
          out.data_ptr(), flags, ptr, size)
    return out


def _linear(x, w, dtype, short_sums):
    """block_mm(block_quant(x), w) that keeps no blocks of x (tide_block_linear)."""
    _matrix(x, "x", _IN_TYPES)
    m, k = x.shape
    _same_device(x.device, w)
    out = _out(None, (m, w.rows), dtype, _PRODUCT_TYPES, x.device, "out")
    flags = _IN_FLAG[x.dtype] | _mm_flags(dtype, short_sums)
    keep, ptr, size = _workspace(_LINEAR, m, w.rows, k, flags, x.device)
    _call(x.device, lib().tide_block_linear, x.data_ptr(), m, k, *w._ptrs, w.rows,
          out.data_ptr(), flags, ptr, size)
    return out


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, anchor, w, dtype, grad, accumulate, short_sums):
        ctx.cols, ctx.x_dtype, ctx.grad, ctx.accumulate = w.cols, x.dtype, grad, accumulate
        if grad is None:         # frozen weights: nothing of x is needed again
            ctx.save_for_backward(w.codes, w.scales)
            return _linear(x, w, dtype, short_sums)
        q = block_quant(x)
        ctx.save_for_backward(w.codes, w.scales, q.codes, q.scales)
        return block_mm(q, w, dtype=dtype, short_sums=short_sums)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        wc, ws, *q = ctx.saved_tensors
        # dy enters the bf16 matrix instruction, as w and q do exactly: an fp32 dy is
        # rounded to 8 significant bits here, where w and q hold 4.
        dy = dy.to(torch.bfloat16).contiguous()
        dx = None
        if ctx.needs_input_grad[0]:
            half = ctx.x_dtype == torch.float16
            dx = block_mm_dx(dy, Blocks(wc, ws, ctx.cols),
                             dtype=torch.float32 if half else ctx.x_dtype)
            dx = dx.to(ctx.x_dtype) if half else dx
        if ctx.grad is not None:
            block_mm_dw(dy, Blocks(*q, ctx.cols), out=ctx.grad, accumulate=ctx.accumulate)
        # the anchor's gradient: an empty tensor of this stream
        da = dy.new_empty(0, dtype=torch.float32) if ctx.needs_input_grad[1] else None
        return dx, da, None, None, None, None, None


def block_linear(x, w, dtype=None, grad=None, accumulate=False, short_sums=False):
    """A linear layer: x [..., k] times w [n, k] (8-bit blocks) -> [..., n].

    x (bf16, fp16 or fp32, contiguous) becomes 8-bit blocks, which are all that
    is kept of it for the backward pass, and only for the weights' gradient.
    dtype: the output's, bf16 or fp32 (default: fp32 for an fp32 x, else bf16).
    short_sums: see block_mm.
    The backward pass takes the output's gradient in bf16, returns x's gradient
    in x's dtype, treating the rounding of x to 8 bits as the identity, and
    writes the weights' gradient to `grad` ([n, k], bf16 or fp32; as the
    reduce-scatter takes it), or adds it there with accumulate.  Without `grad`
    the weights are frozen.  Like other gradients, `grad` is written on the forward
    pass's stream, and the stream that calls backward() waits for it.  w's blocks
    must hold the same values in the backward pass as in the forward pass."""
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
    if torch.is_grad_enabled() and (x.requires_grad or grad is not None):
        # With an x that needs no gradient, this empty leaf is what makes
        # autograd run the backward pass, and with it the weights' gradient.  It
        # lies on x's device, made under the forward pass's stream: autograd joins
        # the stream that calls backward() with those of device leaves, so that
        # `grad` may be read there.
        anchor = None if grad is None else \
            torch.empty(0, dtype=torch.float32, device=x.device, requires_grad=True)
        y = _Linear.apply(x, anchor, w, dtype, grad, accumulate, short_sums)
    else:
        y = _linear(x, w, dtype, short_sums)
    return y if len(lead) == 1 else y.view(*lead, w.rows)


def _words(t):
    """The int32 view of a contiguous byte matrix (its row length divides by 4)."""
    if t.numel() == 0:
        return torch.empty(t.shape[0], t.shape[1] // 4, dtype=torch.int32, device=t.device)
    return t.view(torch.int32)


class _CodesPlan(Plan):
    def __init__(self, plan, select=None):
        self._h = None
        if select is None:
            select = [i for i, s in enumerate(plan.shapes) if len(s) == 2]
        self.select = [int(i) for i in select]
        n = len(self.select)
        arr = (ctypes.c_int32 * max(n, 1))(*self.select)
        h = ctypes.c_void_p()
        self._destroy = lib().tide_plan_destroy
        _check(getattr(lib(), self._create)(plan.handle, n, arr, ctypes.byref(h)))
        self._h = h
        self.world = plan.world
        self.matrices = []
        for i in self.select:
            s = plan.shapes[i]
            self.matrices.append((s[0] if s else 1, _numel(s[1:])))
        kind = self._kind
        self.shapes = [(d, kind._code_cols(c) // 4) for d, c in self.matrices] + \
                      [(d, kind._scale_cols(c) // 4) for d, c in self.matrices]
        self.P = 2 * n
        self.S = int(lib().tide_plan_shard_numel(h))
        self.source_S = plan.S
        self._sig = (self.world, tuple(self.shapes), self.S)

    def empty(self, device="cuda"):
        """A gathered buffer [world, S] of int32 words."""
        return torch.empty(self.world, self.S, dtype=torch.int32, device=device)

    def blocks(self, device="cuda"):
        """One (uninitialised) matrix in blocks per matrix, for ag() to place into."""
        return [self._kind.empty(d, c, device) for d, c in self.matrices]

    def views(self, blocks):
        """The int32 views of a list of such matrices that ag() takes as parameters."""
        if [b.shape for b in blocks] != self.matrices or \
                not all(isinstance(b, self._kind) for b in blocks):
            raise ValueError(f"need one {self._kind.__name__} per matrix, of its shape")
        words = [b.words() for b in blocks]
        return [c for c, _ in words] + [s for _, s in words]


class BlockPlan(_CodesPlan):
    """The plan of an 8-bit gather of `plan`'s matrices (tide_plan_create_blocks).

    select: indices of plan's parameters, by default all 2-D ones.  Its own
    parameters are the codes and then the scales of the selected matrices in
    int32 words, so ag(plan, gathered, plan.views(blocks)) places them."""

    _create, _kind = "tide_plan_create_blocks", Blocks


def block_shard(plan, rank, master, block):
    """Rank `rank`'s fp32 master shard (source_S elements) -> its 8-bit rank
    block (plan.S int32 words, e.g. a row of plan.empty())."""
    _shard(lib().tide_block_shard, plan, rank, master, block)


def _shard(fn, plan, rank, master, block):
    _no_dual(master, "master")
    if master.dtype != torch.float32 or not master.is_cuda or not master.is_contiguous() \
            or master.numel() != plan.source_S:
        raise ValueError(f"master must be a contiguous float32 device tensor of "
                         f"{plan.source_S} elements")
    if block.dtype != torch.int32 or not block.is_cuda or not block.is_contiguous() \
            or block.numel() != plan.S:
        raise ValueError(f"block must be a contiguous int32 device tensor of {plan.S} elements")
    _same_device(master.device, block)
    _call(master.device, fn, plan.handle, int(rank), master.data_ptr(),
          block.data_ptr(), 0)


def _check_unshard(plan, params, device):
    dtype = params[0].dtype
    if dtype not in _OUT_FLAG:
        raise TypeError(f"params must be bfloat16, float16 or float32, got {dtype}")
    for j, (t, s) in enumerate(zip(params, plan.matrices)):
        _no_dual(t, f"params[{j}]")
        if t.dtype != dtype or t.device != device or not t.is_contiguous() \
                or t.numel() != s[0] * s[1]:
            raise ValueError(f"params[{j}] must be a contiguous {dtype} tensor on {device} with "
                             f"{s[0] * s[1]} elements")


def block_unshard(plan, gathered, params):
    """Gathered 8-bit rank blocks (plan.empty()) -> full tensors.

    params: one tensor per matrix of the plan, all bf16, all fp16 or all fp32,
    or a PointerTable of them."""
    _unshard(lib().tide_block_unshard, "block_unshard", plan, gathered, params)


def _unshard(fn, name, plan, gathered, params):
    if gathered.dtype != torch.int32 or not gathered.is_cuda or not gathered.is_contiguous() \
            or gathered.numel() != plan.world * plan.S:
        raise ValueError(f"gathered must be a contiguous int32 device tensor of "
                         f"{plan.world * plan.S} elements")
    if not isinstance(params, PointerTable):
        params = PointerTable(params)
    params.check_len(len(plan.matrices), name)
    device = gathered.device
    params._ensure(plan, name, lambda: _check_unshard(plan, params.tensors, device))
    _same_device(device, params.tensors[0])
    _call(device, fn, plan.handle, gathered.data_ptr(), params.array,
          _OUT_FLAG[params.tensors[0].dtype])


__all__ = ["Blocks", "BlockPlan", "block_quant", "block_dequant", "block_mm", "block_mm_dx",
           "block_mm_dw", "block_linear", "block_shard", "block_unshard"]
