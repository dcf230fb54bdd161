"""Host-side checks of the 8-bit block calls that need no GPU: sizes of the
format, block plans, and every refusal before anything is enqueued."""
import ctypes

import pytest
import torch

import parameter_layout_collectives_amd as tide
from parameter_layout_collectives_amd._lib import lib

E_INVALID, E_UNSUPPORTED = 1, 2
# Never-dereferenced device addresses, 16-byte aligned and far apart.
A, B, C, D, E, W = (0x7F0000000000 + i * (1 << 32) for i in range(6))
P = ctypes.c_void_p


def err():
    return lib().tide_last_error().decode()


def test_sizes():
    L = lib()
    for c in range(0, 2000):
        assert L.tide_block_cols(c) == -(-c // 128) * 128
        assert L.tide_block_scale_cols(c) == -(-c // 512) * 4
    assert L.tide_block_cols(-1) == -1 and L.tide_block_scale_cols(-1) == -1


def quant(x=A, rows=4, cols=200, codes=B, scales=C, flags=0):
    return lib().tide_block_quant(P(x), rows, cols, P(codes), P(scales), flags, None)


def dequant(codes=B, scales=C, rows=4, cols=200, out=A, flags=0):
    return lib().tide_block_dequant(P(codes), P(scales), rows, cols, P(out), flags, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), E_INVALID, "negative"),
    (dict(cols=-1), E_INVALID, "negative"),
    (dict(rows=1 << 31), E_INVALID, "2^31"),
    (dict(cols=1 << 31), E_INVALID, "2^31"),
    (dict(rows=(1 << 31) - 1, cols=(1 << 31) - 1), E_INVALID, "overflow"),
    (dict(flags=0x18), E_INVALID, "both"),
    (dict(flags=0x20), E_UNSUPPORTED, "flag"),
    (dict(flags=0x1), E_UNSUPPORTED, "flag"),
    (dict(x=0), E_INVALID, "x is NULL"),
    (dict(x=A + 1), E_INVALID, "aligned"),
    (dict(x=A + 2, flags=0x10), E_INVALID, "aligned"),
    (dict(codes=0), E_INVALID, "codes are NULL"),
    (dict(scales=0), E_INVALID, "scales are NULL"),
    (dict(codes=B + 8), E_INVALID, "16-byte"),
    (dict(scales=C + 2), E_INVALID, "4-byte"),
    (dict(codes=A + 1584), E_INVALID, "overlaps"),        # x holds 1600 bytes
    (dict(scales=A + 1596), E_INVALID, "overlaps"),
    (dict(scales=B + 1020), E_INVALID, "overlaps"),       # codes hold 1024 bytes
])
def test_quant_refusals(kw, status, needle):
    assert quant(**kw) == status
    assert needle in err()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), E_INVALID, "negative"),
    (dict(flags=0xa0), E_INVALID, "both"),
    (dict(flags=0x8), E_UNSUPPORTED, "flag"),
    (dict(out=0), E_INVALID, "out is NULL"),
    (dict(out=A + 2), E_INVALID, "aligned"),
    (dict(out=A + 1, flags=0x20), E_INVALID, "aligned"),
    (dict(codes=0), E_INVALID, "codes are NULL"),
    (dict(codes=B + 4), E_INVALID, "16-byte"),
    (dict(out=B + 1020), E_INVALID, "overlaps"),
    (dict(out=C + 12), E_INVALID, "overlaps"),            # scales hold 16 bytes
])
def test_dequant_refusals(kw, status, needle):
    assert dequant(**kw) == status
    assert needle in err()


def test_nothing_to_do_is_ok():
    assert quant(x=0, rows=0, codes=0, scales=0) == 0
    assert quant(x=0, cols=0, codes=0, scales=0) == 0
    assert dequant(codes=0, scales=0, rows=0, out=0) == 0
    assert mm(x=0, xs=0, m=0, out=0) == 0
    assert dx(k=0, w=0, ws=0, out=0) == 0
    assert dw(n=0, dy=0, out=0) == 0


def mm(x=A, xs=B, m=4, w=C, ws=D, n=8, k=200, out=E, flags=0, wsp=0, size=0):
    return lib().tide_block_mm(P(x), P(xs), m, P(w), P(ws), n, k, P(out), flags, P(wsp), size, None)


def dx(dy=A, m=4, n=8, w=C, ws=D, k=200, out=E, flags=0, wsp=0, size=0):
    return lib().tide_block_mm_dx(P(dy), m, n, P(w), P(ws), k, P(out), flags, P(wsp), size, None)


def dw(dy=A, m=4, n=8, x=C, xs=D, k=200, out=E, flags=0, wsp=0, size=0):
    return lib().tide_block_mm_dw(P(dy), m, n, P(x), P(xs), k, P(out), flags, P(wsp), size, None)


COMMON = [
    (dict(m=-1), E_INVALID, "negative"),
    (dict(n=-1), E_INVALID, "negative"),
    (dict(k=-1), E_INVALID, "negative"),
    (dict(m=1 << 31), E_INVALID, "2^31"),
    (dict(k=1 << 31), E_INVALID, "2^31"),
    (dict(n=(1 << 22) + 1), E_UNSUPPORTED, "2^22"),
    (dict(k=(1 << 22) + 1), E_UNSUPPORTED, "2^22"),
    (dict(flags=0x80), E_UNSUPPORTED, "flag"),
    (dict(flags=0x1), E_UNSUPPORTED, "flag"),
    (dict(out=0), E_INVALID, "out is NULL"),
    (dict(out=E + 2), E_INVALID, "aligned"),
    (dict(out=E + 1, flags=0x20), E_INVALID, "aligned"),
    (dict(size=-1), E_INVALID, "workspace"),
    (dict(size=64), E_INVALID, "workspace is NULL"),
    (dict(wsp=W + 8, size=64), E_INVALID, "16-byte"),
    (dict(wsp=E, size=64), E_INVALID, "overlaps"),
    (dict(wsp=A, size=64), E_INVALID, "overlaps"),
    (dict(wsp=C, size=64), E_INVALID, "overlaps"),
    (dict(wsp=D, size=64), E_INVALID, "overlaps"),
    (dict(out=A), E_INVALID, "overlaps"),
    (dict(out=C), E_INVALID, "overlaps"),
    (dict(out=D), E_INVALID, "overlaps"),
]


@pytest.mark.parametrize("call", [mm, dx, dw])
@pytest.mark.parametrize("kw,status,needle", COMMON)
def test_product_refusals(call, kw, status, needle):
    assert call(**kw) == status
    assert needle in err()


@pytest.mark.parametrize("call,kw,status,needle", [
    (mm, dict(x=0), E_INVALID, "x's codes are NULL"),
    (mm, dict(xs=0), E_INVALID, "x's scales are NULL"),
    (mm, dict(w=0), E_INVALID, "w's codes are NULL"),
    (mm, dict(ws=D + 1), E_INVALID, "w's scales are not 4-byte"),
    (mm, dict(x=A + 8), E_INVALID, "x's codes are not 16-byte"),
    (mm, dict(flags=0x40), E_UNSUPPORTED, "flag"),          # accumulate: dw only
    (mm, dict(out=B + 12), E_INVALID, "overlaps"),          # x's scales hold 16 bytes
    (dx, dict(dy=0), E_INVALID, "dy is NULL"),
    (dx, dict(dy=A + 1), E_INVALID, "dy is not aligned"),
    (dx, dict(w=0), E_INVALID, "w's codes are NULL"),
    (dx, dict(flags=0x40), E_UNSUPPORTED, "flag"),
    (dw, dict(dy=0), E_INVALID, "dy is NULL"),
    (dw, dict(x=0), E_INVALID, "x's codes are NULL"),
    (dw, dict(x=C + 4), E_INVALID, "x's codes are not 16-byte"),
])
def test_product_operand_refusals(call, kw, status, needle):
    assert call(**kw) == status
    assert needle in err()


def linear(x=A, m=4, k=200, w=C, ws=D, n=8, out=E, flags=0, wsp=0, size=0):
    return lib().tide_block_linear(P(x), m, k, P(w), P(ws), n, P(out), flags, P(wsp), size, None)


@pytest.mark.parametrize("kw,status,needle", [
    c for c in COMMON if c[0] not in (dict(out=A), dict(flags=0x80))] + [
    (dict(flags=0x40), E_UNSUPPORTED, "flag"),
    (dict(flags=0x18), E_INVALID, "both"),
    (dict(x=0), E_INVALID, "x is NULL"),
    (dict(x=A + 1), E_INVALID, "x is not aligned"),
    (dict(x=A + 2, flags=0x10), E_INVALID, "x is not aligned"),
    (dict(w=0), E_INVALID, "w's codes are NULL"),
    (dict(w=C + 8), E_INVALID, "16-byte"),
    (dict(ws=D + 2), E_INVALID, "4-byte"),
    (dict(out=A + 1584), E_INVALID, "overlaps"),
    (dict(m=100), E_INVALID, "x's blocks need"),           # no room for x's blocks
    (dict(m=100, wsp=W, size=256), E_INVALID, "x's blocks need")])
def test_linear_refusals(kw, status, needle):
    assert linear(**kw) == status
    assert needle in err()


def test_linear_of_nothing():
    assert linear(m=0, x=0, out=0) == 0
    assert linear(n=0, w=0, ws=0, out=0) == 0


def test_linear_workspace():
    L = lib()
    assert L.tide_block_workspace(3, 1, 4096, 4096, 0x20) == 0         # in one launch
    assert L.tide_block_workspace(3, 100, 4096, 0, 0x20) == 0
    m, n, k = 100, 4096, 1000
    blocks = (100 * 1024 + 255) // 256 * 256 + (100 * 8 + 255) // 256 * 256
    assert L.tide_block_workspace(3, m, n, k, 0x20) == \
        blocks + L.tide_block_workspace(0, m, n, k, 0x20)


def test_workspace():
    L = lib()
    for op in range(3):
        assert L.tide_block_workspace(op, 8192, 8192, 8192, 0) == 0    # enough tiles
        assert L.tide_block_workspace(op, 0, 0, 0, 0) == 0
    assert L.tide_block_workspace(0, 1, 4096, 4096, 0x20) == 0         # few rows: one kernel
    # a long sum for few tiles, and tiles left over after whole sets
    for op, m, n, k in ((2, 8192, 256, 256), (2, 8192, 14336, 4096)):
        size = L.tide_block_workspace(op, m, n, k, 0)
        assert size > 0 and size % (64 * 64 * 4) == 0
    assert L.tide_block_workspace(4, 1, 1, 1, 0) == -1
    assert L.tide_block_workspace(0, -1, 1, 1, 0) == -1


SHAPES = [(5, 200), (16,), (33, 4), (64, 640)]


def word_shapes(select):
    mats = [(SHAPES[i][0], SHAPES[i][1] if len(SHAPES[i]) > 1 else 1) for i in select]
    return [(d, -(-c // 128) * 32) for d, c in mats] + [(d, -(-c // 512)) for d, c in mats]


@pytest.mark.parametrize("world", [1, 2, 3, 8, 64])
def test_block_plan_is_a_plan_of_words(orc, world):
    plan = tide.Plan(SHAPES, world)
    bp = tide.BlockPlan(plan)
    assert bp.select == [0, 2, 3]
    assert bp.matrices == [(5, 200), (33, 4), (64, 640)]
    g = orc.geometry(word_shapes(bp.select), world, 4)
    assert bp.S == g.S and bp.P == 6 and bp.source_S == plan.S
    for i in range(6):
        assert bp.param(i) == (g.off[i], g.c[i], g.seg[i])
        for r in range(world):
            assert bp.real(r, i) == g.run(r, i)
    assert tide.BlockPlan(plan, [1, 3]).matrices == [(16, 1), (64, 640)]
    assert tide.BlockPlan(tide.Plan([()], 2), [0]).matrices == [(1, 1)]


def create(plan, select, n=None, out=True):
    arr = (ctypes.c_int32 * max(len(select), 1))(*select)
    h = P(1234)
    st = lib().tide_plan_create_blocks(plan.handle if plan else None,
                                       len(select) if n is None else n, arr,
                                       ctypes.byref(h) if out else None)
    return st, h


@pytest.mark.parametrize("select,needle", [
    ([], "n outside"), ([0, 1, 2, 3, 0], "n outside"), ([4], "out of range"),
    ([-1], "out of range"), ([0, 0], "twice")])
def test_block_plan_refusals(select, needle):
    plan = tide.Plan(SHAPES, 2)
    st, h = create(plan, select)
    assert st == E_INVALID and h.value is None and needle in err()


def test_block_plan_refusals_of_plans():
    plan = tide.Plan(SHAPES, 2)
    assert create(None, [0])[0] == E_INVALID and "plan is NULL" in err()
    assert create(tide.BlockPlan(plan), [0])[0] == E_INVALID and "itself" in err()
    assert create(plan, [0], out=False)[0] == E_INVALID
    assert lib().tide_plan_create_blocks(plan.handle, 1, None, ctypes.byref(P())) == E_INVALID
    big = tide.Plan([(1 << 31, 0)], 2)
    assert create(big, [0])[0] == E_INVALID and "2^31" in err()
    with pytest.raises(tide.TideError):
        tide.BlockPlan(tide.Plan([(4,)], 2))             # no matrix to select


def test_shard_refusals():
    plan = tide.Plan([(4, 200), (8, 8)], 2)
    bp = tide.BlockPlan(plan)

    def call(p=bp, rank=0, master=A, block=B, flags=0):
        return lib().tide_block_shard(p.handle if p else None, rank, P(master), P(block), flags,
                                      None)
    for kw, st, needle in [
            (dict(p=None), E_INVALID, "plan is NULL"),
            (dict(p=plan), E_INVALID, "tide_plan_create_blocks"),
            (dict(rank=2), E_INVALID, "rank"), (dict(rank=-1), E_INVALID, "rank"),
            (dict(flags=1), E_UNSUPPORTED, "flag"),
            (dict(master=0), E_INVALID, "master is NULL"),
            (dict(master=A + 2), E_INVALID, "aligned"),
            (dict(block=0), E_INVALID, "block is NULL"),
            (dict(block=B + 8), E_INVALID, "16-byte"),
            (dict(block=A + plan.S * 4 // 16 * 16 - 16), E_INVALID, "overlaps")]:
        assert call(**kw) == st, kw
        assert needle in err(), kw
    empty = tide.BlockPlan(tide.Plan([(0, 5)], 2))
    assert call(p=empty, master=0, block=0) == 0


def test_unshard_refusals():
    plan = tide.Plan([(4, 200), (8, 8), (0, 3)], 2)
    bp = tide.BlockPlan(plan)

    def call(p=bp, gathered=A, params=(B, C, 0), flags=0x20):
        arr = (P * 3)(*params) if params is not None else None
        return lib().tide_block_unshard(p.handle if p else None, P(gathered), arr, flags, None)
    for kw, st, needle in [
            (dict(p=None), E_INVALID, "plan is NULL"),
            (dict(p=plan), E_INVALID, "tide_plan_create_blocks"),
            (dict(flags=0xa0), E_INVALID, "both"),
            (dict(flags=0x1), E_UNSUPPORTED, "flag"),
            (dict(gathered=0), E_INVALID, "gathered is NULL"),
            (dict(gathered=A + 4), E_INVALID, "16-byte"),
            (dict(params=None), E_INVALID, "params array"),
            (dict(params=(B, 0, 0)), E_INVALID, "params[1] is NULL"),
            (dict(params=(B + 1, C, 0)), E_INVALID, "params[0] is not aligned"),
            (dict(params=(B, C + 2, 0), flags=0), E_INVALID, "params[1] is not aligned"),
            (dict(params=(B, B + 1598, 0)), E_INVALID, "overlaps another"),
            (dict(params=(B, A + 16, 0)), E_INVALID, "overlaps the gathered")]:
        assert call(**kw) == st, kw
        assert needle in err(), kw


def test_unshard_of_nothing():
    empty = tide.BlockPlan(tide.Plan([(0, 5), (7, 0)], 2))
    assert lib().tide_block_unshard(empty.handle, None, None, 0x20, None) == 0


class _Stub:
    """A tensor's attributes without memory: what it passes the binding's checks
    with, the library would refuse (address 0)."""

    is_cuda = True
    requires_grad = False

    def __init__(self, shape, dtype, device="cuda:0", contiguous=True):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device(device)
        self._c = contiguous

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._c

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 0


def stub_blocks(rows, cols, device="cuda:0"):
    return tide.Blocks(_Stub((rows, -(-cols // 128) * 128), torch.uint8, device),
                       _Stub((rows, -(-cols // 512) * 4), torch.uint8, device), cols)


def test_binding_refuses_wrong_blocks():
    u8, f8 = torch.uint8, torch.float8_e4m3fn
    good_s = _Stub((4, 4), u8)
    tide.Blocks(_Stub((4, 256), f8), good_s, 200)
    for codes, scales, cols, exc in [
            (_Stub((4, 256), torch.int8), good_s, 200, TypeError),
            (_Stub((4, 256), f8), _Stub((4, 4), torch.int32), 200, TypeError),
            (_Stub((4, 200), f8), good_s, 200, ValueError),
            (_Stub((4, 256), f8), good_s, 257, ValueError),
            (_Stub((4, 256), f8), good_s, 100, ValueError),
            (_Stub((4, 256), f8), _Stub((4, 2), u8), 200, ValueError),
            (_Stub((5, 256), f8), good_s, 200, ValueError),
            (_Stub((1024,), f8), good_s, 200, ValueError),
            (_Stub((4, 256), f8, contiguous=False), good_s, 200, ValueError),
            (_Stub((4, 256), f8, "cuda:1"), good_s, 200, ValueError),
            (torch.zeros(4, 256, dtype=u8), torch.zeros(4, 4, dtype=u8), 200, ValueError)]:
        with pytest.raises(exc):
            tide.Blocks(codes, scales, cols)


def test_binding_refuses_wrong_operands():
    bf = torch.bfloat16
    x, w = stub_blocks(4, 200), stub_blocks(8, 200)
    dy = _Stub((4, 8), bf)
    for call in [
            lambda: tide.block_quant(torch.zeros(4, 4)),                        # host tensor
            lambda: tide.block_quant(_Stub((4, 4), torch.float64)),
            lambda: tide.block_quant(_Stub((4,), bf)),
            lambda: tide.block_quant(_Stub((4, 4), bf, contiguous=False)),
            lambda: tide.block_quant(_Stub((4, 201), bf), out=x),
            lambda: tide.block_quant(_Stub((4, 200), bf, "cuda:1"), out=x),
            lambda: tide.block_dequant(x, dtype=torch.float64),
            lambda: tide.block_dequant(x, out=_Stub((4, 201), bf)),
            lambda: tide.block_dequant(x, out=_Stub((4, 200), bf, "cuda:1")),
            lambda: tide.block_mm(x, stub_blocks(8, 199)),
            lambda: tide.block_mm(x, w, dtype=torch.float16),
            lambda: tide.block_mm(x, w, out=_Stub((8, 4), bf)),
            lambda: tide.block_mm(x, stub_blocks(8, 200, "cuda:1")),
            lambda: tide.block_mm_dx(_Stub((4, 7), bf), w),
            lambda: tide.block_mm_dx(_Stub((4, 8), torch.float16), w),
            lambda: tide.block_mm_dx(dy, w, out=_Stub((4, 200), torch.float16)),
            lambda: tide.block_mm_dw(_Stub((5, 8), bf), x),
            lambda: tide.block_mm_dw(dy, x, accumulate=True),
            lambda: tide.block_mm_dw(dy, x, out=_Stub((8, 201), bf)),
            lambda: tide.block_linear(_Stub((4, 199), bf), w),
            lambda: tide.block_linear(_Stub((4, 200), bf), w, accumulate=True),
            lambda: tide.block_linear(_Stub((4, 200), bf, contiguous=False), w),
            lambda: tide.block_linear(_Stub((4, 200), bf), w, grad=_Stub((8, 199), bf)),
            lambda: tide.block_linear(_Stub((4, 200), bf), w, grad=_Stub((8, 200), torch.float16))]:
        with pytest.raises((ValueError, TypeError)):
            call()


def test_binding_refuses_wrong_gather_buffers():
    plan = tide.Plan([(4, 200), (8, 8)], 2)
    bp = tide.BlockPlan(plan)
    f32, i32, bf = torch.float32, torch.int32, torch.bfloat16
    master, block = _Stub((plan.S,), f32), _Stub((bp.S,), i32)
    for m, b in [(_Stub((plan.S + 1,), f32), block), (_Stub((plan.S,), bf), block),
                 (master, _Stub((bp.S - 1,), i32)), (master, _Stub((bp.S,), f32)),
                 (master, _Stub((bp.S,), i32, "cuda:1")),
                 (torch.zeros(plan.S), block)]:
        with pytest.raises(ValueError):
            tide.block_shard(bp, 0, m, b)
    gathered = _Stub((2, bp.S), i32)
    good = [_Stub((4, 200), bf), _Stub((8, 8), bf)]
    for g, ps in [(_Stub((1, bp.S), i32), good), (_Stub((2, bp.S), f32), good),
                  (gathered, good[:1]), (gathered, [good[0], _Stub((8, 9), bf)]),
                  (gathered, [good[0], _Stub((8, 8), f32)]),
                  (gathered, [good[0], _Stub((8, 8), bf, "cuda:1")]),
                  (gathered, [_Stub((4, 200), torch.int8), good[1]])]:
        with pytest.raises((ValueError, TypeError)):
            tide.block_unshard(bp, g, ps)
    with pytest.raises(ValueError):
        bp.views([stub_blocks(4, 200)])
    with pytest.raises(ValueError):
        bp.views([stub_blocks(4, 200), stub_blocks(8, 9)])


def test_custom_ops_declare_what_they_write():
    import parameter_layout_collectives_amd.torch_ops  # noqa: F401 - registers the ops
    for name, written in [("block_shard", ["Tensor(a3!) block"]),
                          ("block_unshard", ["Tensor(a2!)[] params"]),
                          ("block_quant", ["Tensor(a1!) codes", "Tensor(a2!) scales"]),
                          ("block_dequant", ["Tensor(a2!) out"]),
                          ("block_mm", ["Tensor(a5!) out"]),
                          ("block_mm_dx", ["Tensor(a3!) out"]),
                          ("block_mm_dw", ["Tensor(a3!) out"])]:
        schema = str(getattr(torch.ops.tide, name).default._schema)
        for w in written:
            assert w in schema, (name, schema)
        assert schema.count("!") == len(written), (name, schema)


def test_short_sums_refusals():
    assert mm(flags=0x100) == E_INVALID and "SHORT_SUMS" in err()        # fp32 output
    assert linear(flags=0x100) == E_INVALID and "SHORT_SUMS" in err()
    assert dx(flags=0x120) == E_UNSUPPORTED and "flag" in err()
    assert dw(flags=0x120) == E_UNSUPPORTED and "flag" in err()
    assert dequant(flags=0x120) == E_UNSUPPORTED and "flag" in err()
    assert mm(m=0, x=0, xs=0, out=0, flags=0x120) == 0
