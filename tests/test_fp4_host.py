"""Host-side checks of the 4-bit block calls that need no GPU: sizes of the format,
plans, the reference, and every refusal before anything is enqueued."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fwd

import fp4_ref as ref
import parameter_layout_collectives_amd as tide
from parameter_layout_collectives_amd._lib import lib
from test_blocks_host import _Stub, stub_blocks

E_INVALID, E_UNSUPPORTED = 1, 2
A, B, C, D, E, W = (0x7F0000000000 + i * (1 << 32) for i in range(6))
P = ctypes.c_void_p


def err():
    return lib().tide_last_error().decode()


def test_sizes():
    for c in range(0, 2000):
        assert lib().tide_mx_cols(c) == -(-c // 128) * 128
    assert lib().tide_mx_cols(-1) == -1 and lib().tide_mx_cols(1 << 31) == -1


def quant(x=A, rows=4, cols=200, codes=B, scales=C, flags=0):
    return lib().tide_mx_quant(P(x), rows, cols, P(codes), P(scales), flags, None)


def dequant(codes=B, scales=C, rows=4, cols=200, out=A, flags=0):
    return lib().tide_mx_dequant(P(codes), P(scales), rows, cols, P(out), flags, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), E_INVALID, "negative"),
    (dict(cols=1 << 31), E_INVALID, "2^31"),
    (dict(rows=(1 << 31) - 1, cols=(1 << 31) - 1), E_INVALID, "overflow"),
    (dict(flags=0x18), E_INVALID, "both"),
    (dict(flags=0x200), E_UNSUPPORTED, "flag"),
    (dict(x=0), E_INVALID, "x is NULL"),
    (dict(x=A + 1), E_INVALID, "aligned"),
    (dict(codes=0), E_INVALID, "codes are NULL"),
    (dict(scales=0), E_INVALID, "scales are NULL"),
    (dict(codes=B + 8), E_INVALID, "16-byte"),
    (dict(scales=C + 2), E_INVALID, "4-byte"),
    (dict(codes=A + 1584), E_INVALID, "overlaps"),        # x holds 1600 bytes
    (dict(scales=B + 508), E_INVALID, "overlaps"),        # codes hold 512 bytes
])
def test_quant_refusals(kw, status, needle):
    assert quant(**kw) == status
    assert needle in err() and "tide_mx" in err()


def test_casts_reach_no_further_than_the_format():
    """One byte past the format's is free to be something else."""
    assert quant(rows=0) == 0 and dequant(cols=0) == 0
    for kw, needle in [(dict(out=B + 508), "overlaps"), (dict(out=C + 28), "overlaps"),
                       (dict(out=0), "out is NULL"), (dict(flags=0xa0), "both")]:
        assert dequant(**kw) == E_INVALID and needle in err()


def mm(x=A, xs=B, m=40, w=C, ws=D, n=8, k=200, out=E, flags=0, wsp=0, size=0):
    return lib().tide_mx_mm(P(x), P(xs), m, P(w), P(ws), n, k, P(out), flags, P(wsp), size, None)


def linear(x=A, m=40, w=C, ws=D, n=8, k=200, out=E, flags=0, wsp=0, size=0):
    return lib().tide_mx_linear(P(x), m, k, P(w), P(ws), n, P(out), flags, P(wsp), size, None)


def dx(x=A, m=40, n=8, w=C, ws=D, k=200, out=E, flags=0, wsp=0, size=0):
    return lib().tide_mx_mm_dx(P(x), m, n, P(w), P(ws), k, P(out), flags, P(wsp), size, None)


COMMON = [
    (dict(m=-1), E_INVALID, "negative"),
    (dict(n=-1), E_INVALID, "negative"),
    (dict(k=-1), E_INVALID, "negative"),
    (dict(m=1 << 31), E_INVALID, "2^31"),
    (dict(n=(1 << 22) + 1), E_UNSUPPORTED, "2^22"),
    (dict(k=(1 << 22) + 1), E_UNSUPPORTED, "2^22"),
    (dict(m=(1 << 31) - 1, n=1 << 22, k=1 << 22), E_UNSUPPORTED, "lanes"),
    (dict(flags=0x80), E_UNSUPPORTED, "flag"),
    (dict(flags=0x40), E_UNSUPPORTED, "flag"),
    (dict(out=0), E_INVALID, "out is NULL"),
    (dict(out=E + 2), E_INVALID, "aligned"),
    (dict(out=E + 1, flags=0x20), E_INVALID, "aligned"),
    (dict(size=-1), E_INVALID, "workspace"),
    (dict(size=64), E_INVALID, "workspace is NULL"),
    (dict(wsp=W + 8, size=64), E_INVALID, "16-byte"),
    (dict(wsp=E, size=64), E_INVALID, "overlaps"),
    (dict(wsp=C, size=64), E_INVALID, "overlaps"),
    (dict(wsp=D, size=64), E_INVALID, "overlaps"),
    (dict(wsp=A, size=64), E_INVALID, "overlaps"),
    (dict(out=A), E_INVALID, "overlaps"),
    (dict(out=C), E_INVALID, "overlaps"),
    (dict(out=D), E_INVALID, "overlaps"),
    (dict(x=0), E_INVALID, "NULL"),
    (dict(w=0), E_INVALID, "w's codes are NULL"),
    (dict(ws=0), E_INVALID, "w's scales are NULL"),
    (dict(w=C + 4), E_INVALID, "16-byte"),
    (dict(ws=D + 2), E_INVALID, "4-byte"),
]


@pytest.mark.parametrize("call", [mm, linear, dx])
@pytest.mark.parametrize("kw,status,needle", COMMON)
def test_product_refusals(call, kw, status, needle):
    assert call(**kw) == status
    assert needle in err()


def test_more_product_refusals():
    assert mm(x=A + 8) == E_INVALID and "16-byte" in err()
    assert mm(xs=0) == E_INVALID and "scales" in err()
    assert mm(flags=0x200) == E_UNSUPPORTED and dx(flags=0x200) == E_UNSUPPORTED
    assert linear(x=A + 1) == E_INVALID and "aligned" in err()
    for f in (0x8, 0x10):
        assert linear(flags=f) == E_INVALID and "TIDE_F_QUANT_X" in err()
    assert linear(flags=0x218) == E_INVALID and "both" in err()
    assert linear(flags=0x200) == E_INVALID and "blocks need" in err()
    assert linear(flags=0x200, wsp=W, size=64) == E_INVALID and "blocks need" in err()


def test_nothing_to_do_is_ok():
    assert mm(m=0, x=0, xs=0, out=0) == 0 and linear(n=0, out=0, w=0) == 0 and dx(k=0, out=0) == 0


def test_workspace():
    ws = lib().tide_mx_workspace
    assert ws(3, 1, 1, 1, 0) == -1 and ws(-1, 1, 1, 1, 0) == -1
    for op in range(3):
        assert ws(op, 0, 64, 64, 0) == 0 and ws(op, 64, 64, 0, 0) == 0
        assert ws(op, -1, 64, 64, 0) == -1 and ws(op, 64, 1 << 23, 64, 0) == -1
        assert (ws(op, 64, 64, 64, 0x200) == -1) == (op != 2)
    assert ws(2, 64, 64, 64, 0x8) == -1 and ws(2, 64, 64, 64, 0x208) > 0
    assert ws(2, 1, 64, 4096, 0x200) == 0                # in one launch
    assert ws(2, 40, 64, 1000, 0x200) >= 40 * (512 + 32)     # x's blocks


def test_plans():
    plan = tide.Plan([(5, 7), (16,), (33, 300)], 4)
    fp = tide.Fp4Plan(plan)
    assert fp.select == [0, 2] and fp.matrices == [(5, 7), (33, 300)]
    # 128 and 384 columns: 16 and 48 words of codes, 1 and 3 of scales a row
    assert [fp.param(i)[1:] for i in range(4)] == [(2, 32), (9, 432), (2, 2), (9, 27)]
    assert all(fp.param(i)[0] % 4 == 0 for i in range(4)) and fp.S % 4 == 0
    with pytest.raises(tide.TideError, match="block plan"):
        tide.Fp4Plan(fp)
    with pytest.raises(tide.TideError, match="twice"):
        tide.Fp4Plan(plan, [0, 0])


def test_a_plan_of_the_other_format_is_refused():
    plan = tide.Plan([(8, 200)], 2)
    four, eight = tide.Fp4Plan(plan), tide.BlockPlan(plan)
    L = lib()
    assert L.tide_mx_shard(eight.handle, 0, P(A), P(B), 0, None) == E_INVALID
    assert "tide_plan_create_mx" in err()
    assert L.tide_block_shard(four.handle, 0, P(A), P(B), 0, None) == E_INVALID
    assert "tide_plan_create_blocks" in err()
    arr = (P * 1)(C)
    assert L.tide_mx_unshard(eight.handle, P(A), arr, 0, None) == E_INVALID
    assert L.tide_block_unshard(four.handle, P(A), arr, 0, None) == E_INVALID
    assert L.tide_mx_shard(plan.handle, 0, P(A), P(B), 0, None) == E_INVALID
    with pytest.raises(ValueError, match="Fp4Blocks"):
        four.views([tide.Blocks.empty(8, 200, "cpu")])
    with pytest.raises(ValueError, match="Blocks"):
        eight.views([tide.Fp4Blocks.empty(8, 200, "cpu")])


def stub4(rows, cols, device="cuda:0"):
    nb = -(-cols // 128)
    return tide.Fp4Blocks(_Stub((rows, nb * 64), torch.uint8, device),
                          _Stub((rows, nb * 4), torch.uint8, device), cols)


def test_one_format_in_place_of_the_other_is_refused():
    bf = torch.bfloat16
    four, eight, dy = stub4(8, 200), stub_blocks(8, 200), _Stub((4, 8), bf)
    for call in (lambda: tide.fp4_mm(eight, four), lambda: tide.fp4_mm(four, eight),
                 lambda: tide.fp4_dequant(eight), lambda: tide.fp4_mm_dx(dy, eight)):
        with pytest.raises(TypeError, match="8-bit blocks"):
            call()
    for call in (lambda: four._ptrs, lambda: tide.block_dequant(four, out=None)):
        with pytest.raises((TypeError, RuntimeError)):
            call()


def test_blocks_have_to_fit():
    u8 = torch.uint8
    for codes, scales, cols in [((3, 64), (3, 4), 129), ((3, 64), (2, 4), 100), ((3, 128), (3, 4), 100),
                                ((3, 64), (3, 8), 100), ((3, 64), (3, 4), -1)]:
        with pytest.raises(ValueError):
            tide.Fp4Blocks(_Stub(codes, u8), _Stub(scales, u8), cols)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        tide.Fp4Blocks(_Stub((3, 64), torch.float8_e4m3fn), _Stub((3, 4), u8), 100)
    q = stub4(3, 100)
    with pytest.raises(ValueError):
        q.codes = _Stub((4, 64), u8)
    assert (q.rows, q.cols, q.shape) == (3, 100, (3, 100))


def test_linear_refusals():
    w, bf = stub4(8, 200), torch.bfloat16
    x = torch.zeros(4, 200, dtype=bf)
    for call, error, needle in [
            (lambda: tide.fp4_linear(torch.zeros(4, 100, dtype=bf), w), ValueError, "columns"),
            (lambda: tide.fp4_linear(torch.zeros(200, 4, dtype=bf).t(), w), ValueError, "contiguous"),
            (lambda: tide.fp4_linear(x, w, accumulate=True), ValueError, "accumulate"),
            (lambda: tide.fp4_linear(x.float(), w), TypeError, "float32"),
            (lambda: tide.fp4_linear(x.half(), w), TypeError, "float16"),
            (lambda: tide.fp4_linear(x.double(), w, quant_x=True), TypeError, "float64"),
            (lambda: tide.fp4_linear(x, w), ValueError, "device tensor")]:
        with pytest.raises(error, match=needle):
            call()


def test_dual_tensors_are_refused():
    bf = torch.bfloat16
    w = stub4(8, 200)
    plan = tide.Fp4Plan(tide.Plan([(8, 200)], 2))
    gathered = _Stub((2, plan.S), torch.int32)
    with fwd.dual_level():
        def dual(*shape):
            return fwd.make_dual(torch.zeros(shape, dtype=bf), torch.ones(shape, dtype=bf))
        for call in (lambda: tide.fp4_linear(dual(4, 200), w),
                     lambda: tide.fp4_quant(dual(4, 200)),
                     lambda: tide.fp4_mm_dx(dual(4, 8), w),
                     lambda: tide.fp4_mm(w, w, out=dual(8, 8)),
                     lambda: tide.fp4_dequant(w, out=dual(8, 200)),
                     lambda: tide.fp4_shard(plan, 0, dual(4, 200).float(), None),
                     lambda: tide.fp4_unshard(plan, gathered, [dual(8, 200)])):
            with pytest.raises(NotImplementedError, match="dual"):
                call()


def test_reference_on_worked_blocks():
    """max 7 needs e = 1 (7 > 6): 7 -> 3.5 -> 4 (tie to the even code) -> 8; max 6 keeps
    e = 0 and 5 -> 4, 2.5 -> 2; 0.75 * 2^-125 is the smallest block that is not zeros."""
    x = torch.zeros(4, 33)
    x[0, :4] = torch.tensor([7.0, -0.5, 1.0, 0.4])
    x[1, :4] = torch.tensor([6.0, 5.0, -2.5, 0.25])
    x[2, 32] = 2.0 ** -126
    x[3, 0] = float("inf")
    codes, scales = ref.quant(x)
    v = ref.values(codes, scales, 33)
    assert v[0, :4].tolist() == [8.0, -0.0, 1.0, 0.0] and v[1, :4].tolist() == [6.0, 4.0, -2.0, 0.0]
    assert scales[0, :2].tolist() == [128, 127] and scales[1, 0] == 127
    assert scales[2].tolist() == [127, 2, 127, 127] and v[2, 32] == 2.0 ** -126
    assert scales[3, 0] == 255 and bool(torch.isnan(v[3, :32]).all()) and v[3, 32] == 0
    assert codes[1, :2].tolist() == [7 + 16 * 6, 12]
