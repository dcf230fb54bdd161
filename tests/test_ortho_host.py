"""Host-side checks of tide_ortho that need no GPU: refusals before anything is
enqueued, the workspace's size, and how far the kernels' roundings reach."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fwd

import ortho_ref as ref
import parameter_layout_collectives_amd as tide
from parameter_layout_collectives_amd._lib import lib

E_INVALID, E_UNSUPPORTED = 1, 2
A, B, W = (0x7F0000000000 + i * (1 << 40) for i in range(3))


def err():
    return lib().tide_last_error().decode()


def call(src=(A,), out=(B,), rows=(40,), cols=(70,), steps=5, co=(3.0, -4.0, 2.0), flags=0, ws=W,
         size=None, n=None, null=()):
    n = len(rows) if n is None else n
    r, c = (ctypes.c_int64 * len(rows))(*rows), (ctypes.c_int64 * len(rows))(*cols)
    if size is None:
        size = max(0, lib().tide_ortho_workspace(len(rows), r, c))
    co = list(co) * max(1, steps)
    args = dict(src=(ctypes.c_void_p * len(src))(*src), out=(ctypes.c_void_p * len(out))(*out),
                rows=r, cols=c, co=(ctypes.c_float * len(co))(*co))
    for k in null:
        args[k] = None
    return lib().tide_ortho(n, args["src"], args["out"], args["rows"], args["cols"], steps,
                            args["co"], flags, ctypes.c_void_p(ws), size, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(n=-1), E_INVALID, "n < 0"),
    (dict(n=(1 << 20) + 1), E_UNSUPPORTED, "2^20"),
    (dict(rows=(-1,)), E_INVALID, "negative"),
    (dict(cols=(1 << 31,), size=0), E_INVALID, "2^31"),
    (dict(cols=((1 << 22) + 1,), size=0), E_UNSUPPORTED, "2^22"),
    (dict(rows=((1 << 15) + 1,), cols=((1 << 15) + 1,), size=0), E_UNSUPPORTED, "2^15"),
    (dict(rows=(1 << 12,), cols=(1 << 22,), size=0), E_UNSUPPORTED, "2^33"),
    (dict(steps=0), E_INVALID, "steps"),
    (dict(steps=65), E_INVALID, "steps"),
    (dict(co=(1.0, float("inf"), 0.0)), E_INVALID, "finite"),
    (dict(co=(1.0, float("nan"), 0.0)), E_INVALID, "finite"),
    (dict(flags=0x18), E_INVALID, "both"),
    (dict(flags=0x20), E_UNSUPPORTED, "flag"),
    (dict(src=(0,)), E_INVALID, "src[0] is NULL"),
    (dict(out=(0,)), E_INVALID, "out[0] is NULL"),
    (dict(src=(A + 1,)), E_INVALID, "aligned"),
    (dict(src=(A + 2,), flags=0x10), E_INVALID, "aligned"),
    (dict(out=(B + 1,)), E_INVALID, "aligned"),
    (dict(ws=0), E_INVALID, "workspace is NULL"),
    (dict(ws=W + 64), E_INVALID, "256-byte"),
    (dict(size=256), E_INVALID, "workspace holds"),
    (dict(src=(W + 64,)), E_INVALID, "overlaps the workspace"),
    (dict(out=(W + 64,)), E_INVALID, "overlaps the workspace"),
    (dict(src=(A, A), out=(B, B + 5598), rows=(40, 40), cols=(70, 70)), E_INVALID,
     "overlaps another"),
    (dict(null=("rows",), size=1 << 20), E_INVALID, "NULL"),
    (dict(null=("src",)), E_INVALID, "src is NULL"),
    (dict(null=("out",)), E_INVALID, "out is NULL"),
    (dict(null=("co",)), E_INVALID, "coefficients is NULL"),
])
def test_refusals(kw, status, needle):
    assert call(**kw) == status
    assert needle in err()


def test_nothing_to_do_is_ok():
    assert call(src=(), out=(), rows=(), cols=(), ws=0) == 0
    assert call(src=(0, 0), out=(0, 0), rows=(0, 5), cols=(7, 0), ws=0, size=0) == 0


def test_workspace_holds_what_the_header_says():
    L = lib()
    def ws(*shapes):
        n = len(shapes)
        return L.tide_ortho_workspace(n, (ctypes.c_int64 * n)(*[s[0] for s in shapes]),
                                      (ctypes.c_int64 * n)(*[s[1] for s in shapes]))
    assert ws((0, 9)) == 0 and ws((9, 0), (0, 0)) == 0
    one, two = ws((100, 200)), ws((100, 200), (100, 200))
    # X twice as two fp16 matrices, A and P
    assert one >= 2 * 4 * 128 * 256 + 2 * 128 * 128 + 2 * 128 * 128
    assert one < two < 2 * one + 512
    assert ws((1, 1 << 22)) > 0 and ws((1 << 15, 1 << 15)) > 0
    assert ws((1, (1 << 22) + 1)) == -1 and ws((3, -1)) == -1


class _Stub:
    """Looks like a contiguous device tensor."""

    def __init__(self, shape, dtype=torch.bfloat16, device="cuda:0", contiguous=True, cuda=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.is_cuda, self._contiguous = cuda, contiguous

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._contiguous


@pytest.mark.parametrize("g,kw,error,needle", [
    ([torch.zeros(3, 4)], {}, ValueError, "device tensor"),
    (torch.zeros(3, 4, dtype=torch.float64), {}, TypeError, "float64"),
    (torch.zeros(3, 4), dict(coefficients=(1.0, 2.0)), ValueError, "triples"),
    (torch.zeros(3, 4), dict(coefficients=[(1.0, 2.0, 3.0)] * 2, steps=3), ValueError, "triples"),
    ([], dict(coefficients=[], steps=1), ValueError, "triples"),
])
def test_binding_refusals(g, kw, error, needle):
    with pytest.raises(error, match=needle):
        tide.ortho(g, **kw)


def test_binding_refusals_of_lists(monkeypatch):
    import sys
    mod = sys.modules["parameter_layout_collectives_amd.ortho"]
    monkeypatch.setattr(mod, "_no_dual", lambda t, what: None)
    bf = torch.bfloat16
    for g, kw, error, needle in [
            ([_Stub((3, 4)), _Stub((3, 4), torch.float32)], {}, TypeError, "the others"),
            ([_Stub((3, 4)), _Stub((3, 4), device="cuda:1")], {}, ValueError, "tensors on"),
            ([_Stub((3,))], {}, ValueError, "2-D or 3-D"),
            ([_Stub((3, 4), contiguous=False)], {}, ValueError, "contiguous"),
            ([_Stub((3, 4))], dict(out=[]), ValueError, "outs for"),
            ([_Stub((3, 4))], dict(out=[_Stub((4, 3))]), ValueError, "shape"),
            ([_Stub((3, 4))], dict(out=[_Stub((3, 4), torch.float32)]), TypeError, "float32"),
            ([_Stub((3, 4))], dict(out=[_Stub((3, 4), bf, "cuda:1")]), ValueError, "tensors on")]:
        with pytest.raises(error, match=needle):
            tide.ortho(g, **kw)


def test_empty_list_and_dual():
    assert tide.ortho([]) == []
    with fwd.dual_level():
        d = fwd.make_dual(torch.zeros(3, 4), torch.ones(3, 4))
        with pytest.raises(NotImplementedError, match="dual"):
            tide.ortho(d)


@pytest.mark.parametrize("shape", [(5, 300), (37, 129), (64, 64), (130, 500), (260, 260), (300, 140)])
@pytest.mark.parametrize("kind", ["full", "heavy", "low"])
def test_the_roundings_stay_below_the_output_s(shape, kind):
    """What the fp16 factors cost, before the output is rounded: less than bf16's own
    rounding, 2^-8 / sqrt(12) * 1.47 = 1.66e-3 of the norm for mantissas spread evenly
    over their logarithm."""
    g = ref.gradient(*shape, 7, kind)
    assert ref.off(ref.emulated(g), ref.exact(g)) < 1.66e-3


def test_reference_on_known_singular_values():
    """With G = U S V^T the result is U p(p(...p(S / ||S||))) V^T."""
    gen = torch.Generator().manual_seed(3)
    u, _ = torch.linalg.qr(torch.randn(20, 20, generator=gen, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(50, 20, generator=gen, dtype=torch.float64))
    s = torch.logspace(0, -3, 20, dtype=torch.float64)
    x = s / s.norm()
    for _ in range(5):
        x = 3.4445 * x - 4.7750 * x ** 3 + 2.0315 * x ** 5
    assert ref.off(ref.exact(u @ torch.diag(s) @ v.t()), u @ torch.diag(x) @ v.t()) < 1e-10
    x = torch.logspace(-2.69, 0, 10001, dtype=torch.float64)      # from 2e-3 on
    for _ in range(5):
        x = 3.4445 * x - 4.7750 * x ** 3 + 2.0315 * x ** 5
    assert 0.67 < float(x.min()) and float(x.max()) < 1.21        # as the header says
