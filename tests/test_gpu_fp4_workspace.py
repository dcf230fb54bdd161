"""4-bit products with the workspace that they ask for and with larger ones: the same
bits, at sizes whose large tiles are cut into fewer pieces than the card has room for."""
import ctypes

import pytest
import torch

import parameter_layout_collectives_amd as tide
from gpu_helpers import note
from parameter_layout_collectives_amd._lib import lib
from test_gpu_fp4 import check_products, operands

pytestmark = pytest.mark.gpu
DX, LINEAR = 1, 2


@pytest.mark.parametrize("op,m,n,k", [(DX, 832, 8320, 1920), (DX, 479, 3148, 11218), (DX, 545, 7344, 3000),
                                      (LINEAR, 866, 2400, 6272), (LINEAR, 476, 10771, 2448),
                                      (LINEAR, 40, 4096, 4096)])
def test_any_workspace_from_the_asked_one_on(op, m, n, k):
    note(f"fp4 workspace op={op} {m} x {n} x {k}")
    x, _, w, dy = operands(m, n, k, 9)
    P, L = ctypes.c_void_p, lib()
    stream = P(torch.cuda.current_stream().cuda_stream)
    want = tide.fp4_mm_dx(dy, w, dtype=torch.float32) if op == DX else \
        tide.fp4_linear(x, w, dtype=torch.float32)
    wp = [P(p) for p in w._ptrs4]
    asked = L.tide_mx_workspace(op, m, n, k, 0)
    for more in (0, 256, 64 << 20):
        buf = torch.full((asked + more + 512,), 0xff, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(want)
        ws = (P(buf.data_ptr()), asked + more) if asked + more else (None, 0)
        if op == DX:
            st = L.tide_mx_mm_dx(P(dy.data_ptr()), m, n, *wp, k, P(out.data_ptr()), 0, *ws, stream)
        else:
            st = L.tide_mx_linear(P(x.data_ptr()), m, k, *wp, n, P(out.data_ptr()), 0, *ws, stream)
        assert st == 0
        assert torch.equal(out, want), more
        assert bool((buf[asked + more:] == 0xff).all())


@pytest.mark.parametrize("shape", [(832, 8320, 1920), (866, 2400, 6272), (545, 7344, 3000)])
def test_products(shape):
    check_products(*shape)
