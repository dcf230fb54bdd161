"""tide_ortho of matrices with a smaller side of up to 32 in more than a few steps, on
the GPU, against the steps in 64 bits (ortho_ref.py).

A step raises what is near zero by up to a = 3.4445, so both sides' rounding noise, 16
units of 2^-52 of X's norm for sums of up to 32 terms, grows to 16 * 2^-52 a^steps: that,
the result's half step of bf16, 2^-8 of an entry, and 2^-20 of the largest one for fp32's
on the way are the tolerance.  Beyond about 25 steps the noise is as large as the
result; what holds then is that singular values stay below 1.21, and an entry, which is
no larger than the largest of them, with bf16's rounding below 1.3."""
import ctypes

import pytest
import torch

import ortho_ref as ref
import parameter_layout_collectives_amd as tide
from gpu_helpers import note
from parameter_layout_collectives_amd._lib import lib

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
SHAPES = [(16, 64, 4), (64, 16, 4), (32, 4096, 8), (2, 4, 1), (9, 1, 1), (31, 700, 30), (257, 17, 2),
          (16, 64, 16)]


def matrix(r, c, rank, dtype, seed=1):
    """Of rank `rank` but for its own rounding; with two rows, of equal rows."""
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn(r, rank, generator=gen) @ torch.randn(rank, c, generator=gen)
    if r == 2:
        g = g[:1].expand(2, c).contiguous()
    return g.to(dtype).cuda()


def room(want, steps, growth=3.4445):
    return 2.0 ** -8 * want.abs() + 2.0 ** -20 * want.abs().max() + 16 * 2.0 ** -52 * growth ** steps


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("steps", [7, 8, 9, 12, 16, 17, 20])
def test_low_ranks(steps, dtype):
    note(f"ortho few rows, {steps} steps {dtype}")
    for r, c, rank in SHAPES:
        g = matrix(r, c, rank, dtype)
        buf = torch.full((r * c + 64,), 7.0, dtype=BF, device="cuda")
        out = buf[32:32 + r * c].view(r, c)
        tide.ortho(g, out=out, steps=steps)
        want = ref.exact(g, steps)
        assert bool(((out.double() - want).abs() <= room(want, steps)).all()), (r, c, rank)
        assert bool((buf[:32] == 7.0).all()) and bool((buf[-32:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("steps", [30, 47, 64])
def test_results_stay_bounded(steps, dtype):
    note(f"ortho few rows, {steps} steps {dtype}")
    for r, c, rank in SHAPES:
        for seed in range(3):
            out = tide.ortho(matrix(r, c, rank, dtype, seed), steps=steps)
            assert bool(torch.isfinite(out).all()), (r, c, rank, seed)
            assert float(out.abs().max()) <= 1.3, (r, c, rank, seed)


@pytest.mark.parametrize("coefficients,steps", [
    ((1.5, -0.5, 0.0), 64),
    ((1000.0, 0.0, 0.0), 7),                          # one step between two of X's products
    ([(40000.0, 0.0, 0.0), (3.0, -3.0, 1.0), (0.5, 0.0, 0.0)], 3),
    ([(3.0, -3.2, 1.2)] * 4 + [(1.875, -1.25, 0.375)] * 12, 16),
])
def test_other_coefficients(coefficients, steps):
    note(f"ortho few rows, coefficients {coefficients}")
    for r, c in ((7, 300), (300, 7), (32, 40), (1, 5)):
        g = ref.gradient(r, c, 3, "full", FP, "cuda")
        got = tide.ortho(g, steps=steps, coefficients=coefficients).double()
        want = ref.exact(g, steps, coefficients)
        assert bool(((got - want).abs() <= room(want, 0)).all()), (r, c)


def test_beside_others():
    """In a list with large matrices, in place and as each other's outs, zeros and NaNs
    in their own matrix only, captured and replayed."""
    note("ortho few rows, 20 steps, in lists")
    shapes = [(3, 400, 2), (70, 90, 70), (3, 400, 3), (400, 3, 1), (400, 3, 3), (32, 40, 4)]
    gs = [matrix(*s, BF, i) for i, s in enumerate(shapes)]
    alone = [tide.ortho(g, steps=20) for g in gs]
    assert all(torch.equal(a, b) for a, b in zip(tide.ortho(gs, steps=20), alone))
    x = [g.clone() for g in gs]
    outs = [x[2], x[1], x[0], x[4], x[3], x[5]]
    tide.ortho(x, out=outs, steps=20)
    assert all(torch.equal(a, b) for a, b in zip(outs, alone))
    bad = [g.clone() for g in gs]
    bad[0].zero_()
    bad[2][1, 7], bad[3][399, 2] = float("nan"), float("inf")
    outs = tide.ortho(bad, steps=20)
    assert not bool(outs[0].any())
    assert bool(torch.isnan(outs[2]).all()) and bool(torch.isnan(outs[3]).all())
    assert all(torch.equal(outs[i], alone[i]) for i in (1, 4, 5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = tide.ortho(gs, steps=20)
    for it in range(3):
        for i, g in enumerate(gs):
            g.copy_(matrix(*shapes[i], BF, 20 + 8 * it + i))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, tide.ortho(gs, steps=20)))


def test_workspace_of_exactly_the_asked_size():
    note("ortho few rows, 20 steps, workspace")
    L = lib()
    gs = [matrix(5, 129, 3, BF), matrix(200, 32, 8, BF)]
    want = tide.ortho(gs, steps=20)
    rows, cols = (ctypes.c_int64 * 2)(5, 200), (ctypes.c_int64 * 2)(129, 32)
    size = L.tide_ortho_workspace(2, rows, cols)
    for fill in (0, 0xff):
        buf = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(g) for g in gs]
        co = (ctypes.c_float * 60)(*(ref.QUINTIC * 20))
        ptrs = lambda ts: (ctypes.c_void_p * 2)(*[t.data_ptr() for t in ts])  # noqa: E731
        st = L.tide_ortho(2, ptrs(gs), ptrs(outs), rows, cols, 20, co, 0,
                          ctypes.c_void_p(buf.data_ptr()), size,
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert bool((buf[size:] == fill).all())
