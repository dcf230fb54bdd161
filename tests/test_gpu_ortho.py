"""tide_ortho on the GPU, against Newton-Schulz steps in 64 bits (ortho_ref.py).

Tolerance of a result's norm: rounding to bf16 moves an entry by at most half a step,
2^-8 of it, hence the norm by at most 2^-8 = 3.9e-3; before that the fp16 factors cost
up to 1.66e-3 (test_ortho_host.py pins that for an emulation of them).  Together
5.6e-3.  (1.7e-3 and 1e-3 are usual, but a matrix of one entry can have the worst of
the rounding: 0.7018 becomes 0.6992 or 0.7031, 2.9e-3 apart from the middle.)  A lost
tile, row or term shows as 1e-2 and more."""
import ctypes

import pytest
import torch

import ortho_ref as ref
import parameter_layout_collectives_amd as tide
import parameter_layout_collectives_amd.torch_ops as tops
from gpu_helpers import note
from parameter_layout_collectives_amd._lib import lib

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
TOL = 2.0 ** -8 + 1.66e-3
SHAPES = [(1, 1), (1, 7), (7, 1), (2, 2), (1, 500), (3, 3), (63, 64), (64, 65), (65, 64), (127, 129),
          (128, 300), (129, 300), (300, 129), (256, 256), (257, 255), (255, 1000), (500, 1030),
          (1030, 500), (4100, 65), (65, 4100)]


def check(g, out, what, coefficients=ref.QUINTIC, steps=5):
    want = ref.exact(g.detach(), steps, coefficients)
    err = ref.off(out, want)
    assert err <= TOL, (what, err)
    # no single entry is far off either: an entry's share of the whole error
    worst = float((out.double() - want).abs().max())
    rms = float(want.norm()) / want.numel() ** 0.5
    assert worst <= 2.0 ** -7 * float(want.abs().max()) + 16 * TOL * rms, (what, worst)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", SHAPES)
def test_is_the_definition(shape, dtype):
    note(f"ortho {shape} {dtype}")
    for seed, kind in enumerate(("full", "heavy", "low")):
        g = ref.gradient(*shape, seed, kind, dtype, "cuda")
        n = g.numel()
        buf = torch.full((n + 64,), 7.0, dtype=BF, device="cuda")
        out = buf[32:32 + n].view(shape)
        assert tide.ortho(g, out=out) is out
        check(g, out, kind)
        assert bool((buf[:32] == 7.0).all()) and bool((buf[-32:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", [(1, 1), (1, 2), (2, 1), (2, 2), (2, 3), (3, 2), (29, 2), (3, 259), (4, 4),
                                   (5, 1000), (7, 255), (256, 8), (257, 9), (16, 16), (17, 513), (31, 70),
                                   (32, 32), (32, 4000), (100000, 3), (1, 70000), (70000, 32)])
def test_few_rows_are_exact(shape, dtype):
    """Up to 32 rows the steps run in fp64, and G enters as it is: what is left is the
    result's half step of bf16, 2^-8 of each entry, and fp32's on the way, 2^-24; 2^-20 of
    the largest entry covers fp64's through 5 steps that raise it by up to 500."""
    note(f"ortho few rows {shape} {dtype}")
    for seed in range(6 if shape[0] * shape[1] < 5000 else 2):
        for kind in ("full", "heavy", "low"):
            g = ref.gradient(*shape, seed, kind, dtype, "cuda")
            n = g.numel()
            buf = torch.full((n + 64,), 7.0, dtype=BF, device="cuda")
            out = buf[32:32 + n].view(shape)
            tide.ortho(g, out=out)
            want = ref.exact(g)
            room = 2.0 ** -8 * want.abs() + 2.0 ** -20 * want.abs().max()
            assert bool(((out.double() - want).abs() <= room).all()), (seed, kind)
            assert bool((buf[:32] == 7.0).all()) and bool((buf[-32:] == 7.0).all())


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e30, 3e38])
def test_few_rows_of_any_size_of_numbers(scale):
    note(f"ortho few rows scale {scale}")
    for shape in ((7, 300), (300, 7)):
        g = ref.gradient(*shape, 2, "full", FP, "cuda")
        g = ((g / g.abs().max()).double() * scale).float()
        check(g, tide.ortho(g), (shape, scale))


def test_few_rows_beside_many():
    """Small matrices in a list with large ones: each as alone, zeros, NaNs and
    infinities in their own matrix only, outs that are other matrices' srcs, other
    steps, captured and replayed."""
    note("ortho few rows beside many")
    shapes = [(3, 400), (70, 200), (3, 400), (400, 3), (400, 3), (33, 40), (32, 40), (1, 1)]
    gs = [ref.gradient(*s, i, "heavy", BF, "cuda") for i, s in enumerate(shapes)]
    alone = [tide.ortho(g) for g in gs]
    assert all(torch.equal(a, b) for a, b in zip(tide.ortho(gs), alone))
    x = [g.clone() for g in gs]
    tide.ortho(x, out=[x[2], x[1], x[0], x[4], x[3], *x[5:]])
    got = [x[2], x[1], x[0], x[4], x[3], *x[5:]]
    assert all(torch.equal(a, b) for a, b in zip(got, alone))
    bad = [g.clone() for g in gs]
    bad[0].zero_()
    bad[2][1, 7], bad[3][399, 2] = float("nan"), float("inf")
    outs = tide.ortho(bad)
    assert not bool(outs[0].any())
    assert bool(torch.isnan(outs[2]).all()) and bool(torch.isnan(outs[3]).all())
    for i in (1, 4, 5, 6, 7):
        assert torch.equal(outs[i], alone[i])
    for co, steps in (((1.5, -0.5, 0.0), 64), ((3.4445, -4.775, 2.0315), 1),
                      ([(3.0, -3.0, 1.0), (2.0, -1.5, 0.5)], 2)):
        for g in gs[:1] + gs[3:4]:
            check(g, tide.ortho(g, steps=steps, coefficients=co), steps, co, steps)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        held = tide.ortho(gs)
    for it in range(3):
        for i, g in enumerate(gs):
            g.copy_(ref.gradient(*shapes[i], 20 + 8 * it + i, "full", BF, "cuda"))
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, tide.ortho(gs)))


@pytest.mark.parametrize("shape", [(2050, 4100), (4100, 2050), (3000, 3100)])
def test_large_tiles(shape):
    note(f"ortho large {shape}")
    g = ref.gradient(*shape, 5, "heavy", BF, "cuda")
    check(g, tide.ortho(g), shape)


def test_list_of_many_shapes():
    """More shapes than one launch's arguments hold, more matrices than one table
    launch does, tall and wide, with empty ones in between; each as alone."""
    note("ortho of 300 matrices of 70 shapes")
    shapes = [(1 + 7 * (i % 10), 1 + 11 * (i // 10)) for i in range(70)]
    gs = [ref.gradient(*shapes[i % 70], i, "heavy", FP, "cuda") for i in range(300)]
    gs[5:5] = [torch.zeros(0, 7, device="cuda"), torch.zeros(3, 0, device="cuda")]
    outs = tide.ortho(gs)
    for i, (g, o) in enumerate(zip(gs, outs)):
        assert o.shape == g.shape
        if g.numel():
            check(g, o, (i, g.shape))
    for i in (0, 40, 299):
        assert ref.off(tide.ortho(gs[i]), outs[i].double()) <= 2.0 ** -9, i


@pytest.mark.parametrize("shape", [(3, 70, 130), (5, 130, 70), (1, 40, 40), (0, 4, 4), (4, 0, 3)])
def test_stacks(shape):
    note(f"ortho stack {shape}")
    b, r, c = shape
    g = torch.stack([ref.gradient(r, c, i, "heavy", BF, "cuda") for i in range(b)]) \
        if b and r else torch.zeros(shape, dtype=BF, device="cuda")
    out = tide.ortho(g)
    assert out.shape == g.shape
    if g.numel():
        for i in range(b):
            check(g[i], out[i], i)


@pytest.mark.parametrize("lead", [1, 3])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_any_alignment(lead, dtype):
    note(f"ortho unaligned {lead} {dtype}")
    g = ref.gradient(33, 101, 1, "heavy", dtype, "cuda")
    a = torch.zeros(33 * 101 + 8, dtype=dtype, device="cuda")
    src = a[lead:lead + 33 * 101].view(33, 101)
    src.copy_(g)
    o = torch.full((33 * 101 + 8,), 7.0, dtype=BF, device="cuda")
    dst = o[lead:lead + 33 * 101].view(33, 101)
    tide.ortho(src, out=dst)
    assert torch.equal(dst, tide.ortho(g))
    assert bool((o[:lead] == 7.0).all()) and bool((o[lead + 33 * 101:] == 7.0).all())


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-8, 1e8, 1e30, 3e38])
def test_any_size_of_numbers(scale):
    """The result does not change with G's scale, from subnormal numbers to those
    whose squares overflow."""
    note(f"ortho scale {scale}")
    g = ref.gradient(60, 90, 2, "full", FP, "cuda")
    g = (g / g.abs().max()).double() * scale
    g = g.float()
    check(g, tide.ortho(g), scale)


def test_zeros_and_matrices_that_are_not_finite():
    note("ortho zeros, NaN, inf")
    z = torch.zeros(70, 200, device="cuda")
    ok = ref.gradient(70, 200, 1, "heavy", FP, "cuda")
    nan, inf = ok.clone(), ok.clone()
    nan[3, 5], inf[69, 199] = float("nan"), float("-inf")
    one = torch.zeros(70, 200, device="cuda")
    one[4, 8] = -3.0                                   # of rank 1, in one entry
    outs = tide.ortho([z, nan, ok, inf, one])
    assert not bool(outs[0].any())
    assert bool(torch.isnan(outs[1]).all()) and bool(torch.isnan(outs[3]).all())
    check(ok, outs[2], "beside NaNs")
    check(one, outs[4], "one entry")
    assert int((outs[4] != 0).sum()) == 1


@pytest.mark.parametrize("rank", [1, 4, 30])
def test_low_ranks(rank):
    note(f"ortho rank {rank}")
    gen = torch.Generator().manual_seed(rank)
    g = torch.randn(300, rank, generator=gen) @ torch.randn(rank, 420, generator=gen)
    for dtype in (BF, FP):
        m = g.to(dtype).cuda()
        check(m, tide.ortho(m), (rank, dtype))


@pytest.mark.parametrize("coefficients,steps", [
    ((1.5, -0.5, 0.0), 12),
    ([(8.2, -22.0, 16.0), (4.1, -2.95, 0.55), (3.95, -2.9, 0.55), (3.3, -2.5, 0.51)], 4),
    ((3.4445, -4.7750, 2.0315), 1),
    ((1.0, 0.0, 0.0), 2),
])
def test_other_steps(coefficients, steps):
    note(f"ortho coefficients {coefficients}")
    for shape in ((70, 150), (150, 70), (290, 300)):
        g = ref.gradient(*shape, 3, "full", FP, "cuda")
        check(g, tide.ortho(g, steps=steps, coefficients=coefficients), shape, coefficients, steps)


def test_what_leaves_the_range_is_not_finite():
    """Coefficients under which the singular values grow without end."""
    note("ortho out of range")
    g = ref.gradient(64, 64, 3, "full", FP, "cuda")
    assert not bool(torch.isfinite(tide.ortho(g, steps=6, coefficients=(30.0, 0.0, 0.0))).any())


def test_in_place_and_from_one_another():
    note("ortho in place")
    a, b = (ref.gradient(90, 140, s, "heavy", BF, "cuda") for s in (1, 2))
    want = [tide.ortho(a), tide.ortho(b)]
    x = a.clone()
    assert tide.ortho(x, out=x) is x and torch.equal(x, want[0])
    x, y = a.clone(), b.clone()
    tide.ortho([x, y], out=[y, x])                     # every src is read before any out is written
    assert torch.equal(y, want[0]) and torch.equal(x, want[1])
    u, v = tide.ortho([a, a])                          # the same matrix twice
    assert torch.equal(u, want[0]) and torch.equal(v, want[0])
    with pytest.raises(tide.TideError, match="overlaps another"):
        tide.ortho([a, b], out=[x, x])


def test_same_call_same_bits_on_two_streams():
    note("ortho repeated, two streams")
    gs = [[ref.gradient(300, 700, 1, "heavy", BF, "cuda"), ref.gradient(40, 30, 2, "heavy", BF, "cuda")],
          [ref.gradient(256, 640, 3, "heavy", BF, "cuda")]]
    want = [tide.ortho(g) for g in gs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in gs], []
    for _ in range(4):
        for s, g in zip(streams, gs):
            with torch.cuda.stream(s):
                got.append(tide.ortho(g))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i % 2]))


def test_captured():
    """Two graphs, each with its own workspace; replays between eager calls."""
    note("ortho captured")
    shapes = [(130, 70), (70, 130), (20, 20)]
    ins = [[torch.empty(s, dtype=BF, device="cuda") for s in shapes] for _ in range(2)]
    for k, xs in enumerate(ins):
        for x, s in zip(xs, shapes):
            x.copy_(ref.gradient(*s, k, "heavy", BF))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graphs, outs = [], []
    for xs in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(tide.ortho(xs))
        graphs.append(g)
    for it in range(3):
        for k, xs in enumerate(ins):
            for x, s in zip(xs, shapes):
                x.copy_(ref.gradient(*s, 10 + 2 * it + k, "heavy", BF))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for xs, os in zip(ins, outs):
            assert all(torch.equal(a, b) for a, b in zip(os, tide.ortho(xs)))


def test_workspace_of_exactly_the_asked_size():
    """Nothing past the workspace's end is touched, whatever it held before."""
    note("ortho workspace")
    L = lib()
    gs = [ref.gradient(*s, i, "heavy", BF, "cuda") for i, s in enumerate([(65, 129), (200, 40)])]
    want = tide.ortho(gs)
    rows, cols = (ctypes.c_int64 * 2)(65, 200), (ctypes.c_int64 * 2)(129, 40)
    size = L.tide_ortho_workspace(2, rows, cols)
    for fill in (0, 0xff):
        buf = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(g) for g in gs]
        co = (ctypes.c_float * 15)(*(ref.QUINTIC * 5))
        ptrs = lambda ts: (ctypes.c_void_p * 2)(*[t.data_ptr() for t in ts])  # noqa: E731
        st = L.tide_ortho(2, ptrs(gs), ptrs(outs), rows, cols, 5, co, 0,
                          ctypes.c_void_p(buf.data_ptr()), size,
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert bool((buf[size:] == fill).all())


def test_custom_op():
    note("ortho custom op")
    gs = [ref.gradient(40, 90, 1, "heavy", BF, "cuda"), ref.gradient(90, 40, 2, "heavy", BF, "cuda")]

    def step(g, out):
        torch.ops.tide.ortho(g, out, 5, list(ref.QUINTIC))
        return out[0].float() * 2

    want = tide.ortho(gs)
    assert tops is not None
    for fn in (step, torch.compile(step, backend="aot_eager", fullgraph=True)):
        outs = [torch.zeros_like(g) for g in gs]
        y = fn(gs, outs)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert torch.equal(y, want[0].float() * 2)


UNIT = [(96, 200), (200,), (200, 96), (33, 70), (2, 3, 5)]


def _unit(world, seed=70, **kw):
    from parameter_layout_collectives_amd.fsdp import TideUnit
    full = [ref.gradient(s[0], max(1, torch.Size(s).numel() // s[0]), seed + i, "full", FP, "cuda")
            .mul(50).view(s) for i, s in enumerate(UNIT)]
    unit = TideUnit(UNIT, world, **kw)
    unit.load(full)
    return unit, full


@pytest.mark.parametrize("world", [1, 3, 8])
@pytest.mark.parametrize("nesterov", [False, True])
def test_muon_step_of_a_unit(world, nesterov):
    """Two steps as they would be used - reduce-scatter, muon_step, gather - against
    the formula in 64 bits over the whole matrices."""
    note(f"TideUnit.muon_step world={world} nesterov={nesterov}")
    unit, full = _unit(world)
    lr, mu, wd = 0.02, 0.9, 0.1
    want = [f.double() for f in full]
    buf = [torch.zeros_like(w) for w in want]
    for step in range(2):
        grads = [[ref.gradient(s[0], max(1, torch.Size(s).numel() // s[0]), 100 * step + 10 * r + i,
                               "heavy", BF, "cuda").view(s) for i, s in enumerate(UNIT)]
                 for r in range(world)]
        unit.reduce_scatter(grads)
        unit.muon_step(lr, mu, nesterov, wd)
        for i, s in enumerate(UNIT):
            if len(s) != 2:
                continue
            g = sum(gr[i].double() for gr in grads) / world
            buf[i] = mu * buf[i] + g
            u = (g + mu * buf[i] if nesterov else buf[i]).float().to(BF)
            o = ref.exact(u)
            k = max(1.0, s[0] / s[1]) ** 0.5
            want[i] = (1 - lr * wd) * want[i] - lr * k * o
    unit.all_gather()
    for i, s in enumerate(UNIT):
        off, c, seg = unit.plan.param(i)
        inner = torch.Size(s).numel() // s[0]
        got = unit.master[:, off:off + seg].reshape(-1, inner)[:s[0]].reshape(s)
        if len(s) != 2:
            assert torch.equal(got, full[i])
            continue
        # two updates of O, each off by TOL and (a step in u's rounding) as much again
        o_norm = float((want[i] - full[i].double()).norm())
        assert float((got.double() - want[i]).norm()) <= 4 * TOL * o_norm
        assert torch.equal(unit.params[i], got.to(BF))
        pad = unit.master[:, off:off + seg].reshape(-1, inner)[s[0]:]
        assert not bool(pad.any())


def test_muon_step_of_chosen_parameters():
    note("TideUnit.muon_step select, scale")
    unit, full = _unit(2)
    unit.grad.copy_(torch.randn(unit.grad.shape, generator=torch.Generator().manual_seed(1)))
    before = unit.master.clone()
    unit.muon_step(0.1, select=[4, 0], scale=lambda r, c: 0.5, nesterov=False, momentum=0.0)
    for i in range(len(UNIT)):
        off, _, seg = unit.plan.param(i)
        moved = not torch.equal(unit.master[:, off:off + seg], before[:, off:off + seg])
        assert moved == (i in (0, 4))
    off, c, seg = unit.plan.param(4)                   # [2, 3, 5] is taken as [2, 15]
    g = unit.grad[:, off:off + seg].reshape(2, 15).to(BF)
    delta = (before - unit.master)[:, off:off + seg].reshape(2, 15)
    assert ref.off(delta, 0.05 * ref.exact(g)) <= 2 * TOL
    with pytest.raises(ValueError, match="earlier steps"):
        unit.muon_step(0.1, select=[0])
    unit.muon_step(0.1, select=[])                     # nothing to do
