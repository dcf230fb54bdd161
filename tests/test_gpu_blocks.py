"""8-bit blocks on the GPU: the format, the checkpoint, the gather and the
products against 64-bit references (blocks_ref.py)."""
import pytest
import torch

import blocks_ref as ref
import parameter_layout_collectives_amd as tide
from gpu_helpers import note

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def rand(shape, seed, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * scale
    # channels of very different size, so that blocks get different exponents
    return (x * torch.exp(1.5 * torch.randn(shape[-1], generator=g, device="cuda"))).to(dtype)


def bytes_of(q):
    return q.codes.view(torch.uint8).cpu(), q.scales.view(torch.uint8).cpu()


def filled(rows, cols, byte=0xa5):
    """Blocks whose memory holds a pattern, between guards on both sides."""
    cp, sp = -(-cols // 128) * 128, -(-cols // 512) * 4
    c = torch.full((rows * cp + 64,), byte, dtype=torch.uint8, device="cuda")
    s = torch.full((rows * sp + 64,), byte, dtype=torch.uint8, device="cuda")
    q = tide.Blocks(c[32:32 + rows * cp].view(rows, cp), s[32:32 + rows * sp].view(rows, sp), cols)
    return q, c, s


def guards_whole(buf, byte=0xa5):
    return bool((buf[:32] == byte).all()) and bool((buf[-32:] == byte).all())


SHAPES = [(1, 1), (1, 127), (3, 128), (5, 129), (2, 1000), (33, 513), (7, 4097), (130, 2048)]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", SHAPES)
def test_quant_is_the_definition(shape, dtype):
    note(f"block_quant {shape} {dtype}")
    x = rand(shape, 1, dtype)
    q, c, s = filled(*shape)
    tide.block_quant(x, out=q)
    want = ref.quant(x)
    got = bytes_of(q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert guards_whole(c) and guards_whole(s)


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_quant_of_any_alignment(shift, dtype):
    note(f"block_quant at element {shift} {dtype}")
    base = rand((1, 9 * 264 + 8), 2, dtype).view(-1)
    x = base[shift:shift + 9 * 264].view(9, 264)
    want = ref.quant(x)
    got = bytes_of(tide.block_quant(x))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def special_rows():
    """Rows of 256: the borders of the exponent rule, ties, the ends of the
    range, zeros, subnormals, and infinities and NaNs among finite values."""
    inf, nan = float("inf"), float("nan")
    rows = []
    for top in (448.0, 449.0, 447.0, 2.0 ** 100, 448 * 2.0 ** 119, 3.3e38, 2.0 ** -126, 1e-45,
                2.0 ** -109, 448 * 2.0 ** -117, 1.75, 1.7500001, 0.0):
        r = [top * f for f in (1.0, -0.5, 0.03125, 0.0009765625, 1e-3)]
        rows.append((r + [0.0, -0.0] * 128)[:128] + [1.0, -1.0] * 64)
    # every e4m3 number, every midpoint between two, and their neighbours
    t = ref.e4m3_table()[:127]
    mids = (t[1:] + t[:-1]) / 2
    ties = torch.cat([t, mids, mids * (1 + 2 ** -20), mids * (1 - 2 ** -20)])
    for k in range(0, len(ties), 127):
        part = ties[k:k + 127].tolist()
        rows.append([448.0] + part + [0.0] * (127 - len(part)) + [-v for v in part]
                    + [0.0] * (128 - len(part)))
    rows.append([inf, -inf, nan, 3.0] + [0.125] * 124 + [nan] * 128)
    rows.append([inf] * 128 + [0.0] * 127 + [-inf])
    return torch.tensor(rows, dtype=torch.float64).float()


@pytest.mark.parametrize("dtype", [FP, BF, HF])
def test_quant_of_special_values(dtype):
    note(f"block_quant special values {dtype}")
    x = special_rows().to(dtype).cuda()
    q = tide.block_quant(x)
    want = ref.quant(x)
    got = bytes_of(q)
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0], want[0])
    back = tide.block_dequant(q, dtype=FP).double()
    exact = ref.values(q.codes, q.scales, 256)
    assert torch.equal(torch.isnan(back), torch.isnan(exact))
    assert torch.equal(back.nan_to_num(0), exact.nan_to_num(0))
    assert torch.equal(torch.isnan(back), ~torch.isfinite(x))


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_dequant_of_every_code_and_scale(dtype):
    note(f"block_dequant all codes {dtype}")
    scales = list(range(10, 247, 4)) + [127, 246]
    codes = torch.arange(256, device="cuda").to(torch.uint8).repeat(len(scales), 1)
    sc = torch.full((len(scales), 4), 127, dtype=torch.uint8, device="cuda")
    sc[:, 0] = sc[:, 1] = torch.tensor(scales, dtype=torch.uint8)
    want = ref.values(codes, sc, 256)
    got = tide.block_dequant(tide.Blocks(codes, sc, 256), dtype=dtype)
    # bf16 and fp32 hold every value; fp16 rounds it once
    want = want.to(dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", SHAPES)
def test_dequant_writes_its_matrix_only(shape, dtype):
    note(f"block_dequant {shape} {dtype}")
    q = tide.block_quant(rand(shape, 3))
    n = shape[0] * shape[1]
    for lead in (32, 33):                           # aligned and not
        buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
        tide.block_dequant(q, out=buf[lead:lead + n].view(shape))
        want = ref.values(q.codes, q.scales, shape[1]).to(dtype)
        assert torch.equal(buf[lead:lead + n].view(shape), want)
        assert bool((buf[:lead] == 7.0).all()) and bool((buf[lead + n:] == 7.0).all())


UNITS = [([(5, 7), (16,), (33, 4)], 4, [0, 2]),
         ([(333, 1000), (37, 129), (64, 64)], 6, None),
         ([(9, 260), (3, 640)], 16, None),          # more ranks than rows
         ([(128, 512), (1, 1), (0, 5), (7, 0)], 3, None),
         ([(2, 130)] * 70, 2, None),                # more matrices than a wave has lanes
         ([(1 + i % 4, 120 + i) for i in range(250)], 3, None),   # more than one launch takes
         ([(5, 7)] + [(3, 130), (3, 130), (4, 65)] * 60, 3, None),   # ... that repeat in threes
         ([(2, 130)] * 150 + [(0, 5)] + [(9, 260)] * 4 + [(1, 1)], 5, None),
         ([(7, 20)] + [(6, 136), (6, 136)] * 100, 2, [0, 1, 2, 5] + list(range(8, 190)))]


def shards(shapes, world, seed):
    """Full fp32 matrices and the master shards [world, S] tide_pack makes of them."""
    plan = tide.Plan(shapes, world)
    full = [rand((s[0], s[1]) if len(s) == 2 else (1, s[0]), seed + i, FP).view(s) if
            all(s) else torch.zeros(s, device="cuda") for i, s in enumerate(shapes)]
    master = torch.zeros(world, plan.S, device="cuda")
    if plan.S:
        tide.pack(plan, full, master.view(-1))
    return plan, full, master


@pytest.mark.parametrize("unit", range(len(UNITS)))
def test_gather_in_blocks(unit):
    shapes, world, select = UNITS[unit]
    note(f"block gather unit {unit}")
    plan, full, master = shards(shapes, world, 50)
    bp = tide.BlockPlan(plan, select)
    gathered = bp.empty()
    for r in range(world):
        tide.block_shard(bp, r, master[r], gathered[r])
    weights = bp.blocks()
    tide.ag(bp, gathered, bp.views(weights))
    for dtype in (BF, FP):
        params = [torch.full(m, 7.0, dtype=dtype, device="cuda") for m in bp.matrices]
        tide.block_unshard(bp, gathered, params)
        for j, i in enumerate(bp.select):
            m = full[i].reshape(bp.matrices[j])
            if m.numel() == 0:
                continue
            want = ref.quant(m)
            got = bytes_of(weights[j])
            assert torch.equal(got[0], want[0]), (i, "codes")
            assert torch.equal(got[1], want[1]), (i, "scales")
            assert torch.equal(params[j].double().cpu(), ref.values(*want, m.shape[1])), i


@pytest.mark.parametrize("lead", [0, 1, 8])
@pytest.mark.parametrize("gap", [0, 3])
def test_many_matrices_of_one_tensor(lead, gap):
    """Parameters at fixed distances: experts that are views of one tensor; the
    elements between them stay."""
    note(f"block gather of views, lead {lead}, gap {gap}")
    shapes, world = [(3, 40)] + [(4, 136), (3, 130)] * 70 + [(2, 136)], 3
    plan, full, master = shards(shapes, world, 90)
    bp = tide.BlockPlan(plan)
    gathered = bp.empty()
    for r in range(world):
        tide.block_shard(bp, r, master[r], gathered[r])
    flat = torch.full((lead + sum(a * b + gap for a, b in shapes) + 8,), 7.0, dtype=BF, device="cuda")
    want = flat.cpu()
    params, at = [], lead
    for (a, b), f in zip(shapes, full):
        params.append(flat[at:at + a * b].view(a, b))
        want[at:at + a * b] = ref.values(*ref.quant(f), b).to(BF).view(-1)
        at += a * b + gap
    tide.block_unshard(bp, gathered, params)
    assert torch.equal(flat.cpu(), want)


def test_shard_pads_missing_rows_with_zeros():
    note("block_shard padding rows")
    plan, full, master = shards([(5, 200)], 4, 60)     # 2 rows a rank: rank 2 has 1, rank 3 none
    master.fill_(float("nan"))                         # padding must not be read
    live = [2, 2, 1, 0]
    for r in range(4):
        master[r, :live[r] * 200] = full[0].view(-1)[r * 400:r * 400 + live[r] * 200]
    bp = tide.BlockPlan(plan)
    for r in range(4):
        block = torch.full((bp.S,), -1, dtype=torch.int32, device="cuda")
        tide.block_shard(bp, r, master[r], block)
        codes = block.view(torch.uint8)[:2 * 256].view(2, 256)
        off = bp.param(1)[0] * 4
        scales = block.view(torch.uint8)[off:off + 8].view(2, 4)
        assert not bool(codes[live[r]:].any())
        assert bool((scales[live[r]:] == 127).all())
        if live[r]:
            want = ref.quant(master[r, :live[r] * 200].view(live[r], 200))
            assert torch.equal(codes[:live[r]].cpu(), want[0])
            assert torch.equal(scales[:live[r]].cpu(), want[1])


@pytest.mark.parametrize("dtype", [BF, torch.float16, FP])
@pytest.mark.parametrize("lead", [1, 3])
def test_x_that_starts_anywhere(dtype, lead):
    """The same blocks and products whatever x's alignment, for rows of whole
    vectors and others, made in one kernel (few rows) and in two."""
    note(f"x at element {lead}, {dtype}")
    w = tide.block_quant(rand((40, 264), 95))
    for rows, cols in ((1, 264), (3, 264), (70, 264), (5, 261), (70, 135)):
        x = rand((rows, cols), 96).to(dtype)
        buf = torch.full((lead + rows * cols + 8,), float("nan"), dtype=dtype, device="cuda")
        moved = buf[lead:lead + rows * cols].view(rows, cols)
        moved.copy_(x)
        assert all(torch.equal(a, b) for a, b in zip(bytes_of(tide.block_quant(moved)),
                                                     bytes_of(tide.block_quant(x))))
        if cols == w.cols:
            assert torch.equal(tide.block_linear(moved, w), tide.block_linear(x, w))


def test_unaligned_master_and_params():
    note("block gather unaligned")
    shapes, world = [(6, 136), (5, 136)], 2
    plan, full, master = shards(shapes, world, 70)
    bp = tide.BlockPlan(plan)
    gathered = bp.empty()
    for r in range(world):
        buf = torch.zeros(plan.S + 1, device="cuda")
        buf[1:] = master[r]
        tide.block_shard(bp, r, buf[1:], gathered[r])
    flat = torch.full((11 * 136 + 3,), 7.0, dtype=BF, device="cuda")
    params = [flat[1:1 + 6 * 136].view(6, 136), flat[1 + 6 * 136:1 + 11 * 136].view(5, 136)]
    tide.block_unshard(bp, gathered, params)
    for p, f in zip(params, full):
        assert torch.equal(p.double().cpu(), ref.values(*ref.quant(f), 136))
    assert float(flat[0]) == 7.0 and bool((flat[-2:] == 7.0).all())


# ------------------------------------------------------------------- products

def operands(m, n, k, seed):
    x = tide.block_quant(rand((m, k), seed)) if m * k else tide.Blocks.empty(m, k)
    w = tide.block_quant(rand((n, k), seed + 1, FP, 0.02)) if n * k else tide.Blocks.empty(n, k)
    dy = rand((m, n), seed + 2, BF, 1e-3)
    return x, w, dy


def guarded(shape, dtype):
    n = shape[0] * shape[1]
    buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
    return buf, buf[32:32 + n].view(shape)


def check_guards(buf):
    assert bool((buf[:32] == 7.0).all()) and bool((buf[-32:] == 7.0).all())


def check_products(m, n, k, seed=100):
    note(f"block products m={m} n={n} k={k}")
    x, w, dy = operands(m, n, k, seed)
    xv, wv = ref.values(x.codes, x.scales, k), ref.values(w.codes, w.scales, k)
    dv = dy.double()
    cases = [("mm", lambda o: tide.block_mm(x, w, out=o), (m, n), ref.product(xv, wv), k),
             ("dx", lambda o: tide.block_mm_dx(dy, w, out=o), (m, k),
              ref.product(dv, wv.t().contiguous()), n),
             ("dw", lambda o: tide.block_mm_dw(dy, x, out=o), (n, k),
              ref.product(dv.t().contiguous(), xv.t().contiguous()), m)]
    for name, call, shape, (want, mass), terms in cases:
        for dtype in (BF, FP):
            buf, out = guarded(shape, dtype)
            call(out)
            fast = name == "mm" and dtype == BF
            worst = ref.off(out, want, mass, terms, fast)
            assert worst <= 1.0, (name, dtype, worst)
            check_guards(buf)


@pytest.mark.parametrize("m", [1, 2, 16, 17, 33, 64, 65, 127, 129, 300])
def test_products_over_rows(m):
    check_products(m, 200, 328)


@pytest.mark.parametrize("n", [1, 3, 8, 63, 64, 65, 130, 257, 512])
def test_products_over_outputs(n):
    check_products(70, n, 264)


@pytest.mark.parametrize("k", [1, 7, 127, 128, 129, 511, 512, 513, 1111, 2048])
def test_products_over_inputs(k):
    check_products(66, 72, k)


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 5000, 300), (5000, 1, 300), (300, 300, 5000),
                                   (777, 1000, 1111), (512, 768, 2048), (2, 14336, 4096),
                                   (4100, 260, 130)])
def test_products_of_many_shapes(shape):
    check_products(*shape)


def test_products_over_large_tiles():
    """Enough output for the large tiles of every product, none of it a whole
    number of tiles."""
    check_products(4000, 4104, 3600)


@pytest.mark.parametrize("shape", [(4400, 4200, 4250), (4200, 4400, 2200)])
def test_products_of_tiles_left_over(shape):
    """Whole sets of tiles and some left over, whose sums are cut."""
    check_products(*shape)


def test_accumulate_over_tiles_left_over():
    note("block_mm_dw accumulate, tiles left over")
    m, n, k = 2100, 4400, 4200
    x, _, dy = operands(m, n, k, 7)
    old = rand((n, k), 8, FP, 1e-2)
    out = old.clone()
    tide.block_mm_dw(dy, x, out=out, accumulate=True)
    want, mass = ref.product(dy.double().t().contiguous(),
                             ref.values(x.codes, x.scales, k).t().contiguous())
    assert ref.off(out, want + old.double(), mass + old.double().abs(), m + 1) <= 1.0


def test_products_without_elements():
    note("block products of empty operands")
    x, w, dy = operands(5, 7, 0, 1)
    assert not bool(tide.block_mm(x, w).any())                    # an empty sum
    assert tide.block_mm_dx(dy, w).shape == (5, 0)
    x, w, dy = operands(0, 7, 130, 1)
    assert tide.block_mm(x, w).shape == (0, 7)
    old = torch.ones(7, 130, dtype=FP, device="cuda")
    assert torch.equal(tide.block_mm_dw(dy, x, out=old, accumulate=True), torch.ones_like(old))
    assert not bool(tide.block_mm_dw(dy, x, out=old).any())
    x, w, dy = operands(5, 0, 130, 1)
    assert tide.block_mm(x, w).shape == (5, 0)
    assert not bool(tide.block_mm_dx(dy, w).any())


@pytest.mark.parametrize("shape", [(66, 72, 130), (2000, 40, 136), (600, 768, 2048)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_accumulate(shape, dtype):
    m, n, k = shape
    note(f"block_mm_dw accumulate {shape} {dtype}")
    x, _, dy = operands(m, n, k, 7)
    old = rand((n, k), 8, dtype, 1e-2)
    buf, out = guarded((n, k), dtype)
    out.copy_(old)
    tide.block_mm_dw(dy, x, out=out, accumulate=True)
    want, mass = ref.product(dy.double().t().contiguous(),
                             ref.values(x.codes, x.scales, k).t().contiguous())
    # one more term in the sum: what was there
    assert ref.off(out, want + old.double(), mass + old.double().abs(), m + 1) <= 1.0
    check_guards(buf)


def test_without_workspace_the_sum_is_not_cut():
    note("block products without workspace")
    from parameter_layout_collectives_amd._lib import lib
    import ctypes
    m, n, k = 100, 64, 4096
    x, w, dy = operands(m, n, k, 9)
    assert lib().tide_block_workspace(0, m, n, k, 0) > 0
    out = torch.empty(m, n, device="cuda")
    st = lib().tide_block_mm(*x._ptrs, m, *w._ptrs, n, k, ctypes.c_void_p(out.data_ptr()), 0, None,
                             0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    want, mass = ref.product(ref.values(x.codes, x.scales, k), ref.values(w.codes, w.scales, k))
    assert ref.off(out, want, mass, k) <= 1.0


@pytest.mark.parametrize("m", [9, 200])
def test_a_nan_stays_in_its_row(m):
    """A NaN in one row of x makes that row of y NaN and no other; one in dy its
    row of dx and its column's row of dw."""
    note(f"block products NaN {m}")
    n, k = 136, 392
    xr = rand((m, k), 11)
    xr[4, 300] = float("inf")
    x, w = tide.block_quant(xr), tide.block_quant(rand((n, k), 12))
    for dtype in (BF, FP):
        bad = torch.isnan(tide.block_mm(x, w, dtype=dtype))
        assert bool(bad[4].all()) and int(bad.sum()) == n
    dy = rand((m, n), 13)
    dy[m - 1, n - 1] = float("nan")
    x = tide.block_quant(rand((m, k), 14))
    bad = torch.isnan(tide.block_mm_dx(dy, w))
    assert bool(bad[m - 1].all()) and int(bad.sum()) == k
    bad = torch.isnan(tide.block_mm_dw(dy, x))
    assert bool(bad[n - 1].all()) and int(bad.sum()) == k


@pytest.mark.parametrize("m", [3, 130])
def test_zero_codes_times_what_lies_beyond(m):
    """Rows and columns past the operands' ends never enter a sum, whatever
    the memory there holds: operands lie between NaNs."""
    note(f"block products between NaNs {m}")
    n, k = 40, 200
    x, w, dy = operands(m, n, k, 15)

    def between(q):
        g, c, s = filled(q.rows, q.cols, 0x7f)
        g.codes.copy_(q.codes.view(torch.uint8))
        g.scales.copy_(q.scales)
        return g
    x2, w2 = between(x), between(w)
    buf = torch.full((m * n + 64,), float("nan"), dtype=BF, device="cuda")
    dy2 = buf[32:32 + m * n].view(m, n)
    dy2.copy_(dy)
    for dtype in (BF, FP):
        assert torch.equal(tide.block_mm(x2, w2, dtype=dtype), tide.block_mm(x, w, dtype=dtype))
    assert torch.equal(tide.block_mm_dx(dy2, w2), tide.block_mm_dx(dy, w))
    assert torch.equal(tide.block_mm_dw(dy2, x2), tide.block_mm_dw(dy, x))


@pytest.mark.parametrize("shape", [(50, 61, 131), (130, 200, 260)])
def test_odd_dy_alignment(shape):
    m, n, k = shape
    note(f"block products dy unaligned {shape}")
    x, w, _ = operands(m, n, k, 17)
    base = rand((1, m * n + 1), 18, BF, 1e-3).view(-1)
    dy = base[1:].view(m, n)
    wv, xv, dv = ref.values(w.codes, w.scales, k), ref.values(x.codes, x.scales, k), dy.double()
    want, mass = ref.product(dv, wv.t().contiguous())
    assert ref.off(tide.block_mm_dx(dy, w), want, mass, n) <= 1.0
    want, mass = ref.product(dv.t().contiguous(), xv.t().contiguous())
    assert ref.off(tide.block_mm_dw(dy, x), want, mass, m) <= 1.0


def test_same_call_same_bits():
    note("block products repeated")
    x, w, dy = operands(500, 300, 2000, 19)
    a = [tide.block_mm(x, w), tide.block_mm(x, w, dtype=FP), tide.block_mm_dx(dy, w),
         tide.block_mm_dw(dy, x)]
    for _ in range(3):
        b = [tide.block_mm(x, w), tide.block_mm(x, w, dtype=FP), tide.block_mm_dx(dy, w),
             tide.block_mm_dw(dy, x)]
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_on_two_streams_at_once():
    """The calls share nothing: two streams' products run side by side."""
    note("block products on two streams")
    sets = [operands(300, 200, 3000, 20 + 5 * i) for i in range(2)]
    want = [(tide.block_mm(x, w), tide.block_mm_dw(dy, x)) for x, w, dy in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(4):
        for st, (x, w, dy) in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append((tide.block_mm(x, w), tide.block_mm_dw(dy, x)))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1])


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 72, 4096), (1, 33, 28672), (3, 200, 1111),
                                   (16, 130, 2048), (16, 16, 2049), (17, 64, 700), (8, 100, 4097), (17, 40, 128), (64, 40, 100),
                                   (130, 200, 392), (600, 512, 1000)])
def test_linear_in_one_call(shape, dtype):
    """tide_block_linear equals tide_block_quant and tide_block_mm, bit for bit,
    from any alignment of x."""
    m, n, k = shape
    note(f"block_linear in one call {shape} {dtype}")
    w = tide.block_quant(rand((n, k), 22, FP, 0.02))
    base = rand((1, m * k + 1), 23, dtype).view(-1)
    for lead in (0, 1):
        x = base[lead:lead + m * k].view(m, k)
        for out in (BF, FP):
            got = tide.block_linear(x, w, dtype=out)
            assert torch.equal(got, tide.block_mm(tide.block_quant(x), w, dtype=out)), (lead, out)


def test_linear_in_one_call_of_special_values():
    note("block_linear special values")
    x = special_rows().to(BF).cuda()
    w = tide.block_quant(rand((24, 256), 24, FP, 0.02))
    for rows in (x[:16], x[-16:], x):
        rows = rows.contiguous()
        got, want = tide.block_linear(rows, w), tide.block_mm(tide.block_quant(rows), w)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


# ------------------------------------------------------------------- together

def linear_reference(xq, w, dy, k):
    xv, wv = ref.values(xq.codes, xq.scales, k), ref.values(w.codes, w.scales, k)
    return xv @ wv.t().contiguous(), dy.double() @ wv, dy.double().t().contiguous() @ xv


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("lead", [(40,), (3, 25), ()])
def test_linear_through_autograd(dtype, lead):
    note(f"block_linear {dtype} {lead}")
    n, k = 72, 264
    x = rand((*lead, k) if lead else (1, k), 30, dtype).view(*lead, k).requires_grad_()
    w = tide.block_quant(rand((n, k), 31, FP, 0.02))
    dw = torch.full((n, k), 7.0, device="cuda")
    y = tide.block_linear(x, w, grad=dw)
    assert y.shape == (*lead, n) and y.dtype == (FP if dtype == FP else BF)
    dy = rand((1, y.numel()), 32, BF, 1e-3).view(y.shape).to(y.dtype)
    y.backward(dy)
    x2, dy2 = x.detach().reshape(-1, k), dy.reshape(-1, n).to(BF)
    m = x2.shape[0]
    xq = tide.block_quant(x2)
    xv, wv = ref.values(xq.codes, xq.scales, k), ref.values(w.codes, w.scales, k)
    want, mass = ref.product(xv, wv)
    assert ref.off(y.detach().reshape(m, n), want, mass, k, fast=True) <= 1.0
    want, mass = ref.product(dy2.double(), wv.t().contiguous())
    assert x.grad.dtype == dtype
    # an fp16 gradient is rounded twice: to fp32 sums, then to fp16
    assert ref.off(x.grad.reshape(m, k), want, mass, n + 1) <= 1.0
    want, mass = ref.product(dy2.double().t().contiguous(), xv.t().contiguous())
    assert ref.off(dw, want, mass, m) <= 1.0


def test_linear_gradient_against_differences():
    """<dy, y(x + t d) - y(x - t d)> / 2t = <dx, d> for a layer whose x passes
    the rounding unchanged (x and d on the block's grid, so y is linear there)."""
    note("block_linear differences")
    m, n, k = 20, 64, 256
    g = torch.Generator(device="cuda").manual_seed(33)
    # whole numbers up to 8 in blocks that all hold one 256: 2^0 steps are exact
    x = torch.randint(-4, 5, (m, k), generator=g, device="cuda").float()
    x[:, ::128] = 256.0
    d = torch.randint(-1, 2, (m, k), generator=g, device="cuda").float()
    d[:, ::128] = 0.0
    w = tide.block_quant(rand((n, k), 34, FP, 0.02))
    dy = rand((m, n), 35, BF, 1.0).float()
    xl = x.clone().requires_grad_()
    dw = torch.empty(n, k, device="cuda")
    y = tide.block_linear(xl, w, grad=dw)
    dx, = torch.autograd.grad(y, xl, dy)
    wv = ref.values(w.codes, w.scales, k)

    def f(z):
        return tide.block_linear(z, w).double()
    with torch.no_grad():
        diff = (dy.double() * (f(x + d) - f(x - d)) / 2).sum()
    got = (dx.double() * d.double()).sum()
    # fp32 outputs: k products and sums of half a unit each, over m * n terms
    mass = (dy.double().abs() * ((x.abs() + d.abs()).double() @ wv.abs().t())).sum()
    mass += (d.double().abs() * (dy.double().abs() @ wv.abs())).sum()
    assert abs(float(diff - got)) <= float(mass) * k * 2.0 ** -23


def test_linear_with_frozen_parts():
    note("block_linear frozen parts")
    m, n, k = 33, 40, 130
    x = rand((m, k), 36)
    w = tide.block_quant(rand((n, k), 37, FP, 0.02))
    dy = rand((m, n), 38, BF, 1e-3)
    dw = torch.full((n, k), 7.0, device="cuda")
    tide.block_linear(x, w, grad=dw).backward(dy)             # x needs no gradient
    assert torch.equal(dw, tide.block_mm_dw(dy, tide.block_quant(x), dtype=FP))
    xl = x.clone().requires_grad_()
    tide.block_linear(xl, w).backward(dy)                     # frozen weights
    assert torch.equal(xl.grad, tide.block_mm_dx(dy, w))
    assert not tide.block_linear(x, w).requires_grad
    with torch.no_grad():
        assert not tide.block_linear(xl, w, grad=dw).requires_grad
    # a sum over two micro-batches, through a broadcast output gradient
    tide.block_linear(xl, w, grad=dw).sum().backward()
    tide.block_linear(xl, w, grad=dw, accumulate=True).sum().backward()
    ones = torch.ones(m, n, dtype=BF, device="cuda")
    once = tide.block_mm_dw(ones, tide.block_quant(x), dtype=FP)
    assert torch.equal(dw, once + once)


@pytest.mark.parametrize("m", [1, 130])
def test_captured_linear(m):
    """Forward and backward captured into two graphs with their own workspaces;
    replays with eager work between them equal the eager results."""
    note(f"block_linear captured {m}")
    n, k = 200, 2600
    w = tide.block_quant(rand((n, k), 40, FP, 0.02))
    xs = [torch.empty(m, k, dtype=BF, device="cuda") for _ in range(2)]
    dy = rand((m, n), 41, BF, 1e-3)
    outs, graphs = [], []

    def step(x):
        q = tide.block_quant(x)
        y = tide.block_mm(q, w)
        return y, tide.block_mm_dx(dy, w), tide.block_mm_dw(dy, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x in xs:
        x.copy_(rand((m, k), 42))
    torch.cuda.synchronize()
    for x in xs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(step(x))
        graphs.append(gr)
    for it in range(3):
        for i, x in enumerate(xs):
            x.copy_(rand((m, k), 50 + 2 * it + i))
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(xs):
            for got, want in zip(outs[i], step(x)):
                assert torch.equal(got, want)


def test_captured_backward_through_autograd():
    """Forward and backward through autograd in a graph, over a leaf that no live
    eager graph holds; eager passes over other leaves run between the replays."""
    note("block_linear autograd captured")
    m, n, k = 70, 96, 640
    w = tide.block_quant(rand((n, k), 43, FP, 0.02))
    dy = rand((m, n), 44, BF, 1e-3)
    x, dw = rand((m, k), 45), torch.zeros(n, k, device="cuda")

    def step(leaf, grad):
        y = tide.block_linear(leaf, w, grad=grad, accumulate=True)
        dx, = torch.autograd.grad(y, leaf, dy)
        return y.detach(), dx
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x.clone().requires_grad_(), torch.zeros_like(dw))    # one pass outside the capture
    torch.cuda.current_stream().wait_stream(side)
    leaf = x.clone().requires_grad_()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        y, dx = step(leaf, dw)
    total = torch.zeros_like(dw)
    dw.zero_()
    for it in range(3):
        new = rand((m, k), 46 + it)
        with torch.no_grad():
            leaf.copy_(new)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        want = step(new.clone().requires_grad_(), total)
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1]) and torch.equal(dw, total)


def test_custom_ops():
    import parameter_layout_collectives_amd.torch_ops as tops
    note("block custom ops")
    ops = torch.ops.tide
    m, n, k = 70, 48, 200
    x, wr, dy = rand((m, k), 60), rand((n, k), 61, FP, 0.02), rand((m, n), 62, BF, 1e-3)
    q, w = tide.Blocks.empty(m, k), tide.Blocks.empty(n, k)
    ops.block_quant(x, q.codes, q.scales)
    ops.block_quant(wr, w.codes, w.scales)
    y, dx = torch.empty(m, n, dtype=BF, device="cuda"), torch.empty(m, k, dtype=BF, device="cuda")
    dw, back = torch.zeros(n, k, device="cuda"), torch.empty(m, k, dtype=BF, device="cuda")
    ops.block_mm(q.codes, q.scales, w.codes, w.scales, k, y)
    ops.block_mm_dx(dy, w.codes, w.scales, dx)
    ops.block_mm_dw(dy, q.codes, q.scales, dw)
    ops.block_mm_dw(dy, q.codes, q.scales, dw, True)
    ops.block_dequant(q.codes, q.scales, back)
    once = tide.block_mm_dw(dy, q, dtype=FP)
    assert torch.equal(y, tide.block_mm(q, w)) and torch.equal(dx, tide.block_mm_dx(dy, w))
    assert torch.equal(dw, once + once) and torch.equal(back, tide.block_dequant(q))
    plan, full, master = shards([(9, 130), (4, 4)], 2, 63)
    pid = tops.register_plan(tide.BlockPlan(plan))
    try:
        bp = tops._PLANS[pid]
        gathered = bp.empty()
        for r in range(2):
            ops.block_shard(pid, r, master[r], gathered[r])
        params = [torch.empty(s, dtype=BF, device="cuda") for s in bp.matrices]
        ops.block_unshard(pid, gathered, params)
        for p, f in zip(params, full):
            assert torch.equal(p, tide.block_dequant(tide.block_quant(f)))
    finally:
        tops.unregister_plan(pid)


UNIT = [(96, 200), (200,), (200, 96), (40, 200)]


def unit_with_weights(world, blocks, seed=70):
    from parameter_layout_collectives_amd.fsdp import TideUnit
    full = [rand((1, s[0]) if len(s) == 1 else s, seed + i, FP, 0.05).view(s)
            for i, s in enumerate(UNIT)]
    unit = TideUnit(UNIT, world, blocks=blocks)
    unit.load(full)
    return unit, full


@pytest.mark.parametrize("world", [1, 3, 8])
@pytest.mark.parametrize("kw", [{}, {"small": True}, {"copy_engine": True}])
def test_unit_gathers_matrices_in_blocks(world, kw):
    note(f"TideUnit blocks world={world} {kw}")
    unit, full = unit_with_weights(world, [0, 2])
    unit.all_gather(**kw)
    torch.cuda.synchronize()
    for i, f in enumerate(full):
        if i in (0, 2):
            want = ref.quant(f)
            got = bytes_of(unit.params[i])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        else:
            assert torch.equal(unit.params[i], f.to(BF))
    every, _ = unit_with_weights(world, range(4))          # the vector as a column too
    assert torch.equal(tide.block_dequant(every.params[1], dtype=FP).view(-1),
                       tide.block_dequant(tide.block_quant(full[1].view(-1, 1)), dtype=FP).view(-1))
    with pytest.raises(ValueError):
        unit.linear(3, torch.empty(1, 200, device="cuda"))


def test_unit_trains_through_blocks():
    """A step of a two-layer unit as it would be used: gather in blocks on a side
    stream, forward and backward of every rank's micro-batch through linear(),
    reduce-scatter of the gradients, an update of the master shards, gather.
    Gradients are the formula's at the gathered weights, and the update is what
    the next gather holds."""
    note("TideUnit blocks training step")
    N, m = 4, 33
    unit, full = unit_with_weights(N, [0, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    unit.all_gather(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    w0, w2 = unit.params[0], unit.params[2]
    grads, want = [], []
    for r in range(N):
        g = [torch.zeros(s, device="cuda") for s in UNIT]
        x = rand((m, 200), 80 + r, BF, 0.5).requires_grad_()
        h = unit.linear(0, x, grad=g[0])
        a = torch.relu(h)
        y = unit.linear(2, a, grad=g[2], dtype=FP)
        dy = rand((m, 200), 90 + r, BF, 1e-2).float()
        y.backward(dy)
        grads.append(g)
        aq = tide.block_quant(a.detach())
        da = tide.block_mm_dx(dy.to(BF), w2)
        dh = da * (h.detach() > 0)
        assert torch.equal(x.grad, tide.block_mm_dx(dh, w0))
        want.append((tide.block_mm_dw(dh, tide.block_quant(x.detach()), dtype=FP),
                     tide.block_mm_dw(dy.to(BF), aq, dtype=FP)))
    for g, (d0, d2) in zip(grads, want):
        assert torch.equal(g[0], d0) and torch.equal(g[2], d2)
    unit.reduce_scatter(grads)
    unit.master -= 0.1 * unit.grad
    unit.all_gather()
    for i, k in ((0, 0), (2, 1)):
        total = want[0][k]
        for r in range(1, N):
            total = total + want[r][k]
        new = full[i] - 0.1 * (total / N)
        q = tide.block_quant(new)
        assert torch.equal(bytes_of(unit.params[i])[0], bytes_of(q)[0])
        assert torch.equal(bytes_of(unit.params[i])[1], bytes_of(q)[1])
