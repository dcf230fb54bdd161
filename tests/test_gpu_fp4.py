"""4-bit blocks on the GPU: the format, the gather and the products against 64-bit
references (fp4_ref.py).  Products' tolerances are blocks_ref.off's: exact products,
one unit of fp32 per addition, one rounding of the result."""
import ctypes

import pytest
import torch

import blocks_ref
import fp4_ref as ref
import parameter_layout_collectives_amd as tide
import parameter_layout_collectives_amd.torch_ops as tops
from gpu_helpers import note
from parameter_layout_collectives_amd._lib import lib
from test_gpu_blocks import UNITS, check_guards, guarded, rand, shards

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def bytes_of(q):
    return q.codes.view(torch.uint8).cpu(), q.scales.view(torch.uint8).cpu()


def filled(rows, cols, byte=0xa5):
    """4-bit blocks whose memory holds a pattern, between guards on both sides."""
    cp, sp = -(-cols // 128) * 64, -(-cols // 128) * 4
    c = torch.full((rows * cp + 64,), byte, dtype=torch.uint8, device="cuda")
    s = torch.full((rows * sp + 64,), byte, dtype=torch.uint8, device="cuda")
    q = tide.Fp4Blocks(c[32:32 + rows * cp].view(rows, cp), s[32:32 + rows * sp].view(rows, sp), cols)
    return q, c, s


def guards_whole(buf, byte=0xa5):
    return bool((buf[:32] == byte).all()) and bool((buf[-32:] == byte).all())


def val(q):
    return ref.values(q.codes, q.scales, q.cols)


# ------------------------------------------------------------------- the format

SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (3, 128), (5, 129), (2, 1000), (7, 513), (20, 300)]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", SHAPES)
def test_quant_is_the_definition(shape, dtype):
    note(f"fp4_quant {shape} {dtype}")
    x = rand(shape, 1, dtype)
    q, c, s = filled(*shape)
    assert tide.fp4_quant(x, out=q) is q
    got, want = bytes_of(q), ref.quant(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert guards_whole(c) and guards_whole(s)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("lead", [1, 3])
def test_x_that_starts_anywhere(dtype, lead):
    note(f"fp4_quant unaligned {dtype} {lead}")
    x = rand((9, 137), 2, dtype)
    flat = torch.zeros(9 * 137 + 8, dtype=dtype, device="cuda")
    view = flat[lead:lead + 9 * 137].view(9, 137)
    view.copy_(x)
    a, b = tide.fp4_quant(view), tide.fp4_quant(x)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_quant_of_special_values(dtype):
    """Every midpoint and its neighbours, both signs and zeros, under every exponent
    the type has; blocks at the border of an exponent; subnormal and largest numbers;
    infinities and NaNs, which take their block of 32 and no other."""
    note(f"fp4_quant special {dtype}")
    m = torch.tensor([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 0.1])
    info = torch.finfo(dtype)
    rows = []
    lowest = -14 - 10 if dtype == HF else -133 if dtype == BF else -149
    top = 15 if dtype == HF else 127
    for e in list(range(lowest, top - 2, 7)) + [top - 2, top - 3, lowest + 1]:
        v = m.double() * 2.0 ** e
        rows.append(torch.cat([v, -v]))
        rows.append(torch.cat([v * (1 - info.eps), -v * (1 + info.eps)]).clamp(-info.max, info.max))
    for a in (info.max, info.max / 2, info.tiny, info.smallest_normal * info.eps, 6.0, 6.0 * (1 + info.eps)):
        rows.append(torch.full((32,), float(a), dtype=torch.float64) * torch.linspace(-1, 1, 32).double())
    rows.append(torch.full((32,), -0.0, dtype=torch.float64))
    x = torch.stack(rows).to(dtype)
    x = torch.cat([x, x.flip(0), x], 1)[:, :90].contiguous()
    x[0, 5], x[1, 40], x[2, 89] = float("inf"), float("nan"), float("-inf")
    got, want = bytes_of(tide.fp4_quant(x.cuda())), ref.quant(x)
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0], want[0])
    back = tide.fp4_dequant(tide.fp4_quant(x.cuda()), dtype=FP).cpu()
    nan = torch.isnan(back)
    assert bool(nan[0, :32].all()) and bool(nan[1, 32:64].all()) and bool(nan[2, 64:].all())
    assert int(nan.sum()) == 32 + 32 + 26


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_dequant_of_every_code_and_scale(dtype):
    note(f"fp4_dequant all codes {dtype}")
    scales = torch.tensor(list(range(2, 253)) + [255], dtype=torch.uint8)
    codes = torch.arange(256, dtype=torch.uint8).repeat(len(scales), 1)       # 512 columns
    q = tide.Fp4Blocks(codes.cuda(), scales.view(-1, 1).repeat(1, 16).cuda(), 512)
    for cols in (512, 511, 385):
        q = tide.Fp4Blocks(codes[:, :-(-cols // 128) * 64].contiguous().cuda(),
                           scales.view(-1, 1).repeat(1, -(-cols // 128) * 4).contiguous().cuda(), cols)
        got = tide.fp4_dequant(q, dtype=dtype)
        want = val(q).to(dtype)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", [(3, 31), (5, 130), (2, 1001)])
def test_dequant_writes_its_matrix_only(shape, dtype):
    note(f"fp4_dequant guards {shape} {dtype}")
    q = tide.fp4_quant(rand(shape, 3, FP))
    n = shape[0] * shape[1]
    for lead in (1, 8):
        buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
        tide.fp4_dequant(q, out=buf[lead:lead + n].view(shape))
        assert torch.equal(buf[lead:lead + n].view(shape), val(q).to(dtype))
        assert bool((buf[:lead] == 7.0).all()) and bool((buf[lead + n:] == 7.0).all())


# ------------------------------------------------------------------- the gather

@pytest.mark.parametrize("unit", range(len(UNITS)))
def test_gather(unit):
    shapes, world, select = UNITS[unit]
    note(f"fp4 gather unit {unit}")
    plan, full, master = shards(shapes, world, 50)
    fp = tide.Fp4Plan(plan, select)
    gathered = fp.empty()
    for r in range(world):
        tide.fp4_shard(fp, r, master[r], gathered[r])
    weights = fp.blocks()
    tide.ag(fp, gathered, fp.views(weights))
    for dtype in (BF, HF, FP):
        params = [torch.full(m, 7.0, dtype=dtype, device="cuda") for m in fp.matrices]
        tide.fp4_unshard(fp, gathered, params)
        for j, i in enumerate(fp.select):
            m = full[i].reshape(fp.matrices[j])
            if m.numel() == 0:
                continue
            q = tide.fp4_quant(m)              # the definition's, by the tests above
            assert torch.equal(weights[j].codes, q.codes), (i, "codes")
            assert torch.equal(weights[j].scales, q.scales), (i, "scales")
            assert torch.equal(params[j], val(q).to(dtype)), i


def test_shard_pads_missing_rows_with_zeros():
    note("fp4_shard padding rows")
    plan, full, master = shards([(5, 200)], 4, 60)     # 2 rows a rank: rank 2 has 1, rank 3 none
    master.fill_(float("nan"))                         # padding must not be read
    live = [2, 2, 1, 0]
    for r in range(4):
        master[r, :live[r] * 200] = full[0].view(-1)[r * 400:r * 400 + live[r] * 200]
    fp = tide.Fp4Plan(plan)
    for r in range(4):
        block = torch.full((fp.S,), -1, dtype=torch.int32, device="cuda")
        tide.fp4_shard(fp, r, master[r], block)
        codes = block.view(torch.uint8)[:2 * 128].view(2, 128)
        off = fp.param(1)[0] * 4
        scales = block.view(torch.uint8)[off:off + 16].view(2, 8)
        assert not bool(codes[live[r]:].any())
        assert bool((scales[live[r]:] == 127).all())
        if live[r]:
            want = ref.quant(master[r, :live[r] * 200].view(live[r], 200))
            assert torch.equal(codes[:live[r]].cpu(), want[0])
            assert torch.equal(scales[:live[r]].cpu(), want[1])


# ------------------------------------------------------------------- products

def operands(m, n, k, seed):
    x = rand((m, k), seed)
    xq = tide.fp4_quant(x) if m * k else tide.Fp4Blocks.empty(m, k)
    w = tide.fp4_quant(rand((n, k), seed + 1, FP, 0.02)) if n * k else tide.Fp4Blocks.empty(n, k)
    return x, xq, w, rand((m, n), seed + 2, BF, 1e-3)


def linear(x, w, out, quant):
    out.copy_(tide.fp4_linear(x, w, dtype=out.dtype, quant_x=quant))


def check_products(m, n, k, seed=100):
    note(f"fp4 products m={m} n={n} k={k}")
    x, xq, w, dy = operands(m, n, k, seed)
    xv, wv = val(xq), val(w)
    four = blocks_ref.product(xv, wv)
    cases = [("mm", lambda o: tide.fp4_mm(xq, w, out=o), (m, n), four, k),
             ("linear", lambda o: linear(x, w, o, False), (m, n), blocks_ref.product(x.double(), wv), k),
             ("quant", lambda o: linear(x, w, o, True), (m, n), four, k),
             ("dx", lambda o: tide.fp4_mm_dx(dy, w, out=o), (m, k),
              blocks_ref.product(dy.double(), wv.t().contiguous()), n)]
    for name, call, shape, (want, mass), terms in cases:
        for dtype in (BF, FP):
            buf, out = guarded(shape, dtype)
            call(out)
            worst = blocks_ref.off(out, want, mass, terms)
            assert worst <= 1.0, (name, dtype, worst)
            check_guards(buf)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 127, 129, 300])
def test_products_over_rows(m):
    check_products(m, 72, 392)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 129, 300])
def test_products_over_outputs(n):
    check_products(70, n, 264)
    check_products(3, n, 264)


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 63, 65, 127, 128, 129, 255, 256, 257, 384, 511, 513, 640,
                               1000, 1280, 2049])
def test_products_over_inputs(k):
    check_products(70, 40, k)
    check_products(5, 40, k)


@pytest.mark.parametrize("shape", [(1, 14336, 4096), (16, 100, 28672), (1, 33, 30000), (4, 64, 7000),
                                   (200, 1000, 5000), (500, 300, 9000), (1500, 1510, 460),
                                   (2050, 2056, 1100), (777, 1001, 1111), (131, 201, 392),
                                   (100, 512, 8200), (130, 5000, 600)])
def test_products_of_many_shapes(shape):
    check_products(*shape)


@pytest.mark.parametrize("shape", [(4000, 4104, 1100), (4100, 1104, 4000), (4200, 4400, 2210),
                                   (250, 8200, 8200)])
def test_products_over_large_tiles(shape):
    check_products(*shape)


# one to 64 rows of x by matrices of 2^21 numbers and more: sums in one piece and in
# several, units of 128 columns that end inside a group, rows that end inside a strip
STRIPS = [(17, 2000, 1100), (1, 33000, 4100), (5, 20000, 4100), (16, 5000, 28700), (20, 1030, 2100),
          (33, 4099, 520), (48, 129, 20000), (64, 70, 30001), (32, 300, 7040), (32, 1300, 26000),
          (18, 33000, 1050), (9, 40000, 900)]


@pytest.mark.parametrize("shape", STRIPS)
def test_products_of_some_rows(shape):
    check_products(*shape)


@pytest.mark.parametrize("shape", STRIPS)
def test_some_rows_between_nans(shape):
    """Nothing past a row's end or a matrix' end enters a sum: rows in turn NaN."""
    note(f"fp4 some rows between NaNs {shape}")
    m, n, k = shape
    x, xq, w, _ = operands(m, n, k, 51)
    y, y4 = tide.fp4_linear(x, w, dtype=FP), tide.fp4_mm(xq, w, dtype=FP)
    c, s = w.codes.clone(), w.scales.clone()
    s[::2] = 255
    odd = tide.Fp4Blocks(c, s, k)
    for got, want in ((tide.fp4_linear(x, odd, dtype=FP), y), (tide.fp4_mm(xq, odd, dtype=FP), y4)):
        assert torch.equal(got[:, 1::2], want[:, 1::2])
        assert bool(torch.isnan(got[:, ::2]).all())
    x[m // 2, k - 1] = float("nan")
    bad = torch.isnan(tide.fp4_linear(x, w, dtype=FP))
    assert bool(bad[m // 2].all()) and int(bad.sum()) == n


def test_products_without_elements():
    note("fp4 products without elements")
    for m, n, k in [(0, 5, 40), (5, 0, 40), (5, 6, 0), (0, 0, 0), (40, 6, 0)]:
        x, xq, w, dy = operands(m, n, k, 5)
        assert tide.fp4_mm(xq, w).shape == (m, n) and not bool(tide.fp4_mm(xq, w).any())
        for quant in (False, True):
            y = tide.fp4_linear(x, w, quant_x=quant)
            assert y.shape == (m, n) and not bool(y.any())
        dx = tide.fp4_mm_dx(dy, w)
        assert dx.shape == (m, k) and not bool(dx.any())


@pytest.mark.parametrize("shape", [(40, 130, 1000), (300, 257, 5000), (2, 40, 700), (2, 33000, 4100),
                                   (40, 1030, 2100)])
def test_without_workspace(shape):
    """A call without workspace runs another way, where it can."""
    note(f"fp4 products without workspace {shape}")
    m, n, k = shape
    x, xq, w, dy = operands(m, n, k, 6)
    P, L = ctypes.c_void_p, lib()
    st = P(torch.cuda.current_stream().cuda_stream)
    out, dx = torch.empty(m, n, device="cuda"), torch.empty(m, k, device="cuda")
    wp, o = [P(p) for p in w._ptrs4], P(out.data_ptr())
    assert L.tide_mx_mm(*[P(p) for p in xq._ptrs4], m, *wp, n, k, o, 0, None, 0, st) == 0
    want, mass = blocks_ref.product(val(xq), val(w))
    assert blocks_ref.off(out, want, mass, k) <= 1.0
    assert L.tide_mx_linear(P(x.data_ptr()), m, k, *wp, n, o, 0, None, 0, st) == 0
    want, mass = blocks_ref.product(x.double(), val(w))
    assert blocks_ref.off(out, want, mass, k) <= 1.0
    assert L.tide_mx_mm_dx(P(dy.data_ptr()), m, n, *wp, k, P(dx.data_ptr()), 0, None, 0, st) == 0
    want, mass = blocks_ref.product(dy.double(), val(w).t().contiguous())
    assert blocks_ref.off(dx, want, mass, n) <= 1.0
    if m > 16:
        assert L.tide_mx_linear(P(x.data_ptr()), m, k, *wp, n, o, 0x200, None, 0, st) == 1
        assert b"workspace" in L.tide_last_error()


@pytest.mark.parametrize("shape", [(3, 40, 700), (40, 130, 1000), (300, 260, 520), (20, 40, 8200)])
def test_sums_are_held_in_fp32(shape):
    """Whole numbers whose sums stay below 2^24 come out exactly, in every kernel and
    beside products that cancel: blocks of 6 * 6 * 2^16 in pairs of opposite sign."""
    note(f"fp4 exact sums {shape}")
    m, n, k = shape
    gen = torch.Generator(device="cuda").manual_seed(9)
    def whole(r):
        t = torch.randint(0, 16, (r, -(-k // 128) * 128), generator=gen, device="cuda", dtype=torch.uint8)
        t[:, k:] = 0
        return t
    def pack(t, s):
        return tide.Fp4Blocks((t[:, 0::2] + 16 * t[:, 1::2]).contiguous(), s, k)
    a, b = whole(m), whole(n)
    sa = torch.full((m, a.shape[1] // 32), 128, dtype=torch.uint8, device="cuda")   # 2 * e2m1: whole
    sb = torch.full((n, b.shape[1] // 32), 128, dtype=torch.uint8, device="cuda")
    a[:, 5], b[:, 5], a[:, 37], b[:, 37] = 7, 7, 7, 15          # 6 * 6 and 6 * -6
    for t in (a, b):
        t[:, :5], t[:, 6:32], t[:, 32:37], t[:, 38:64] = 0, 0, 0, 0
    sa[:, :2] = 128 + 16
    x, w = pack(a, sa), pack(b, sb)
    want = val(x) @ val(w).t().contiguous()
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(tide.fp4_mm(x, w, dtype=FP).double(), want)
    xv = tide.fp4_dequant(x)
    assert torch.equal(tide.fp4_linear(xv, w, dtype=FP).double(), want)
    assert torch.equal(tide.fp4_linear(xv, w, dtype=FP, quant_x=True).double(), want)


@pytest.mark.parametrize("m", [3, 16, 130])
def test_a_nan_stays_where_it_is(m):
    """A NaN in x makes its row of y NaN, one in W its row of W a column of y and,
    through dX, the 32 columns of its block."""
    note(f"fp4 NaN {m}")
    n, k = 136, 392
    x = rand((m, k), 11)
    x[2, 300] = float("inf")
    wr = rand((n, k), 12)
    w = tide.fp4_quant(wr)
    for dtype in (BF, FP):
        for y in (tide.fp4_mm(tide.fp4_quant(x), w, dtype=dtype),
                  tide.fp4_linear(x, w, dtype=dtype, quant_x=True)):
            bad = torch.isnan(y)
            assert bool(bad[2].all()) and int(bad.sum()) == n
    wr[7, 33] = float("nan")
    w = tide.fp4_quant(wr)
    x = rand((m, k), 13)
    for y in (tide.fp4_mm(tide.fp4_quant(x), w), tide.fp4_linear(x, w),
              tide.fp4_linear(x, w, quant_x=True)):
        bad = torch.isnan(y)
        assert bool(bad[:, 7].all()) and int(bad.sum()) == m
    bad = torch.isnan(tide.fp4_mm_dx(rand((m, n), 14), w))
    assert bool(bad[:, 32:64].all()) and int(bad.sum()) == 32 * m


@pytest.mark.parametrize("shape", [(3, 40, 200), (130, 40, 200), (130, 300, 900), (16, 33, 130)])
def test_operands_between_nans(shape):
    """Rows and columns past the operands' ends never enter a sum, whatever the memory
    there holds (0xff: NaN scales)."""
    note(f"fp4 products between NaNs {shape}")
    m, n, k = shape
    x, xq, w, dy = operands(m, n, k, 15)

    def between(q):
        g, c, s = filled(q.rows, q.cols, 0xff)
        g.codes.copy_(q.codes)
        g.scales.copy_(q.scales)
        return g

    def nan_around(t):
        buf = torch.full((t.numel() + 64,), float("nan"), dtype=BF, device="cuda")
        v = buf[32:32 + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    x2, q2, w2, dy2 = nan_around(x), between(xq), between(w), nan_around(dy)
    for dtype in (BF, FP):
        assert torch.equal(tide.fp4_mm(q2, w2, dtype=dtype), tide.fp4_mm(xq, w, dtype=dtype))
        for quant in (False, True):
            assert torch.equal(tide.fp4_linear(x2, w2, dtype=dtype, quant_x=quant),
                               tide.fp4_linear(x, w, dtype=dtype, quant_x=quant))
    assert torch.equal(tide.fp4_mm_dx(dy2, w2), tide.fp4_mm_dx(dy, w))


@pytest.mark.parametrize("shape", [(5, 61, 131), (50, 61, 131), (130, 200, 260), (16, 40, 256),
                                   (9, 24, 20000), (20, 1030, 2100), (33, 2050, 1024), (13, 8200, 4096),
                                   (250, 8200, 8200)])
def test_x_and_dy_of_any_alignment(shape):
    note(f"fp4 products unaligned {shape}")
    m, n, k = shape
    _, _, w, _ = operands(m, n, k, 17)
    dy = rand((1, m * n + 1), 18, BF, 1e-3).view(-1)[1:].view(m, n)
    x = rand((1, m * k + 1), 19, BF).view(-1)[1:].view(m, k)
    want, mass = blocks_ref.product(dy.double(), val(w).t().contiguous())
    assert blocks_ref.off(tide.fp4_mm_dx(dy, w), want, mass, n) <= 1.0
    want, mass = blocks_ref.product(x.double(), val(w))
    assert blocks_ref.off(tide.fp4_linear(x, w), want, mass, k) <= 1.0
    want, mass = blocks_ref.product(val(tide.fp4_quant(x)), val(w))
    assert blocks_ref.off(tide.fp4_linear(x, w, quant_x=True), want, mass, k) <= 1.0


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("shape", [(1, 33, 4096), (1, 40, 28672), (1, 40, 28800), (16, 40, 1700),
                                   (16, 40, 1900), (17, 64, 700), (200, 100, 4097), (20, 1030, 2101),
                                   (9, 20000, 900), (31, 2050, 1024)])
def test_linear_rounds_x_as_quant_does(shape, dtype):
    note(f"fp4_linear quant_x {shape} {dtype}")
    m, n, k = shape
    x = rand((m, k), 21, dtype)
    w = tide.fp4_quant(rand((n, k), 22, FP, 0.02))
    want, mass = blocks_ref.product(val(tide.fp4_quant(x)), val(w))
    for out in (BF, FP):
        y = tide.fp4_linear(x, w, dtype=out, quant_x=True)
        assert blocks_ref.off(y, want, mass, k) <= 1.0


@pytest.mark.parametrize("shape", [(300, 200, 9000), (50, 2050, 4100), (4200, 600, 4300)])
def test_same_call_same_bits_on_two_streams(shape):
    note(f"fp4 products on two streams {shape}")
    sets = [operands(*shape, 20 + 5 * i) for i in range(2)]

    def both(x, xq, w, dy):
        return [tide.fp4_mm(xq, w), tide.fp4_linear(x, w), tide.fp4_linear(x, w, quant_x=True),
                tide.fp4_mm_dx(dy, w), tide.fp4_linear(x[:3], w)]
    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for _ in range(4):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(both(*s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("n,k,m", [(24, 1 << 22, 3), (24, 1 << 22, 40), (70, (1 << 22) - 1, 17)])
def test_longest_rows(n, k, m):
    note(f"fp4 longest rows {n} {k} {m}")
    x = torch.zeros(m, k, dtype=BF, device="cuda")
    wr = torch.zeros(n, k, device="cuda")
    at = torch.tensor([0, 31, 4096, k // 2, k - 130, k - 1], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x[:, at] = torch.randint(-4, 5, (m, 6), generator=gen, device="cuda").to(BF)
    wr[:, at] = torch.tensor([1.0, -2.0, 4.0, 3.0, 6.0, -0.5], device="cuda")
    w = tide.fp4_quant(wr)
    del wr
    want = x[:, at].double() @ torch.tensor([1.0, -2.0, 4.0, 3.0, 6.0, -0.5], device="cuda").double()
    for quant in (False, True):
        y = tide.fp4_linear(x, w, dtype=FP, quant_x=quant)
        assert torch.equal(y.double(), want.view(m, 1).expand(m, n))
    dy = torch.zeros(m, n, dtype=BF, device="cuda")
    dy[:, n - 1] = 2.0
    dx = tide.fp4_mm_dx(dy, w)
    assert torch.equal(dx[:, at], torch.tensor([2.0, -4, 8, 6, 12, -1], device="cuda").to(BF).expand(m, 6))
    assert int((dx != 0).sum()) == 6 * m


def test_longest_sums_in_dx():
    note("fp4 dx over 2^22 rows")
    n, m, k = 1 << 22, 20, 40
    w = tide.Fp4Blocks(torch.zeros(n, 64, dtype=torch.uint8, device="cuda"),
                       torch.full((n, 4), 127, dtype=torch.uint8, device="cuda"), k)
    dy = torch.zeros(m, n, dtype=BF, device="cuda")
    for r, c in ((0, 2), (n // 2, 4), (n - 1, 6)):
        w.codes[r, :20] = c + 16 * c
        dy[:, r] = 1.0
    assert torch.equal(tide.fp4_mm_dx(dy, w, dtype=FP), torch.full((m, k), 7.0, device="cuda"))


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("lead", [(40,), (3, 25), ()])
def test_linear_through_autograd(dtype, lead, quant):
    if not quant and dtype != BF:
        with pytest.raises(TypeError, match="bfloat16"):
            tide.fp4_linear(torch.zeros(2, 264, dtype=dtype, device="cuda"), tide.Fp4Blocks.empty(3, 264))
        return
    note(f"fp4_linear {dtype} {lead} {quant}")
    n, k = 72, 264
    x = rand((*lead, k) if lead else (1, k), 30, dtype).view(*lead, k).requires_grad_()
    w = tide.fp4_quant(rand((n, k), 31, FP, 0.02))
    dw = torch.full((n, k), 7.0, device="cuda")
    y = tide.fp4_linear(x, w, quant_x=quant, grad=dw)
    assert y.shape == (*lead, n) and y.dtype == (FP if dtype == FP else BF)
    dy = rand((1, y.numel()), 32, BF, 1e-3).view(y.shape).to(y.dtype)
    y.backward(dy)
    x2, dy2 = x.detach().reshape(-1, k), dy.reshape(-1, n).to(BF)
    m = x2.shape[0]
    xv = val(tide.fp4_quant(x2)) if quant else x2.double()
    want, mass = blocks_ref.product(xv, val(w))
    assert blocks_ref.off(y.detach().reshape(m, n), want, mass, k) <= 1.0
    want, mass = blocks_ref.product(dy2.double(), val(w).t().contiguous())
    assert x.grad.dtype == dtype
    # an fp16 gradient is rounded twice: to fp32 sums, then to fp16
    assert blocks_ref.off(x.grad.reshape(m, k), want, mass, n + 1) <= 1.0
    q8 = tide.block_quant(x2)                          # the weights' gradient reads 8 bits of x
    x8 = blocks_ref.values(q8.codes, q8.scales, k)
    want, mass = blocks_ref.product(dy2.double().t().contiguous(), x8.t().contiguous())
    assert blocks_ref.off(dw, want, mass, m) <= 1.0


def test_linear_gradient_against_differences():
    """<dy, y(x + d) - y(x - d)> / 2 = <dx, d>: y is linear in a bf16 x."""
    note("fp4_linear differences")
    m, n, k = 20, 64, 256
    g = torch.Generator(device="cuda").manual_seed(33)
    x = torch.randint(-60, 61, (m, k), generator=g, device="cuda").to(BF)
    d = torch.randint(-1, 2, (m, k), generator=g, device="cuda").to(BF)
    w = tide.fp4_quant(rand((n, k), 34, FP, 0.02))
    dy = rand((m, n), 35, BF, 1.0)
    xl = x.clone().requires_grad_()
    dx, = torch.autograd.grad(tide.fp4_linear(xl, w, dtype=FP), xl, dy.float())
    def f(z):
        return tide.fp4_linear(z, w, dtype=FP).double()
    diff = (dy.double() * (f(x + d) - f(x - d)) / 2).sum()
    got = (dx.double() * d.double()).sum()
    wv = val(w).abs()
    mass = (dy.double().abs() * ((x.abs() + d.abs()).double() @ wv.t())).sum()
    # fp32 sums on both sides, and dx rounded to bf16
    back = (d.double().abs() * (dy.double().abs() @ wv)).sum()
    assert abs(float(diff - got)) <= float(mass + back) * k * 2.0 ** -23 + float(back) * 2.0 ** -8


def test_linear_with_frozen_parts():
    note("fp4_linear frozen parts")
    m, n, k = 33, 40, 130
    x = rand((m, k), 36)
    w = tide.fp4_quant(rand((n, k), 37, FP, 0.02))
    dy = rand((m, n), 38, BF, 1e-3)
    dw = torch.full((n, k), 7.0, device="cuda")
    tide.fp4_linear(x, w, grad=dw).backward(dy)               # x needs no gradient
    assert torch.equal(dw, tide.block_mm_dw(dy, tide.block_quant(x), dtype=FP))
    xl = x.clone().requires_grad_()
    tide.fp4_linear(xl, w).backward(dy)                       # frozen weights
    assert torch.equal(xl.grad, tide.fp4_mm_dx(dy, w))
    assert not tide.fp4_linear(x, w).requires_grad
    with torch.no_grad():
        assert not tide.fp4_linear(xl, w, grad=dw).requires_grad
    tide.fp4_linear(xl, w, grad=dw).sum().backward()          # a broadcast output gradient
    tide.fp4_linear(xl, w, grad=dw, accumulate=True).sum().backward()
    ones = torch.ones(m, n, dtype=BF, device="cuda")
    once = tide.block_mm_dw(ones, tide.block_quant(x), dtype=FP)
    assert torch.equal(dw, once + once)


def test_weight_gradient_is_ordered_before_the_caller():
    """Forward on a side stream, backward() called from another one that reads `grad`
    right away."""
    note("fp4_linear backward from another stream")
    m, n, k = 200, 264, 392
    x, _, w, dy = operands(m, n, k, 39)
    big = rand((4096, 4096), 4)

    def passes(stream):
        grad = torch.full((n, k), 7.0, device="cuda")
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            y = tide.fp4_linear(x, w, grad=grad)
            for _ in range(20):
                big @ big
        y.backward(dy)
        return grad.clone()
    want = passes(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = passes(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not bool((want == 7.0).any())


@pytest.mark.parametrize("m", [1, 16, 130])
def test_captured(m):
    """Quantisation, products and the gather captured into two graphs with their own
    workspaces; replays with eager work between them equal the eager results."""
    note(f"fp4 captured {m}")
    n, k = 200, 5000
    _, _, w, dy = operands(m, n, k, 40)
    plan, _, master = shards([(40, 200), (7, 33)], 2, 44)
    fp = tide.Fp4Plan(plan)
    xs = [rand((m, k), 42 + i) for i in range(2)]

    def step(x):
        gathered = fp.empty()
        for r in range(2):
            tide.fp4_shard(fp, r, master[r], gathered[r])
        params = [torch.empty(s, dtype=BF, device="cuda") for s in fp.matrices]
        tide.fp4_unshard(fp, gathered, params)
        q = tide.fp4_quant(x)
        return [tide.fp4_mm(q, w), tide.fp4_linear(x, w), tide.fp4_linear(x, w, quant_x=True),
                tide.fp4_mm_dx(dy, w), tide.fp4_dequant(q), *params]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    outs, graphs = [], []
    for x in xs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(step(x))
        graphs.append(gr)
    for it in range(3):
        for i, x in enumerate(xs):
            x.copy_(rand((m, k), 50 + 2 * it + i))
        master.mul_(1.5)
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(xs):
            for got, want in zip(outs[i], step(x)):
                assert torch.equal(got, want)


@pytest.mark.parametrize("shape", [(40, 2050, 4100), (20, 2050, 1024), (4200, 700, 4200)])
def test_captured_in_several_launches(shape):
    """Sums in pieces, padded x and turned operands, in two graphs that replay in turn."""
    note(f"fp4 captured launches {shape}")
    m, n, k = shape
    _, xq, w, dy = operands(m, n, k, 48)
    xs = [rand((m, k), 60 + i) for i in range(2)]

    def step(x):
        return [tide.fp4_linear(x, w), tide.fp4_linear(x, w, quant_x=True),
                tide.fp4_mm(tide.fp4_quant(x), w), tide.fp4_mm_dx(dy, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    outs, graphs = [], []
    for x in xs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(step(x))
        graphs.append(gr)
    for it in range(3):
        for i, x in enumerate(xs):
            x.copy_(rand((m, k), 70 + 2 * it + i))
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(xs):
            for got, want in zip(outs[i], step(x)):
                assert torch.equal(got, want)


def test_captured_backward_through_autograd():
    """Over a leaf that no live eager graph holds; eager passes over others between."""
    note("fp4_linear autograd captured")
    m, n, k = 70, 96, 640
    _, _, w, dy = operands(m, n, k, 43)
    x, dw = rand((m, k), 45), torch.zeros(n, k, device="cuda")

    def step(leaf, grad):
        y = tide.fp4_linear(leaf, w, grad=grad, accumulate=True, quant_x=True)
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
    """The operators, eager and in a compiled step, give the binding's bits."""
    note("fp4 custom ops")
    plan, full, master = shards([(72, 264), (9, 130)], 3, 80)
    pid = tops.register_plan(tide.Fp4Plan(plan))
    ops = torch.ops.tide
    try:
        fp = tops._PLANS[pid]
        m, n, k = 70, 72, 264
        w = tide.fp4_quant(full[0])
        x, dy = rand((m, k), 81), rand((m, n), 82, BF, 1e-3)

        def step(master, gathered, params, x, dy, codes, scales, y, back, dx):
            for r in range(3):
                ops.fp4_shard(pid, r, master[r], gathered[r])
            ops.fp4_unshard(pid, gathered, params)
            ops.fp4_quant(x, codes, scales)
            ops.fp4_dequant(codes, scales, back)
            ops.fp4_mm(codes, scales, w.codes, w.scales, k, y)
            ops.fp4_mm_dx(dy, w.codes, w.scales, dx)
            z = ops.fp4_linear(x.view(7, 10, k), w.codes, w.scales, torch.float32, False)
            return z * 2.0

        for fn in (step, torch.compile(step, backend="aot_eager", fullgraph=True)):
            q = tide.Fp4Blocks.empty(m, k)
            params = [torch.zeros(s, dtype=BF, device="cuda") for s in fp.matrices]
            y, back, dx = (torch.zeros(s, dtype=BF, device="cuda") for s in ((m, n), (m, k), (m, k)))
            z = fn(master, fp.empty().zero_(), params, x, dy, q.codes, q.scales, y, back, dx)
            xq = tide.fp4_quant(x)
            assert torch.equal(z, 2 * tide.fp4_linear(x.view(7, 10, k), w, dtype=FP))
            assert torch.equal(q.codes, xq.codes) and torch.equal(q.scales, xq.scales)
            assert torch.equal(y, tide.fp4_mm(xq, w)) and torch.equal(back, tide.fp4_dequant(xq))
            assert torch.equal(dx, tide.fp4_mm_dx(dy, w))
            assert torch.equal(params[0], tide.fp4_dequant(w))
    finally:
        tops.unregister_plan(pid)


def test_weights_released_and_restored():
    """An FSDP unit releases gathered weights' storage and restores it elsewhere."""
    note("fp4 storage released and restored")
    x, _, w, _ = operands(5, 40, 300, 90)
    want, codes = tide.fp4_linear(x, w), w.codes.clone()
    size = w.codes.untyped_storage().nbytes()
    w.codes.untyped_storage().resize_(0)
    with pytest.raises(tide.TideError, match="codes are NULL"):
        tide.fp4_linear(x, w)
    hold = torch.empty(size, dtype=torch.uint8, device="cuda")
    w.codes.untyped_storage().resize_(size)
    w.codes.copy_(codes)
    assert torch.equal(tide.fp4_linear(x, w), want)
    w.codes = codes
    assert torch.equal(tide.fp4_linear(x, w), want)
    del hold


UNIT = [(96, 200), (200,), (200, 96), (40, 200)]


@pytest.mark.parametrize("world", [1, 3, 8])
@pytest.mark.parametrize("kw", [{}, {"small": True}, {"copy_engine": True}])
def test_unit_gathers_matrices_in_both_formats(world, kw):
    from parameter_layout_collectives_amd.fsdp import TideUnit
    note(f"TideUnit fp4 world={world} {kw}")
    full = [rand((1, s[0]) if len(s) == 1 else s, 70 + i, FP, 0.05).view(s) for i, s in enumerate(UNIT)]
    unit = TideUnit(UNIT, world, blocks=[2], fp4=[3, 0])
    unit.load(full)
    unit.all_gather(**kw)
    torch.cuda.synchronize()
    for i in (0, 3):
        q = tide.fp4_quant(full[i])
        assert torch.equal(unit.params[i].codes, q.codes) and torch.equal(unit.params[i].scales, q.scales)
    assert torch.equal(tide.block_dequant(unit.params[2]), tide.block_dequant(tide.block_quant(full[2])))
    assert torch.equal(unit.params[1], full[1].to(BF))
    x = rand((5, 200), 3)
    assert torch.equal(unit.linear(0, x), tide.fp4_linear(x, tide.fp4_quant(full[0])))
    assert torch.equal(unit.linear(3, x, quant_x=True),
                       tide.fp4_linear(x, tide.fp4_quant(full[3]), quant_x=True))
    for bad in (lambda: unit.linear(1, x), lambda: unit.linear(0, x, short_sums=True),
                lambda: unit.linear(2, rand((5, 96), 4), quant_x=True)):
        with pytest.raises(ValueError):
            bad()


def test_unit_trains_behind_4_bit_products():
    """A run as it would be used: gather in 4 bits, forward and backward of every
    rank's micro-batch, reduce-scatter, a Muon step on the master shards, gather."""
    from parameter_layout_collectives_amd.fsdp import TideUnit
    import ortho_ref
    note("TideUnit fp4 + muon training step")
    N, m, shapes = 4, 33, [(96, 200), (200, 96)]
    full = [rand(s, 70 + i, FP, 0.05) for i, s in enumerate(shapes)]
    unit = TideUnit(shapes, N, fp4=[0, 1])
    unit.load(full)
    grads, want = [], []
    for r in range(N):
        g = [torch.zeros(s, device="cuda") for s in shapes]
        x = rand((m, 200), 80 + r, BF, 0.5).requires_grad_()
        h = unit.linear(0, x, grad=g[0], quant_x=True)
        a = torch.relu(h)
        y = unit.linear(1, a, grad=g[1], dtype=FP)
        dy = rand((m, 200), 90 + r, BF, 1e-2).float()
        y.backward(dy)
        grads.append(g)
        da = tide.fp4_mm_dx(dy.to(BF), unit.params[1])
        dh = da * (h.detach() > 0)
        assert torch.equal(x.grad, tide.fp4_mm_dx(dh, unit.params[0]))
        want.append((tide.block_mm_dw(dh, tide.block_quant(x.detach()), dtype=FP),
                     tide.block_mm_dw(dy.to(BF), tide.block_quant(a.detach()), dtype=FP)))
    for g, d in zip(grads, want):
        assert torch.equal(g[0], d[0]) and torch.equal(g[1], d[1])
    unit.reduce_scatter(grads)
    unit.muon_step(0.02, momentum=0.9)
    unit.all_gather()
    for i, s in enumerate(shapes):
        mean = sum(w[i].double() for w in want) / N
        u = (mean.float() * 1.9).to(BF)
        new = full[i].double() - 0.02 * max(1.0, s[0] / s[1]) ** 0.5 * ortho_ref.exact(u)
        off, _, seg = unit.plan.param(i)
        got = unit.master[:, off:off + seg].reshape(-1, s[1])[:s[0]]
        moved = float((new - full[i].double()).norm())
        # O is off by 2^-8 of its norm, and as much again by a step in u's rounding
        assert float((got.double() - new).norm()) <= 2 * 2.0 ** -8 * moved
        q = tide.fp4_quant(got.contiguous())
        assert torch.equal(unit.params[i].codes, q.codes) and torch.equal(unit.params[i].scales, q.scales)
