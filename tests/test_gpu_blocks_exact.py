"""Products of 8-bit blocks over whole numbers: every product and every partial
sum is a whole number below 2^24, so sums held in fp32 are exact in any order and
a result equals the exact one rounded once to its type, bit for bit.  Columns in
pairs whose products are large and cancel hide nothing of the small ones."""
import pytest
import torch

import blocks_ref as ref
import parameter_layout_collectives_amd as tide
from gpu_helpers import note

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def small(shape, gen):
    return torch.randint(-4, 5, shape, generator=gen, device="cuda").float()


def operands(m, n, k, seed):
    """x [m, k], w [n, k] and dy [m, n] in whole numbers of at most 448: mostly
    below 5, with large pairs along each product's sum: 448 * 448 - 448 * 448."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w, dy = small((m, k), g), small((n, k), g), small((m, n), g)
    # along k, for x w^T
    at = torch.randperm(max(k // 2, 1), generator=g, device="cuda")[:12] * 2
    at = at[at + 1 < k]
    x[:, at] = x[:, at + 1] = 448.0
    w[:, at], w[:, at + 1] = 448.0, -448.0
    # along n, for dy w: rows of w that are each other's negative
    at = torch.randperm(max(n // 2, 1), generator=g, device="cuda")[:6] * 2
    at = at[at + 1 < n]
    w[at + 1] = -w[at]
    # (in a few rows of dy: in all of them dy^T x would pass 2^24)
    dy[:8, at] = dy[:8, at + 1] = 256.0
    # along m, for dy^T x
    at = torch.randperm(max(m // 2, 1), generator=g, device="cuda")[:6] * 2
    at = at[at + 1 < m]
    dy[at + 1] = -dy[at]
    x[at + 1] = x[at]
    return x, w, dy.to(BF)


def check(name, got, a, b):
    want, mass = ref.product(a, b)
    assert float(mass.max()) < 2 ** 24                 # every partial sum is exact
    assert torch.equal(got, want.float().to(got.dtype)), \
        (name, got.dtype, float((got.double() - want).abs().max()))


def check_products(m, n, k, seed=1, shift=0):
    """`shift`: dy starts that many elements into its memory."""
    note(f"exact block products m={m} n={n} k={k} dy at {shift}")
    xr, wr, dy = operands(m, n, k, seed)
    if shift:
        buf = torch.empty(m * n + shift, dtype=BF, device="cuda")
        buf[shift:].copy_(dy.view(-1))
        dy = buf[shift:].view(m, n)
    x, w = tide.block_quant(xr), tide.block_quant(wr)
    assert torch.equal(tide.block_dequant(x, dtype=FP), xr)        # whole numbers stay
    assert torch.equal(tide.block_dequant(w, dtype=FP), wr)
    xd, wd, dd = xr.double(), wr.double(), dy.double()
    wt, xt, dt = wd.t().contiguous(), xd.t().contiguous(), dd.t().contiguous()
    for dtype in (FP, BF):
        check("dx", tide.block_mm_dx(dy, w, dtype=dtype), dd, wt)
        check("dw", tide.block_mm_dw(dy, x, dtype=dtype), dt, xt)
        check("mm", tide.block_mm(x, w, dtype=dtype), xd, wd)
        check("linear", tide.block_linear(xr, w, dtype=dtype), xd, wd)
        old = small((n, k), torch.Generator(device="cuda").manual_seed(seed + 9)).to(dtype)
        got = tide.block_mm_dw(dy, x, out=old.clone(), accumulate=True)
        want = (ref.product(dt, xt)[0] + old.double()).float().to(dtype)
        assert torch.equal(got, want), ("accumulate", dtype)


@pytest.mark.parametrize("shape", [(1, 40, 300), (16, 200, 700), (17, 200, 700), (40, 130, 1111),
                                   (64, 300, 520), (65, 72, 2048), (130, 200, 392)])
def test_products_of_few_rows(shape):
    check_products(*shape)


@pytest.mark.parametrize("shape", [(24, 8192, 4099), (25, 8192, 4099), (33, 8192, 4099)])
def test_products_of_a_large_w(shape):
    check_products(*shape)


# Every tile, cut and whole, with dy's rows in whole vectors and not: which shape
# takes which is pinned in tests/sanitize/block_checks.cpp.
@pytest.mark.parametrize("shape,shift", [
    ((130, 200, 392), 0), ((131, 201, 392), 0), ((130, 200, 392), 1),          # 64
    ((1500, 1510, 2060), 0), ((1500, 1510, 440), 0),                           # 128
    ((2050, 2049, 2060), 0), ((2050, 2056, 2060), 0), ((2050, 2056, 2060), 1),
    ((4100, 1101, 4000), 0), ((4100, 1104, 4000), 0), ((1101, 4100, 4000), 0),  # 256
    ((4000, 4104, 1100), 0), ((4400, 4200, 4250), 0), ((4200, 2200, 4400), 0),
    ((2200, 4200, 4400), 0)])
def test_products_over_tiles(shape, shift):
    check_products(*shape, shift=shift)


def between_nans(t, rows, byte):
    """t with `rows` rows of the byte on either side of it in memory."""
    u = t.view(torch.uint8)
    buf = torch.full((u.shape[0] + 2 * rows, u.shape[1]), byte, dtype=torch.uint8, device="cuda")
    mid = buf[rows:rows + u.shape[0]]
    mid.copy_(u)
    return mid.view(t.dtype)


@pytest.mark.parametrize("shape", [(17, 40, 200), (131, 200, 520), (2050, 2056, 2060),
                                   (4100, 1104, 4010), (4009, 4104, 1040), (2200, 4200, 4400)])
def test_operands_between_nans(shape):
    """Whole tiles of NaNs before and behind every operand: what a tile or a step
    has past the operand's end never enters a sum."""
    m, n, k = shape
    note(f"block products between 300 rows of NaNs {shape}")
    xr, wr, dy = operands(m, n, k, 5)
    x, w = tide.block_quant(xr), tide.block_quant(wr)
    x2, w2 = (tide.Blocks(between_nans(q.codes, 304, 0x7f), between_nans(q.scales, 304, 0xf6), k)
              for q in (x, w))
    dy2 = between_nans(dy, 304, 0x7f)
    assert dy2.data_ptr() % 16 == 0
    for dtype in (FP, BF):
        assert torch.equal(tide.block_mm(x2, w2, dtype=dtype), tide.block_mm(x, w, dtype=dtype))
        assert torch.equal(tide.block_mm_dx(dy2, w2, dtype=dtype),
                           tide.block_mm_dx(dy, w, dtype=dtype))
        assert torch.equal(tide.block_mm_dw(dy2, x2, dtype=dtype),
                           tide.block_mm_dw(dy, x, dtype=dtype))
    assert torch.equal(tide.block_mm(x2, w2, short_sums=True), tide.block_mm(x, w, short_sums=True))


@pytest.mark.parametrize("shape", [(17, 64, 700), (40, 5000, 4099), (130, 200, 392), (500, 300, 2000),
                                   (2100, 1100, 1300), (4000, 4104, 1100)])
def test_short_sums(shape):
    """The 8-bit instruction's sums, where the caller asks for them, on normal data
    and through every entry point."""
    m, n, k = shape
    note(f"block products with short sums {shape}")
    g = torch.Generator(device="cuda").manual_seed(3)
    xr = torch.randn(m, k, generator=g, device="cuda").to(BF)
    wr = 0.02 * torch.randn(n, k, generator=g, device="cuda")
    x, w = tide.block_quant(xr), tide.block_quant(wr)
    want, mass = ref.product(ref.values(x.codes, x.scales, k), ref.values(w.codes, w.scales, k))
    got = tide.block_mm(x, w, short_sums=True)
    assert ref.off(got, want, mass, k, fast=True) <= 1.0
    assert torch.equal(got, tide.block_linear(xr, w, short_sums=True))
    leaf = xr.clone().requires_grad_()
    assert torch.equal(got, tide.block_linear(leaf, w, short_sums=True).detach())
    import parameter_layout_collectives_amd.torch_ops  # noqa: F401 - registers the ops
    out = torch.empty(m, n, dtype=BF, device="cuda")
    torch.ops.tide.block_mm(x.codes, x.scales, w.codes, w.scales, k, out, True)
    assert torch.equal(got, out)
    for call in (lambda: tide.block_mm(x, w, dtype=FP, short_sums=True),
                 lambda: tide.block_linear(xr, w, dtype=FP, short_sums=True)):
        with pytest.raises(ValueError):
            call()


def scaled_exponents(v):
    """The exponent that each e4m3 value stands under: subnormals under -6."""
    return torch.where(v == 0, -1000, (torch.frexp(v)[1] - 1).clamp_min(-6)).float()


def short_bound(x, w):
    """What short sums may lose of x w^T, codes under the scale 2^0: of 8 neighbouring
    products those that lie below 2^-13 of the largest exponent's power, 7 of them."""
    ex, ew = scaled_exponents(x), scaled_exponents(w)
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for k in range(0, x.shape[1], 8):
        e = (ex[:, None, k:k + 8] + ew[None, :, k:k + 8]).amax(2).double()
        total += 7 * 2.0 ** -13 * torch.exp2(e)
    return total


def code_blocks(v):
    """Blocks whose codes are v itself, under the scale 2^0."""
    q = tide.Blocks.empty(*v.shape)
    q.codes.view(torch.uint8).zero_()
    q.scales.fill_(127)
    q.codes.view(torch.uint8)[:, :v.shape[1]] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return q


@pytest.mark.parametrize("large", [(448.0, 448.0), (256.0, 256.0), (1.0, 1.0), (256.0, 2.0 ** -9),
                                   (2.0 ** -9, 2.0 ** -9)])
@pytest.mark.parametrize("k,apart", [(128, 1), (128, 64), (1100, 8)])
def test_short_sums_lose_what_is_documented(large, k, apart):
    """Large products that cancel, inside a group of 8 and across groups, beside
    every pair of codes: what is lost stays within the documented bound."""
    note(f"short sums beside {large}, k={k}, {apart} apart")
    t = ref.e4m3_table()[:127].float().cuda()
    x, w = t[:, None].repeat(1, k), t[:, None].repeat(1, k)
    for at in range(0, k - 127, 128):
        x[:, at] = x[:, at + apart] = large[0]
        w[:, at], w[:, at + apart] = large[1], -large[1]
    q, r = code_blocks(x), code_blocks(w)
    want, mass = ref.product(x.double(), w.double())
    got = tide.block_mm(q, r, short_sums=True)
    tol = short_bound(x, w) + mass * k * 2.0 ** -23
    tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((got.double() - want).abs() <= tol).all())
    # sums in fp32 keep what a sum of k products in fp32 keeps
    assert ref.off(tide.block_mm(q, r), want, mass, k) <= 1.0
    assert ref.off(tide.block_mm(q, r, dtype=FP), want, mass, k) <= 1.0
