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
    """The 8-bit instruction's sums, where the caller asks for them: within the
    documented 2^-12 of the products' magnitudes, through every entry point."""
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
