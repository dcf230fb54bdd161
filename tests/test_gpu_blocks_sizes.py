"""8-bit blocks at the size limits: n and k of 2^22, where the bytes of a tile's rows
fill 31 bits, and matrices of more than 2^31 elements.

Products are over whole numbers that are zero but in a few rows and columns along
the sum, so that the reference is a small product in 64 bits and exact."""
import gc

import pytest
import torch

import blocks_ref as ref
import parameter_layout_collectives_amd as tide
from gpu_helpers import note
from test_gpu_blocks import HF, UNITS, shards
from test_gpu_blocks_exact import check, small

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
MOST = 1 << 22


@pytest.fixture(autouse=True)
def free():
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def picked(count, of, seed):
    """`count` of `of` places, the first and the last few among them, ascending."""
    ends = torch.cat([torch.arange(5), torch.arange(of - 70, of)])
    rest = torch.randperm(of, generator=torch.Generator().manual_seed(seed))[:count]
    return torch.unique(torch.cat([ends, rest])).cuda()


def sparse_blocks(rows, cols, places, seed, along):
    """Blocks [rows, cols] of whole numbers, zero but in the rows (along=0) or the
    columns (along=1) `places`, and the values there in fp32."""
    q = tide.Blocks.empty(rows, cols)
    q.codes.view(torch.uint8).zero_()
    q.scales.fill_(127)
    if along == 0:
        v = small((len(places), cols), gen(seed))
        part = tide.block_quant(v)
        q.codes.view(torch.uint8)[places] = part.codes.view(torch.uint8)
        q.scales[places] = part.scales
    else:
        v = small((rows, len(places)), gen(seed))
        # whole numbers below 5 under the scale 2^0
        q.codes.view(torch.uint8)[:, places] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return q, v


@pytest.mark.parametrize("m,n", [(1, 300), (40, 130), (300, 260), (2900, 4100)])
def test_longest_rows_in_mm(m, n):
    """k = 2^22; 2900 x 4100 takes tiles of 256 rows, of 2^30 bytes."""
    note(f"block_mm k=2^22 {m}x{n}")
    at = picked(1500, MOST, 1)
    x, xv = sparse_blocks(m, MOST, at, 2, 1)
    w, wv = sparse_blocks(n, MOST, at, 3, 1)
    for dtype in (FP, BF):
        check("mm", tide.block_mm(x, w, dtype=dtype), xv.double(), wv.double())
    got = tide.block_mm(x, w, short_sums=True)      # small numbers: nothing is cut
    want, mass = ref.product(xv.double(), wv.double())
    assert ref.off(got, want, mass, len(at), fast=True) <= 1.0


@pytest.mark.parametrize("n,m,k", [(MOST, 3, 130), (MOST, 130, 200), (MOST - 3, 130, 200),
                                   (MOST - 3, 2050, 2060), (MOST, 4000, 2900)])
def test_longest_sums_in_dx(n, m, k):
    """n = 2^22; 4000 x 2900 takes tiles of 256 rows, of 2^31 bytes of dy."""
    note(f"block_mm_dx n={n} {m}x{k}")
    at = picked(1500, n, 4)
    w, wv = sparse_blocks(n, k, at, 5, 0)
    dy = torch.zeros(m, n, dtype=BF, device="cuda")
    dv = small((m, len(at)), gen(6))
    dy[:, at] = dv.to(BF)
    for dtype in (FP, BF):
        check("dx", tide.block_mm_dx(dy, w, dtype=dtype), dv.double(), wv.double().t().contiguous())


def whole(rows, cols, seed):
    v = small((rows, cols), gen(seed))
    return tide.block_quant(v), v


@pytest.mark.parametrize("n,m,k", [(MOST, 70, 264), (MOST - 3, 70, 200)])
def test_most_rows_in_dw(n, m, k):
    note(f"block_mm_dw n={n} {m}x{k}")
    x, xv = whole(m, k, 7)
    dy = torch.randint(-4, 5, (m, n), generator=gen(8), device="cuda").to(BF)
    got = tide.block_mm_dw(dy, x)
    for lo in (0, n // 2 + 1, n - 4096):
        check("dw", got[lo:lo + 4096], dy[:, lo:lo + 4096].double().t().contiguous(),
              xv.double().t().contiguous())


def test_most_columns_in_dx_and_dw():
    note("block_mm_dx, block_mm_dw k=2^22")
    m, n = 70, 72
    x, xv = whole(m, MOST, 9)
    w, wv = whole(n, MOST, 10)
    dy = small((m, n), gen(11)).to(BF)
    dx, dw = tide.block_mm_dx(dy, w), tide.block_mm_dw(dy, x)
    d = dy.double()
    for lo in (0, MOST // 2 + 1, MOST - 4096):
        part = slice(lo, lo + 4096)
        check("dx", dx[:, part], d, wv[:, part].double().t().contiguous())
        check("dw", dw[:, part], d.t().contiguous(), xv[:, part].double().t().contiguous())


def test_a_sum_over_many_rows():
    note("block_mm_dw m=2^24+3")
    m, n, k = (1 << 24) + 3, 9, 130
    at = picked(3000, m, 12)
    x, xv = sparse_blocks(m, k, at, 13, 0)
    dy = torch.zeros(m, n, dtype=BF, device="cuda")
    dv = small((len(at), n), gen(14))
    dy[at] = dv.to(BF)
    for dtype in (FP, BF):
        check("dw", tide.block_mm_dw(dy, x, dtype=dtype), dv.double().t().contiguous(),
              xv.double().t().contiguous())


@pytest.mark.parametrize("cols", [8200, 8187])
def test_blocks_of_more_than_2g_elements(cols):
    """The same bytes as its rows give in smaller calls, there and back."""
    note(f"block_quant, block_dequant 2^18+5 x {cols}")
    rows = (1 << 18) + 261
    assert rows * cols > 1 << 31
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    x.normal_(generator=gen(15))
    q = tide.block_quant(x)
    back = tide.block_dequant(q)
    for lo in (0, rows // 2 + 1, rows - 300):
        part = tide.block_quant(x[lo:lo + 300])
        assert torch.equal(q.codes[lo:lo + 300].view(torch.uint8), part.codes.view(torch.uint8))
        assert torch.equal(q.scales[lo:lo + 300], part.scales)
        assert torch.equal(back[lo:lo + 300], tide.block_dequant(part))


def test_gather_of_more_than_2g_elements():
    """Rank blocks and matrices past 2^31 elements, beside small ones."""
    note("block gather of 2^31 elements")
    shapes, world = [(5, 200), ((1 << 18) + 261, 8200), (33, 130)], 3
    plan = tide.Plan(shapes, world)
    bp = tide.BlockPlan(plan)
    master = torch.empty(world, plan.S, device="cuda").normal_(generator=gen(16))
    gathered = bp.empty()
    for r in range(world):
        tide.block_shard(bp, r, master[r], gathered[r])
    params = [torch.empty(s, dtype=BF, device="cuda") for s in shapes]
    tide.block_unshard(bp, gathered, params)
    for i, (d0, cols) in enumerate(shapes):
        off, c, _ = plan.param(i)
        for row in sorted({0, 1, c - 1, c, 2 * c - 1, 2 * c, d0 - 1}):
            r = row // c
            if row >= d0:
                continue
            src = master[r, off + (row - r * c) * cols:][:cols].view(1, cols)
            assert torch.equal(params[i][row:row + 1], tide.block_dequant(tide.block_quant(src)))


@pytest.mark.parametrize("unit", range(len(UNITS)))
def test_gather_in_blocks_to_fp16(unit):
    """Values rounded once to fp16, to infinity past 65504 and to its subnormals."""
    shapes, world, select = UNITS[unit]
    note(f"block gather to fp16 unit {unit}")
    plan, full, master = shards(shapes, world, 50)
    master *= 3e4
    master[:, ::7] *= 1e-10
    bp = tide.BlockPlan(plan, select)
    gathered = bp.empty()
    for r in range(world):
        tide.block_shard(bp, r, master[r], gathered[r])
    exact = [torch.empty(m, device="cuda") for m in bp.matrices]
    got = [torch.full(m, 7.0, dtype=HF, device="cuda") for m in bp.matrices]
    tide.block_unshard(bp, gathered, exact)
    tide.block_unshard(bp, gathered, got)
    for g, e in zip(got, exact):
        assert torch.equal(g, e.to(HF))
