"""Two more steps of an FSDP unit as timed cases: the update that its optimizer makes of a
gathered gradient (orthogonalised by Newton-Schulz products), and weights held in microscaled
4-bit floating point (their sharded gather, the products that read them, and the gradient that
passes through them).

A matrix [R, C] in 4-bit blocks has, for each row and each run of 32 columns, one power of two
2^e and 32 e2m1 numbers (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  e is the smallest
integer with max|x| <= 6 * 2^e (within -125..125; 0 where there is none but zeros), and every x
becomes the e2m1 number nearest to x / 2^e, ties to the even code.

A matrix G [r, c] is orthogonalised from X = G / ||G||_F by steps of
X <- a X + b (X X^T) X + c (X X^T)^2 X, which bring all its singular values near 1.

Kinds of cases (every size is that of the matrices as a user has them):
  gather    fp32 master shards of all ranks -> 4-bit rank blocks -> full bf16 parameters
  forward   y = x w^T, w in 4-bit blocks, x as it is (bf16) or quantised to 4 bits on the way
  backward  dx = dy w, w in 4-bit blocks
  tune      forward and backward of one layer of frozen 4-bit weights through autograd
  ortho     matrices, or stacks of equal ones, orthogonalised in five steps
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)

# The matrices of a Llama-3-8B-shaped decoder layer, as the repository's own workloads list
# them (the norms stay out: they are not matrices).
LAYER_8B = "4096x4096*2+1024x4096*2+14336x4096*2+4096x14336"
# An eighth of the experts of a Qwen3-30B-A3B-shaped MoE layer, as equal matrices in two stacks.
EXPERTS = "768x2048*32+2048x768*16"


def listed():
    return [
        # a unit of small matrices whose rows do not divide by the ranks and whose rows end
        # inside a block: the shortest gather
        {"name": "gather, small odd unit", "kind": "gather", "shapes": "333x1000+37x129+64x64",
         "world": 6},
        # a dense decoder layer over one node, for a frozen base model or for serving
        {"name": "gather, 8B layer", "kind": "gather", "shapes": LAYER_8B, "world": 8},
        # one token through the 8B layer's gate projection: a serving step, W's bytes bound it
        {"name": "forward, one token", "kind": "forward", "m": 1, "n": 14336, "k": 4096,
         "type": "bf16", "quant": False, "out": "bf16"},
        # a decode batch of 32 through the 70B layer's down projection
        {"name": "forward, 32 rows", "kind": "forward", "m": 32, "n": 8192, "k": 28672,
         "type": "bf16", "quant": False, "out": "bf16"},
        # a ragged micro-batch through an odd matrix, both in 4 bits, fp32 in and out
        {"name": "forward, odd", "kind": "forward", "m": 777, "n": 1000, "k": 1111,
         "type": "fp32", "quant": True, "out": "fp32"},
        # 8K tokens of a prompt through the 70B layer's gate projection, both in 4 bits
        {"name": "forward, 70B gate", "kind": "forward", "m": 8192, "n": 28672, "k": 8192,
         "type": "bf16", "quant": True, "out": "bf16"},
        # one frozen expert's share of a micro-batch in the MoE layer
        {"name": "backward, expert", "kind": "backward", "m": 509, "n": 768, "k": 2048,
         "out": "fp32"},
        # 4K tokens through the 70B layer's frozen output projection and back
        {"name": "tune, 70B o_proj", "kind": "tune", "m": 4096, "n": 8192, "k": 8192,
         "quant": False, "out": "bf16"},
        # the smallest unit: three matrices in which only the latency counts
        {"name": "ortho, small odd unit", "kind": "ortho", "shapes": "333x1000+37x129+64x64",
         "type": "fp32"},
        # one attention projection of the 8B layer
        {"name": "ortho, 8B q_proj", "kind": "ortho", "shapes": "4096x4096", "type": "bf16"},
        # experts: many equal matrices, wide and tall
        {"name": "ortho, experts", "kind": "ortho", "shapes": EXPERTS, "type": "bf16"},
        # every matrix of the 8B layer: an optimizer's step of one unit
        {"name": "ortho, 8B layer", "kind": "ortho", "shapes": LAYER_8B, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["gather", "forward", "forward", "backward", "tune", "ortho", "ortho"])
    if kind == "gather":
        shapes = ["%dx%d" % (_log(rng, 1, 8192), _log(rng, 1, 8192))
                  for _ in range(rng.randint(1, 6))]
        return {"kind": kind, "shapes": "+".join(shapes), "world": _log(rng, 1, 64)}
    if kind == "ortho":
        # at most the listed layer's multiplications
        while True:
            shapes = []
            for _ in range(rng.randint(1, 4)):
                r, c = _log(rng, 1, 8192), _log(rng, 1, 8192)
                shapes.append("%dx%d*%d" % (r, c, _log(rng, 1, 16)))
            c = {"kind": kind, "shapes": "+".join(shapes),
                 "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
            if work(c)["flops"] <= work({"kind": kind, "shapes": LAYER_8B, "type": "bf16"})["flops"]:
                return c
    # at most the largest listed product's multiplications
    most = 8192 * 28672 * 8192 // (2 if kind == "tune" else 1)
    while True:
        m, n, k = _log(rng, 1, 8192), _log(rng, 1, 28672), _log(rng, 1, 28672)
        if n * k <= 28672 * 8192 and m * n * k <= most:
            break
    c = {"kind": kind, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "fp32"])}
    if kind in ("forward", "tune"):
        c["quant"] = rng.choice([False, True])
    if kind == "forward":
        c["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"]) if c["quant"] else "bf16"
    return c


def _shapes(case):
    """[(rows, cols, how many)]"""
    out = []
    for item in case["shapes"].split("+"):
        dims, _, count = item.partition("*")
        out.append(tuple(int(d) for d in dims.split("x")) + (int(count or 1),))
    return out


def _each(case):
    return [(r, c) for r, c, b in _shapes(case) for _ in range(b)]


def _segments(shapes, world):
    """[(d0, inner, rows a rank holds, offset in a rank block)] and the block's size."""
    segs, off = [], 0
    for d0, inner in shapes:
        c = -(-d0 // world)
        segs.append((d0, inner, c, off))
        off += c * inner
    return segs, off


def _starts(shapes):
    """Where each parameter starts in one flat buffer (at multiples of 64), and its size."""
    at, pos = [], 0
    for d0, inner in shapes:
        at.append(pos)
        pos += -(-(d0 * inner) // 64) * 64
    return at, pos


def _activation(gen, rows, cols, dtype):
    """Normal values with a few outlier channels, as hidden states have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.7 * torch.randn(cols, generator=gen, device="cuda"))
    return x.to(dtype)


def _gradients(gen, b, r, c, dtype):
    """Momenta as training has them: a few directions far above a floor whose rows and
    columns differ in size."""
    few = max(1, min(r, c) // 64)
    g = torch.randn(b, r, c, generator=gen, device="cuda")
    g *= torch.exp(0.5 * torch.randn(b, r, 1, generator=gen, device="cuda"))
    g *= torch.exp(0.5 * torch.randn(b, 1, c, generator=gen, device="cuda"))
    left = torch.randn(b, r, few, generator=gen, device="cuda")
    right = torch.randn(b, few, c, generator=gen, device="cuda")
    g += torch.matmul(left, right) * (2.0 / math.sqrt(few))
    return (g * 1e-3).to(dtype)


# ------------------------------------------------------------------- plain form

def _pow2(e):
    """2^e in fp32 for whole e in -126..127, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _round_blocks(x):
    """The values of x's 4-bit blocks as e2m1 numbers [R, nb, 32] and exponents [R, nb]."""
    R, C = x.shape
    nb = -(-C // 128) * 4
    t = torch.zeros(R, nb * 32, device=x.device)
    t[:, :C] = x
    t = t.view(R, nb, 32)
    amax = t.abs().amax(-1)
    m, ex = torch.frexp(amax)
    e = torch.where(amax > 0, ex - torch.where(m <= 0.75, 3, 2), 0).clamp(-125, 125)
    y = t * _pow2(-e).unsqueeze(-1)
    a = y.abs().clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, y), e


def _blocks(x):
    """x [R, C] in 4-bit blocks: code bytes [R, Cp / 2] (two e2m1 codes each, the even column
    in the low half) and e8m0 scale bytes [R, Cp / 32]."""
    v, e = _round_blocks(x)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(x.shape[0], -1)
    return code[:, 0::2] + 16 * code[:, 1::2], (e + 127).to(torch.uint8)


def _values(codes, scales, cols):
    """The fp32 values that 4-bit blocks stand for, [R, cols]."""
    R = codes.shape[0]
    code = torch.stack([codes & 15, codes >> 4], -1).view(R, -1)
    m = (code & 7).float()
    v = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(code > 7, -v, v).view(R, -1, 32)
    return (v * _pow2(scales.to(torch.int32) - 127).unsqueeze(-1)).view(R, -1)[:, :cols]


def _rounded(x):
    """x as its 4-bit blocks hold it, in fp32."""
    v, e = _round_blocks(x)
    return (v * _pow2(e).unsqueeze(-1)).view(x.shape[0], -1)[:, :x.shape[1]]


def _ortho(g):
    """A stack [b, r, c] orthogonalised in fp32."""
    a, b, c = COEFFICIENTS
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / x.square().sum((1, 2), keepdim=True).sqrt()
    for _ in range(STEPS):
        p = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    if tall:
        x = x.transpose(1, 2).contiguous()
    return x.to(torch.bfloat16)


# ------------------------------------------------------------------- cases

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = case["kind"]
    s = {"case": dict(case), "kept": {}}
    if kind == "gather":
        shapes, world = _each(case), case["world"]
        segs, S = _segments(shapes, world)
        master = torch.randn(world, S, generator=gen, device="cuda").mul_(0.02)
        for d0, inner, c, off in segs:
            if c * world != d0:         # rows past the end of the parameter are zeros
                rows = master[:, off:off + c * inner].reshape(world * c, inner)
                rows[d0:] = 0
                master[:, off:off + c * inner] = rows.view(world, c * inner)
        s["master"] = master
        return s
    if kind == "ortho":
        s["g"] = [_gradients(gen, b, r, c, TYPES[case["type"]]) for r, c, b in _shapes(case)]
        return s
    m, n, k = case["m"], case["n"], case["k"]
    w = torch.randn(n, k, generator=gen, device="cuda").mul_(0.02)
    s["w"] = _blocks(w)
    if kind in ("forward", "tune"):
        x = _activation(gen, m, k, TYPES[case.get("type", "bf16")])
        s["x"] = x.requires_grad_() if kind == "tune" else x
    if kind in ("backward", "tune"):
        dy = torch.randn(m, n, generator=gen, device="cuda").mul_(1e-3)
        dy *= torch.exp(torch.randn(m, 1, generator=gen, device="cuda"))
        s["dy"] = dy.to(torch.bfloat16)
    return s


def _kept(s, name, make):
    """What a user's program makes once and keeps: plans and buffers."""
    if name not in s["kept"]:
        s["kept"][name] = make()
    return s["kept"][name]


def _flat_params(shapes):
    at, size = _starts(shapes)
    flat = torch.zeros(size, dtype=torch.bfloat16, device="cuda")
    return flat, [flat[a:a + d0 * inner].view(d0, inner) for a, (d0, inner) in zip(at, shapes)]


def _run_own(s):
    import parameter_layout_collectives_amd as tide
    case = s["case"]
    kind = case["kind"]
    if kind == "gather":
        shapes, world = _each(case), case["world"]
        plan = _kept(s, "plan", lambda: tide.Fp4Plan(tide.Plan(shapes, world)))
        gathered = _kept(s, "gathered", lambda: plan.empty(device="cuda"))
        flat, params = _kept(s, "params", lambda: _flat_params(shapes))
        for r in range(world):
            tide.fp4_shard(plan, r, s["master"][r], gathered[r])
        tide.fp4_unshard(plan, gathered, params)
        return flat
    if kind == "ortho":
        return tide.ortho(s["g"], steps=STEPS, coefficients=COEFFICIENTS)
    w = tide.Fp4Blocks(*s["w"], cols=case["k"])
    if kind == "forward":
        return tide.fp4_linear(s["x"], w, dtype=TYPES[case["out"]], quant_x=case["quant"])
    if kind == "backward":
        return tide.fp4_mm_dx(s["dy"], w, dtype=TYPES[case["out"]])
    y = tide.fp4_linear(s["x"], w, dtype=TYPES[case["out"]], quant_x=case["quant"])
    dx, = torch.autograd.grad(y, s["x"], s["dy"].to(y.dtype))
    return {"y": y.detach(), "dx": dx}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    kind = case["kind"]
    if kind == "gather":
        shapes, world = _each(case), case["world"]
        segs, _ = _segments(shapes, world)
        flat, params = _flat_params(shapes)
        for (d0, inner, c, off), p in zip(segs, params):
            full = s["master"][:, off:off + c * inner].reshape(world * c, inner)[:d0]
            p.copy_(_rounded(full))
        return flat
    if kind == "ortho":
        return [_ortho(g) for g in s["g"]]
    w = _values(*s["w"], case["k"])
    out = TYPES[case["out"]]
    if kind == "backward":
        return (s["dy"].float() @ w).to(out)
    x = s["x"].detach()
    x = _rounded(x) if case["quant"] else x.float()
    y = (x @ w.t()).to(out)
    if kind == "forward":
        return y
    return {"y": y, "dx": (s["dy"].float() @ w).to(torch.bfloat16)}


def work(case):
    kind = case["kind"]
    if kind == "gather":
        each = _each(case)
        psi = sum(a * b for a, b in each)
        blk = sum(a * (-(-b // 2) + -(-b // 32)) for a, b in each)
        # masters read, 4-bit blocks written and read, bf16 parameters written
        return {"bytes": 4 * psi + 2 * blk + 2 * psi, "flops": 0}
    if kind == "ortho":
        nbytes = flops = 0
        for r, c, b in _shapes(case):
            lo, hi = min(r, c), max(r, c)
            nbytes += b * r * c * (SIZE[case["type"]] + 2)
            # X X^T and its square are symmetric: half of their products suffice
            flops += STEPS * b * (lo * lo * hi + lo ** 3 + 2 * lo * lo * hi)
        return {"bytes": nbytes, "flops": flops}
    m, n, k, es = case["m"], case["n"], case["k"], SIZE[case["out"]]
    wb = n * (-(-k // 2) + -(-k // 32))
    flops = 2 * m * n * k
    if kind == "forward":
        return {"bytes": m * k * SIZE[case["type"]] + wb + m * n * es, "flops": flops}
    if kind == "backward":
        return {"bytes": m * n * 2 + wb + m * k * es, "flops": flops}
    # x in, y out, dy in, dx out, W twice
    return {"bytes": 2 * m * k * 2 + m * n * (es + 2) + 2 * wb, "flops": 2 * flops}


# ------------------------------------------------------------------- 64 bits

_POWERS = [2.0 ** j for j in range(-400, 401)]
_MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_values(x):
    """The values of x's 4-bit blocks in 64 bits, from the definition: the exponent by
    comparison with 6 * 2^e, the rounding by counting the midpoints below a value."""
    p2 = torch.tensor(_POWERS, dtype=torch.float64, device=x.device)
    mags = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=x.device)
    R, C = x.shape
    nb = -(-C // 32)
    v = torch.nn.functional.pad(x.double(), (0, nb * 32 - C)).view(R, nb, 32)
    top = v.abs().amax(-1)
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -200) / 6)).long() - 1
    for _ in range(3):
        e = e + (top > 6 * p2[e + 400]).long()
    e = torch.where(top > 0, e.clamp(-125, 125), torch.zeros_like(e))
    s = p2[e + 400].unsqueeze(-1)
    a = (v.abs() / s).contiguous()
    mids = (mags[1:] + mags[:-1]) / 2
    # a midpoint goes up from an odd code and stays with an even one
    up = torch.searchsorted(mids, a, right=True)
    down = torch.searchsorted(mids, a, right=False)
    code = torch.where(up % 2 == 0, up, down)
    return (torch.sign(v) * mags[code] * s).view(R, nb * 32)[:, :C]


def _exact_stored(codes, scales, cols):
    """Stored blocks in 64 bits, by a table of the 16 codes."""
    p2 = torch.tensor(_POWERS, dtype=torch.float64, device=codes.device)
    table = torch.tensor(_MAGNITUDES + [-v for v in _MAGNITUDES], dtype=torch.float64,
                         device=codes.device)
    col = torch.arange(cols, device=codes.device)
    byte = codes[:, col // 2].long()
    code = torch.where(col % 2 == 0, byte % 16, byte // 16)
    return table[code] * p2[scales[:, col // 32].long() - 127 + 400]


def _exact_ortho(g):
    """One matrix orthogonalised in 64 bits."""
    a, b, c = COEFFICIENTS
    x = g.double()
    x = x / torch.sqrt(torch.sum(x * x))
    wide = x.shape[0] <= x.shape[1]
    for _ in range(STEPS):
        p = torch.matmul(x, x.t()) if wide else torch.matmul(x.t(), x)
        q = b * p + c * torch.matmul(p, p)
        x = a * x + (torch.matmul(q, x) if wide else torch.matmul(x, q))
    return x


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "gather":
        shapes, world = _each(case), case["world"]
        segs, _ = _segments(shapes, world)
        at, size = _starts(shapes)
        flat = torch.zeros(size, dtype=torch.float64, device="cuda")
        for (d0, inner, c, off), a in zip(segs, at):
            rows = [s["master"][r, off:off + c * inner].view(c, inner) for r in range(world)]
            full = torch.cat(rows)[:d0]
            flat[a:a + d0 * inner] = _exact_values(full).reshape(-1)
        return flat
    if kind == "ortho":
        return [torch.stack([_exact_ortho(m) for m in g]) for g in s["g"]]
    w = _exact_stored(*s["w"], case["k"])
    if kind == "backward":
        return torch.matmul(s["dy"].double(), w)
    x = s["x"].detach()
    x = _exact_values(x) if case["quant"] else x.double()
    y = torch.matmul(x, w.t())
    if kind == "forward":
        return y
    return {"y": y, "dx": torch.matmul(s["dy"].double(), w)}
