"""The 8-bit block operators of an FSDP unit as timed cases: the gather of sharded weights
in 8 bits, the activation checkpoint, the product that reads 8-bit weights, and its backward.

A matrix [R, C] in 8-bit blocks has, for each row and each run of 128 columns, one power of
two 2^e and 128 e4m3 numbers.  e is the smallest integer with max|x| <= 448 * 2^e over the
finite values of the run (within -117..119; 0 where there is none but zeros), and every x
becomes the e4m3 number nearest to x / 2^e, ties to even.

Kinds of cases (every size is that of the matrices as a user has them):
  gather      fp32 master shards of all ranks -> 8-bit rank blocks -> full bf16 parameters
  checkpoint  an activation saved in 8-bit blocks and restored
  forward     y = q(x) w^T, x quantised on the way, w held in 8-bit blocks
  backward    dx = dy w and dw = dy^T x, with w and the checkpoint x in 8-bit blocks
  step        forward and backward of one linear layer through autograd
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}

# The matrices of a Llama-3-8B-shaped decoder layer and of a Qwen3-30B-A3B-shaped MoE layer,
# as the repository's own workloads list them (the norms stay out: they are not matrices).
LAYER_8B = "4096x4096*2+1024x4096*2+14336x4096*2+4096x14336"
LAYER_MOE = "4096x2048+512x2048*2+2048x4096+128x2048+768x2048*256+2048x768*128"


def listed():
    return [
        # a unit of small matrices whose rows do not divide by the ranks and whose rows end
        # inside a block: the shortest gather
        {"name": "gather, small odd unit", "kind": "gather", "shapes": "333x1000+37x129+64x64",
         "world": 6},
        # a dense decoder layer over one node
        {"name": "gather, 8B layer", "kind": "gather", "shapes": LAYER_8B, "world": 8},
        # 389 matrices over two nodes: many short segments
        {"name": "gather, MoE layer", "kind": "gather", "shapes": LAYER_MOE, "world": 16},
        # one token's activation, where only the latency counts
        {"name": "checkpoint, one row", "kind": "checkpoint", "rows": 1, "cols": 4096,
         "type": "bf16"},
        # the hidden states of 8K tokens of a 70B-shaped layer
        {"name": "checkpoint, 8K tokens", "kind": "checkpoint", "rows": 8192, "cols": 8192,
         "type": "bf16"},
        # one token through the 8B layer's gate projection: a serving step, W's bytes bound it
        {"name": "forward, one token", "kind": "forward", "m": 1, "n": 14336, "k": 4096,
         "type": "bf16", "out": "bf16"},
        # a decode batch of 32 through the 70B layer's down projection
        {"name": "forward, 32 rows", "kind": "forward", "m": 32, "n": 8192, "k": 28672,
         "type": "bf16", "out": "bf16"},
        # a ragged micro-batch through an odd matrix, fp32 in and out
        {"name": "forward, odd", "kind": "forward", "m": 777, "n": 1000, "k": 1111,
         "type": "fp32", "out": "fp32"},
        # 8K tokens through the 70B layer's gate projection: the largest product
        {"name": "forward, 70B gate", "kind": "forward", "m": 8192, "n": 28672, "k": 8192,
         "type": "bf16", "out": "bf16"},
        # one expert's share of a micro-batch in the MoE layer, fp32 weight gradient
        {"name": "backward, expert", "kind": "backward", "m": 509, "n": 768, "k": 2048,
         "out": "fp32"},
        # 8K tokens back through the 8B layer's gate projection
        {"name": "backward, 8B gate", "kind": "backward", "m": 8192, "n": 14336, "k": 4096,
         "out": "bf16"},
        # a training step of the 70B layer's output projection on 4K tokens
        {"name": "step, 70B o_proj", "kind": "step", "m": 4096, "n": 8192, "k": 8192,
         "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["gather", "checkpoint", "forward", "forward", "backward", "step"])
    if kind == "gather":
        shapes = ["%dx%d" % (_log(rng, 1, 8192), _log(rng, 1, 8192))
                  for _ in range(rng.randint(1, 6))]
        return {"kind": kind, "shapes": "+".join(shapes), "world": _log(rng, 1, 64)}
    if kind == "checkpoint":
        return {"kind": kind, "rows": _log(rng, 1, 8192), "cols": _log(rng, 1, 8192),
                "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    # at most the largest listed product's multiplications (a backward pass makes two
    # products, a step three)
    most = 8192 * 28672 * 8192 // {"forward": 1, "backward": 2, "step": 3}[kind]
    while True:
        m, n, k = _log(rng, 1, 8192), _log(rng, 1, 28672), _log(rng, 1, 28672)
        if n * k <= 28672 * 8192 and m * n * k <= most:
            break
    c = {"kind": kind, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "fp32"])}
    if kind == "forward":
        c["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return c


def _shapes(case):
    out = []
    for item in case["shapes"].split("+"):
        dims, _, count = item.partition("*")
        out += [tuple(int(d) for d in dims.split("x"))] * int(count or 1)
    return out


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


# ------------------------------------------------------------------- plain form

def _pow2(e):
    """2^e in fp32 for whole e in -126..127, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _blocks(x):
    """x [R, C] in 8-bit blocks: e4m3 codes [R, Cp] and e8m0 scale bytes [R, Sp]."""
    R, C = x.shape
    nb = -(-C // 128)
    t = torch.zeros(R, nb * 128, device=x.device)
    t[:, :C] = x
    t = t.view(R, nb, 128)
    finite = torch.isfinite(t)
    amax = torch.where(finite, t.abs(), torch.zeros_like(t)).amax(-1)
    m, ex = torch.frexp(amax)
    e = torch.where(amax > 0, ex - torch.where(m <= 0.875, 9, 8), 0).clamp(-117, 119)
    scaled = (t * _pow2(-e).unsqueeze(-1)).clamp(-448.0, 448.0)
    scaled = torch.where(finite, scaled, torch.full_like(scaled, math.nan))
    codes = scaled.to(torch.float8_e4m3fn).view(R, nb * 128)
    scales = torch.full((R, -(-nb // 4) * 4), 127, dtype=torch.uint8, device=x.device)
    scales[:, :nb] = (e + 127).to(torch.uint8)
    return codes, scales


def _values(codes, scales, cols):
    """The fp32 values that 8-bit blocks stand for, [R, cols]."""
    R, cp = codes.shape
    e = scales[:, :cp // 128].to(torch.int32) - 127
    return (codes.float().view(R, cp // 128, 128) * _pow2(e).unsqueeze(-1)).view(R, cp)[:, :cols]


# ------------------------------------------------------------------- cases

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = case["kind"]
    s = {"case": dict(case), "kept": {}}
    if kind == "gather":
        shapes, world = _shapes(case), case["world"]
        segs, S = _segments(shapes, world)
        master = torch.randn(world, S, generator=gen, device="cuda").mul_(0.02)
        for d0, inner, c, off in segs:
            if c * world != d0:         # rows past the end of the parameter are zeros
                rows = master[:, off:off + c * inner].reshape(world * c, inner)
                rows[d0:] = 0
                master[:, off:off + c * inner] = rows.view(world, c * inner)
        s["master"] = master
        return s
    if kind == "checkpoint":
        s["x"] = _activation(gen, case["rows"], case["cols"], TYPES[case["type"]])
        return s
    m, n, k = case["m"], case["n"], case["k"]
    x = _activation(gen, m, k, TYPES[case.get("type", "bf16")])
    w = torch.randn(n, k, generator=gen, device="cuda").mul_(0.02)
    s["w"] = _blocks(w)
    if kind == "backward":
        s["x"] = _blocks(x)
    else:
        s["x"] = x.requires_grad_() if kind == "step" else x
    if kind in ("backward", "step"):
        dy = torch.randn(m, n, generator=gen, device="cuda").mul_(1e-3)
        dy *= torch.exp(torch.randn(m, 1, generator=gen, device="cuda"))
        s["dy"] = dy.to(torch.bfloat16)
    return s


def _kept(s, name, make):
    """What a user's program makes once and keeps: plans and buffers."""
    if name not in s["kept"]:
        s["kept"][name] = make()
    return s["kept"][name]


def _run_own(s):
    import parameter_layout_collectives_amd as tide
    case = s["case"]
    kind = case["kind"]
    if kind == "gather":
        shapes, world = _shapes(case), case["world"]
        plan = _kept(s, "plan", lambda: tide.BlockPlan(tide.Plan(shapes, world)))
        gathered = _kept(s, "gathered", lambda: plan.empty(device="cuda"))
        flat, params = _kept(s, "params", lambda: _flat_params(shapes))
        for r in range(world):
            tide.block_shard(plan, r, s["master"][r], gathered[r])
        tide.block_unshard(plan, gathered, params)
        return flat
    if kind == "checkpoint":
        return tide.block_dequant(tide.block_quant(s["x"]), dtype=s["x"].dtype)
    w = tide.Blocks(*s["w"], cols=case["k"])
    if kind == "forward":
        return tide.block_linear(s["x"], w, dtype=TYPES[case["out"]])
    if kind == "backward":
        x = tide.Blocks(*s["x"], cols=case["k"])
        return {"dx": tide.block_mm_dx(s["dy"], w),
                "dw": tide.block_mm_dw(s["dy"], x, dtype=TYPES[case["out"]])}
    dw = torch.empty(case["n"], case["k"], dtype=TYPES[case["out"]], device="cuda")
    y = tide.block_linear(s["x"], w, grad=dw)
    dx, = torch.autograd.grad(y, s["x"], s["dy"])
    return {"y": y, "dx": dx, "dw": dw}


def _flat_params(shapes):
    at, size = _starts(shapes)
    flat = torch.zeros(size, dtype=torch.bfloat16, device="cuda")
    return flat, [flat[a:a + d0 * inner].view(d0, inner) for a, (d0, inner) in zip(at, shapes)]


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    kind = case["kind"]
    if kind == "gather":
        shapes, world = _shapes(case), case["world"]
        segs, _ = _segments(shapes, world)
        flat, params = _flat_params(shapes)
        for (d0, inner, c, off), p in zip(segs, params):
            full = s["master"][:, off:off + c * inner].reshape(world * c, inner)[:d0]
            p.copy_(_values(*_blocks(full), inner))
        return flat
    if kind == "checkpoint":
        return _values(*_blocks(s["x"]), case["cols"]).to(s["x"].dtype)
    w = _values(*s["w"], case["k"])
    if kind == "backward":
        x = _values(*s["x"], case["k"])
    else:
        x = _values(*_blocks(s["x"].detach()), case["k"])
    out = TYPES[case["out"]]
    if kind == "forward":
        return (x @ w.t()).to(out)
    dy = s["dy"].float()
    r = {"dx": (dy @ w).to(torch.bfloat16), "dw": (dy.t() @ x).to(out)}
    if kind == "step":
        r["y"] = (x @ w.t()).to(torch.bfloat16)
    return r


def work(case):
    kind = case["kind"]
    if kind == "gather":
        psi = sum(a * b for a, b in _shapes(case))
        blk = sum(a * (b + -(-b // 128)) for a, b in _shapes(case))
        # masters read, 8-bit blocks written and read, bf16 parameters written
        return {"bytes": 4 * psi + 2 * blk + 2 * psi, "flops": 0}
    if kind == "checkpoint":
        r, c, es = case["rows"], case["cols"], SIZE[case["type"]]
        return {"bytes": r * (2 * es * c + 2 * (c + -(-c // 128))), "flops": 0}
    m, n, k, es = case["m"], case["n"], case["k"], SIZE[case["out"]]
    kb = k + -(-k // 128)
    flops = 2 * m * n * k
    if kind == "forward":
        return {"bytes": m * k * SIZE[case["type"]] + n * kb + m * n * es, "flops": flops}
    back = m * n * 2 + n * kb + m * kb + m * k * 2 + n * k * es
    if kind == "backward":
        return {"bytes": back, "flops": 2 * flops}
    # x in, its checkpoint out and in again, W twice, dy, y, dx and dw
    return {"bytes": back + m * k * 2 + m * kb + n * kb + m * n * 2, "flops": 3 * flops}


# ------------------------------------------------------------------- 64 bits

_POWERS = [2.0 ** j for j in range(-400, 401)]


def _exact_values(x, block=128):
    """The values of x's 8-bit blocks in 64 bits, from the definition: the exponent by
    comparison with 448 * 2^e, the rounding by the spacing of e4m3 numbers."""
    p2 = torch.tensor(_POWERS, dtype=torch.float64, device=x.device)
    R, C = x.shape
    nb = -(-C // block)
    v = torch.nn.functional.pad(x.double(), (0, nb * block - C)).view(R, nb, block)
    a = v.abs()
    top = torch.where(torch.isfinite(a), a, 0.0).amax(-1)
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -200) / 448)).long() - 1
    for _ in range(3):
        e = e + (top > 448 * p2[e + 400]).long()
    e = torch.where(top > 0, e.clamp(-117, 119), torch.zeros_like(e))
    s = p2[e + 400].unsqueeze(-1)
    a = (a / s).clamp_max(448.0)
    lead = torch.frexp(a)[1].long() - 1
    step = p2[lead.clamp_min(-6) - 3 + 400]
    q = torch.sign(v) * torch.round(a / step) * step * s
    q = torch.where(torch.isfinite(v), q, math.nan)
    return q.view(R, nb * block)[:, :C]


def _exact_stored(codes, scales, cols):
    """Stored blocks in 64 bits, read bit by bit: sign, 4 exponent and 3 fraction bits."""
    p2 = torch.tensor(_POWERS, dtype=torch.float64, device=codes.device)
    b = torch.arange(256, device=codes.device)
    ex, fr = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(ex == 0, fr * 2.0 ** -9, (8 + fr) * p2[ex - 10 + 400])
    table = torch.where(b >= 128, -mag, mag)
    table[127] = table[255] = math.nan
    v = table[codes.view(torch.uint8).long()[:, :cols]]
    s = p2[scales.long() - 127 + 400].repeat_interleave(128, dim=1)[:, :cols]
    return v * s


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "gather":
        shapes, world = _shapes(case), case["world"]
        segs, _ = _segments(shapes, world)
        at, size = _starts(shapes)
        flat = torch.zeros(size, dtype=torch.float64, device="cuda")
        for (d0, inner, c, off), a in zip(segs, at):
            rows = [s["master"][r, off:off + c * inner].view(c, inner) for r in range(world)]
            full = torch.cat(rows)[:d0]
            flat[a:a + d0 * inner] = _exact_values(full).reshape(-1)
        return flat
    if kind == "checkpoint":
        return _exact_values(s["x"])
    k = case["k"]
    w = _exact_stored(*s["w"], k)
    if kind == "backward":
        x = _exact_stored(*s["x"], k)
    else:
        x = _exact_values(s["x"].detach())
    if kind == "forward":
        return torch.matmul(x, w.t())
    dy = s["dy"].double()
    r = {"dx": torch.matmul(dy, w), "dw": torch.matmul(dy.t(), x)}
    if kind == "step":
        r["y"] = torch.matmul(x, w.t())
    return r
