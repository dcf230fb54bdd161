"""One FSDP unit with TIDE's collectives in place of FSDP2's layout copies.

FSDP2 keeps every parameter (and its gradient) as its own tensor, while its
collectives work on one flat rank-major buffer, so each step packs the
gradients into that buffer before the reduce-scatter and copies the
all-gathered buffer back out into the parameters ("FSDP通信终局：TIDE零拷贝
集合通信优化", §"FSDP2通信开销的根源").  TIDE folds both layout changes into
the collectives' addressing (§"TIDE的设计思路").  TideUnit holds one unit's
state laid out that way on one device, for N ranks:

    master   [N, S] fp32   rank r's shard of the master weights = row r
    grad     [N, S] fp32   rank r's reduced gradient shard = row r
    gathered [N*S]  bf16   the all-gather buffer (rank-major)
    params   P tensors     the unsharded parameters, each its own tensor

reduce_scatter() runs tide_rs for every rank straight from the per-parameter
gradients (fp32 reduction, the mean by default: tqpw.cn "FSDP技术演进全景图"
§3.2 reduces in fp32; apxml "Communication volume analysis" §"分片中的通信
原语" averages).  all_gather() casts the master shards into the gathered
buffer and places it with tide_ag.  The optimizer updates `master` from
`grad` in between, shard by shard.  With all N ranks in one device's memory
this is one GPU's emulation of the data-parallel group; across GPUs each
rank would hold only its rows and its peers' blocks would arrive over the
network.

With `blocks`, the matrices named there are gathered in 8-bit blocks instead:
all_gather() casts their master shards into 8-bit rank blocks and places those,
half the bytes of a bf16 gather, and params holds them as Blocks, which
linear() multiplies by without ever making them bf16.  Its backward pass reads
an 8-bit checkpoint of the layer's input and writes the weight gradient that
reduce_scatter() takes.  `fp4` does the same with 4-bit blocks, about a quarter of
the bytes, for weights that are frozen, serve, or train behind 4-bit products.

muon_step() is the optimizer's step in between for the unit's matrices: momentum
on the shards, the update gathered as parameters are, orthogonalised (ortho.py) and
scattered back onto the master shards.
"""
import contextlib

import torch

from . import (BlockPlan, Fp4Plan, Plan, ag, block_linear, block_shard, fp4_linear, fp4_shard,
               grad_table, ortho, pack, rs)
from .ortho import COEFFICIENTS, check_steps


class TideUnit:
    def __init__(self, shapes, world, device="cuda", align=1, param_dtype=torch.bfloat16,
                 blocks=(), fp4=()):
        self.plan = Plan(shapes, world, align)
        N, S = world, self.plan.S
        self.shapes = [tuple(s) for s in shapes]
        self.world = N
        self.param_dtype = param_dtype
        self.master = torch.zeros(N, S, dtype=torch.float32, device=device)
        self.grad = torch.zeros(N, S, dtype=torch.float32, device=device)
        self.blocks = [int(i) for i in blocks]
        self.fp4 = [int(i) for i in fp4]
        if set(self.blocks) & set(self.fp4):
            raise ValueError("a parameter is named in blocks and in fp4")
        # the parameters gathered in param_dtype, and their plan
        coded = self.blocks + self.fp4
        self.rest = [i for i in range(len(self.shapes)) if i not in coded]
        self.rest_plan = self.plan
        self.params = [None] * len(self.shapes)
        # (indices, plan, gathered buffer, shard call) of the matrices in blocks
        self._coded = []
        if self.blocks:
            self.block_plan = BlockPlan(self.plan, self.blocks)
            self.block_gathered = self.block_plan.empty(device)
            self._coded.append((self.blocks, self.block_plan, self.block_gathered, block_shard))
        if self.fp4:
            self.fp4_plan = Fp4Plan(self.plan, self.fp4)
            self.fp4_gathered = self.fp4_plan.empty(device)
            self._coded.append((self.fp4, self.fp4_plan, self.fp4_gathered, fp4_shard))
        if coded:
            self.rest_plan = Plan([self.shapes[i] for i in self.rest], N, align) \
                if self.rest else None
        S = self.rest_plan.S if self.rest_plan is not None else 0
        self.gathered = torch.zeros(N * S, dtype=param_dtype, device=device)
        for i in self.rest:
            self.params[i] = torch.empty(self.shapes[i], dtype=param_dtype, device=device)
        for indices, plan, _, _ in self._coded:
            for i, w in zip(indices, plan.blocks(device)):
                self.params[i] = w
        self.momentum = None     # [N, S] fp32, made by the first muon_step
        self._muon = None        # its matrices and their plan

    def load(self, full):
        """Shard full fp32 tensors into the master rows (tide_pack of 4-byte
        elements; padding stays 0) and place them into `params`."""
        tensors = [t.detach().to(device=self.master.device, dtype=torch.float32).contiguous()
                   for t in full]
        pack(self.plan, tensors, self.master.view(-1))
        self.all_gather()

    def reduce_scatter(self, grads, avg=True, small=False, stream=None):
        """grads[r][i] = rank r's gradient of parameter i (bf16, fp16 or fp32,
        one dtype): row r of `grad` becomes rank r's reduced shard."""
        table = grad_table(self.plan, grads)
        for R in range(self.world):
            rs(self.plan, R, table, self.grad[R], small=small, avg=avg, stream=stream)

    def all_gather(self, small=False, copy_engine=False, stream=None):
        """Master shards -> param dtype into the gathered buffer -> params, and
        for the matrices of `blocks` and `fp4` 8-bit or 4-bit rank blocks -> Blocks or
        Fp4Blocks."""
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            if not self._coded:
                self.gathered.view(self.world, self.plan.S).copy_(self.master)
            else:
                for _, plan, gathered, shard in self._coded:
                    for r in range(self.world):
                        shard(plan, r, self.master[r], gathered[r])
                if self.rest:
                    self._copy_segments(self.master, self.rest, self.rest_plan,
                                        self.gathered.view(self.world, self.rest_plan.S))
        for indices, plan, gathered, _ in self._coded:
            ag(plan, gathered, plan.views([self.params[i] for i in indices]), small=small,
               copy_engine=copy_engine, stream=stream)
        if self.rest:
            ag(self.rest_plan, self.gathered, [self.params[i] for i in self.rest], small=small,
               copy_engine=copy_engine, stream=stream)

    def _copy_segments(self, shards, select, plan, out):
        """The shards of the parameters `select`, cast, each at its place in the rank
        blocks `out` of their own plan."""
        for j, i in enumerate(select):
            src, _, seg = self.plan.param(i)
            dst, _, _ = plan.param(j)
            out[:, dst:dst + seg].copy_(shards[:, src:src + seg])

    def muon_step(self, lr, momentum=0.95, nesterov=True, weight_decay=0.0, select=None,
                  scale=None, steps=5, coefficients=COEFFICIENTS):
        """One Muon step on the master shards, from `grad` as reduce_scatter() left it:

            buf <- momentum * buf + grad            (fp32, on the shards)
            u    = grad + momentum * buf, or buf without nesterov
            O    = ortho(u), the whole matrix in bf16
            W   <- (1 - lr * weight_decay) W - lr * scale(rows, cols) * O

        select: the parameters that are updated, by default all 2-D ones, the same in
        every call; others are left as they are, for another optimizer.  A parameter of
        more dimensions is taken as the matrix [dim0, inner].  scale: by default
        sqrt(max(1, rows / cols)).  all_gather() then makes params of the new W.  A call
        that is refused leaves the unit as it was."""
        if select is None:
            select = [i for i, s in enumerate(self.shapes) if len(s) == 2]
        select = [int(i) for i in select]
        if not select:
            return
        if not all(0 <= i < len(self.shapes) for i in select):
            raise ValueError(f"select {select} holds an index out of range")
        if len(set(select)) != len(select):
            raise ValueError(f"select {select} holds an index twice")
        if self._muon is not None and self._muon[0] != select:
            raise ValueError(f"earlier steps updated parameters {self._muon[0]}, not {select}")
        check_steps(steps, coefficients)
        lr, momentum, weight_decay = float(lr), float(momentum), float(weight_decay)
        factors = [self._muon_factor(i, lr, scale) for i in select]
        if self._muon is None:
            plan = Plan([self.shapes[i] for i in select], self.world, self.plan.align)
            self.momentum = torch.zeros_like(self.master)
            self._muon = select, plan
        plan, device = self._muon[1], self.master.device
        if not plan.S:           # matrices without elements only
            return
        u = torch.zeros(self.world, plan.S, dtype=torch.bfloat16, device=device)
        for j, i in enumerate(select):
            src, _, seg = self.plan.param(i)
            dst, _, _ = plan.param(j)
            buf, g = self.momentum[:, src:src + seg], self.grad[:, src:src + seg]
            buf.mul_(momentum).add_(g)
            u[:, dst:dst + seg].copy_(torch.add(g, buf, alpha=momentum) if nesterov else buf)
        full = [torch.empty(self.shapes[i], dtype=torch.bfloat16, device=device) for i in select]
        ag(plan, u.view(-1), full)
        mats = [t.view(t.shape[0] if t.dim() else 1, -1) for t in full if t.numel()]
        ortho(mats, out=mats, steps=steps, coefficients=coefficients)
        pack(plan, full, u.view(-1))
        for j, i in enumerate(select):
            src, _, seg = self.plan.param(i)
            dst, _, _ = plan.param(j)
            if not seg:
                continue
            w = self.master[:, src:src + seg]
            if weight_decay:
                w.mul_(1 - lr * weight_decay)
            w.add_(u[:, dst:dst + seg], alpha=factors[j])

    def _muon_factor(self, i, lr, scale):
        shape = self.shapes[i]
        rows, cols = shape[0] if shape else 1, torch.Size(shape[1:]).numel()
        if not rows or not cols:
            return 0.0
        k = scale(rows, cols) if scale is not None else max(1.0, rows / cols) ** 0.5
        return -lr * float(k)

    def linear(self, i, x, grad=None, accumulate=False, dtype=None, short_sums=False,
               quant_x=False):
        """x [..., k] times parameter i (one of `blocks` or `fp4`, [n, k]) -> [..., n]:
        see block_linear (short_sums) and fp4_linear (quant_x).  grad: where the
        backward pass writes the weight gradient ([n, k], bf16 or fp32), e.g. the
        tensor that reduce_scatter() will read."""
        if i in self.fp4:
            if short_sums:
                raise ValueError("short_sums is for parameters in 8-bit blocks")
            return fp4_linear(x, self.params[i], dtype=dtype, quant_x=quant_x, grad=grad,
                              accumulate=accumulate)
        if i not in self.blocks:
            raise ValueError(f"parameter {i} is not gathered in blocks")
        if quant_x:
            raise ValueError("quant_x is for parameters in 4-bit blocks")
        return block_linear(x, self.params[i], dtype=dtype, grad=grad, accumulate=accumulate,
                            short_sums=short_sums)
