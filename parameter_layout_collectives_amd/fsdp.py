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
reduce_scatter() takes.
"""
import contextlib

import torch

from . import BlockPlan, Plan, ag, block_linear, block_shard, grad_table, pack, rs


class TideUnit:
    def __init__(self, shapes, world, device="cuda", align=1, param_dtype=torch.bfloat16,
                 blocks=()):
        self.plan = Plan(shapes, world, align)
        N, S = world, self.plan.S
        self.shapes = [tuple(s) for s in shapes]
        self.world = N
        self.param_dtype = param_dtype
        self.master = torch.zeros(N, S, dtype=torch.float32, device=device)
        self.grad = torch.zeros(N, S, dtype=torch.float32, device=device)
        self.blocks = [int(i) for i in blocks]
        # the parameters gathered in param_dtype, and their plan
        self.rest = [i for i in range(len(self.shapes)) if i not in self.blocks]
        self.rest_plan = self.plan
        if self.blocks:
            self.block_plan = BlockPlan(self.plan, self.blocks)
            self.block_gathered = self.block_plan.empty(device)
            weights = self.block_plan.blocks(device)
            self.rest_plan = Plan([self.shapes[i] for i in self.rest], N, align) \
                if self.rest else None
        S = self.rest_plan.S if self.rest_plan is not None else 0
        self.gathered = torch.zeros(N * S, dtype=param_dtype, device=device)
        self.params = [None] * len(self.shapes)
        for i in self.rest:
            self.params[i] = torch.empty(self.shapes[i], dtype=param_dtype, device=device)
        for j, i in enumerate(self.blocks):
            self.params[i] = weights[j]

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
        for the matrices of `blocks` 8-bit rank blocks -> Blocks."""
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            if not self.blocks:
                self.gathered.view(self.world, self.plan.S).copy_(self.master)
            else:
                for r in range(self.world):
                    block_shard(self.block_plan, r, self.master[r], self.block_gathered[r])
                self._copy_rest()
        if self.blocks:
            views = self.block_plan.views([self.params[i] for i in self.blocks])
            ag(self.block_plan, self.block_gathered, views, small=small, copy_engine=copy_engine,
               stream=stream)
        if self.rest:
            ag(self.rest_plan, self.gathered, [self.params[i] for i in self.rest], small=small,
               copy_engine=copy_engine, stream=stream)

    def _copy_rest(self):
        """The master shards of the parameters outside `blocks`, cast, each at its
        place in the rank blocks of the rest's plan."""
        if not self.rest:
            return
        out = self.gathered.view(self.world, self.rest_plan.S)
        for j, i in enumerate(self.rest):
            src, _, seg = self.plan.param(i)
            dst, _, _ = self.rest_plan.param(j)
            out[:, dst:dst + seg].copy_(self.master[:, src:src + seg])

    def linear(self, i, x, grad=None, accumulate=False, dtype=None, short_sums=False):
        """x [..., k] times parameter i (one of `blocks`, [n, k]) -> [..., n]: see
        block_linear.  grad: where the backward pass writes the weight gradient
        ([n, k], bf16 or fp32), e.g. the tensor that reduce_scatter() will read."""
        if i not in self.blocks:
            raise ValueError(f"parameter {i} is not gathered in blocks")
        return block_linear(x, self.params[i], dtype=dtype, grad=grad, accumulate=accumulate,
                            short_sums=short_sums)
