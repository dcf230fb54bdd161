"""The weights' gradient of block_linear, the streams of its passes, and what it keeps."""
import pytest
import torch

import parameter_layout_collectives_amd as tide
from gpu_helpers import note
from test_gpu_blocks import BF, FP, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x_grad", [False, True])
@pytest.mark.parametrize("two", [False, True])
def test_weight_gradient_is_ordered_before_the_caller(x_grad, two):
    """Forward on a side stream, backward() called from another one, which reads
    `grad` right away: much work is queued on the side stream before the backward
    pass's, so an unordered read would find the old values."""
    note(f"block_linear backward from another stream, x_grad={x_grad}, two layers={two}")
    m, n, k = 200, 264, 392
    w, w2 = (tide.block_quant(rand(s, 2 + i, FP, 0.02)) for i, s in enumerate([(n, k), (k, n)]))
    dy = rand((m, k if two else n), 3, BF, 1e-3)
    big = rand((4096, 4096), 4)
    x = rand((m, k), 1)

    def passes(stream, grads):
        xl = x.clone().requires_grad_(x_grad)
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            y = tide.block_linear(xl, w, grad=grads[0])
            if two:
                y = tide.block_linear(y, w2, grad=grads[1])
            for _ in range(20):
                big @ big
        y.backward(dy)
        return [g.clone() for g in grads] + ([xl.grad.clone()] if x_grad else [])

    here = torch.cuda.current_stream()
    shapes = [(n, k), (k, n)]
    want = passes(here, [torch.full(s, 7.0, device="cuda") for s in shapes])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    grads = [torch.full(s, 7.0, device="cuda") for s in shapes]
    got = passes(side, grads)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not bool((want[0] == 7.0).any())


@pytest.mark.parametrize("m", [3, 40, 200])
def test_frozen_weights_keep_nothing_of_x(m):
    note(f"block_linear with frozen weights keeps no checkpoint {m}")
    n, k = 72, 264
    w = tide.block_quant(rand((n, k), 2, FP, 0.02))
    x, dy = rand((m, k), 1).requires_grad_(), rand((m, n), 3, BF, 1e-3)
    kept = []

    def pack(t):
        kept.append(t.data_ptr())
        return t
    weights = [w.codes.data_ptr(), w.scales.data_ptr()]
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        y = tide.block_linear(x, w)
        assert kept == weights
        dw = torch.empty(n, k, device="cuda")
        same = tide.block_linear(x, w, grad=dw)
    assert kept[2:4] == weights and len(kept) == 6
    assert torch.equal(y, same)
    y.backward(dy)
    assert torch.equal(x.grad, tide.block_mm_dx(dy, w))


def test_weight_gradient_of_autograd_grad():
    """The same through torch.autograd.grad(), which runs no leaf's accumulation."""
    note("block_linear autograd.grad from another stream")
    m, n, k = 200, 264, 392
    w, dy, x = tide.block_quant(rand((n, k), 2, FP, 0.02)), rand((m, n), 3, BF, 1e-3), rand((m, k), 1)
    big = rand((4096, 4096), 4)
    want = tide.block_mm_dw(dy, tide.block_quant(x), dtype=FP)
    dw = torch.full((n, k), 7.0, device="cuda")
    xl = x.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = tide.block_linear(xl * 1.0, w, grad=dw)
        for _ in range(20):
            big @ big
    dx, = torch.autograd.grad(y, xl, dy)
    got, dx = dw.clone(), dx.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(dx, tide.block_mm_dx(dy, w))


def test_captured_weight_gradient_alone():
    """A captured forward and backward pass over an x that needs no gradient."""
    note("block_linear captured, x without gradient")
    m, n, k = 70, 96, 640
    w, dy = tide.block_quant(rand((n, k), 43, FP, 0.02)), rand((m, n), 44, BF, 1e-3)
    x, dw = rand((m, k), 45), torch.zeros(n, k, device="cuda")

    def step(grad):
        y = tide.block_linear(x, w, grad=grad, accumulate=True)
        y.backward(dy)
        return y.detach()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(torch.zeros_like(dw))                     # one pass outside the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        y = step(dw)
    total = torch.zeros_like(dw)
    dw.zero_()
    for it in range(3):
        x.copy_(rand((m, k), 46 + it))
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step(total)) and torch.equal(dw, total)
