"""The training step's operators together, as a program uses them: the example of a block with
experts against autograd, the same work captured into graphs and replayed over changed inputs and
spoilt buffers, on other streams, two calls at once, and runs that repeat bit for bit."""
import importlib.util
import os

import pytest
import torch

import gradient_reduction_gb300 as dpr
from tests import gpu_helpers as H
from tests.test_gpu_operators import BF, F32, gen

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("experts_step",
                                                  os.path.join(ROOT, "examples", "experts_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("hidden,out,experts,ranks,tokens", [(256, 320, 4, 2, 200), (200, 136, 5, 4, 77),
                                                             (512, 256, 16, 2, 40)])
def test_block_with_experts(hidden, out, experts, ranks, tokens):
    """Gradients and norm against fp32 autograd.  A step of the 8-bit format is at most 1/63.75 of its
    block's peak and errors are even over it, so their root mean square is at most peak / 221; the
    peak of 32 normal numbers is about 2.2 of their deviations (above 3.5 in 1.5% of blocks), which
    makes 1.0% (1.6%) of the activations' norm, and of their products' with gradients that do not
    depend on the errors; bf16's roundings (2^-8 an element at most) add in squares."""
    H.device()
    m = example()
    g = torch.Generator(device="cuda").manual_seed(1)
    block = m.Block(hidden, out, experts, ranks, g)
    data = m.data(block, tokens, g)
    for max_norm in (1e-2, 1e3):
        parts, outs = m.step(block, data, max_norm)
        norm, grads, dxs = m.autograd(block, data, max_norm)
        assert abs(block.norm.item() - norm) <= 0.02 * norm
        for got, want in zip(block.gradients(parts.view(-1)), grads):
            assert m.relative(got, want) < 0.02
        for (h, z, dx), want, (x, residual, expert, dz, dh) in zip(outs, dxs, data):
            assert torch.equal(h, (x.float() + residual.float()).to(BF))
            assert m.relative(dx, want) < 0.02
        # a second step over the same data: the same bits
        first = [parts.clone(), block.norm.clone()]
        parts, _ = m.step(block, data, max_norm)
        assert torch.equal(parts, first[0]) and torch.equal(block.norm, first[1])


def test_tokens_are_sorted_without_waiting_for_the_device():
    H.device()
    m = example()
    expert = torch.tensor([3, 0, 3, 5, 0, 0, 2], device="cuda")
    m.sort_tokens(expert, 7)                 # what is loaded once is loaded
    torch.cuda.set_sync_debug_mode("error")
    try:
        order, offsets = m.sort_tokens(expert, 7)
    finally:
        torch.cuda.set_sync_debug_mode("default")
    assert order.tolist() == [1, 4, 5, 6, 0, 2, 3]
    assert offsets.dtype == torch.int32 and offsets.tolist() == [0, 3, 3, 4, 6, 6, 7, 7]


class Work:
    """Buffers of all operators, and a pass through them."""

    def __init__(self, rows=300, hidden=264, out=136, seed=0, odd=False):
        pad = 3 if odd else 0                # rows that have to be copied for the tensor core
        def t(r, w, dtype=BF, scale=1.0, s=0):
            v = (scale * torch.randn(r, w + pad, generator=gen(seed + s))).to(dtype).cuda()
            return v[:, :w]
        self.x, self.residual = t(rows, hidden, s=1), t(rows, hidden, s=2)
        self.dz, self.dh = t(rows, out, scale=1e-2, s=3), t(rows, hidden, scale=1e-2, s=4)
        self.weight = t(1, hidden, s=5)[0].contiguous()
        self.linear = t(3 * out, hidden, s=6).unflatten(0, (3, out))
        self.offsets = torch.tensor([0, 100, 110, rows], dtype=torch.int32, device="cuda")
        self.h, self.y, self.dx, self.dy = (t(rows, hidden, s=7) for _ in range(4))
        self.rstd = torch.empty(rows, device="cuda")
        self.h_saved, self.y_saved = (dpr.dpr_checkpoint_empty(rows, hidden) for _ in range(2))
        self.z = t(rows, out, F32, s=8)
        self.dweight = torch.empty(hidden, dtype=BF, device="cuda")
        self.dlinear, self.dlinear8 = (torch.empty(3, out, hidden, device="cuda") for _ in range(2))
        self.clipped = torch.zeros(2 * 3 * out * hidden, device="cuda")
        self.norm = torch.empty(1, device="cuda")
        n = 3 * out * hidden
        self.plan = dpr.dpr_grad_plan_create([self.dlinear, self.dlinear8, self.dweight],
                                             [self.clipped[:n], self.clipped[n:], self.dweight])

    def run(self, **kw):
        dpr.dpr_rmsnorm_forward(self.x, self.weight, 1e-6, self.y, self.rstd, self.residual, self.h,
                                self.h_saved, self.y_saved, **kw)
        dpr.dpr_grouped_linear(self.y, self.offsets, self.linear, self.z, **kw)
        dpr.dpr_grouped_linear_weight_grad(self.dz, self.offsets, self.y, self.dlinear, **kw)
        dpr.dpr_grouped_linear_weight_grad(self.dz, self.offsets, self.y_saved, self.dlinear8, **kw)
        dpr.dpr_grouped_linear_input_grad(self.dz, self.offsets, self.linear, self.dy, **kw)
        dpr.dpr_rmsnorm_backward(self.dy, self.h_saved, self.weight, self.rstd, self.dx, self.dweight,
                                 dh=self.dh, **kw)
        dpr.dpr_grad_norm_clip(self.plan, self.norm, 0.5, scale=0.25, **kw)

    def outputs(self):
        return [self.h, self.y, self.rstd, self.z, self.dlinear, self.dlinear8, self.dy, self.dx,
                self.dweight, self.norm, self.clipped, self.h_saved.codes, self.h_saved.steps,
                self.y_saved.codes, self.y_saved.steps]

    def spoil(self):
        for t in self.outputs():
            t.fill_(float("nan") if t.is_floating_point() else 77)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.outputs()]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("odd", [False, True], ids=["aligned", "odd"])
@pytest.mark.parametrize("programmatic", [True, False])
def test_chains_over_spoilt_buffers(programmatic, odd):
    """A call reads what the call before wrote, on a side stream with and without programmatic
    launches, many times over."""
    H.device()
    w = Work(odd=odd)
    w.run()
    want = w.results()
    old = dpr.dpr_set_programmatic_launch(programmatic)
    try:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(20):
                w.spoil()
                w.run()
        assert same(w.results(), want)
    finally:
        dpr.dpr_set_programmatic_launch(old)


@pytest.mark.parametrize("odd", [False, True], ids=["aligned", "odd"])
def test_captured_and_replayed(odd):
    """Two graphs of the same calls, each with scratch memory of its own, replayed in turn and at
    once with eager calls in between, over inputs that change."""
    H.device()
    a, b = Work(odd=odd), Work(rows=301, seed=40, odd=odd)
    graphs, side = [], torch.cuda.Stream()
    for w in (a, b):
        w.run()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            w.run()
        graphs.append(g)
    for turn in range(3):
        for w in (a, b):
            w.x.copy_(torch.randn(w.x.shape, generator=gen(90 + turn)))
            w.offsets[1] = 60 + 10 * turn
        wants = []
        for w in (a, b):
            w.run()
            wants.append(w.results())
            w.spoil()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        assert same(a.results(), wants[0]) and same(b.results(), wants[1])


def test_streams_given_with_the_call():
    H.device()
    w = Work()
    w.run()
    want = w.results()
    for stream in (torch.cuda.Stream(), 0, torch.cuda.Stream().cuda_stream):
        w.spoil()
        torch.cuda.synchronize()
        w.run(stream=stream)
        assert same(w.results(), want)


def test_two_calls_at_once():
    """The same inputs, plan tensors apart, on two streams at the same time."""
    H.device()
    a, b = Work(seed=5), Work(seed=5)
    a.run()
    want = a.results()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a.spoil()
        b.spoil()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            a.run()
        with torch.cuda.stream(t):
            b.run()
    assert same(a.results(), want) and same(b.results(), want)


def test_no_wait_ran_out():
    H.device()
    assert dpr.dpr_device_wait_failures() == 0
