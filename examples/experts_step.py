"""One training step of a block with experts on K data-parallel ranks (simulated as K buffers of one
GPU), from the norm to the clipped gradients:

    forward   h = x + residual, y = rmsnorm(h)   both saved in 8 bits in the same pass
              tokens sorted by expert, z = y W_e^T
    backward  dW_e = dz^T y~                     from y's checkpoint, into the rank's bucket
              dy = dz W_e, back in token order
              dx, dweight                        from h's checkpoint; dx adds the residual stream's gradient
    reduce    the K buckets' mean, scattered as fp32 partitions
    clip      the global norm of the partitions, and the partitions scaled to a largest norm

    python examples/experts_step.py [--ranks 2] [--tokens 4096] [--hidden 4096] [--out 4096] [--experts 8]

prints the norm and how far the clipped gradients are from those of an fp32 autograd pass.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gradient_reduction_gb300 as dpr  # noqa: E402

EPS = 1e-6
BF = torch.bfloat16


class Block:
    """Parameters of the block, their places in a rank's flat bucket, and the plan of the clipping."""

    def __init__(self, hidden: int, out: int, experts: int, ranks: int, gen: torch.Generator):
        self.hidden, self.out, self.experts, self.ranks = hidden, out, experts, ranks
        self.weight = (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).to(BF)
        self.linear = (torch.randn(experts, out, hidden, generator=gen, device="cuda") / hidden ** 0.5).to(BF)
        # arrival order of a backward pass; places are multiples of 16 elements (32 bytes)
        n = experts * out * hidden
        self.places = [(0, (experts, out, hidden)), (-(-n // 16) * 16, (hidden,))]
        unit = 16 * ranks
        self.numel = -(-(self.places[1][0] + hidden) // unit) * unit
        self.parts = torch.zeros(ranks, self.numel // ranks, device="cuda")
        self.norm = torch.empty(1, device="cuda")
        self.plan = dpr.dpr_grad_plan_create(list(self.parts))

    def gradients(self, bucket: torch.Tensor):
        """Views of a bucket: the gradients of linear and weight."""
        return [bucket[at:at + torch.Size(shape).numel()].view(shape) for at, shape in self.places]


def sort_tokens(expert: torch.Tensor, experts: int):
    """The order that sorts tokens by expert, and the experts' offsets, without leaving the device."""
    by_expert, order = torch.sort(expert, stable=True)
    # (torch.bincount would wait for the device: the length of its result is the largest value's)
    return order, torch.searchsorted(by_expert, torch.arange(experts + 1, device="cuda"), out_int32=True)


def forward(block: Block, x: torch.Tensor, residual: torch.Tensor, expert: torch.Tensor):
    """(h, z in token order), and what the backward pass needs."""
    rows = x.shape[0]
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    h_saved, y_saved = (dpr.dpr_checkpoint_empty(rows, block.hidden) for _ in range(2))
    dpr.dpr_rmsnorm_forward(x, block.weight, EPS, y, rstd, residual, h, h_saved, y_saved)
    order, offsets = sort_tokens(expert, block.experts)
    z = torch.empty(rows, block.out, dtype=BF, device="cuda")
    dpr.dpr_grouped_linear(y[order], offsets, block.linear, z)
    back = torch.empty_like(z)
    back[order] = z
    return h, back, (h_saved, y_saved, rstd, order, offsets)


def backward(block: Block, dz: torch.Tensor, dh: torch.Tensor, kept, bucket: torch.Tensor):
    """dx, the gradient of x and of the residual; the parameters' gradients go into `bucket`."""
    h_saved, y_saved, rstd, order, offsets = kept
    dlinear, dweight = block.gradients(bucket)
    dz = dz[order]
    sorted_y = dpr.Checkpoint(y_saved.codes[order], y_saved.steps[order])
    dpr.dpr_grouped_linear_weight_grad(dz, offsets, sorted_y, dlinear)
    dy = torch.empty(dz.shape[0], block.hidden, dtype=BF, device="cuda")
    dpr.dpr_grouped_linear_input_grad(dz, offsets, block.linear, dy)
    dx = torch.empty_like(dy)
    dx[order] = dy
    dpr.dpr_rmsnorm_backward(dx, h_saved, block.weight, rstd, dx, dweight, dh=dh)
    return dx


def step(block: Block, ranks, max_norm: float):
    """The clipped fp32 partitions of the mean gradient, and each rank's (h, z, dx)."""
    buckets = torch.zeros(block.ranks, block.numel, dtype=BF, device="cuda")
    outs = []
    for r, (x, residual, expert, dz, dh) in enumerate(ranks):
        h, z, kept = forward(block, x, residual, expert)
        outs.append((h, z, backward(block, dz, dh, kept, buckets[r])))
    dpr.dpr_reduce_scatter(buckets, block.ranks, 1, block.numel, block.parts)
    dpr.dpr_grad_norm_clip(block.plan, block.norm, max_norm)
    return block.parts, outs


def autograd(block: Block, ranks, max_norm: float):
    """The norm, the clipped mean gradients of (linear, weight) and each rank's dx, in fp32."""
    params = [p.float().requires_grad_() for p in (block.linear, block.weight)]
    dxs = []
    for x, residual, expert, dz, dh in ranks:
        h = (x.float() + residual.float()).requires_grad_()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * params[1]
        loss = (h * dh.float()).sum()
        for e in range(block.experts):
            mine = expert == e
            loss = loss + ((y[mine] @ params[0][e].t()) * dz[mine].float()).sum()
        loss.backward()
        dxs.append(h.grad)
    grads = [p.grad / block.ranks for p in params]
    norm = torch.sqrt(sum(g.double().square().sum() for g in grads))
    factor = min(1.0, max_norm / float(norm))
    return float(norm), [g * factor for g in grads], dxs


def data(block: Block, tokens: int, gen: torch.Generator):
    def randn(width, scale):
        return (scale * torch.randn(tokens, width, generator=gen, device="cuda")).to(BF)

    out = []
    for _ in range(block.ranks):
        # some experts are busier than others
        expert = (block.experts * torch.rand(tokens, generator=gen, device="cuda") ** 1.5).long()
        out.append((randn(block.hidden, 1.0), randn(block.hidden, 2.0), expert.clamp(max=block.experts - 1),
                    randn(block.out, 1e-3), randn(block.hidden, 1e-3)))
    return out


def relative(got: torch.Tensor, want: torch.Tensor) -> float:
    return float((got.float() - want).norm() / want.norm())


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--ranks", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--out", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=8)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)
    block = Block(a.hidden, a.out, a.experts, a.ranks, gen)
    ranks = data(block, a.tokens, gen)
    parts, outs = step(block, ranks, 1.0)
    norm, grads, dxs = autograd(block, ranks, 1.0)
    print(f"norm     {block.norm.item():.6f} (autograd: {norm:.6f})")
    for name, got, want in zip(("linear", "weight"), block.gradients(parts.view(-1)), grads):
        print(f"d{name:7s} off by {relative(got, want):.2e} of its norm")
    print(f"dx       off by {max(relative(o[2], w) for o, w in zip(outs, dxs)):.2e} of its norm")


if __name__ == "__main__":
    main()
