"""One training step of a pre-norm linear block on K data-parallel ranks
(simulated as K buffers of one GPU), with the activations of the forward pass
kept in 8 bits and every gradient written straight into its place in the flat
bucket that the reduce-scatter takes:

    forward   y = layernorm(x)          both checkpoints written in the same pass
              z = y W^T                 (the x and y of 16 bits may be dropped now)
    backward  dW = dz^T y~              from y's checkpoint, into the bucket
              dy = dz W
              dx, dweight, dbias        from x's checkpoint, the latter into the bucket
    reduce    the K buckets' mean, scattered as fp32 partitions

    python examples/norm_linear_step.py [--ranks 4] [--tokens 4096] [--hidden 4096] [--out 4096]

prints the sizes kept for the backward pass and how far the reduced gradients
are from those of an fp32 autograd pass over the same data.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gradient_reduction_gb300 as dpr  # noqa: E402

EPS = 1e-5
BF = torch.bfloat16


class Block:
    """Parameters of the block, and their places in a rank's flat bucket."""

    def __init__(self, hidden: int, out: int, ranks: int, gen: torch.Generator):
        self.hidden, self.out, self.ranks = hidden, out, ranks
        self.weight = (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).to(BF)
        self.bias = (0.1 * torch.randn(hidden, generator=gen, device="cuda")).to(BF)
        self.linear = (torch.randn(out, hidden, generator=gen, device="cuda") / hidden ** 0.5).to(BF)
        # arrival order of a backward pass; places are multiples of 16 elements (32 bytes)
        self.places, at = [], 0
        for shape in ((out, hidden), (hidden,), (hidden,)):
            n = torch.Size(shape).numel()
            self.places.append((at, shape))
            at += -(-n // 16) * 16
        unit = 16 * ranks
        self.numel = -(-at // unit) * unit

    def gradients(self, bucket: torch.Tensor):
        """Views of a bucket: the gradients of linear, weight and bias."""
        return [bucket[at:at + torch.Size(shape).numel()].view(shape) for at, shape in self.places]


def forward(block: Block, x: torch.Tensor):
    """z, and what the backward pass needs: two checkpoints and two numbers a token."""
    rows = x.shape[0]
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    x_saved, y_saved = (dpr.dpr_checkpoint_empty(rows, block.hidden) for _ in range(2))
    dpr.dpr_layernorm_forward(x, block.weight, block.bias, EPS, y, mean, rstd, x_saved, y_saved)
    return y @ block.linear.t(), (x_saved, y_saved, mean, rstd)


def backward(block: Block, dz: torch.Tensor, kept, bucket: torch.Tensor) -> torch.Tensor:
    """dx; the parameters' gradients go into `bucket`."""
    x_saved, y_saved, mean, rstd = kept
    dlinear, dweight, dbias = block.gradients(bucket)
    dpr.dpr_linear_weight_grad(dz, y_saved, dlinear)
    dy = dz @ block.linear
    dpr.dpr_layernorm_backward(dy, x_saved, block.weight, mean, rstd, dy, dweight, dbias)
    return dy


def step(block: Block, xs, dzs):
    """The fp32 partitions of the mean gradient, [ranks, numel / ranks], and each rank's dx."""
    ranks = block.ranks
    buckets = torch.zeros(ranks, block.numel, dtype=BF, device="cuda")
    dxs, kept_bytes = [], 0
    for r in range(ranks):
        _, kept = forward(block, xs[r])
        kept_bytes += sum(t.nbytes if isinstance(t, dpr.Checkpoint) else t.numel() * 4 for t in kept)
        dxs.append(backward(block, dzs[r], kept, buckets[r]))
    parts = torch.empty(ranks, block.numel // ranks, device="cuda")
    dpr.dpr_reduce_scatter(buckets, ranks, 1, block.numel, parts)
    return parts, dxs, kept_bytes


def autograd(block: Block, xs, dzs):
    """Mean gradients of (linear, weight, bias) and each rank's dx, in fp32."""
    params = [p.float().requires_grad_() for p in (block.linear, block.weight, block.bias)]
    dxs = []
    for x, dz in zip(xs, dzs):
        x = x.float().requires_grad_()
        y = torch.nn.functional.layer_norm(x, (block.hidden,), params[1], params[2], EPS)
        (y @ params[0].t()).backward(dz.float())
        dxs.append(x.grad)
    return [p.grad / block.ranks for p in params], dxs


def data(block: Block, tokens: int, gen: torch.Generator):
    xs, dzs = [], []
    for _ in range(block.ranks):
        xs.append((torch.randn(tokens, block.hidden, generator=gen, device="cuda") + 0.3).to(BF))
        dzs.append((1e-3 * torch.randn(tokens, block.out, generator=gen, device="cuda")).to(BF))
    return xs, dzs


def relative(got: torch.Tensor, want: torch.Tensor) -> float:
    return float((got.float() - want).norm() / want.norm())


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--out", type=int, default=4096)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)
    block = Block(a.hidden, a.out, a.ranks, gen)
    xs, dzs = data(block, a.tokens, gen)
    parts, dxs, kept = step(block, xs, dzs)
    grads, want_dx = autograd(block, xs, dzs)
    full = 2 * 2 * a.ranks * a.tokens * a.hidden
    print(f"kept for the backward pass: {kept / 2 ** 20:.1f} MiB (bf16 x and y: {full / 2 ** 20:.1f} MiB)")
    for name, got, want in zip(("linear", "weight", "bias"), block.gradients(parts.view(-1)), grads):
        print(f"d{name:7s} off by {relative(got, want):.2e} of its norm")
    print(f"dx       off by {max(relative(g, w) for g, w in zip(dxs, want_dx)):.2e} of its norm")


if __name__ == "__main__":
    main()
