"""The operators of a training step (RMS norm, products grouped by expert, gradient clipping)
in 64 bits, written from their definitions, and the error bounds the tests hold the kernels to.

u = 2^-24 is fp32's rounding unit; a sum of n terms added along chains of at most D additions is
off by at most D u (1 + o(1)) sum|terms| (Higham, Accuracy and Stability of Numerical Algorithms,
section 4.2)."""
import torch

from tests.operators_reference import ROUND, TINY, U, weight_grad_chunk_bound


def rms_forward(h, w, eps):
    h = h.double()
    rstd = 1 / torch.sqrt(h.square().mean(1) + eps)
    return h * rstd[:, None] * w.double(), rstd


def rms_forward_bounds(h, w, eps, dtype):
    """Bounds on the errors of (y, rstd): chains of at most 32 squares a thread and two warp-wide
    trees (64 covers both), one more per 1024 channels for longer rows."""
    D = 64 + h.shape[1] // 1024
    y, rstd = rms_forward(h, w, eps)
    # the mean's square sum by the chain, its division and the addition of eps; the root halves it
    relative = (D + 4) * U / 2 * 1.01 + 4 * U
    d_y = (relative + 3 * U) * y.abs()
    return d_y + ROUND[dtype] * (y.abs() + d_y) + TINY[dtype], relative * rstd


def rms_backward(dy, h, w, rstd, dh=None):
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    g, n = dy * w, h * r
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * n).sum(0)


def rms_backward_bounds(dy, h, w, rstd, dh, dtype, grad_dtype):
    """Row sums along chains of at most 64 additions and one more per 256 channels; column sums
    along chains of at most rows / 8 + 384 (a thread's rows, the block's groups, the slices)."""
    dx, dw = rms_backward(dy, h, w, rstd, dh)
    rows, width = dy.shape
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    D = 64 + width // 256
    g = (dy * w).abs()
    # c = rstd^3 avg(g h): the products' and the chain's roundings, and five of the scaling
    c = r ** 3 * (g * h.abs()).mean(1, keepdim=True)
    d_c = (D + 7) * U * c
    add = 0 if dh is None else dh.double().abs()
    d_dx = h.abs() * d_c + 5 * U * (r * g + h.abs() * c + add)
    d_dx = d_dx + ROUND[dtype] * (dx.abs() + d_dx) + TINY[dtype]
    d_dw = (rows / 8 + 384 + 2) * U * (dy.abs() * h.abs() * r).sum(0)
    return d_dx, d_dw + ROUND[grad_dtype] * (dw.abs() + d_dw) + TINY[grad_dtype]


def spans(offsets, rows):
    """(begin, end) of every expert, limited as the calls take them: to the rows, and to no less than
    the offsets before."""
    edges = []
    for a in offsets:
        edges.append(max(min(max(a, 0), rows), edges[-1] if edges else 0))
    return list(zip(edges, edges[1:]))


def product(x, offsets, weight, transpose):
    """Rows of x times W_e^T (or, transposed, W_e), and the sums of the terms' magnitudes; NaN
    where no expert owns the row."""
    x, weight = x.double(), weight.double()
    width = weight.shape[2] if transpose else weight.shape[1]
    out = torch.full((x.shape[0], width), float("nan"), dtype=torch.float64)
    size = torch.zeros_like(out)
    for (a, b), w in zip(spans(offsets, x.shape[0]), weight):
        w = w if transpose else w.t()
        out[a:b] = x[a:b] @ w
        size[a:b] = x[a:b].abs() @ w.abs()
    return out, size


def weight_grads(dy, offsets, x):
    dy, x = dy.double(), x.double()
    parts = [(dy[a:b].t() @ x[a:b], dy[a:b].abs().t() @ x[a:b].abs())
             for a, b in spans(offsets, dy.shape[0])]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def sum_bound(want, size, length, dtype, parts=1):
    """A sum of `length` exact products with the terms' magnitudes `size`, as the tensor core makes
    it (weight_grad_chunk_bound), in at most `parts` parts (a GB300 has 76 pairs of SMs), rounded to
    dtype."""
    d = weight_grad_chunk_bound(max(length, 1), parts) * size
    return d + ROUND[dtype] * (want.abs() + d) + TINY[dtype]


def clip(grads, scale, max_norm):
    """norm, and the gradients times the factor."""
    total = sum(float(g.double().square().sum()) for g in grads)
    norm = scale * total ** 0.5
    factor = scale * (1.0 if norm <= max_norm else max_norm / norm)
    return norm, [g.double() * factor for g in grads]


# 16 squares along chains of at most 16 additions, whose sum's relative error the root halves; the
# sums of those are exact far beyond fp32; the root's and the scale's rounding
NORM_ERROR = (16 / 2 + 2) * U


def clip_bound(want, dtype):
    """The factor's error: the norm's, a division and two products; the output's rounding."""
    d = (NORM_ERROR + 3 * U) * want.abs()
    return d + ROUND[dtype] * (want.abs() + d) + TINY[dtype]
