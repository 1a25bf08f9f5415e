"""The backward-pass operators in 64 bits, written from their definitions, and
the error bounds the tests hold the fp32 kernels to.

Everything here is CPU torch in float64.  u = 2^-24 is fp32's rounding unit;
a sum of n terms added along chains of at most D additions is off by at most
D u (1 + o(1)) sum|terms| (Higham, Accuracy and Stability of Numerical
Algorithms, section 4.2)."""
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: U}   # 2^-p, p significant bits
# below this, rounding is absolute (subnormals)
TINY = {torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


def encode(x):
    """(codes, steps) of a [rows, width] float64 tensor, block by block."""
    rows, width = x.shape
    blocks = -(-width // 32)
    codes = torch.zeros(rows, width, dtype=torch.int8)
    steps = torch.zeros(rows, blocks, dtype=torch.uint8)
    for b in range(blocks):
        v = x[:, 32 * b:32 * b + 32]
        peak = v.abs().amax(1)
        bad = ~torch.isfinite(v).all(1)
        zero = (peak == 0) & ~bad
        p = torch.where(bad | zero, torch.ones_like(peak), peak)
        # smallest e with p < 127.5 * 2^e, from p = m * 2^k with m in [0.5, 1)
        m, k = torch.frexp(p)
        e = torch.where(m * 128 >= 127.5, k - 6, k - 7).clamp(-126, 121)
        q = torch.round(v / torch.ldexp(torch.ones_like(p), e)[:, None]).clamp(-127, 127)
        q = torch.where((bad | zero)[:, None], torch.zeros_like(q), q)
        codes[:, 32 * b:32 * b + 32] = q.to(torch.int8)
        s = torch.where(zero, 0, torch.where(bad, 255, e + 127))
        steps[:, b] = s.to(torch.uint8)
    return codes, steps


def decode(codes, steps):
    s = steps.to(torch.int64)
    value = torch.ldexp(torch.ones_like(s, dtype=torch.float64), s - 127)
    value = torch.where(s == 0, 0.0, torch.where(s == 255, float("nan"), value))
    return codes.double() * value.repeat_interleave(32, 1)[:, :codes.shape[1]]


def norm_forward(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    return (x - mean[:, None]) * rstd[:, None] * w.double() + b.double(), mean, rstd


def norm_forward_bounds(x, w, b, eps, dtype):
    """Bounds on the errors of (y, mean, rstd): chains of at most 64 additions
    for rows held in registers (32 a thread, two warp-wide trees), and one
    more per 1024 channels for longer rows."""
    x, w, b = x.double(), w.double(), b.double()
    D = 64 + x.shape[1] // 1024
    y, mean, rstd = norm_forward(x, w, b, eps)
    d_mean = (D + 2) * U * x.abs().mean(1)
    # centred values are off by d_mean and a rounding; their squares' sum by
    # the chain; the division and root add a few units
    centred = (x - mean[:, None]).abs()
    d_c = d_mean[:, None] + U * centred
    d_var = (2 * centred * d_c + d_c * d_c).mean(1) + (D + 4) * U * centred.square().mean(1)
    d_rstd = rstd * (d_var / (2 * (1 / rstd ** 2))) * 1.01 + 4 * U * rstd
    d_y = (d_c * rstd[:, None] + centred * d_rstd[:, None]) * w.abs()
    d_y = d_y + 4 * U * (centred * rstd[:, None] * w.abs() + b.abs())
    d_y = d_y + ROUND[dtype] * (y.abs() + d_y) + TINY[dtype]
    return d_y, d_mean + U * mean.abs() + TINY[torch.float32], d_rstd


def norm_backward(dy, x, w, mean, rstd):
    dy, x, w = dy.double(), x.double(), w.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def norm_backward_bounds(dy, x, w, mean, rstd, dtype, grad_dtype):
    """Row sums as in the forward; column sums along chains of at most
    rows / 8 + 384 additions."""
    dx, dw, db = norm_backward(dy, x, w, mean, rstd)
    dy, x, w = dy.double(), x.double(), w.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    rows, width = dy.shape
    D = 64 + width // 256
    h = (x - mean).abs() * rstd
    d_h = 3 * U * h                       # one subtraction, one product
    g = (dy * w).abs()
    d_g = U * g
    d_avg1 = d_g.mean(1, keepdim=True) + (D + 2) * U * g.mean(1, keepdim=True)
    gh = g * h
    d_avg2 = (g * d_h + d_g * h).mean(1, keepdim=True) + (D + 2) * U * gh.mean(1, keepdim=True)
    a2 = gh.mean(1, keepdim=True)
    d_dx = rstd * (d_g + d_avg1 + d_h * a2 + h * d_avg2
                   + 6 * U * (g + g.mean(1, keepdim=True) + h * a2))
    d_dx = d_dx + ROUND[dtype] * (dx.abs() + d_dx) + TINY[dtype]
    C = rows / 8 + 384
    d_dw = (dy.abs() * d_h).sum(0) + C * U * (dy.abs() * h).sum(0)
    d_dw = d_dw + ROUND[grad_dtype] * (dw.abs() + d_dw) + TINY[grad_dtype]
    d_db = C * U * dy.abs().sum(0)
    d_db = d_db + ROUND[grad_dtype] * (db.abs() + d_db) + TINY[grad_dtype]
    return d_dx, d_dw, d_db


def weight_grad(dy, restored):
    return dy.double().t() @ restored


def weight_grad_bounds(dy, restored, dtype):
    """Products of a bf16 number and an 8-bit code are exact; a chain of at
    most rows + 64 additions, each within one unit in the last place (2 u,
    which covers truncating adders)."""
    out = weight_grad(dy, restored)
    d = 2 * U * (dy.shape[0] + 64) * (dy.double().abs().t() @ restored.abs())
    return d + ROUND[dtype] * (out.abs() + d) + TINY[dtype]


def weight_grad_chunk_bound(rows, parts):
    """Error of a weight gradient in fp32 relative to the sum of its terms' magnitudes.  Terms are
    exact; 16 of them at a time are added to an accumulator that truncates, each time off by less
    than a unit in the last place (2 u) of a running sum that is at most the accumulator's
    magnitudes; after 1024 tokens the accumulator is added to the sum of its part, rounded (u of a
    running sum), and the at most `parts` parts to each other likewise.  (First order in u.)"""
    truncated = -(-min(rows, 1024) // 16)
    rounded = -(-rows // 1024) + parts + 1
    return 2 * U * truncated + U * rounded


def check(got, want, bound, what):
    """Elementwise |got - want| <= bound; NaN matches NaN, infinities themselves."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, want {tuple(want.shape)}"
    odd = ~torch.isfinite(want)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(same[odd].all()), f"{what}: non-finite values differ"
    err = torch.where(odd, torch.zeros_like(want), (got - want).abs())
    ok = (err <= bound) | odd
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(
            f"{what}: {int((~ok).sum())} of {ok.numel()} out of bounds; first at {i}: got "
            f"{got.flatten()[i]!r} want {want.flatten()[i]!r} bound {bound.flatten()[i]!r}")
