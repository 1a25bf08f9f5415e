"""The layer norm, activation-checkpoint and weight-gradient operators as a
training step calls them, beside their plain forms in elementary torch
operations.

A case is one call (or one save with its restore) of a size:

  norm_forward   layer norm of `rows` rows of `width` channels; with
                 `checkpoint`, the 8-bit checkpoints of its input and of its
                 output are written in the same call and restored afterwards
  norm_backward  its backward pass, from the stored input or (`checkpoint`)
                 from the input's 8-bit checkpoint: dx, dweight, dbias
  checkpoint     an activation saved in 8 bits and restored
  weight_grad    a linear layer's weight gradient dY^T X from the 8-bit
                 checkpoint of X

`pad` is the number of unused elements between rows (a slice of a wider
activation).  bf16 activations have bf16 parameters and parameter gradients
(fragments of a bf16 gradient bucket), fp32 ones fp32.
"""
import torch

own = False

EPS = 1e-5
BLOCK = 32               # channels that share a step


# --- the cases ---------------------------------------------------------------

def _norm(op, rows, width, dtype, checkpoint, pad=0, name=None):
    c = {"op": op, "rows": rows, "width": width, "dtype": dtype, "checkpoint": checkpoint, "pad": pad}
    return dict(c, name=name) if name else c


def _save(rows, width, dtype, pad=0, name=None):
    c = {"op": "checkpoint", "rows": rows, "width": width, "dtype": dtype, "pad": pad}
    return dict(c, name=name) if name else c


def _grad(rows, out_features, in_features, dtype, pad=0, name=None):
    c = {"op": "weight_grad", "rows": rows, "out_features": out_features,
         "in_features": in_features, "dtype": dtype, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a layer norm of the hidden-4096 transformer: latency
        _norm("norm_forward", 1, 4096, "bf16", False, name="forward, one token"),
        # a training micro-batch of four sequences of 2048 tokens, checkpoints taken
        _norm("norm_forward", 8192, 4096, "bf16", True, name="forward, checkpointed step"),
        # fp32 activations whose rows start at every 4-byte offset
        _norm("norm_forward", 4099, 1001, "fp32", False, name="forward, ragged fp32"),
        # the last few sequences of a ragged batch
        _norm("norm_backward", 64, 4096, "bf16", False, name="backward, few rows"),
        # a training micro-batch of eight sequences, read from the checkpoint
        _norm("norm_backward", 16384, 4096, "bf16", True, name="backward, checkpointed step"),
        # fp32, odd width, a slice of a wider activation
        _norm("norm_backward", 3001, 1003, "fp32", False, 5, name="backward, ragged fp32"),
        # the activation of the feed-forward layer (11008 channels)
        _save(8192, 11008, "bf16", name="checkpoint, feed-forward"),
        # a width whose last block of 32 holds one channel
        _save(515, 4097, "fp32", name="checkpoint, ragged fp32"),
        # a small projection's gradient: few tiles, latency and the split over tokens
        _grad(256, 512, 512, "bf16", name="weight gradient, small"),
        # an attention projection of the hidden-4096 transformer, fp32 gradients
        _grad(8192, 4096, 4096, "fp32", name="weight gradient, attention"),
        # the feed-forward projection into 11008 channels
        _grad(4096, 11008, 4096, "bf16", name="weight gradient, feed-forward"),
        # odd sizes in all three directions
        _grad(2047, 1001, 1003, "bf16", name="weight gradient, ragged"),
    ]


def _size(rng, lo, hi):
    """A size whose logarithm is spread over [lo, hi]; as often any number as a multiple of 64."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    return max(64, n // 64 * 64) if rng.random() < 0.5 and hi > 64 and n >= 64 else max(1, n)


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "checkpoint", "weight_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    pad = rng.choice([0, 0, 0, 8, 3])
    if op == "weight_grad":
        while True:
            t, o, i = _size(rng, 1, 16384), _size(rng, 64, 11008), _size(rng, 64, 11008)
            if 2 * t * o * i <= 2 * 4096 * 11008 * 4096:
                return _grad(t, o, i, dtype, pad)
    while True:
        rows, width = _size(rng, 1, 16384), _size(rng, 64, 16384)
        if rows * width <= 8192 * 4096:
            break
    if op == "checkpoint":
        return _save(rows, width, dtype, pad)
    return _norm(op, rows, width, dtype, rng.random() < 0.5, pad)


# --- what a program has in hand before the call --------------------------------

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _rows(rows, width, pad, dtype, fill):
    """A [rows, width] view of a buffer whose rows are `pad` elements longer."""
    full = torch.empty(rows, width + pad, dtype=dtype, device="cuda")
    view = full[:, :width]
    if fill is not None:
        view.copy_(fill)
    return view


def _activation(rows, width, gen):
    """Token activations: a spread of channel magnitudes, a few channels far larger than the rest, and a mean that differs by token."""
    x = torch.randn(rows, width, generator=gen, device="cuda")
    magnitude = torch.exp(0.5 * torch.randn(width, generator=gen, device="cuda"))
    large = torch.rand(width, generator=gen, device="cuda") < 0.005
    x *= torch.where(large, 20 * magnitude, magnitude)
    x += 0.5 + 0.25 * torch.randn(rows, 1, generator=gen, device="cuda")
    return x


def _checkpoint_buffers(rows, width):
    """Codes and step bytes, rows padded to 16 bytes."""
    codes = torch.empty(rows, -(-width // 16) * 16, dtype=torch.int8, device="cuda")
    blocks = -(-width // BLOCK)
    steps = torch.empty(rows, -(-blocks // 16) * 16, dtype=torch.uint8, device="cuda")
    return codes[:, :width], steps[:, :blocks]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, pad = case["op"], case["rows"], case["pad"]
    dtype = _TYPES[case["dtype"]]
    s = {"op": op, "dtype": dtype}
    if op == "weight_grad":
        o, i = case["out_features"], case["in_features"]
        dy = 1e-3 * torch.randn(rows, o, generator=gen, device="cuda")
        s["dy"] = _rows(rows, o, pad, torch.bfloat16, dy)
        s["codes"], s["steps"] = _checkpoint_buffers(rows, i)
        _plain_save(_activation(rows, i, gen), s["codes"], s["steps"])
        s["dweight"] = torch.empty(o, i, dtype=dtype, device="cuda")
        return s
    width = case["width"]
    x = _rows(rows, width, pad, dtype, _activation(rows, width, gen))
    s["x"] = x
    if op == "checkpoint":
        s["codes"], s["steps"] = _checkpoint_buffers(rows, width)
        s["restored"] = torch.empty(rows, width, dtype=dtype, device="cuda")
        return s
    s["checkpoint"] = case["checkpoint"]
    s["weight"] = (1 + 0.1 * torch.randn(width, generator=gen, device="cuda")).to(dtype)
    s["bias"] = (0.1 * torch.randn(width, generator=gen, device="cuda")).to(dtype)
    if op == "norm_forward":
        s["y"] = torch.empty(rows, width, dtype=dtype, device="cuda")
        s["mean"] = torch.empty(rows, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        if s["checkpoint"]:
            s["x_codes"], s["x_steps"] = _checkpoint_buffers(rows, width)
            s["y_codes"], s["y_steps"] = _checkpoint_buffers(rows, width)
            s["x_restored"] = torch.empty(rows, width, dtype=dtype, device="cuda")
            s["y_restored"] = torch.empty(rows, width, dtype=dtype, device="cuda")
        return s
    xf = x.float()
    s["mean"] = xf.mean(1)
    s["rstd"] = torch.rsqrt(xf.var(1, correction=0) + EPS)
    s["dy"] = _rows(rows, width, pad, dtype, 1e-3 * torch.randn(rows, width, generator=gen, device="cuda"))
    s["dx"] = torch.empty(rows, width, dtype=dtype, device="cuda")
    s["dweight"] = torch.empty(width, dtype=dtype, device="cuda")
    s["dbias"] = torch.empty(width, dtype=dtype, device="cuda")
    if s["checkpoint"]:
        s["codes"], s["steps"] = _checkpoint_buffers(rows, width)
        _plain_save(xf, s["codes"], s["steps"])
        del s["x"]
    return s


# --- the plain forms -------------------------------------------------------------

def _power_of_two(e):
    """2^e in fp32 for integers e in [-126, 127], from the exponent field."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_save(x, codes, steps):
    """Blocks of 32 channels: the step is the smallest power of two (2^-126 to 2^121) that keeps max|x| / step below 127.5."""
    rows, width = x.shape
    blocks = steps.shape[1]
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - width)).view(rows, blocks, BLOCK)
    peak = v.abs().amax(2)
    finite = torch.isfinite(peak)
    safe = torch.where(finite, peak, 0.0)
    e = (torch.frexp(safe).exponent - 7).clamp(-126, 121)
    e = torch.where(safe * _power_of_two(-e) >= 127.5, e + 1, e).clamp(-126, 121)
    q = torch.round(torch.where(finite[..., None], v, 0.0) * _power_of_two(-e)[..., None])
    codes.copy_(q.clamp(-127, 127).to(torch.int8).view(rows, blocks * BLOCK)[:, :width])
    steps.copy_(torch.where(finite, torch.where(peak > 0, e + 127, 0), 255).to(torch.uint8))


def _plain_load(codes, steps):
    """codes x step in fp32; the step is the fp32 number whose exponent field is the byte."""
    step = (steps.to(torch.int32) << 23).view(torch.float32)
    return codes.float() * step.repeat_interleave(BLOCK, 1)[:, : codes.shape[1]]


def _plain(s):
    op, dtype = s["op"], s["dtype"]
    if op == "weight_grad":
        return (s["dy"].float().t() @ _plain_load(s["codes"], s["steps"])).to(dtype)
    if op == "checkpoint":
        _plain_save(s["x"], s["codes"], s["steps"])
        return _plain_load(s["codes"], s["steps"]).to(dtype)
    w, b = s["weight"].float(), s["bias"].float()
    if op == "norm_forward":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        centred = x - mean
        rstd = torch.rsqrt(centred.square().mean(1, keepdim=True) + EPS)
        y = (centred * rstd * w + b).to(dtype)
        out = [y, mean[:, 0], rstd[:, 0]]
        if s["checkpoint"]:
            _plain_save(x, s["x_codes"], s["x_steps"])
            _plain_save(y, s["y_codes"], s["y_steps"])
            out += [_plain_load(s["x_codes"], s["x_steps"]).to(dtype),
                    _plain_load(s["y_codes"], s["y_steps"]).to(dtype)]
        return out
    x = _plain_load(s["codes"], s["steps"]) if s["checkpoint"] else s["x"].float()
    dy = s["dy"].float()
    normed = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - normed * (g * normed).mean(1, keepdim=True))
    return [dx.to(dtype), (dy * normed).sum(0).to(dtype), dy.sum(0).to(dtype)]


# --- the framework's calls ---------------------------------------------------------

def _framework(s):
    import gradient_reduction_gb300 as dpr
    op = s["op"]
    if op == "weight_grad":
        dpr.dpr_linear_weight_grad(s["dy"], dpr.Checkpoint(s["codes"], s["steps"]), s["dweight"])
        return s["dweight"]
    if op == "checkpoint":
        saved = dpr.Checkpoint(s["codes"], s["steps"])
        dpr.dpr_checkpoint_save(s["x"], saved)
        dpr.dpr_checkpoint_load(saved, s["restored"])
        return s["restored"]
    if op == "norm_forward":
        out = [s["y"], s["mean"], s["rstd"]]
        if not s["checkpoint"]:
            dpr.dpr_layernorm_forward(s["x"], s["weight"], s["bias"], EPS, *out)
            return out
        x_saved = dpr.Checkpoint(s["x_codes"], s["x_steps"])
        y_saved = dpr.Checkpoint(s["y_codes"], s["y_steps"])
        dpr.dpr_layernorm_forward(s["x"], s["weight"], s["bias"], EPS, *out,
                                  x_checkpoint=x_saved, y_checkpoint=y_saved)
        dpr.dpr_checkpoint_load(x_saved, s["x_restored"])
        dpr.dpr_checkpoint_load(y_saved, s["y_restored"])
        return out + [s["x_restored"], s["y_restored"]]
    x = dpr.Checkpoint(s["codes"], s["steps"]) if s["checkpoint"] else s["x"]
    dpr.dpr_layernorm_backward(s["dy"], x, s["weight"], s["mean"], s["rstd"],
                               s["dx"], s["dweight"], s["dbias"])
    return [s["dx"], s["dweight"], s["dbias"]]


def run(state):
    return _framework(state) if own else _plain(state)


# --- the definitions in 64 bits ------------------------------------------------------

def _exact_restored(x):
    """What a saved activation stands for, block by block, from the definition."""
    rows, width = x.shape
    out = torch.empty_like(x)
    for first in range(0, width, BLOCK):
        v = x[:, first:first + BLOCK]
        peak = v.abs().max(dim=1, keepdim=True).values
        # the smallest step 2^e with peak < 127.5 * 2^e
        e = torch.floor(torch.log2(torch.clamp(peak, min=2.0 ** -149) / 127.5)) + 1
        e = torch.clamp(e, -126, 121)
        step = torch.exp2(e)
        out[:, first:first + BLOCK] = torch.clamp(torch.round(v / step), -127, 127) * step
    return out


def _exact_steps(codes, steps):
    step = torch.exp2(steps.double() - 127)
    return codes.double() * torch.repeat_interleave(step, BLOCK, dim=1)[:, : codes.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "weight_grad":
        return torch.einsum("to,ti->oi", s["dy"].double(), _exact_steps(s["codes"], s["steps"]))
    if op == "checkpoint":
        return _exact_restored(s["x"].double())
    w, b = s["weight"].double(), s["bias"].double()
    if op == "norm_forward":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = (x - mean[:, None]) * rstd[:, None] * w + b
        if not case["checkpoint"]:
            return [y, mean, rstd]
        # the output's checkpoint is of the output as stored, so it has a value only where the output is not rounded first
        return [y, mean, rstd, _exact_restored(x), _exact_restored(y) if s["dtype"] == torch.float32 else None]
    x = _exact_steps(s["codes"], s["steps"]) if case["checkpoint"] else s["x"].double()
    dy = s["dy"].double()
    n = case["width"]
    r = s["rstd"].double()[:, None]
    normed = (x - s["mean"].double()[:, None]) * r
    dweight = torch.einsum("rc,rc->c", dy, normed)
    g = dy * w
    dx = r * g - r / n * g.sum(1, keepdim=True) - r * normed / n * (g * normed).sum(1, keepdim=True)
    return [dx, dweight, dy.sum(0)]


def work(case):
    """Each input read once and each output written once; a checkpoint is 1 byte a value and 1 byte a block."""
    op, rows = case["op"], case["rows"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "weight_grad":
        o, i = case["out_features"], case["in_features"]
        saved = rows * (i + -(-i // BLOCK))
        return {"bytes": 2 * rows * o + saved + size * o * i, "flops": 2 * rows * o * i}
    n = rows * case["width"]
    saved = n + rows * -(-case["width"] // BLOCK)
    if op == "checkpoint":
        return {"bytes": 2 * (size * n + saved), "flops": 4 * n}
    if op == "norm_forward":
        b = 2 * size * n + 2 * size * case["width"] + 8 * rows
        if case["checkpoint"]:
            b += 4 * saved + 2 * size * n       # both written, read back and restored
        return {"bytes": b, "flops": 8 * n}
    b = 2 * size * n + (saved if case["checkpoint"] else size * n) + 3 * size * case["width"] + 8 * rows
    return {"bytes": b, "flops": 14 * n}
