"""The operators around a step of a transformer block with experts, as a
training program calls them, beside their plain forms in elementary torch
operations.

A case is one call (or one call and the restoring of what it saved in 8 bits):

  clip           the global norm of a list of gradients, and the gradients
                 scaled to a largest norm, written into a flat buffer of the
                 type that the optimizer step takes
  rms_forward    h = x + residual, y = h / rms(h) * weight; with `checkpoint`
                 the 8-bit checkpoints of h and y are written in the same call
                 and restored afterwards
  rms_backward   its backward pass, from h or (`checkpoint`) from the 8-bit
                 checkpoint of h: dx (with the residual stream's own gradient
                 added) and dweight
  grouped        y = x W_e^T for tokens sorted by expert
  grouped_input  its input gradient dx = dy W_e
  grouped_weight its weight gradients dW_e = dy_e^T x_e, from x or
                 (`checkpoint`) from the 8-bit checkpoint of x

`pad` is the number of unused elements between rows (a slice of a wider
activation).  Activations of the norms are bf16 or fp32 and their parameters
alike; the products take bf16 operands and give `dtype`.
"""
import random

import torch

own = False

EPS = 1e-6
BLOCK = 32               # channels that share a step of a checkpoint


# --- the cases ---------------------------------------------------------------

def _clip(sizes, tensors, elements, dtype, out, max_norm, shares=0, name=None):
    c = {"op": "clip", "sizes": sizes, "tensors": tensors, "elements": elements, "dtype": dtype, "out": out,
         "max_norm": max_norm, "shares": shares}
    return dict(c, name=name) if name else c


def _rms(op, rows, width, dtype, residual, checkpoint, pad=0, name=None):
    c = {"op": op, "rows": rows, "width": width, "dtype": dtype, "residual": residual,
         "checkpoint": checkpoint, "pad": pad}
    return dict(c, name=name) if name else c


def _grouped(op, rows, experts, out_features, in_features, dtype, skew, checkpoint=False, pad=0, name=None):
    c = {"op": op, "rows": rows, "experts": experts, "out_features": out_features, "in_features": in_features,
         "dtype": dtype, "skew": skew, "checkpoint": checkpoint, "pad": pad}
    return dict(c, name=name) if name else c


_LAYERS = 7 * (2 * 4096 + 4 * 4096 * 4096 + 2 * 4096 * 11008)


def listed():
    return [
        # the four fp32 partitions of a bucket of 4096 elements: latency
        _clip("even", 4, 4096, "fp32", "fp32", 0.02, name="clip, four small partitions"),
        # the 56 bf16 gradients of seven transformer layers of hidden 4096, to fp32 for the step
        _clip("layers", 56, _LAYERS, "bf16", "fp32", 1.0, name="clip, seven layers"),
        # one token through the norm in front of a block: latency
        _rms("rms_forward", 1, 4096, "bf16", True, False, name="rms norm, one token"),
        # a training micro-batch of four sequences of 2048 tokens, activations kept in 8 bits
        _rms("rms_forward", 8192, 4096, "bf16", True, True, name="rms norm, checkpointed step"),
        # fp32, odd width, a slice of a wider activation
        _rms("rms_backward", 3001, 1003, "fp32", False, False, 5, name="rms norm backward, ragged fp32"),
        # a training micro-batch of eight sequences, read from the checkpoint
        _rms("rms_backward", 16384, 4096, "bf16", True, True, name="rms norm backward, checkpointed step"),
        # 16 tokens sent to two of eight experts each: every expert's weights are read for a few rows
        _grouped("grouped", 32, 8, 11008, 4096, "bf16", 0.5, name="experts, few tokens"),
        # 8192 tokens sent to two of eight experts each, the busiest with several times the rows of the idlest
        _grouped("grouped", 16384, 8, 11008, 4096, "bf16", 0.7, name="experts, training step"),
        # small experts, some of them without a token
        _grouped("grouped_input", 300, 16, 512, 512, "bf16", 2.0, name="input gradient, small experts"),
        # the same training step's other product, half as many tokens
        _grouped("grouped_input", 8192, 8, 11008, 4096, "bf16", 0.7, name="input gradient, training step"),
        # odd sizes in all three directions, from the checkpoint
        _grouped("grouped_weight", 2047, 5, 1001, 1003, "bf16", 1.0, True, name="weight gradients, ragged"),
        # square projections of every expert, fp32 gradients
        _grouped("grouped_weight", 16384, 8, 4096, 4096, "fp32", 0.7, name="weight gradients, training step"),
    ]


_LARGEST_PRODUCT = 16384 * 11008 * 4096
_LARGEST_WEIGHTS = 8 * 11008 * 4096


def _size(rng, lo, hi):
    """A size whose logarithm is spread over [lo, hi]; as often any number as a multiple of 64."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    return max(64, n // 64 * 64) if rng.random() < 0.5 and hi > 64 and n >= 64 else max(1, n)


def draw(rng):
    op = rng.choice(["clip", "rms_forward", "rms_backward", "grouped", "grouped_input", "grouped_weight"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "clip":
        count = _size(rng, 1, 600)
        total = _size(rng, 4096, _LAYERS // 4)
        return _clip("spread", count, total, dtype, rng.choice(["bf16", "fp32"]), rng.choice([0.02, 0.5, 8.0]),
                     rng.randrange(1 << 30))
    pad = rng.choice([0, 0, 0, 8, 3])
    if op in ("rms_forward", "rms_backward"):
        while True:
            rows, width = _size(rng, 1, 16384), _size(rng, 64, 16384)
            if rows * width <= 8192 * 4096:
                return _rms(op, rows, width, dtype, rng.random() < 0.6, rng.random() < 0.5, pad)
    while True:
        rows, experts = _size(rng, 1, 16384), rng.choice([1, 2, 3, 5, 8, 16, 31, 64])
        o, i = _size(rng, 64, 11008), _size(rng, 64, 11008)
        if rows * o * i <= _LARGEST_PRODUCT and experts * o * i <= _LARGEST_WEIGHTS:
            return _grouped(op, rows, experts, o, i, dtype, rng.choice([0.0, 0.7, 1.5, 3.0]),
                            op == "grouped_weight" and rng.random() < 0.5, pad)


# --- what a case's texts and numbers stand for ----------------------------------

def _numels(case):
    """The gradients' lengths."""
    count, total = case["tensors"], case["elements"]
    if case["sizes"] == "even":
        return [total // count] * count
    if case["sizes"] == "layers":
        square, wide = 4096 * 4096, 4096 * 11008
        return [4096, square, square, square, square, 4096, wide, wide] * (count // 8)
    rng = random.Random(case["shares"])
    share = [rng.random() ** 4 + 1e-6 for _ in range(count)]     # few large ones, many small ones
    return [max(1, int(total * s / sum(share))) for s in share]


def _counts(case):
    """Tokens of each expert, falling with its rank as rank^-skew; the last ones may have none."""
    e = case["experts"]
    share = [(r + 1.0) ** -case["skew"] for r in range(e)]
    edges, at = [0], 0.0
    for s in share:
        at += s / sum(share)
        edges.append(min(case["rows"], int(at * case["rows"] + 0.5)))
    edges[-1] = case["rows"]
    return [b - a for a, b in zip(edges, edges[1:])]


# --- what a program has in hand before the call --------------------------------

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _rows(rows, width, pad, dtype, fill):
    """A [rows, width] view of a buffer whose rows are `pad` elements longer."""
    full = torch.empty(rows, width + pad, dtype=dtype, device="cuda")
    view = full[:, :width]
    view.copy_(fill)
    return view


def _activation(rows, width, gen):
    """Token activations: a spread of channel magnitudes, a few channels far larger than the rest."""
    x = torch.randn(rows, width, generator=gen, device="cuda")
    magnitude = torch.exp(0.5 * torch.randn(width, generator=gen, device="cuda"))
    large = torch.rand(width, generator=gen, device="cuda") < 0.005
    return x * torch.where(large, 20 * magnitude, magnitude)


def _checkpoint_buffers(rows, width):
    """Codes and step bytes, rows padded to 16 bytes."""
    codes = torch.empty(rows, -(-width // 16) * 16, dtype=torch.int8, device="cuda")
    blocks = -(-width // BLOCK)
    steps = torch.empty(rows, -(-blocks // 16) * 16, dtype=torch.uint8, device="cuda")
    return codes[:, :width], steps[:, :blocks]


def _place(numel):
    """A gradient's room in the flat buffer of the step: multiples of 16 elements."""
    return -(-numel // 16) * 16


def _views(flat, grads):
    views, at = [], 0
    for g in grads:
        views.append(flat[at:at + g.numel()])
        at += _place(g.numel())
    return views


def _prepare_clip(case, gen):
    dtype, out = _TYPES[case["dtype"]], _TYPES[case["out"]]
    grads = []
    for n in _numels(case):
        g = torch.empty(n, dtype=dtype, device="cuda")
        # tensors of a model differ in the size of their gradients
        spread = 1e-3 * torch.exp(torch.randn((), generator=gen, device="cuda"))
        for a in range(0, n, 1 << 26):
            part = g[a:a + (1 << 26)]
            part.copy_(torch.randn(part.numel(), generator=gen, device="cuda") * spread)
        grads.append(g)
    flat = torch.zeros(sum(_place(g.numel()) for g in grads), dtype=out, device="cuda")
    s = {"grads": grads, "flat": flat, "outs": _views(flat, grads), "norm": torch.empty(1, device="cuda"),
         "max_norm": case["max_norm"], "scale": 0.5}
    if own:
        import gradient_reduction_gb300 as dpr
        s["plan"] = dpr.dpr_grad_plan_create(s["grads"], s["outs"])
    return s


def _prepare_rms(case, gen):
    op, rows, width, pad = case["op"], case["rows"], case["width"], case["pad"]
    dtype = _TYPES[case["dtype"]]
    s = {"weight": (1 + 0.1 * torch.randn(width, generator=gen, device="cuda")).to(dtype)}
    x = _activation(rows, width, gen)
    if op == "rms_forward":
        s["x"] = _rows(rows, width, pad, dtype, x)
        s["residual"] = None
        s["h"] = s["x"]
        if case["residual"]:
            s["residual"] = _rows(rows, width, pad, dtype, _activation(rows, width, gen))
            s["h"] = torch.empty(rows, width, dtype=dtype, device="cuda")
        s["y"] = torch.empty(rows, width, dtype=dtype, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        if case["checkpoint"]:
            s["h_codes"], s["h_steps"] = _checkpoint_buffers(rows, width)
            s["y_codes"], s["y_steps"] = _checkpoint_buffers(rows, width)
            s["h_restored"] = torch.empty(rows, width, dtype=dtype, device="cuda")
            s["y_restored"] = torch.empty(rows, width, dtype=dtype, device="cuda")
        return s
    s["h"] = _rows(rows, width, pad, dtype, x)
    s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
    s["dy"] = _rows(rows, width, pad, dtype, 1e-3 * torch.randn(rows, width, generator=gen, device="cuda"))
    s["dh"] = None
    if case["residual"]:
        s["dh"] = _rows(rows, width, pad, dtype, 1e-3 * torch.randn(rows, width, generator=gen, device="cuda"))
    s["dx"] = torch.empty(rows, width, dtype=dtype, device="cuda")
    s["dweight"] = torch.empty(width, dtype=dtype, device="cuda")
    if case["checkpoint"]:
        s["codes"], s["steps"] = _checkpoint_buffers(rows, width)
        _plain_save(s["h"], s["codes"], s["steps"])
        del s["h"]
    return s


def _prepare_grouped(case, gen, seed):
    op, rows, pad = case["op"], case["rows"], case["pad"]
    e, o, i = case["experts"], case["out_features"], case["in_features"]
    dtype = _TYPES[case["dtype"]]
    counts = _counts(case)
    random.Random(seed).shuffle(counts)         # which expert is busy differs from batch to batch
    edges = [0]
    for c in counts:
        edges.append(edges[-1] + c)
    s = {"edges": edges, "offsets": torch.tensor(edges, dtype=torch.int32, device="cuda")}
    if op != "grouped":
        s["dy"] = _rows(rows, o, pad, torch.bfloat16, 1e-3 * torch.randn(rows, o, generator=gen, device="cuda"))
    if op != "grouped_input":
        s["x"] = _rows(rows, i, pad, torch.bfloat16, _activation(rows, i, gen))
    if op == "grouped_weight":
        s["dweight"] = torch.empty(e, o, i, dtype=dtype, device="cuda")
        if case["checkpoint"]:
            s["codes"], s["steps"] = _checkpoint_buffers(rows, i)
            _plain_save(s["x"], s["codes"], s["steps"])
            del s["x"]
        return s
    s["weight"] = torch.empty(e, o, i, dtype=torch.bfloat16, device="cuda")
    for w in s["weight"]:
        w.copy_(torch.randn(o, i, generator=gen, device="cuda") / i ** 0.5)
    s["out"] = torch.empty(rows, o if op == "grouped" else i, dtype=dtype, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "clip":
        s = _prepare_clip(case, gen)
    elif op in ("rms_forward", "rms_backward"):
        s = _prepare_rms(case, gen)
    else:
        s = _prepare_grouped(case, gen, seed)
    s["op"], s["dtype"], s["checkpoint"] = op, _TYPES[case["dtype"]], case.get("checkpoint", False)
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


def _plain_clip(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        total = total + g.float().square().sum(dtype=torch.float64)      # up to 10^9 terms
    norm = (s["scale"] * total.sqrt()).float()
    factor = s["scale"] * torch.where(norm <= s["max_norm"], 1.0, s["max_norm"] / norm)
    s["norm"].copy_(norm)
    for g, out in zip(s["grads"], s["outs"]):
        out.copy_(g.float() * factor)
    return [s["norm"], s["flat"]]


def _plain_rms_forward(s):
    dtype, h = s["dtype"], s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)
    y = (f * rstd * s["weight"].float()).to(dtype)
    out = [h, y, rstd[:, 0]]
    if s["checkpoint"]:
        _plain_save(h, s["h_codes"], s["h_steps"])
        _plain_save(y, s["y_codes"], s["y_steps"])
        out += [_plain_load(s["h_codes"], s["h_steps"]).to(dtype), _plain_load(s["y_codes"], s["y_steps"]).to(dtype)]
    return out


def _plain_rms_backward(s):
    dtype = s["dtype"]
    h = _plain_load(s["codes"], s["steps"]) if s["checkpoint"] else s["h"].float()
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    normed = h * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - normed * (g * normed).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return [dx.to(dtype), (dy * normed).sum(0).to(dtype)]


def _plain_grouped(s):
    op, edges = s["op"], s["edges"]
    if op == "grouped_weight":
        x = _plain_load(s["codes"], s["steps"]) if s["checkpoint"] else s["x"]
        for e, (a, b) in enumerate(zip(edges, edges[1:])):
            s["dweight"][e].copy_(s["dy"][a:b].float().t() @ x[a:b].float())
        return s["dweight"]
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        if a < b:
            w = s["weight"][e].float()
            s["out"][a:b].copy_(s["x"][a:b].float() @ w.t() if op == "grouped" else s["dy"][a:b].float() @ w)
    return s["out"]


_PLAIN = {"clip": _plain_clip, "rms_forward": _plain_rms_forward, "rms_backward": _plain_rms_backward}


# --- the framework's calls ---------------------------------------------------------

def _framework(s):
    import gradient_reduction_gb300 as dpr
    op = s["op"]
    if op == "clip":
        dpr.dpr_grad_norm_clip(s["plan"], s["norm"], s["max_norm"], scale=s["scale"])
        return [s["norm"], s["flat"]]
    if op == "rms_forward":
        out = [s["h"], s["y"], s["rstd"]]
        added = {} if s["residual"] is None else {"residual": s["residual"], "h": s["h"]}
        if not s["checkpoint"]:
            dpr.dpr_rmsnorm_forward(s["x"], s["weight"], EPS, s["y"], s["rstd"], **added)
            return out
        h_saved = dpr.Checkpoint(s["h_codes"], s["h_steps"])
        y_saved = dpr.Checkpoint(s["y_codes"], s["y_steps"])
        dpr.dpr_rmsnorm_forward(s["x"], s["weight"], EPS, s["y"], s["rstd"], **added,
                                h_checkpoint=h_saved, y_checkpoint=y_saved)
        dpr.dpr_checkpoint_load(h_saved, s["h_restored"])
        dpr.dpr_checkpoint_load(y_saved, s["y_restored"])
        return out + [s["h_restored"], s["y_restored"]]
    if op == "rms_backward":
        h = dpr.Checkpoint(s["codes"], s["steps"]) if s["checkpoint"] else s["h"]
        dpr.dpr_rmsnorm_backward(s["dy"], h, s["weight"], s["rstd"], s["dx"], s["dweight"], dh=s["dh"])
        return [s["dx"], s["dweight"]]
    if op == "grouped":
        dpr.dpr_grouped_linear(s["x"], s["offsets"], s["weight"], s["out"])
        return s["out"]
    if op == "grouped_input":
        dpr.dpr_grouped_linear_input_grad(s["dy"], s["offsets"], s["weight"], s["out"])
        return s["out"]
    x = dpr.Checkpoint(s["codes"], s["steps"]) if s["checkpoint"] else s["x"]
    dpr.dpr_grouped_linear_weight_grad(s["dy"], s["offsets"], x, s["dweight"])
    return s["dweight"]


def run(state):
    return _framework(state) if own else _PLAIN.get(state["op"], _plain_grouped)(state)


# --- the definitions in 64 bits ------------------------------------------------------

def _exact_restored(x):
    """What a saved activation stands for, block by block, from the definition."""
    out = torch.empty_like(x)
    for first in range(0, x.shape[1], BLOCK):
        v = x[:, first:first + BLOCK]
        peak = v.abs().max(dim=1, keepdim=True).values
        # the smallest step 2^e with peak < 127.5 * 2^e
        e = torch.floor(torch.log2(torch.clamp(peak, min=2.0 ** -149) / 127.5)) + 1
        step = torch.exp2(torch.clamp(e, -126, 121))
        out[:, first:first + BLOCK] = torch.clamp(torch.round(v / step), -127, 127) * step
    return out


def _exact_steps(codes, steps):
    step = torch.exp2(steps.double() - 127)
    return codes.double() * torch.repeat_interleave(step, BLOCK, dim=1)[:, : codes.shape[1]]


def _dot_self(g):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for part in torch.split(g, 1 << 26):
        d = part.double()
        total += torch.dot(d, d)
    return total


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = s["scale"] * torch.sqrt(torch.stack([_dot_self(g) for g in s["grads"]]).sum())
        factor = s["scale"] * min(1.0, s["max_norm"] / float(norm))
        flat = torch.zeros(s["flat"].shape, dtype=torch.float64, device="cuda")
        for view, g in zip(_views(flat, s["grads"]), s["grads"]):
            view.copy_(g).mul_(factor)
        return [norm.reshape(1), flat]
    if op == "rms_forward":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(s["dtype"]).double()     # the sum as it is stored
        rstd = 1 / torch.sqrt(torch.einsum("rc,rc->r", h, h) / case["width"] + EPS)
        y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].double())
        if not case["checkpoint"]:
            return [h, y, rstd]
        # the output's checkpoint is of the output as stored, so it has a value only where the output is not rounded first
        return [h, y, rstd, _exact_restored(h), _exact_restored(y) if s["dtype"] == torch.float32 else None]
    if op == "rms_backward":
        h = _exact_steps(s["codes"], s["steps"]) if case["checkpoint"] else s["h"].double()
        dy, r, w = s["dy"].double(), s["rstd"].double(), s["weight"].double()
        along = torch.einsum("rc,c,rc->r", dy, w, h) / case["width"]
        dx = r[:, None] * dy * w - (r ** 3 * along)[:, None] * h
        if s["dh"] is not None:
            dx += s["dh"].double()
        return [dx, torch.einsum("rc,rc,r->c", dy, h, r)]
    edges = s["edges"]
    if op == "grouped_weight":
        x = _exact_steps(s["codes"], s["steps"]) if case["checkpoint"] else s["x"]
        out = torch.zeros(s["dweight"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            mine = slice(edges[e], edges[e + 1])
            out[e] = torch.einsum("to,ti->oi", s["dy"][mine].double(), x[mine].double())
        return out
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        mine = slice(edges[e], edges[e + 1])
        w = s["weight"][e].double()
        if op == "grouped":
            out[mine] = torch.einsum("ti,oi->to", s["x"][mine].double(), w)
        else:
            out[mine] = torch.einsum("to,oi->ti", s["dy"][mine].double(), w)
    return out


def work(case):
    """Each input read once and each output written once; a checkpoint is 1 byte a value and 1 byte a block."""
    op = case["op"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "clip":
        n = sum(_numels(case))
        return {"bytes": n * (size + (2 if case["out"] == "bf16" else 4)) + 4, "flops": 3 * n}
    rows = case["rows"]
    if op in ("rms_forward", "rms_backward"):
        width = case["width"]
        n = rows * width
        saved = n + rows * -(-width // BLOCK)
        if op == "rms_forward":
            b = (2 + 2 * case["residual"]) * size * n + size * width + 4 * rows
            if case["checkpoint"]:
                b += 4 * saved + 2 * size * n       # both written, read back and restored
            return {"bytes": b, "flops": 6 * n}
        b = (2 + case["residual"]) * size * n + (saved if case["checkpoint"] else size * n)
        return {"bytes": b + 2 * size * width + 4 * rows, "flops": 11 * n}
    o, i = case["out_features"], case["in_features"]
    used = sum(c > 0 for c in _counts(case))
    if op == "grouped_weight":
        x = rows * (i + -(-i // BLOCK)) if case["checkpoint"] else 2 * rows * i
        b = 2 * rows * o + x + size * case["experts"] * o * i
    else:
        read, written = (i, o) if op == "grouped" else (o, i)
        b = 2 * rows * read + 2 * used * o * i + size * rows * written
    return {"bytes": b + 4 * (case["experts"] + 1), "flops": 2 * rows * o * i}
