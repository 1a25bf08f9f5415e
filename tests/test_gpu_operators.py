"""Layer norm, 8-bit activation checkpoints and the weight gradient against
their definitions in 64 bits (tests/operators_reference.py), with bounds
derived from the summation lengths: widths from one channel to rows too long
for registers, every access width, odd strides and addresses, in-place forms,
masks of infinities and NaN, empty calls, streams, graphs, guard bytes."""
import pytest
import torch

import gradient_reduction_gb300 as dpr
from tests import gpu_helpers as H
from tests import operators_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def gen(seed):
    return torch.Generator().manual_seed(seed)


def activation(rows, width, seed, dtype):
    """Tokens with a mean of their own, channels of different magnitude, one in 64 far larger."""
    g = gen(seed)
    x = torch.randn(rows, width, generator=g)
    scale = torch.exp(torch.randn(width, generator=g))
    scale[torch.rand(width, generator=g) < 1 / 64] *= 30
    return (x * scale + torch.randn(rows, 1, generator=g)).to(dtype)


class Placed:
    """A [rows, width] view inside a larger buffer of sentinel bytes: rows
    `pad` elements apart beyond the width, starting `shift` elements in."""

    def __init__(self, rows, width, dtype, pad=0, shift=0, fill=None):
        size = torch.empty(0, dtype=dtype).element_size()
        self.n = 64 + shift + rows * (width + pad) + 64
        self.raw = torch.full((self.n * size,), 0xA5, dtype=torch.uint8, device="cuda")
        flat = self.raw.view(dtype)
        self.view = flat[64 + shift:64 + shift + rows * (width + pad)].view(
            rows, width + pad)[:, :width]
        self.mask = torch.ones(self.n, dtype=torch.bool, device="cuda")
        self.mask[64 + shift:64 + shift + rows * (width + pad)].view(
            rows, width + pad)[:, :width] = False
        if fill is not None:
            self.view.copy_(fill)
        self.size = size

    def check_guards(self, what):
        torch.cuda.synchronize()
        around = self.raw.view(self.n, self.size)[self.mask]
        assert bool((around == 0xA5).all()), f"{what}: bytes outside the view changed"


def checkpoint(rows, width, pad=None, shift=0):
    """A checkpoint in guarded buffers: 16-byte rows, or `pad` odd bytes between rows."""
    blocks = -(-width // 32)
    if pad is None:
        codes = Placed(rows, width, torch.int8, -width % 16, shift)
        steps = Placed(rows, blocks, torch.uint8, -blocks % 16, shift)
    else:
        codes = Placed(rows, width, torch.int8, pad, shift)
        steps = Placed(rows, blocks, torch.uint8, pad, shift)
    return codes, steps, dpr.Checkpoint(codes.view, steps.view)


# (pad, shift) in elements: aligned rows, 16-byte rows (bf16), odd rows, odd addresses
LAYOUTS = {"plain": (0, 0), "wide": (32, 0), "half": (8, 8), "odd": (3, 0), "shifted": (0, 1)}
WIDTHS = [1, 2, 31, 32, 33, 48, 96, 100, 512, 1000, 1001, 1024, 2064, 4096, 4097, 11008, 16400,
          33000]


# --- checkpoints -------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 31), (2, 32), (5, 33), (4, 96), (7, 1000),
                                        (3, 4097), (2, 11008)])
def test_save_and_load_match_the_format(rows, width, layout, dtype):
    H.device()
    pad, shift = LAYOUTS[layout]
    x = activation(rows, width, rows * width, dtype)
    want_codes, want_steps = R.encode(x.double())
    src = Placed(rows, width, dtype, pad, shift, x)
    codes, steps, saved = checkpoint(rows, width, None if layout == "plain" else pad,
                                     0 if layout == "plain" else shift)
    dpr.dpr_checkpoint_save(src.view, saved)
    assert torch.equal(codes.view.cpu(), want_codes)
    assert torch.equal(steps.view.cpu(), want_steps)
    out = Placed(rows, width, dtype, pad, shift)
    dpr.dpr_checkpoint_load(saved, out.view)
    assert torch.equal(out.view.cpu().double(), R.decode(want_codes, want_steps))
    for b, what in ((src, "x"), (codes, "codes"), (steps, "steps"), (out, "out")):
        b.check_guards(what)


def _special_values(dtype):
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).tiny
    inf, nan = float("inf"), float("nan")
    ramp = torch.arange(32, dtype=torch.float64)
    blocks = [
        torch.zeros(32), -torch.zeros(32), ramp, -ramp, torch.full((32,), big),
        torch.full((32,), -big), ramp / 32 * big, torch.full((32,), tiny), ramp * tiny,
        ramp * tiny / 64, ramp * 2.0 ** -100, torch.where(ramp == 5, inf, ramp),
        torch.where(ramp == 31, -inf, ramp), torch.where(ramp == 0, nan, ramp),
        torch.where(ramp == 17, torch.tensor(127.5), torch.tensor(0.5)),
        torch.where(ramp == 17, torch.tensor(127.0), torch.tensor(2.5)),
        torch.where(ramp == 17, torch.tensor(64.0), torch.tensor(-1.5)),
        torch.where(ramp == 3, torch.tensor(255.0 * 2 ** 30), torch.tensor(1.0)),
    ]
    return torch.stack([b.double() for b in blocks]).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [32, 64, 33])
def test_save_special_values(dtype, width):
    """Zeros of both signs, the largest and smallest numbers, ties, infinities, NaN: a block's
    neighbours keep their values, and infinities and NaN come back as NaN."""
    H.device()
    s = _special_values(dtype)
    x = torch.cat([s, s.flip(0)], 1)[:, :width].contiguous()
    want_codes, want_steps = R.encode(x.double())
    saved = dpr.dpr_checkpoint_empty(x.shape[0], width)
    dpr.dpr_checkpoint_save(x.cuda(), saved)
    assert torch.equal(saved.codes.cpu(), want_codes)
    assert torch.equal(saved.steps.cpu(), want_steps)
    out = torch.empty(x.shape, dtype=dtype, device="cuda")
    dpr.dpr_checkpoint_load(saved, out)
    want = R.decode(want_codes, want_steps)
    got = out.cpu().double()
    assert bool(((got == want) | (got.isnan() & want.isnan())).all())


def test_restored_values_are_exact_in_bf16_for_every_code_and_step():
    H.device()
    codes = torch.arange(-127, 128, dtype=torch.int8).repeat(249, 1)
    steps = torch.arange(249, dtype=torch.uint8)[:, None].repeat(1, 8)
    saved = dpr.Checkpoint(codes.cuda(), steps.cuda())
    want = R.decode(codes, steps)
    for dtype in (BF, F32):
        out = torch.empty(249, 255, dtype=dtype, device="cuda")
        dpr.dpr_checkpoint_load(saved, out)
        # from byte 243 up large codes pass fp32's range
        assert torch.equal(out.cpu()[:243].double(), want[:243])
        assert bool((out.cpu()[243:].double() == want[243:].float().double()).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_saving_is_within_half_a_step_and_idempotent(dtype):
    H.device()
    x = activation(64, 1000, 3, dtype).cuda()
    saved, again = (dpr.dpr_checkpoint_empty(64, 1000) for _ in range(2))
    out = torch.empty_like(x)
    dpr.dpr_checkpoint_save(x, saved)
    dpr.dpr_checkpoint_load(saved, out)
    step = torch.exp2(saved.steps.double() - 127).repeat_interleave(32, 1)[:, :1000]
    assert bool(((out.double() - x.double()).abs() <= step / 2).all())
    dpr.dpr_checkpoint_save(out, again)
    back = torch.empty_like(x)
    dpr.dpr_checkpoint_load(again, back)
    assert torch.equal(out, back)


# --- layer norm, forward -----------------------------------------------------

def _forward(rows, width, dtype, pdtype, layout="plain", in_place=False, ckpt=False, affine=True):
    pad, shift = LAYOUTS[layout]
    x = activation(rows, width, rows + width, dtype)
    g = gen(7)
    w = (1 + 0.2 * torch.randn(width, generator=g)).to(pdtype)
    b = (0.3 * torch.randn(width, generator=g)).to(pdtype)
    px = Placed(rows, width, dtype, pad, shift, x)
    py = px if in_place else Placed(rows, width, dtype, pad, shift)
    mean, rstd = Placed(1, rows, F32), Placed(1, rows, F32)
    guarded = [px, py, mean, rstd]
    saved = []
    if ckpt:
        for _ in range(2):
            codes, steps, c = checkpoint(rows, width, None if layout != "odd" else 5)
            guarded += [codes, steps]
            saved.append(c)
    dpr.dpr_layernorm_forward(px.view, w.cuda() if affine else None, b.cuda() if affine else None,
                              EPS, py.view, mean.view[0], rstd.view[0],
                              *(saved if ckpt else (None, None)))
    if not affine:
        w, b = torch.ones(width), torch.zeros(width)
    wy, wm, wr = R.norm_forward(x, w, b, EPS)
    by, bm, br = R.norm_forward_bounds(x, w, b, EPS, dtype)
    R.check(py.view, wy, by, "y")
    R.check(mean.view[0], wm, bm, "mean")
    R.check(rstd.view[0], wr, br, "rstd")
    for p in guarded:
        p.check_guards("forward")
    if ckpt:   # bit for bit what saving x, and y as stored, gives
        for c, src in zip(saved, (x, py.view.cpu())):
            codes, steps = R.encode(src.double())
            assert torch.equal(c.codes.cpu(), codes)
            assert torch.equal(c.steps.cpu(), steps)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_forward_widths(width, dtype, ckpt):
    H.device()
    _forward(5, width, dtype, dtype, ckpt=ckpt)


@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("width", [96, 1024, 33000])
def test_norm_forward_layouts(width, layout, dtype, pdtype):
    H.device()
    _forward(3, width, dtype, pdtype, layout, ckpt=True)


# where a rule changes the kernel: vectors of 8, 48 channels a thread, three reads of a row, the
# staged, register and two-pass backward kernels
EDGES = [510, 512, 520, 528, 4104, 5136, 8192, 8200, 10240, 12288, 16376, 24576, 24592]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", EDGES)
def test_norm_at_the_edges_of_the_rules(width, dtype):
    H.device()
    _forward(6, width, dtype, dtype, ckpt=True)
    _backward(6, width, dtype, dtype)
    _backward(6, width, dtype, dtype, source="saved")


@pytest.mark.parametrize("rows,width", [(1300, 528), (2500, 1024), (700, 4096), (900, 8192),
                                        (600, 8208), (500, 11008), (2200, 4128), (2048, 5120), (310, 16384), (155, 24576),
                                        (4000, 64), (1250, 16), (9000, 8)])
def test_norm_many_rows_per_block(rows, width):
    """Several rows to every block of the GPU: loops, rings and prefetches go round."""
    H.device()
    for dtype in (BF, F32):
        _forward(rows, width, dtype, F32, ckpt=True)
        _backward(rows, width, dtype, F32)
        _backward(rows, width, dtype, F32, source="saved", into="dy")


@pytest.mark.parametrize("shift", [0, 8, 1])
@pytest.mark.parametrize("pdtype", [BF, F32])
def test_norm_parameters_at_any_address(shift, pdtype):
    """Weight and bias 32-byte, 16-byte (bf16) and element aligned give the same bits."""
    H.device()
    x, dy = (activation(40, 1056, k, BF).cuda() for k in range(2))
    w0, b0 = (activation(1, 1056, 5 + k, pdtype)[0] for k in range(2))
    mean, rstd = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    got = []
    for s in (0, shift):
        w, b = (Placed(1, 1056, pdtype, 0, s, t[None]).view[0] for t in (w0, b0))
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dw, db = torch.empty(1056, device="cuda"), torch.empty(1056, device="cuda")
        dpr.dpr_layernorm_forward(x, w, b, EPS, y, mean, rstd)
        dpr.dpr_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db)
        got.append((y, dx, dw, db))
    assert _equal(*got)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 33, 300])
def test_norm_forward_rows(rows):
    H.device()
    _forward(rows, 160, BF, BF, ckpt=True)
    _forward(rows, 33, F32, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [96, 97, 4096, 40000])
def test_norm_forward_in_place_and_without_affine(width, dtype):
    H.device()
    _forward(4, width, dtype, dtype, in_place=True, ckpt=True)
    _forward(4, width, dtype, dtype, affine=False)


@pytest.mark.parametrize("width", [64, 100, 40000])
def test_norm_forward_constant_and_nonfinite_rows(width):
    """A constant row has y = bias exactly (variance 0); a NaN or an infinity spoils its own row only."""
    H.device()
    x = activation(5, width, 1, F32)
    x[1] = 3.0
    x[2, width // 2] = float("nan")
    x[3, 0] = float("inf")
    w, b = torch.full((width,), 2.0), torch.linspace(-1, 1, width)
    y = torch.empty(5, width, device="cuda")
    mean, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    dpr.dpr_layernorm_forward(x.cuda(), w.cuda(), b.cuda(), EPS, y, mean, rstd)
    assert torch.equal(y[1].cpu(), b)
    assert bool(y[2].isnan().all()) and bool(y[3].isnan().all())
    keep = [0, 4]
    wy, _, _ = R.norm_forward(x[keep], w, b, EPS)
    by, _, _ = R.norm_forward_bounds(x[keep], w, b, EPS, F32)
    R.check(y[keep], wy, by, "neighbours")


def test_norm_forward_large_mean():
    """A mean 1000 times the spread: the centred second pass keeps the variance."""
    H.device()
    x = torch.randn(8, 4096, generator=gen(2)) + 1000
    w, b = torch.ones(4096), torch.zeros(4096)
    y = torch.empty(8, 4096, device="cuda")
    dpr.dpr_layernorm_forward(x.cuda(), None, None, EPS, y)
    wy, _, _ = R.norm_forward(x, w, b, EPS)
    by, _, _ = R.norm_forward_bounds(x, w, b, EPS, F32)
    R.check(y, wy, by, "y")


# --- layer norm, backward ----------------------------------------------------

def _backward(rows, width, dtype, gdtype, layout="plain", source="x", into=None, accumulate=False,
              affine=True, pdtype=None):
    pad, shift = LAYOUTS[layout]
    x = activation(rows, width, rows + width, dtype)
    g = gen(11)
    dy = (1e-2 * torch.randn(rows, width, generator=g)).to(dtype)
    w = (1 + 0.2 * torch.randn(width, generator=g)).to(pdtype or dtype)
    _, mean, rstd = R.norm_forward(x, w, w, EPS)
    mean, rstd = mean.float(), rstd.float()
    px = Placed(rows, width, dtype, pad, shift, x)
    pd = Placed(rows, width, dtype, pad, shift, dy)
    po = {None: None, "dy": pd, "x": px}[into] or Placed(rows, width, dtype, pad, shift)
    pw, pb = Placed(1, width, gdtype), Placed(1, width, gdtype)
    old_w, old_b = (torch.randn(width, generator=g).to(gdtype) for _ in range(2))
    pw.view[0].copy_(old_w)
    pb.view[0].copy_(old_b)
    guarded = [px, pd, po, pw, pb]
    src, xx = px.view, x.double()
    if source == "saved":
        codes, steps, src = checkpoint(rows, width, None if layout != "odd" else 5)
        guarded += [codes, steps]
        c, s = R.encode(x.double())
        codes.view.copy_(c)
        steps.view.copy_(s)
        xx = R.decode(c, s)
    dpr.dpr_layernorm_backward(pd.view, src, w.cuda() if affine else None, mean.cuda(), rstd.cuda(),
                               po.view, pw.view[0], pb.view[0], accumulate)
    if not affine:
        w = torch.ones(width)
    want = list(R.norm_backward(dy, xx, w, mean, rstd))
    bound = list(R.norm_backward_bounds(dy, xx, w, mean, rstd, dtype, gdtype))
    if accumulate:
        for i, old in ((1, old_w), (2, old_b)):
            want[i] = want[i] + old.double()
            bound[i] = bound[i] + R.U * want[i].abs() + R.ROUND[gdtype] * old.double().abs()
    for got, wv, bv, what in zip((po.view, pw.view[0], pb.view[0]), want, bound,
                                 ("dx", "dweight", "dbias")):
        R.check(got, wv, bv, what)
    for p in guarded:
        p.check_guards("backward")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("source", ["x", "saved"])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_backward_widths(width, source, dtype):
    H.device()
    _backward(5, width, dtype, dtype, source=source)


@pytest.mark.parametrize("dtype,pdtype,gdtype", [(BF, BF, BF), (BF, F32, F32), (F32, BF, BF),
                                                 (F32, F32, F32)])
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("width", [96, 1024, 33000])
def test_norm_backward_layouts(width, layout, dtype, pdtype, gdtype):
    H.device()
    _backward(3, width, dtype, gdtype, layout, pdtype=pdtype)
    _backward(3, width, dtype, gdtype, layout, "saved", pdtype=pdtype)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 100, 1000, 5000])
@pytest.mark.parametrize("width", [40, 160, 1056])
def test_norm_backward_rows(rows, width):
    H.device()
    _backward(rows, width, BF, F32, source="saved")
    _backward(rows, width, F32, F32)


@pytest.mark.parametrize("into", ["dy", "x"])
@pytest.mark.parametrize("width", [96, 97, 4096, 33000])
def test_norm_backward_in_place(width, into):
    H.device()
    _backward(20, width, BF, BF, into=into)
    _backward(20, width, F32, F32, into=into)


@pytest.mark.parametrize("gdtype", [BF, F32])
@pytest.mark.parametrize("width", [97, 512])
def test_norm_backward_accumulates(width, gdtype):
    H.device()
    _backward(40, width, BF, gdtype, accumulate=True)
    _backward(40, width, BF, gdtype, accumulate=True, affine=False)


def test_norm_backward_no_rows_and_unwanted_gradients():
    H.device()
    dw = torch.ones(96, device="cuda")
    db = torch.ones(96, dtype=F32, device="cuda")
    empty = torch.empty(0, 96, device="cuda")
    stat = torch.empty(0, device="cuda")
    dpr.dpr_layernorm_backward(empty, empty, None, stat, stat, empty, dw, db, accumulate=True)
    assert bool((dw == 1).all()) and bool((db == 1).all())
    dpr.dpr_layernorm_backward(empty, empty, None, stat, stat, empty, dw, db)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    dpr.dpr_layernorm_forward(empty, None, None, EPS, empty.clone())
    x, dy = activation(6, 96, 0, F32).cuda(), activation(6, 96, 1, F32).cuda()
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    y, dx, dx2 = (torch.empty_like(x) for _ in range(3))
    dpr.dpr_layernorm_forward(x, None, None, EPS, y, mean, rstd)
    dpr.dpr_layernorm_backward(dy, x, None, mean, rstd, dx, dw, db)
    only = torch.full((96,), 9.0, device="cuda")
    dpr.dpr_layernorm_backward(dy, x, None, mean, rstd, dx2, None, only)
    assert torch.equal(only, db) and torch.equal(dx, dx2)
    dpr.dpr_layernorm_backward(dy, x, None, mean, rstd, dx2, only, None)
    assert torch.equal(only, dw)
    dpr.dpr_layernorm_backward(dy, x, None, mean, rstd, dx2)
    assert torch.equal(dx, dx2)


def test_norm_backward_broadcast_rows():
    """dy of a mean over tokens: one row, stride 0."""
    H.device()
    x = activation(30, 256, 5, F32).cuda()
    row = activation(1, 256, 6, F32).cuda()
    mean, rstd = torch.empty(30, device="cuda"), torch.empty(30, device="cuda")
    y = torch.empty_like(x)
    dpr.dpr_layernorm_forward(x, None, None, EPS, y, mean, rstd)
    got = [torch.empty_like(x), torch.empty(256, device="cuda"), torch.empty(256, device="cuda")]
    want = [torch.empty_like(t) for t in got]
    dpr.dpr_layernorm_backward(row.expand(30, 256), x, None, mean, rstd, *got)
    dpr.dpr_layernorm_backward(row.expand(30, 256).contiguous(), x, None, mean, rstd, *want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_norm_backward_saved_nan_block_reaches_the_gradients():
    H.device()
    x = activation(8, 256, 5, F32)
    x[3, 70] = float("inf")
    saved = dpr.dpr_checkpoint_empty(8, 256)
    dpr.dpr_checkpoint_save(x.cuda(), saved)
    dy = activation(8, 256, 6, F32).cuda()
    mean, rstd = torch.zeros(8, device="cuda"), torch.ones(8, device="cuda")
    dx, dw, db = torch.empty_like(dy), torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
    dpr.dpr_layernorm_backward(dy, saved, None, mean, rstd, dx, dw, db)
    assert bool(dx[3].isnan().all()) and not bool(dx[[0, 1, 2, 4, 5, 6, 7]].isnan().any())
    assert bool(dw[64:96].isnan().all()) and not bool(dw[:64].isnan().any())
    assert not bool(dw[96:].isnan().any()) and not bool(db.isnan().any())


@pytest.mark.parametrize("width", [40, 1001])
def test_norm_backward_against_differences(width):
    """<gradient, v> against (L(. + h v) - L(. - h v)) / 2h of L = sum dy * y, the forward's
    definition in 64 bits.  With h = 1e-5 times the data's spread the difference quotient is
    off by about h^2 = 1e-10 relative to sum|terms|; the kernel's fp32 gradient by 1e-5."""
    H.device()
    rows = 12
    g = gen(21)
    x = activation(rows, width, 9, F32)
    dy = torch.randn(rows, width, generator=g)
    w = 1 + 0.2 * torch.randn(width, generator=g)
    b = torch.randn(width, generator=g)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y, dx = torch.empty(rows, width, device="cuda"), torch.empty(rows, width, device="cuda")
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    dpr.dpr_layernorm_forward(x.cuda(), w.cuda(), b.cuda(), EPS, y, mean, rstd)
    dpr.dpr_layernorm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd, dx, dw, db)
    X, W, B, DY = x.double(), w.double(), b.double(), dy.double()

    def loss(x, w, b):
        return (DY * R.norm_forward(x, w, b, EPS)[0]).sum()

    h = 1e-5
    for k in range(3):
        v = torch.randn(rows, width, generator=gen(30 + k), dtype=torch.float64)
        quotient = (loss(X + h * v, W, B) - loss(X - h * v, W, B)) / (2 * h)
        terms = dx.cpu().double() * v
        assert abs(quotient - terms.sum()) <= 2e-5 * terms.abs().sum()
        v = v[0]
        for grad, at in ((dw, lambda s: loss(X, W + s * v, B)), (db, lambda s: loss(X, W, B + s * v))):
            terms = grad.cpu().double() * v
            assert abs((at(h) - at(-h)) / (2 * h) - terms.sum()) <= 2e-5 * terms.abs().sum()


# --- the weight gradient ------------------------------------------------------

def _weight_grad(rows, o, i, dtype, layout="plain", accumulate=False, exact=False, seed=0):
    """`exact`: integers whose sums stay below 2^24, so fp32 sums are exact in any order."""
    pad, shift = LAYOUTS[layout]
    g = gen(100 + seed + rows + o + i)
    if exact:
        dy = torch.randint(-3, 4, (rows, o), generator=g).to(BF)
        x = torch.randint(-127, 128, (rows, i), generator=g).double()
    else:
        dy = (1e-2 * torch.randn(rows, o, generator=g)).to(BF)
        x = activation(rows, i, seed, F32).double()
    c, s = R.encode(x)
    pd = Placed(rows, o, BF, pad, shift, dy)
    codes, steps, saved = checkpoint(rows, i, None if layout in ("plain", "wide") else pad,
                                     0 if layout in ("plain", "wide") else shift)
    codes.view.copy_(c)
    steps.view.copy_(s)
    pw = Placed(o, i, dtype, pad, shift)
    old = (torch.randint(-50, 50, (o, i), generator=g) if exact
           else torch.randn(o, i, generator=g)).to(dtype)
    pw.view.copy_(old)
    dpr.dpr_linear_weight_grad(pd.view, saved, pw.view, accumulate)
    xx = R.decode(c, s)
    want = R.weight_grad(dy, xx)
    if accumulate:
        want = want + old.double()
    if exact:
        assert float(want.abs().max()) < 2 ** 24
        assert torch.equal(pw.view.cpu(), want.to(dtype)), "integer sums differ"
    else:
        bound = R.weight_grad_bounds(dy, xx, dtype)
        if accumulate:
            bound = bound + R.U * want.abs() + R.ROUND[dtype] * old.double().abs()
        R.check(pw.view, want, bound, "dweight")
    for p in (pd, codes, steps, pw):
        p.check_guards("weight gradient")


SIZES = [(1, 1, 1), (1, 8, 16), (2, 64, 33), (3, 70, 1100), (4, 257, 2050), (5, 257, 2050),
         (15, 8, 128), (16, 128, 128), (17, 256, 160),
         (63, 100, 100), (64, 256, 128), (65, 264, 144), (128, 512, 512), (200, 1000, 48),
         (500, 72, 1008), (1025, 136, 272), (333, 257, 511)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,o,i", SIZES)
def test_weight_grad_sizes(rows, o, i, dtype):
    H.device()
    _weight_grad(rows, o, i, dtype)
    _weight_grad(rows, o, i, dtype, exact=True)


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,o,i", [(70, 136, 144), (33, 65, 97), (3, 65, 97)])
def test_weight_grad_layouts(rows, o, i, dtype, layout):
    H.device()
    _weight_grad(rows, o, i, dtype, layout)
    _weight_grad(rows, o, i, dtype, layout, accumulate=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,o,i", [(4096, 256, 384), (5000, 128, 128), (16384, 64, 64),
                                      (2048, 1024, 1152)])
def test_weight_grad_long(rows, o, i, dtype):
    H.device()
    _weight_grad(rows, o, i, dtype, exact=True)
    _weight_grad(rows, o, i, dtype, exact=True, accumulate=True)
    _weight_grad(rows, o, i, dtype)


@pytest.mark.parametrize("rows,o,i,dtype", [(200, 2304, 2304, F32), (1100, 2310, 2305, BF),
                                            (65, 5000, 1100, BF), (3, 3001, 1030, F32)])
def test_weight_grad_more_tiles_than_pairs(rows, o, i, dtype):
    """Whole waves of tiles and a dealt-out rest in one call."""
    H.device()
    _weight_grad(rows, o, i, dtype, exact=True)
    _weight_grad(rows, o, i, dtype, exact=True, accumulate=True, layout="odd")
    _weight_grad(rows, o, i, dtype)


def test_weight_grad_no_rows():
    H.device()
    saved = dpr.dpr_checkpoint_empty(0, 96)
    dy = torch.empty(0, 40, dtype=BF, device="cuda")
    for dtype in (BF, F32):
        dw = torch.ones(40, 96, dtype=dtype, device="cuda")
        dpr.dpr_linear_weight_grad(dy, saved, dw, accumulate=True)
        assert bool((dw == 1).all())
        dpr.dpr_linear_weight_grad(dy, saved, dw)
        assert bool((dw == 0).all())


@pytest.mark.parametrize("o,i", [(64, 128), (61, 127)])
def test_weight_grad_nonfinite(o, i):
    """A spoilt block of the checkpoint spoils its channels' gradients, a spoilt dy its
    output's, and nothing else; an infinity of dy against zeros is NaN as in any product."""
    H.device()
    rows = 70
    x = activation(rows, i, 4, F32)
    x[5, 40] = float("nan")
    saved = dpr.dpr_checkpoint_empty(rows, i)
    dpr.dpr_checkpoint_save(x.cuda(), saved)
    dy = (1e-2 * torch.randn(rows, o, generator=gen(3))).to(BF)
    dy[9, 2] = float("inf")
    dy[11, 7] = float("nan")
    dw = torch.empty(o, i, device="cuda")
    dpr.dpr_linear_weight_grad(dy.cuda(), saved, dw)
    want = R.weight_grad(dy, R.decode(saved.codes.cpu(), saved.steps.cpu()))
    bound = R.weight_grad_bounds(torch.nan_to_num(dy, 0, 0, 0),
                                 torch.nan_to_num(R.decode(saved.codes.cpu(), saved.steps.cpu())), F32)
    R.check(dw, want, bound, "dweight")


def test_weight_grad_against_differences():
    """dL/dW of L = sum dy * (x~ W^T) by differences along random directions (L is linear in W)."""
    H.device()
    rows, o, i = 100, 72, 96
    x, dy = activation(rows, i, 4, F32), (torch.randn(rows, o, generator=gen(3))).to(BF)
    saved = dpr.dpr_checkpoint_empty(rows, i)
    dpr.dpr_checkpoint_save(x.cuda(), saved)
    dw = torch.empty(o, i, device="cuda")
    dpr.dpr_linear_weight_grad(dy.cuda(), saved, dw)
    xx = R.decode(saved.codes.cpu(), saved.steps.cpu())
    W = torch.randn(o, i, generator=gen(4), dtype=torch.float64)

    def loss(w):
        return (dy.double() * (xx @ w.t())).sum()

    for k in range(3):
        v = torch.randn(o, i, generator=gen(40 + k), dtype=torch.float64)
        terms = dw.cpu().double() * v
        assert abs((loss(W + v) - loss(W - v)) / 2 - terms.sum()) <= 1e-5 * terms.abs().sum()


# --- together ------------------------------------------------------------------

def _step(stream, x, dy, w, b, buffers):
    """Forward with both checkpoints, then the backward pass from them, on `stream`."""
    y, mean, rstd, xs, ys, dx, dw, db, dlin = buffers
    dpr.dpr_layernorm_forward(x, w, b, EPS, y, mean, rstd, xs, ys, stream=stream)
    dpr.dpr_layernorm_backward(dy, xs, w, mean, rstd, dx, dw, db, stream=stream)
    dpr.dpr_linear_weight_grad(dx, ys, dlin, stream=stream)


def _buffers(rows, width):
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")
    return (e(rows, width), e(rows, dtype=F32), e(rows, dtype=F32),
            dpr.dpr_checkpoint_empty(rows, width), dpr.dpr_checkpoint_empty(rows, width),
            e(rows, width), e(width), e(width), e(width, width))


def _tensors(buffers):
    out = []
    for t in buffers:
        out += [t.codes.clone(), t.steps.clone()] if isinstance(t, dpr.Checkpoint) else [t.clone()]
    return out


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rows,width", [(300, 256), (77, 100)])
@pytest.mark.parametrize("programmatic", [True, False])
def test_chains_on_side_streams_and_graphs_repeat_bit_for_bit(rows, width, programmatic):
    """Calls that feed each other on a stream of their own, launched back to back without waits,
    as an int handle, and replayed from a graph give what the default stream gives."""
    H.device()
    old = dpr.dpr_set_programmatic_launch(programmatic)
    try:
        x, dy = activation(rows, width, 1, BF).cuda(), activation(rows, width, 2, BF).cuda()
        w, b = activation(1, width, 3, BF)[0].cuda(), activation(1, width, 4, BF)[0].cuda()
        first, second = _buffers(rows, width), _buffers(rows, width)
        _step(None, x, dy, w, b, first)
        torch.cuda.synchronize()
        want = _tensors(first)
        side = torch.cuda.Stream()
        for handle in (side, side.cuda_stream):
            for t in _tensors(second):
                pass
            for _ in range(5):
                _step(handle, x, dy, w, b, second)
            side.synchronize()
            assert _equal(_tensors(second), want)
        graph = torch.cuda.CUDAGraph()
        third = _buffers(rows, width)
        with torch.cuda.graph(graph, stream=side):
            _step(None, x, dy, w, b, third)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert _equal(_tensors(third), want)
    finally:
        dpr.dpr_set_programmatic_launch(old)


def test_scratch_memory_is_shared_safely():
    """Calls of different sizes on one stream, on two streams at once and inside a capture, each
    with the library's own scratch memory, give what separate workspaces give."""
    H.device()
    sizes = [(40, 1056), (3, 8192), (700, 512), (40, 1056), (64, 4096)]

    def make(rows, width, seed):
        x, dy = (activation(rows, width, seed + k, F32).cuda() for k in range(2))
        mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        out = [torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")]
        return (dy, x, None, mean, rstd, *out), out

    calls = [make(r, w, 10 * i) for i, (r, w) in enumerate(sizes)]
    want = []
    for args, out in calls:
        dpr.dpr_layernorm_backward(*args, workspace=torch.empty(16 << 20, dtype=torch.uint8, device="cuda"))
        want.append([t.clone() for t in out])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for args, out in calls[:3]:
            dpr.dpr_layernorm_backward(*args)
        with torch.cuda.stream(side):
            for args, out in calls[3:]:
                dpr.dpr_layernorm_backward(*args)
    torch.cuda.synchronize()
    for (args, out), w in zip(calls, want):
        assert _equal(out, w)
        for t in out:
            t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for args, out in calls:
            dpr.dpr_layernorm_backward(*args)
    dpr.dpr_layernorm_backward(*make(5000, 8192, 99)[0])       # grows the kept memory
    graph.replay()
    torch.cuda.synchronize()
    for (args, out), w in zip(calls, want):
        assert _equal(out, w)


def test_binding_refusals():
    H.device()
    x = torch.zeros(8, 64, device="cuda")
    half = x.to(torch.float16)
    saved = dpr.dpr_checkpoint_empty(8, 64)
    stat, vec = torch.zeros(8, device="cuda"), torch.zeros(64, device="cuda")
    bad = pytest.raises(ValueError)
    with bad:
        dpr.dpr_layernorm_forward(half, None, None, EPS, half)                    # dtype
    with bad:
        dpr.dpr_layernorm_forward(x, None, None, EPS, x[:4].clone())              # shape
    with bad:
        dpr.dpr_layernorm_forward(x, None, None, EPS, x.bfloat16())               # y's dtype
    with bad:
        dpr.dpr_layernorm_forward(x, vec[:32], None, EPS, x.clone())              # weight's length
    with bad:
        dpr.dpr_layernorm_forward(x, vec, vec.bfloat16(), EPS, x.clone())         # mixed dtypes
    with bad:
        dpr.dpr_layernorm_forward(x, None, None, EPS, x.clone(), stat.bfloat16())
    with bad:
        dpr.dpr_layernorm_forward(x, None, None, EPS, x.clone(), x_checkpoint=x)  # no Checkpoint
    with bad:
        dpr.dpr_layernorm_forward(x, None, None, EPS, x.clone(),
                                  y_checkpoint=dpr.dpr_checkpoint_empty(8, 32))
    with bad:
        dpr.dpr_layernorm_forward(x.t(), None, None, EPS, x.t())                  # inner stride
    with bad:
        dpr.dpr_layernorm_forward(x.cpu(), None, None, EPS, x)
    with pytest.raises(dpr.DprError):
        dpr.dpr_layernorm_forward(x, None, None, -1.0, x.clone())
    with pytest.raises(dpr.DprError):
        dpr.dpr_layernorm_forward(x[:4], None, None, EPS, x[2:6])                 # overlap
    args = (x, x.clone(), None, stat, stat.clone())
    with bad:
        dpr.dpr_layernorm_backward(*args, x[:, :32].clone())
    with bad:
        dpr.dpr_layernorm_backward(x, x.bfloat16(), None, stat, stat, x.clone())
    with bad:
        dpr.dpr_layernorm_backward(x, x, None, None, stat, x.clone())
    with bad:
        dpr.dpr_layernorm_backward(*args, x.clone(), vec, vec.bfloat16())
    with bad:
        dpr.dpr_layernorm_backward(*args, x.clone(), vec, vec.clone(),
                                   workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dpr.DprError):
        dpr.dpr_layernorm_backward(*args, x.clone(), vec, vec)                    # one for both
    with bad:
        dpr.dpr_checkpoint_save(x, dpr.Checkpoint(saved.codes, saved.steps[:, :1]))
    with bad:
        dpr.dpr_checkpoint_save(x, dpr.Checkpoint(saved.codes.view(torch.uint8), saved.steps))
    with bad:
        dpr.dpr_checkpoint_load(saved, torch.zeros(8, 32, device="cuda"))
    dy = torch.zeros(8, 40, dtype=BF, device="cuda")
    with bad:
        dpr.dpr_linear_weight_grad(dy.float(), saved, torch.zeros(40, 64, device="cuda"))
    with bad:
        dpr.dpr_linear_weight_grad(dy, saved, torch.zeros(64, 40, device="cuda"))
    with bad:
        dpr.dpr_linear_weight_grad(dy[:4], saved, torch.zeros(40, 64, device="cuda"))
    with bad:
        dpr.dpr_linear_weight_grad(dy, saved, torch.zeros(40 * 64, device="cuda"))


def test_leading_dimensions_merge():
    H.device()
    x = activation(24, 160, 1, BF).cuda()
    flat, deep = torch.empty_like(x), torch.empty(2, 3, 4, 160, dtype=BF, device="cuda")
    dpr.dpr_layernorm_forward(x, None, None, EPS, flat)
    dpr.dpr_layernorm_forward(x.view(2, 3, 4, 160), None, None, EPS, deep)
    assert torch.equal(flat, deep.view(24, 160))


def test_offsets_past_32_bits():
    """Rows 2^30 elements apart: the last starts at element 5 * 2^30 (byte 10 * 2^30 for bf16)."""
    H.device()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of free device memory")
    rows, width, far = 6, 64, 1 << 30

    def spread(dtype, n):
        return torch.empty(5 * far + n, dtype=dtype, device="cuda").as_strided((rows, n), (far, 1))

    x, dy = activation(rows, width, 1, BF), activation(rows, width, 2, BF)
    fx, fdy, fy = spread(BF, width), spread(BF, width), spread(BF, width)
    fx.copy_(x)
    fdy.copy_(dy)
    saved = dpr.Checkpoint(spread(torch.int8, width), spread(torch.uint8, 2))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpr.dpr_layernorm_forward(fx, None, None, EPS, fy, mean, rstd, saved)
    codes, steps = R.encode(x.double())
    assert torch.equal(saved.codes.cpu(), codes) and torch.equal(saved.steps.cpu(), steps)
    ones, zeros = torch.ones(width), torch.zeros(width)
    R.check(fy, R.norm_forward(x, ones, zeros, EPS)[0],
            R.norm_forward_bounds(x, ones, zeros, EPS, BF)[0], "y")
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    dpr.dpr_layernorm_backward(fdy, saved, None, mean, rstd, fy, dw, db)
    xx = R.decode(codes, steps)
    args = (dy, xx, ones, mean.cpu(), rstd.cpu())
    for got, want, bound in zip((fy, dw, db), R.norm_backward(*args),
                                R.norm_backward_bounds(*args, BF, F32)):
        R.check(got, want, bound, "backward")
    dpr.dpr_checkpoint_load(saved, fy)
    assert torch.equal(fy.cpu().double(), xx)
    lin = torch.empty(width, width, device="cuda")
    dpr.dpr_linear_weight_grad(fdy, saved, lin)
    R.check(lin, R.weight_grad(dy, xx), R.weight_grad_bounds(dy, xx, F32), "dweight")


def test_no_wait_ran_out():
    H.device()
    assert dpr.dpr_device_wait_failures() == 0


@pytest.mark.parametrize("ranks,tokens,hidden,out", [(2, 300, 256, 200), (4, 130, 200, 72)])
def test_step_of_a_block_into_the_bucket(ranks, tokens, hidden, out):
    """The example's step: gradients of the block written into flat buckets from 8-bit
    activations and reduce-scattered, against an fp32 autograd pass.  An activation is off by
    at most half a step, step <= max|x| / 63.5: relative to the norm of a block of normal
    values (max about 3 rms) an rms error of at most 3 / 63.5 / sqrt(12) = 1.4e-2; the
    gradients read them once, and bf16 rounding adds 2^-8."""
    H.device()
    from examples import norm_linear_step as ex
    g = torch.Generator(device="cuda").manual_seed(5)
    block = ex.Block(hidden, out, ranks, g)
    xs, dzs = ex.data(block, tokens, g)
    parts, dxs, kept = ex.step(block, xs, dzs)
    grads, want_dx = ex.autograd(block, xs, dzs)
    assert kept < 0.56 * 4 * ranks * tokens * hidden
    for got, want in zip(block.gradients(parts.view(-1)), grads):
        assert ex.relative(got, want) < 2.5e-2
    for got, want in zip(dxs, want_dx):
        assert ex.relative(got, want) < 2.5e-2
    # the bucket's gaps stay zero
    used = torch.zeros(block.numel, dtype=torch.bool)
    for t in block.gradients(used):
        t.fill_(True)
    assert bool((parts.view(-1).cpu()[~used] == 0).all())


def test_step_matches_its_own_calls_bit_for_bit():
    """The partitions are the exact ring mean of the gradients that the calls give on their own."""
    H.device()
    from examples import norm_linear_step as ex
    from oracle import ring
    g = torch.Generator(device="cuda").manual_seed(6)
    block = ex.Block(160, 96, 2, g)
    xs, dzs = ex.data(block, 77, g)
    parts, _, _ = ex.step(block, xs, dzs)
    buckets = torch.zeros(2, block.numel, dtype=BF, device="cuda")
    for r in range(2):
        _, kept = ex.forward(block, xs[r])
        ex.backward(block, dzs[r], kept, buckets[r])
    want, _ = ring.reduce_scatter([H.bits(b) for b in buckets], 2, 1, ring.RING_FP32, 0.5)
    for j in range(2):
        H.assert_f32_equal(parts[j].cpu().numpy(), want[j])
