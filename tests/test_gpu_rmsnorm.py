"""RMS norm with the residual's addition, forward and backward, against its definition in 64 bits
(tests/step_reference.py): every access width, odd strides and addresses, rows from one channel to
ones too long for registers, in-place forms, infinities and NaN, empty calls, guard bytes."""
import pytest
import torch

import gradient_reduction_gb300 as dpr
from tests import gpu_helpers as H
from tests import operators_reference as R
from tests import step_reference as S
from tests.test_gpu_operators import BF, F32, LAYOUTS, Placed, activation, checkpoint, gen

pytestmark = pytest.mark.gpu

EPS = 1e-6
WIDTHS = [1, 2, 31, 32, 33, 48, 96, 100, 512, 520, 1000, 1001, 2064, 4096, 4097, 8192, 11008, 16384,
          16400, 33000]


def weight_of(width, dtype, seed=5):
    return (1 + 0.2 * torch.randn(width, generator=gen(seed))).to(dtype)


def added(x, residual):
    """x + residual in their type, rounded once (fp32's sum of two bf16 numbers, then bf16)."""
    return (x.float() + residual.float()).to(x.dtype)


def same_saved(got, of):
    codes, steps = R.encode(of.double())
    assert torch.equal(got.codes.cpu(), codes) and torch.equal(got.steps.cpu(), steps)


# --- forward -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("width", WIDTHS)
def test_forward(width, layout, dtype):
    H.device()
    pad, shift = LAYOUTS[layout]
    rows = 3 if width > 8192 else 7
    x, r = activation(rows, width, width, dtype), activation(rows, width, width + 1, dtype)
    w = weight_of(width, dtype)
    h = added(x, r)
    px, pr = (Placed(rows, width, dtype, pad, shift, t) for t in (x, r))
    ph, py = Placed(rows, width, dtype, pad, shift), Placed(rows, width, dtype, pad, shift)
    ps = Placed(1, rows, F32)
    hc, hs, h_saved = checkpoint(rows, width, None if layout == "plain" else pad, shift)
    yc, ys, y_saved = checkpoint(rows, width, None if layout == "plain" else pad, shift)
    dpr.dpr_rmsnorm_forward(px.view, w.cuda(), EPS, py.view, ps.view[0], pr.view, ph.view, h_saved,
                            y_saved)
    want, rstd = S.rms_forward(h, w, EPS)
    d_y, d_rstd = S.rms_forward_bounds(h, w, EPS, dtype)
    assert torch.equal(ph.view.cpu(), h)
    R.check(py.view, want, d_y, "y")
    R.check(ps.view[0], rstd, d_rstd, "rstd")
    same_saved(h_saved, h)
    same_saved(y_saved, py.view.cpu())
    for p, what in ((px, "x"), (pr, "residual"), (ph, "h"), (py, "y"), (ps, "rstd"), (hc, "codes"),
                    (hs, "steps"), (yc, "codes"), (ys, "steps")):
        p.check_guards(what)
    # the same without what is optional: y from x alone, y in 8 bits alone (the order of a row's sum
    # goes by the layouts, so that the bits are the same where those are)
    y = torch.empty(rows, width, dtype=dtype, device="cuda")
    dpr.dpr_rmsnorm_forward(ph.view, w.cuda(), EPS, y)
    R.check(y, want, d_y, "y alone")
    alone = dpr.dpr_checkpoint_empty(rows, width)
    dpr.dpr_rmsnorm_forward(px.view, w.cuda(), EPS, residual=pr.view, y_checkpoint=alone)
    if layout == "plain":
        assert torch.equal(y, py.view)
        assert torch.equal(alone.codes, y_saved.codes) and torch.equal(alone.steps, y_saved.steps)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [100, 1001, 4096, 20000])
@pytest.mark.parametrize("places", ["h is residual", "h is x", "y is x", "y is residual",
                                    "h is residual, y is x", "h is x, y is residual"])
def test_forward_in_place(places, width, dtype):
    H.device()
    x, r = (activation(9, width, s, dtype).cuda() for s in (1, 2))
    w = weight_of(width, F32).cuda()
    want_h, want_y = torch.empty_like(x), torch.empty_like(x)
    dpr.dpr_rmsnorm_forward(x, w, EPS, want_y, residual=r, h=want_h)
    h = x if "h is x" in places else r if "h is residual" in places else torch.empty_like(x)
    y = x if "y is x" in places else r if "y is residual" in places else torch.empty_like(x)
    dpr.dpr_rmsnorm_forward(x, w, EPS, y, residual=r, h=h)
    assert torch.equal(h, want_h) and torch.equal(y, want_y)


@pytest.mark.parametrize("rows", [0, 1, 2, 33, 1000, 70001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_rows(rows, dtype):
    """Short rows that share warps and blocks, an expanded (broadcast) residual, no weight."""
    H.device()
    for width in (8, 40, 64):
        x, r = activation(rows, width, rows, dtype), activation(1, width, 3, dtype)
        y, rstd = torch.empty(rows, width, dtype=dtype, device="cuda"), torch.empty(rows, device="cuda")
        dpr.dpr_rmsnorm_forward(x.cuda(), None, EPS, y, rstd, r.cuda().expand(rows, width))
        h = added(x, r.expand(rows, width))
        want, want_rstd = S.rms_forward(h, torch.ones(width), EPS)
        d_y, d_rstd = S.rms_forward_bounds(h, torch.ones(width), EPS, dtype)
        R.check(y, want, d_y, "y")
        R.check(rstd, want_rstd, d_rstd, "rstd")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [64, 1001, 4096, 20000])
def test_infinities_and_nan_stay_in_their_row(width, dtype):
    H.device()
    x = activation(6, width, 4, dtype)
    x[1, width // 2] = float("inf")
    x[3, 0] = float("nan")
    x[4] = 0
    w = weight_of(width, dtype)
    y, rstd = torch.empty(6, width, dtype=dtype, device="cuda"), torch.empty(6, device="cuda")
    dpr.dpr_rmsnorm_forward(x.cuda(), w.cuda(), EPS, y, rstd)
    want, want_rstd = S.rms_forward(x, w, EPS)
    d_y, d_rstd = S.rms_forward_bounds(x, w, EPS, dtype)
    R.check(y, want, d_y, "y")
    R.check(rstd, want_rstd, d_rstd, "rstd")
    dy = (1e-2 * torch.randn(6, width, generator=gen(6))).to(dtype)
    dy[2, width - 1] = float("nan")
    dx = torch.empty_like(y)
    dpr.dpr_rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd, dx)
    bad = [1, 2, 3]
    ok = [0, 4, 5]
    assert bool(dx[3].isnan().all()) and bool(dx[2].isnan().all()) and bool(dx[1].isnan().any())
    want, _ = S.rms_backward(dy[ok], x[ok], w, rstd.cpu()[ok])
    bound, _ = S.rms_backward_bounds(dy[ok], x[ok], w, rstd.cpu()[ok], None, dtype, dtype)
    R.check(dx[ok], want, bound, f"rows beside {bad}")


@pytest.mark.parametrize("layout", ["plain", "half", "odd"])
@pytest.mark.parametrize("width", [96, 1000, 1001, 4096, 5000])
def test_forward_of_many_bf16_rows_with_checkpoints(width, layout):
    """From 1024 rows on a thread takes 32 channels."""
    H.device()
    pad, shift = LAYOUTS[layout]
    rows = 1100
    x, r = activation(rows, width, width, BF), activation(rows, width, width + 1, BF)
    w = weight_of(width, BF)
    h = added(x, r)
    px, pr = (Placed(rows, width, BF, pad, shift, t) for t in (x, r))
    ph, py = Placed(rows, width, BF, pad, shift), Placed(rows, width, BF, pad, shift)
    rstd = torch.empty(rows, device="cuda")
    hc, hs, h_saved = checkpoint(rows, width, None if layout == "plain" else pad, shift)
    yc, ys, y_saved = checkpoint(rows, width, None if layout == "plain" else pad, shift)
    dpr.dpr_rmsnorm_forward(px.view, w.cuda(), EPS, py.view, rstd, pr.view, ph.view, h_saved, y_saved)
    want, want_rstd = S.rms_forward(h, w, EPS)
    d_y, d_rstd = S.rms_forward_bounds(h, w, EPS, BF)
    assert torch.equal(ph.view.cpu(), h)
    R.check(py.view, want, d_y, "y")
    R.check(rstd, want_rstd, d_rstd, "rstd")
    same_saved(h_saved, h)
    same_saved(y_saved, py.view.cpu())
    for p, what in ((px, "x"), (pr, "residual"), (ph, "h"), (py, "y"), (hc, "codes"), (hs, "steps"),
                    (yc, "codes"), (ys, "steps")):
        p.check_guards(what)


# --- backward ------------------------------------------------------------------

def run_backward(rows, width, dtype, pad, shift, saved, with_dh, grad_dtype=F32, accumulate=False):
    h = activation(rows, width, rows + width, dtype)
    dy, dh = ((1e-2 * torch.randn(rows, width, generator=gen(s))).to(dtype) for s in (11, 12))
    w = weight_of(width, dtype)
    _, rstd = S.rms_forward(h, w, EPS)
    rstd = rstd.float()
    source, hh = Placed(rows, width, dtype, pad, shift, h), h.double()
    placed = [(source, "h")]
    source = source.view
    if saved:
        pc, ps, source = checkpoint(rows, width, None if pad == 0 else pad, shift)
        codes, steps = R.encode(h.double())
        pc.view.copy_(codes)
        ps.view.copy_(steps)
        hh = R.decode(codes, steps)
        placed += [(pc, "codes"), (ps, "steps")]
    pd, pe = (Placed(rows, width, dtype, pad, shift, t) for t in (dy, dh))
    po, pw = Placed(rows, width, dtype, pad, shift), Placed(1, width, grad_dtype)
    old = torch.randn(width, generator=gen(9)).to(grad_dtype)
    pw.view[0].copy_(old)
    dpr.dpr_rmsnorm_backward(pd.view, source, w.cuda(), rstd.cuda(), po.view, pw.view[0],
                             dh=pe.view if with_dh else None, accumulate=accumulate)
    dx, dw = S.rms_backward(dy, hh, w, rstd, dh if with_dh else None)
    d_dx, d_dw = S.rms_backward_bounds(dy, hh, w, rstd, dh if with_dh else None, dtype, grad_dtype)
    if accumulate:
        dw = dw + old.double()
        d_dw = d_dw + (R.ROUND[grad_dtype] + R.U) * (dw.abs() + old.double().abs())
    R.check(po.view, dx, d_dx, "dx")
    R.check(pw.view[0], dw, d_dw, "dweight")
    for p, what in placed + [(pd, "dy"), (pe, "dh"), (po, "dx"), (pw, "dweight")]:
        p.check_guards(what)


@pytest.mark.parametrize("saved", [False, True], ids=["stored", "saved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("width", WIDTHS)
def test_backward(width, layout, dtype, saved):
    H.device()
    pad, shift = LAYOUTS[layout]
    run_backward(3 if width > 8192 else 11, width, dtype, pad, shift, saved, width % 2 == 0)


@pytest.mark.parametrize("saved", [False, True], ids=["stored", "saved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,width", [(1, 4096), (305, 768), (700, 2048), (1300, 4096), (913, 5120),
                                        (457, 8192), (311, 12288), (9001, 24), (4000, 130)])
def test_backward_many_rows(rows, width, dtype, saved):
    """Every block with several turns, groups whose rows end at different turns."""
    H.device()
    run_backward(rows, width, dtype, 0, 0, saved, True)
    run_backward(rows, width, dtype, 8, 8, saved, False, BF, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [100, 1001, 4096, 20000])
@pytest.mark.parametrize("place", ["dy", "dh", "h"])
def test_backward_in_place(place, width, dtype):
    H.device()
    t = {n: (activation(200, width, s, dtype) * (1 if n == "h" else 1e-2)).cuda()
         for n, s in (("dy", 1), ("dh", 2), ("h", 3))}
    w, rstd = weight_of(width, dtype).cuda(), torch.rand(200, generator=gen(4)).cuda() + 0.5
    want, want_w = torch.empty_like(t["dy"]), torch.empty(width, device="cuda")
    dpr.dpr_rmsnorm_backward(t["dy"], t["h"], w, rstd, want, want_w, dh=t["dh"])
    dw = torch.empty(width, device="cuda")
    dpr.dpr_rmsnorm_backward(t["dy"], t["h"], w, rstd, t[place], dw, dh=t["dh"])
    assert torch.equal(t[place], want) and torch.equal(dw, want_w)


def test_backward_without_rows_or_outputs():
    H.device()
    none = torch.empty(0, 64, device="cuda")
    dw = torch.full((64,), 3.0, device="cuda")
    rstd = torch.empty(0, device="cuda")
    dpr.dpr_rmsnorm_backward(none, none, None, rstd, none, dw, accumulate=True)
    assert bool((dw == 3).all())
    dpr.dpr_rmsnorm_backward(none, none, None, rstd, none, dw)
    assert not dw.any()


def test_gradient_against_differences():
    """The forward's own outputs in fp32, differenced along random directions: the sum of their
    rounding errors (2 * 3 u |y dy| summed) over the step's length, and the third derivative's part,
    of the order step^2, are below 1e-3 of the slope."""
    H.device()
    rows, width, step = 5, 300, 2.0 ** -6
    h, v = torch.randn(rows, width, generator=gen(1)), torch.randn(rows, width, generator=gen(2))
    w, u = weight_of(width, F32), torch.randn(width, generator=gen(3))
    dy = torch.randn(rows, width, generator=gen(4))

    def value(h, w):
        y, rstd = torch.empty(rows, width, device="cuda"), torch.empty(rows, device="cuda")
        dpr.dpr_rmsnorm_forward(h.cuda(), w.cuda(), EPS, y, rstd)
        return float((y.cpu().double() * dy.double()).sum()), rstd
    _, rstd = value(h, w)
    dx, dw = torch.empty(rows, width, device="cuda"), torch.empty(width, device="cuda")
    dpr.dpr_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd, dx, dw)
    for slope, (a, b) in (((dx.cpu() * v).double().sum(), ((h + step * v, w), (h - step * v, w))),
                          ((dw.cpu() * u).double().sum(), ((h, w + step * u), (h, w - step * u)))):
        measured = (value(*a)[0] - value(*b)[0]) / (2 * step)
        size = float((dy.abs()).sum()) * 1e-3
        assert abs(float(slope) - measured) < size


@pytest.mark.parametrize("width", [40, 300, 1001])
def test_gradient_against_differences_along_the_row(width):
    """The forward's fp32 outputs differenced along the row itself, where the slope is none but for
    eps: the term that takes the part along the row away makes up for all the rest.  And along the
    weight.  The bound is the sum of the same difference quotient's distance from the slope in 64
    bits, of the outputs' errors over the step's length, and of the gradients' own errors."""
    H.device()
    rows, step = 5, 2.0 ** -6
    h, w = torch.randn(rows, width, generator=gen(1)), weight_of(width, F32)
    dy = h * torch.rand(rows, width, generator=gen(2))          # a gradient along the row
    u = w * torch.rand(width, generator=gen(3))
    _, rstd = S.rms_forward(h, w, EPS)
    rstd = rstd.float()
    want, want_w = S.rms_backward(dy, h, w, rstd)
    d_dx, d_dw = S.rms_backward_bounds(dy, h, w, rstd, None, F32, F32)
    kept = rstd.double()[:, None] * dy.double() * w.double()    # without that term
    dx, dw = torch.empty(rows, width, device="cuda"), torch.empty(width, device="cuda")
    dpr.dpr_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dx, dw)
    for got, exact, error, ends in ((dx.cpu().double() * h.double(), want * h.double(), d_dx * h.double().abs(),
                                     [(h + a * step * h, w) for a in (1, -1)]),
                                    (dw.cpu().double() * u.double(), want_w * u.double(), d_dw * u.double().abs(),
                                     [(h, w + a * step * u) for a in (1, -1)])):
        measured, in64, rounding = 0.0, 0.0, 0.0
        for sign, (a, b) in zip((1, -1), ends):
            y = torch.empty(rows, width, device="cuda")
            dpr.dpr_rmsnorm_forward(a.cuda(), b.cuda(), EPS, y)
            measured += sign * float((y.cpu().double() * dy.double()).sum()) / (2 * step)
            in64 += sign * float((S.rms_forward(a, b, EPS)[0] * dy.double()).sum()) / (2 * step)
            rounding += float((S.rms_forward_bounds(a, b, EPS, F32)[0] * dy.double().abs()).sum()) / (2 * step)
        bound = abs(in64 - float(exact.sum())) + rounding + float(error.sum())
        assert abs(float(got.sum()) - measured) <= bound
        if got.dim() == 2:
            assert float(((kept - want) * h.double()).sum()) > 1000 * bound


def test_rows_past_32_bits():
    """Elements past 2^32 of a matrix: the last rows of 300000 x 16384."""
    H.device()
    rows, width = 300000, 16384
    x = torch.zeros(rows, width, dtype=BF, device="cuda")
    tail = activation(3, width, 1, BF)
    x[-3:] = tail.cuda()
    w = weight_of(width, BF)
    rstd = torch.empty(rows, device="cuda")
    dpr.dpr_rmsnorm_forward(x, w.cuda(), EPS, x, rstd)
    want, want_rstd = S.rms_forward(tail, w, EPS)
    d_y, d_rstd = S.rms_forward_bounds(tail, w, EPS, BF)
    R.check(x[-3:], want, d_y, "y")
    R.check(rstd[-3:], want_rstd, d_rstd, "rstd")
    assert not x[:-3].any()


@pytest.mark.parametrize("saved", [False, True], ids=["stored", "saved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [24, 100, 1001, 4096, 8192, 12288, 20000])
@pytest.mark.parametrize("size,grad", [(2.0 ** 57, 2.0 ** -50), (2.0 ** 40, 2.0 ** -60), (2.0 ** 40, 2.0 ** -90),
                                       (2.0 ** -62, 16.0)])
def test_backward_of_large_and_small_rows(size, grad, width, dtype, saved):
    """Rows whose rstd^2 leaves fp32 or takes small gradients out of it, while the outputs are in it.
    (Only the last operation on dx may round a subnormal number: half of TINY.)"""
    H.device()
    rows = 40
    h = (activation(rows, width, 1, F32) * size).to(dtype)
    dy = (torch.randn(rows, width, generator=gen(2)) * grad).to(dtype)
    w = weight_of(width, dtype)
    rstd = S.rms_forward(h, w, 0.0)[1].float()
    source, hh = h.cuda(), h.double()
    if saved:
        source = dpr.dpr_checkpoint_empty(rows, width)
        dpr.dpr_checkpoint_save(h.cuda(), source)
        hh = R.decode(source.codes.cpu(), source.steps.cpu())
    dx, dw = torch.empty(rows, width, dtype=dtype, device="cuda"), torch.empty(width, device="cuda")
    dpr.dpr_rmsnorm_backward(dy.cuda(), source, w.cuda(), rstd.cuda(), dx, dw)
    want, want_w = S.rms_backward(dy, hh, w, rstd)
    d_dx, d_dw = S.rms_backward_bounds(dy, hh, w, rstd, None, dtype, F32)
    R.check(dw, want_w, d_dw, "dweight")
    R.check(dx, want, d_dx, "dx")


@pytest.mark.parametrize("pad", [0, 3], ids=["staged", "odd"])
def test_backward_of_rows_past_32_bits(pad):
    """The last rows of more than 2^32 elements; a broadcast dh; the others' gradient is dh."""
    H.device()
    rows, width = 300000, 16384 - 8 + pad
    tail = activation(3, width, 1, BF)
    dy = torch.zeros(rows, width, dtype=BF, device="cuda")
    dy[-3:] = tail.flip(0).cuda()
    h = torch.zeros(rows, width, dtype=BF, device="cuda")
    h[-3:] = tail.cuda()
    dh = (1e-2 * torch.randn(1, width, generator=gen(2))).to(BF)
    w, rstd = weight_of(width, BF), torch.rand(rows, generator=gen(3)) + 0.5
    dw = torch.empty(width, device="cuda")
    dpr.dpr_rmsnorm_backward(dy, h, w.cuda(), rstd.cuda(), dy, dw, dh=dh.cuda().expand(rows, width))
    args = tail.flip(0), tail, w, rstd[-3:], dh.expand(3, width)
    want, want_w = S.rms_backward(*args)
    bound, bound_w = S.rms_backward_bounds(*args, BF, F32)
    R.check(dy[-3:], want, bound, "dx")
    R.check(dw, want_w, bound_w, "dweight")
    for at in (0, 131072, 262144, rows - 4):
        assert torch.equal(dy[at].cpu(), dh[0])
