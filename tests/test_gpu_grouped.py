"""Linear layers of experts against their definitions in 64 bits (tests/step_reference.py): sizes
that end inside tiles, experts without tokens, rows that belong to nobody (left as they were,
whatever they hold), odd strides and addresses, checkpoints, accumulation, empty calls."""
import pytest
import torch

import gradient_reduction_gb300 as dpr
from tests import gpu_helpers as H
from tests import operators_reference as R
from tests import step_cases as C
from tests import step_reference as S
from tests.test_gpu_operators import BF, F32, Placed, checkpoint, gen

pytestmark = pytest.mark.gpu

NAN = float("nan")


def offsets_of(counts, first=0):
    out = [first]
    for c in counts:
        out.append(out[-1] + c)
    return out


def device_offsets(offs):
    return torch.tensor(offs, dtype=torch.int32, device="cuda")


def randn(*shape, seed=0, scale=1.0):
    return (scale * torch.randn(*shape, generator=gen(seed))).to(BF)


# (tokens of each expert, out_features, in_features): one token, tiles that end inside, several
# tiles an expert, empty experts at both ends, sums of several accumulators
SIZES = [
    ((1,), 8, 8), ((1,), 1, 1), ((3,), 40, 72), ((64,), 256, 64), ((65, 1), 264, 120),
    ((0, 5, 0, 0, 257, 31, 0), 136, 200), ((256, 256), 512, 256), ((513, 100), 96, 1032),
    ((33,) * 9, 300, 24), ((1000, 24), 256, 2056), ((2, 3000), 72, 64), ((0, 0, 7), 1001, 1003),
    ((129, 0, 1), 67, 515),
    # few tiles of long sums, along the tokens and along the features: dealt out in parts
    ((3000,), 184, 412), ((0, 1500, 0, 7, 2600, 0), 200, 104), ((40,), 96, 6000), ((5, 0, 20), 3001, 2003),
    ((700,), 2056, 5000),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,o,i", SIZES)
@pytest.mark.parametrize("input_grad", [False, True], ids=["product", "input_grad"])
def test_product(input_grad, counts, o, i, dtype):
    H.device()
    offs = offsets_of(counts, 2)
    rows = offs[-1] + 3                      # rows in front of the first expert and behind the last
    have, give = (o, i) if input_grad else (i, o)
    x, w = randn(rows, have, seed=1), randn(len(counts), o, i, seed=2)
    x[:2] = NAN
    x[offs[-1]:] = NAN
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = NAN
    px, pw = Placed(rows, have, BF, -have % 8, 0, x), Placed(len(counts) * o, i, BF, -i % 8, 0,
                                                             w.view(-1, i))
    py = Placed(rows, give, dtype, 3)
    py.view.fill_(7)
    f = dpr.dpr_grouped_linear_input_grad if input_grad else dpr.dpr_grouped_linear
    f(px.view, device_offsets(offs), pw.view.unflatten(0, (len(counts), o)), py.view)
    want, size = S.product(x, offs, w, input_grad)
    mine = slice(offs[0], offs[-1])
    R.check(py.view[mine], want[mine], S.sum_bound(want, size, have, dtype, 76)[mine], "out")
    assert bool((py.view[:2] == 7).all()) and bool((py.view[offs[-1]:] == 7).all())
    for p, what in ((px, "x"), (pw, "weight"), (py, "out")):
        p.check_guards(what)


@pytest.mark.parametrize("saved", [False, True], ids=["stored", "saved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,o,i", SIZES)
def test_weight_gradient(counts, o, i, dtype, saved):
    H.device()
    offs = offsets_of(counts, 2)
    rows, experts = offs[-1] + 3, len(counts)
    dy, x = randn(rows, o, seed=1), randn(rows, i, seed=2)
    for t in (dy, x):
        t[:2] = NAN
        t[offs[-1]:] = NAN
    pd, px = Placed(rows, o, BF, -o % 8, 0, dy), Placed(rows, i, BF, -i % 8, 0, x)
    source, xx = px.view, x.double()
    if saved:
        pc, ps, source = checkpoint(rows, i)
        codes, steps = R.encode(x.double())
        pc.view.copy_(codes)
        ps.view.copy_(steps)
        xx = R.decode(codes, steps)
    pw = Placed(experts * o, i, dtype, 5)
    dw = pw.view.unflatten(0, (experts, o))
    dw.fill_(NAN)
    dpr.dpr_grouped_linear_weight_grad(pd.view, device_offsets(offs), source, dw)
    want, size = S.weight_grads(dy, offs, xx)
    bound = S.sum_bound(want, size, max(counts), dtype, 76)
    R.check(dw, want, bound, "dweight")
    old = torch.randn(experts, o, i, generator=gen(3)).to(dtype)
    dw.copy_(old)
    dpr.dpr_grouped_linear_weight_grad(pd.view, device_offsets(offs), source, dw, accumulate=True)
    total = want + old.double()
    R.check(dw, total, bound + (R.ROUND[dtype] + R.U) * (total.abs() + old.double().abs()), "added")
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e].cpu(), old[e])
    for p, what in ((pd, "dy"), (px, "x"), (pw, "dweight")):
        p.check_guards(what)


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (0, 1), (5, 7)])
def test_strides_and_addresses(pad, shift):
    """Rows that TMA reads where they are and rows that are copied first, for every operand; weights
    whose matrices lie apart, and one matrix for all experts."""
    H.device()
    counts, o, i = (70, 0, 9), 136, 264
    offs, rows, experts = offsets_of(counts), sum(counts), len(counts)
    x, dy, w = randn(rows, i, seed=1), randn(rows, o, seed=2), randn(experts, o, i, seed=3)
    px, pd = Placed(rows, i, BF, pad, shift, x), Placed(rows, o, BF, pad, shift, dy)
    apart = Placed(experts, (o + 1) * (i + pad), BF, 16, shift)
    pw = apart.view.unflatten(1, (o + 1, i + pad))[:, 1:, :i]
    pw.copy_(w)
    at = device_offsets(offs)
    for f, p, tr, give in ((dpr.dpr_grouped_linear, px, False, o),
                           (dpr.dpr_grouped_linear_input_grad, pd, True, i)):
        out = Placed(rows, give, F32, pad, shift)
        f(p.view, at, pw, out.view)
        want, size = S.product(p.view.cpu(), offs, w, tr)
        R.check(out.view, want, S.sum_bound(want, size, 264, F32), "out")
        out.check_guards("out")
        f(p.view, at, pw[:1].expand(experts, o, i), out.view)
        want, size = S.product(p.view.cpu(), offs, w[:1].expand(experts, o, i), tr)
        R.check(out.view, want, S.sum_bound(want, size, 264, F32), "shared weight")
    pc, ps, saved = checkpoint(rows, i, pad, shift)
    codes, steps = R.encode(x.double())
    pc.view.copy_(codes)
    ps.view.copy_(steps)
    for source, xx in ((px.view, x.double()), (saved, R.decode(codes, steps))):
        dw = apart.view.unflatten(1, (o + 1, i + pad))[:, :o, :i]
        dpr.dpr_grouped_linear_weight_grad(pd.view, at, source, dw)
        want, size = S.weight_grads(dy, offs, xx)
        R.check(dw, want, S.sum_bound(want, size, 70, BF), "dweight")
    apart.check_guards("weights")


# widths whose rows start anywhere: rows of all experts follow one another, experts' first rows lie
# anywhere too; one tile and several, sums in parts, fewer rows or channels than a step
ODD = [((3, 0, 20), 136, 67, 0), ((40,), 96, 6001, 1), ((5, 0, 300), 257, 129, 3), ((1,), 64, 65, 0),
       ((0, 0, 7, 2), 67, 515, 5), ((70, 1), 300, 1003, 2), ((2,), 4097, 701, 7), ((33,) * 9, 75, 65, 1),
       ((600, 0, 900), 200, 331, 4), ((9, 4), 40, 71, 1), ((9,), 63, 71, 1), ((9, 4), 70, 61, 1),
       ((130, 5, 64), 192, 256, 1), ((17, 3), 128, 65, 6), ((5000,), 72, 131, 1)]


@pytest.mark.parametrize("input_grad", [False, True], ids=["product", "input_grad"])
@pytest.mark.parametrize("counts,o,i,shift", ODD)
def test_weights_at_any_address(counts, o, i, shift, input_grad):
    """Without padding, between NaN, next to experts whose weights are NaN."""
    H.device()
    offs, experts = offsets_of(counts), len(counts)
    have, give = (o, i) if input_grad else (i, o)
    x, w = randn(offs[-1], have, seed=1), randn(experts, o, i, seed=2)
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = NAN
    memory = torch.full((experts * o * i + 64,), NAN, dtype=BF, device="cuda")
    pw = memory[16 + shift:16 + shift + w.numel()].view(experts, o, i)
    pw.copy_(w)
    for dtype in (BF, F32):
        out = Placed(offs[-1], give, dtype, 3)
        f = dpr.dpr_grouped_linear_input_grad if input_grad else dpr.dpr_grouped_linear
        f(x.cuda(), device_offsets(offs), pw, out.view)
        want, size = S.product(x, offs, w, input_grad)
        R.check(out.view, want, S.sum_bound(want, size, have, dtype, 76), "out")
        out.check_guards("out")


# more tiles than pairs of SMs, and a last round that is not full
@pytest.mark.parametrize("counts,o,i", [((300, 0, 1, 520, 256), 6300, 2200), ((700, 90), 5000, 4200),
                                        ((513, 2, 0), 9000, 2240), ((400, 300), 5003, 4201)])
@pytest.mark.parametrize("input_grad", [False, True], ids=["product", "input_grad"])
def test_several_rounds_of_tiles(counts, o, i, input_grad):
    H.device()
    offs, experts = offsets_of(counts), len(counts)
    have, give = (o, i) if input_grad else (i, o)
    x, w = randn(offs[-1], have, seed=1), randn(experts, o, i, seed=2)
    f = dpr.dpr_grouped_linear_input_grad if input_grad else dpr.dpr_grouped_linear
    want, size = S.product(x, offs, w, input_grad)
    xs, ws = x.cuda(), w.cuda()
    for dtype in (BF, F32):
        out = Placed(offs[-1], give, dtype, 3)
        f(xs, device_offsets(offs), ws, out.view)
        R.check(out.view, want, S.sum_bound(want, size, have, dtype, 76), "out")
        out.check_guards("out")


@pytest.mark.parametrize("odd", [False, True], ids=["aligned", "odd"])
@pytest.mark.parametrize("case", range(len(C.PRODUCTS_IN_PARTS)))
@pytest.mark.parametrize("input_grad", [False, True], ids=["product", "input_grad"])
def test_products_dealt_out_over_experts(input_grad, case, odd):
    H.device()
    counts, along, to = (C.ODD_PRODUCTS_IN_PARTS if odd else C.PRODUCTS_IN_PARTS)[case]
    o, i = (along, to) if input_grad else (to, along)
    offs, experts = offsets_of(counts, 2), len(counts)
    rows = offs[-1] + 3
    x, w = randn(rows, along, seed=1), randn(experts, o, i, seed=2)
    x[:2] = NAN
    x[offs[-1]:] = NAN
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = NAN
    px = Placed(rows, along, BF, -along % 8, 0, x)
    f = dpr.dpr_grouped_linear_input_grad if input_grad else dpr.dpr_grouped_linear
    want, size = S.product(x, offs, w, input_grad)
    mine = slice(offs[0], offs[-1])
    for dtype in (BF, F32):
        out = Placed(rows, to, dtype, 3)
        out.view.fill_(7)
        f(px.view, device_offsets(offs), w.cuda(), out.view)
        R.check(out.view[mine], want[mine], S.sum_bound(want, size, along, dtype, 76)[mine], "out")
        assert bool((out.view[:2] == 7).all()) and bool((out.view[offs[-1]:] == 7).all())
        out.check_guards("out")


@pytest.mark.parametrize("saved", [False, True], ids=["stored", "saved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,o,i", C.GRADS_IN_PARTS)
def test_weight_gradients_dealt_out_over_experts(counts, o, i, dtype, saved):
    H.device()
    offs, experts = offsets_of(counts, 2), len(counts)
    rows = offs[-1] + 3
    dy, x = randn(rows, o, seed=1), randn(rows, i, seed=2)
    for t in (dy, x):
        t[:2] = NAN
        t[offs[-1]:] = NAN
    pd, px = Placed(rows, o, BF, -o % 8, 0, dy), Placed(rows, i, BF, -i % 8, 0, x)
    source, xx = px.view, x.double()
    if saved:
        source = dpr.dpr_checkpoint_empty(rows, i)
        dpr.dpr_checkpoint_save(x.cuda(), source)
        xx = R.decode(source.codes.cpu(), source.steps.cpu())
    pw = Placed(experts * o, i, dtype, 5)
    dw = pw.view.unflatten(0, (experts, o))
    dw.fill_(NAN)
    dpr.dpr_grouped_linear_weight_grad(pd.view, device_offsets(offs), source, dw)
    want, size = S.weight_grads(dy, offs, xx)
    bound = S.sum_bound(want, size, max(counts), dtype, 76)
    R.check(dw, want, bound, "dweight")
    first = dw.clone()
    dpr.dpr_grouped_linear_weight_grad(pd.view, device_offsets(offs), source, dw)
    assert torch.equal(dw, first)
    old = torch.randn(experts, o, i, generator=gen(3)).to(dtype)
    dw.copy_(old)
    dpr.dpr_grouped_linear_weight_grad(pd.view, device_offsets(offs), source, dw, accumulate=True)
    total = want + old.double()
    R.check(dw, total, bound + (R.ROUND[dtype] + R.U) * (total.abs() + old.double().abs()), "added")
    pw.check_guards("dweight")


def test_one_row_for_all_tokens():
    H.device()
    w, x = randn(2, 72, 64, seed=1), randn(1, 64, seed=2)
    out = torch.empty(40, 72, device="cuda")
    dpr.dpr_grouped_linear(x.cuda().expand(40, 64), device_offsets([0, 10, 40]), w.cuda(), out)
    want, size = S.product(x.expand(40, 64), [0, 10, 40], w, False)
    R.check(out, want, S.sum_bound(want, size, 64, F32), "out")


def test_offsets_are_limited_to_the_rows():
    """What a broken router leaves is read and written within the rows that there are."""
    H.device()
    x, w = randn(10, 64, seed=1), randn(5, 72, 64, seed=2)
    for offs in ([-5, 3, 3, 100, 50, 2 ** 31 - 1], [-2 ** 31, -1, 0, 10, 10, 10], [20, 30, 5, 5, 5, 5]):
        out = Placed(10, 72, F32)
        out.view.fill_(7)
        dpr.dpr_grouped_linear(x.cuda(), device_offsets(offs), w.cuda(), out.view)
        want, size = S.product(x, offs, w, False)
        owned = ~want[:, 0].isnan()
        R.check(out.view[owned.cuda()], want[owned], S.sum_bound(want, size, 64, F32)[owned], "out")
        assert bool((out.view[~owned.cuda()] == 7).all())
        out.check_guards("out")
        dw = torch.empty(5, 72, 64, device="cuda")
        dpr.dpr_grouped_linear_weight_grad(out.view.to(BF), device_offsets(offs), x.cuda(), dw)
        want, size = S.weight_grads(out.view.to(BF).cpu(), offs, x)
        R.check(dw, want, S.sum_bound(want, size, 10, F32), "dweight")


def test_infinities_and_nan_stay_with_their_tokens():
    """A token's NaN reaches its own output row alone, and of the weight gradients its expert's
    alone, also where its neighbours share the step of the sum that the experts' border cuts."""
    H.device()
    offs = [0, 70, 100, 130]
    x, dy, w = randn(130, 72, seed=1), randn(130, 80, seed=2), randn(3, 80, 72, seed=3)
    x[75, 3], x[80, 5], dy[90, 7] = NAN, float("inf"), NAN
    out = torch.empty(130, 80, device="cuda")
    dpr.dpr_grouped_linear(x.cuda(), device_offsets(offs), w.cuda(), out)
    want, size = S.product(x, offs, w, False)
    ok = torch.ones(130, dtype=torch.bool)
    ok[[75, 80]] = False
    R.check(out.cpu()[ok], want[ok], S.sum_bound(want, size, 72, F32)[ok], "out")
    assert bool(out[75].isnan().all()) and not bool(out[80].isfinite().any())
    dw = torch.empty(3, 80, 72, device="cuda")
    saved = dpr.dpr_checkpoint_empty(130, 72)
    dpr.dpr_checkpoint_save(x.cuda(), saved)
    restored = torch.empty(130, 72, dtype=BF, device="cuda")
    dpr.dpr_checkpoint_load(saved, restored)
    for source, xx in ((x.cuda(), x), (saved, restored.cpu())):
        dpr.dpr_grouped_linear_weight_grad(dy.cuda(), device_offsets(offs), source, dw)
        want, size = S.weight_grads(dy, offs, xx)
        for e in (0, 2):
            R.check(dw[e], want[e], S.sum_bound(want[e], size[e], 70, F32), f"expert {e}")
        assert bool(dw[1, 7].isnan().all()) and bool(dw[1, :, 3].isnan().all())


def test_calls_without_tokens():
    H.device()
    w = randn(3, 72, 64).cuda()
    at = device_offsets([0, 0, 0, 0])
    none, y = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, 72, device="cuda")
    dpr.dpr_grouped_linear(none, at, w, y)
    dpr.dpr_grouped_linear_input_grad(y.to(BF), at, w, none)
    dw = torch.full((3, 72, 64), 5.0, device="cuda")
    dpr.dpr_grouped_linear_weight_grad(y.to(BF), at, none, dw, accumulate=True)
    assert bool((dw == 5).all())
    dpr.dpr_grouped_linear_weight_grad(y.to(BF), at, none, dw)
    assert not dw.any()
    # rows, but no expert has any
    x = torch.full((40, 64), NAN, dtype=BF, device="cuda")
    y = torch.full((40, 72), 7.0, device="cuda")
    dpr.dpr_grouped_linear(x, at, w, y)
    assert bool((y == 7).all())
    for source in (x, dpr.dpr_checkpoint_empty(40, 64)):
        dw.fill_(5)
        dpr.dpr_grouped_linear_weight_grad(y.to(BF), at, source, dw)
        assert not dw.any()


def test_many_experts():
    """The most that a call takes, most of them with a token or none."""
    H.device()
    counts = [(e * 7) % 4 for e in range(1024)]
    offs = offsets_of(counts)
    x, w = randn(offs[-1], 64, seed=1), randn(1024, 72, 64, seed=2)
    out = torch.empty(offs[-1], 72, device="cuda")
    dpr.dpr_grouped_linear(x.cuda(), device_offsets(offs), w.cuda(), out)
    want, size = S.product(x, offs, w, False)
    R.check(out, want, S.sum_bound(want, size, 64, F32), "out")
    dw = torch.empty(1024, 72, 64, device="cuda")
    dpr.dpr_grouped_linear_weight_grad(out.to(BF), device_offsets(offs), x.cuda(), dw)
    want, size = S.weight_grads(out.to(BF).cpu(), offs, x)
    R.check(dw, want, S.sum_bound(want, size, 3, F32), "dweight")


def test_binding_refusals():
    H.device()
    x, w = randn(8, 64).cuda(), randn(2, 72, 64).cuda()
    y, at = torch.empty(8, 72, device="cuda"), device_offsets([0, 3, 8])
    for bad in ((x, at.long(), w, y), (x, at[:2], w, y), (x, at, w[0], y), (x[:, :63], at, w, y),
                (x, at, w, y[:7]), (x, at, w, y[:, :71]), (x.float(), at, w, y),
                (x, at, w.float(), y), (x, at, w, y.half()), (x, at.cpu(), w, y)):
        with pytest.raises(ValueError):
            dpr.dpr_grouped_linear(*bad)
    dw = torch.empty(2, 72, 64, device="cuda")
    dy = torch.empty(8, 72, dtype=BF, device="cuda")
    for bad in ((dy, at, x[:7], dw), (dy, at, x.float(), dw), (dy[:, :71], at, x, dw),
                (dy, at, x, dw[:1]), (dy, at, x, dw.transpose(1, 2))):
        with pytest.raises(ValueError):
            dpr.dpr_grouped_linear_weight_grad(*bad)


@pytest.mark.parametrize("wide", [4096, 4099], ids=["aligned", "odd"])
def test_activations_past_32_bits(wide):
    """Inputs and outputs of more than 2^32 elements; an expert with the last rows alone, one with none,
    and one with the rows around element 2^32."""
    H.device()
    rows, narrow = (1 << 20) + 5000, 72
    offs = [(1 << 20) - 300, (1 << 20) + 300, (1 << 20) + 300, rows - 77, rows - 70, rows]
    mine = [slice(offs[0], offs[1]), slice(offs[3], rows)]
    w = randn(5, wide, narrow, seed=1, scale=0.1)
    x = torch.full((rows, narrow), NAN, dtype=BF)
    for k, m in enumerate(mine):
        x[m] = randn(m.stop - m.start, narrow, seed=2 + k)
    offs[2:4] = [offs[1], rows - 77]             # expert 2 has the many rows between: NaN
    y = torch.full((rows, wide), 7.0, dtype=BF, device="cuda")
    dpr.dpr_grouped_linear(x.cuda(), device_offsets(offs), w.cuda(), y)
    assert bool((y[:offs[0]] == 7).all())
    back = torch.empty(rows, narrow, device="cuda")
    dpr.dpr_grouped_linear_input_grad(y, device_offsets(offs), w.cuda(), back)
    dw = torch.empty(5, wide, narrow, device="cuda")
    dpr.dpr_grouped_linear_weight_grad(y, device_offsets(offs), x.cuda(), dw)
    for e, m in ((0, mine[0]), (3, slice(rows - 77, rows - 70)), (4, slice(rows - 70, rows))):
        got = y[m].cpu()
        n = m.stop - m.start
        want, size = S.product(x[m], [0, n], w[e:e + 1], False)
        R.check(got, want, S.sum_bound(want, size, narrow, BF, 76), "y")
        want, size = S.product(got, [0, n], w[e:e + 1], True)
        R.check(back[m], want, S.sum_bound(want, size, wide, F32, 76), "dx")
        want, size = S.weight_grads(got, [0, n], x[m])
        R.check(dw[e], want[0], S.sum_bound(want, size, n, F32, 76)[0], "dweight")


@pytest.mark.parametrize("dtype,wide", [(BF, 4096), (F32, 4096), (F32, 4095)])
def test_weights_past_32_bits(dtype, wide):
    """Experts' matrices of more than 2^32 elements in all: gradients of the last, products with them."""
    H.device()
    experts, o = 260, 4100
    rows, counts = 37, [0] * experts
    counts[0], counts[257], counts[259] = 5, 12, 20
    offs = offsets_of(counts)
    dy, x = randn(rows, o, seed=1), randn(rows, wide, seed=2)
    dw = torch.empty(experts, o, wide, dtype=dtype, device="cuda")
    dw[1].fill_(NAN)
    dw[258].fill_(NAN)
    dpr.dpr_grouped_linear_weight_grad(dy.cuda(), device_offsets(offs), x.cuda(), dw)
    assert not dw[1].any() and not dw[258].any()
    for e in (0, 257, 259):
        m = slice(offs[e], offs[e + 1])
        want, size = S.weight_grads(dy[m], [0, counts[e]], x[m])
        R.check(dw[e], want[0], S.sum_bound(want, size, counts[e], dtype, 76)[0], "dweight")
    if dtype == F32:
        return
    y = torch.empty(rows, o, device="cuda")
    dpr.dpr_grouped_linear(x.cuda(), device_offsets(offs), dw, y)
    for e in (0, 257, 259):
        m = slice(offs[e], offs[e + 1])
        want, size = S.product(x[m], [0, counts[e]], dw[e:e + 1].cpu(), False)
        R.check(y[m], want, S.sum_bound(want, size, wide, F32, 76), "y")


def test_missing_tensors():
    H.device()
    x, w = randn(8, 64).cuda(), randn(2, 72, 64).cuda()
    y, at = torch.empty(8, 72, device="cuda"), device_offsets([0, 3, 8])
    for f, a, b in ((dpr.dpr_grouped_linear, x, y), (dpr.dpr_grouped_linear_input_grad, y.to(BF), x)):
        for bad in ((a, None, w, b), (a, at, None, b), (a, at, w, None)):
            with pytest.raises(ValueError, match="needed"):
                f(*bad)
    for bad in ((y.to(BF), None, x, torch.empty(2, 72, 64, device="cuda")), (y.to(BF), at, x, None)):
        with pytest.raises(ValueError, match="needed"):
            dpr.dpr_grouped_linear_weight_grad(*bad)


def test_no_wait_ran_out():
    H.device()
    assert dpr.dpr_device_wait_failures() == 0
