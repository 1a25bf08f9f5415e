"""The global gradient norm and clipping against their definitions in 64 bits: lists of odd lengths
and addresses, every pair of types, in place, extreme magnitudes, infinities and NaN, empty lists."""
import pytest
import torch

import gradient_reduction_gb300 as dpr
from tests import gpu_helpers as H
from tests import operators_reference as R
from tests import step_reference as S
from tests.test_gpu_operators import BF, F32, Placed, gen

pytestmark = pytest.mark.gpu

LISTS = {
    "one element": [1], "one small": [1000], "four tiles": [8192] * 4, "five tiles": [8192] * 5,
    "ragged": [1, 0, 17, 8191, 8193, 31, 33, 16, 15, 0, 100001], "one large": [3_000_001],
    "many": [(7 * k * k) % 5003 for k in range(300)],
}


def grads_of(sizes, dtype, shift, seed=0):
    g = gen(seed)
    out = []
    for k, n in enumerate(sizes):
        out.append((1e-3 * 2.0 ** (k % 5) * torch.randn(n, generator=g)).to(dtype))
    return out, [Placed(1, n, dtype, 0, shift, t) for n, t in zip(sizes, out)]


@pytest.mark.parametrize("shift,out_shift", [(0, 0), (1, 1), (8, 0), (3, 8), (16, 16)])
@pytest.mark.parametrize("src,dst", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("sizes", list(LISTS.values()), ids=list(LISTS))
def test_norm_and_clip(sizes, src, dst, shift, out_shift):
    H.device()
    grads, placed = grads_of(sizes, src, shift)
    outs = [Placed(1, n, dst, 0, out_shift) for n in sizes]
    total, _ = S.clip(grads, 0.5, 1e30)
    norm = torch.full((3,), -1.0, device="cuda")
    with dpr.dpr_grad_plan_create([p.view[0] for p in placed], [p.view[0] for p in outs]) as plan:
        for max_norm in (total / 3, total * 3):
            want, clipped = S.clip(grads, 0.5, max_norm)
            dpr.dpr_grad_norm_clip(plan, norm[1:2], max_norm, scale=0.5)
            assert abs(norm[1].item() - want) <= S.NORM_ERROR * want
            assert norm[0].item() == norm[2].item() == -1
            first = [p.view.clone() for p in outs]
            for p, w in zip(outs, clipped):
                R.check(p.view[0], w, S.clip_bound(w, dst), "out")
                p.check_guards("out")
            # the two halves by themselves give the same bits
            alone = torch.empty(1, device="cuda")
            dpr.dpr_grad_norm(plan, alone, scale=0.5)
            assert torch.equal(alone, norm[1:2])
            for p in outs:
                p.view.fill_(9)
            dpr.dpr_grad_clip(plan, alone, max_norm, scale=0.5)
            assert all(torch.equal(p.view, f) for p, f in zip(outs, first))
    for p in placed:
        p.check_guards("grads")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [[100, 3000], [8192 * 9 + 5, 77, 0, 4096]])
def test_in_place(sizes, dtype):
    H.device()
    grads, placed = grads_of(sizes, dtype, 2)
    total, _ = S.clip(grads, 1.0, 1e30)
    norm = torch.empty(1, device="cuda")
    with dpr.dpr_grad_plan_create([p.view[0] for p in placed]) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, 2 * total)               # nothing to do
        assert all(torch.equal(p.view[0].cpu(), g) for p, g in zip(placed, grads))
        dpr.dpr_grad_norm_clip(plan, norm, total / 2)
        for p, w in zip(placed, S.clip(grads, 1.0, total / 2)[1]):
            R.check(p.view[0], w, S.clip_bound(w, dtype), "clipped")
            p.check_guards("clipped")
        dpr.dpr_grad_norm(plan, norm)                                # of what it left
        left = S.clip([p.view[0].cpu() for p in placed], 1.0, 1e30)[0]
        assert abs(norm.item() - left) <= S.NORM_ERROR * left


def test_lists_of_both_types_and_places():
    """bf16 and fp32 gradients in one list, some in place, some cast into a flat buffer."""
    H.device()
    a, b, c = (torch.randn(n, generator=gen(n)).cuda() for n in (5000, 40000, 300))
    a, c = a.to(BF), c.to(BF)
    flat = torch.zeros(5000 + 304, device="cuda")
    grads = [a.cpu(), b.cpu(), c.cpu()]
    norm = torch.empty(1, device="cuda")
    plan = dpr.dpr_grad_plan_create([a, b, c], [flat[:5000], b, flat[5000:5300]])
    dpr.dpr_grad_norm_clip(plan, norm, 1.0, scale=0.25)
    want, clipped = S.clip(grads, 0.25, 1.0)
    assert abs(norm.item() - want) <= S.NORM_ERROR * want
    for got, w in zip((flat[:5000], b, flat[5000:5300]), clipped):
        R.check(got, w, S.clip_bound(w, F32), "out")
    assert torch.equal(a.cpu(), grads[0]) and not flat[5300:].any()
    dpr.dpr_grad_plan_destroy(plan)
    with pytest.raises(ValueError, match="closed"):
        dpr.dpr_grad_norm(plan, norm)


@pytest.mark.parametrize("value", [2.0 ** -149, 2.0 ** -120, 1e-25, 2.0 ** -50, 2.0 ** -49, 1e9,
                                   2.0 ** 30, 1e25, 3e38])
@pytest.mark.parametrize("n", [16, 9000, 100000])
def test_magnitudes_whose_squares_leave_fp32(value, n):
    """All gradients of one tiny or huge magnitude, and among ordinary ones."""
    H.device()
    t = torch.full((n,), value)
    mixed = t.clone()
    mixed[::3] = 1.0
    for g in (t, mixed):
        norm, out = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
        with dpr.dpr_grad_plan_create([g.cuda()], [out]) as plan:
            dpr.dpr_grad_norm(plan, norm)
            want = float(g.double().square().sum()) ** 0.5
            if want > 3.4e38:
                assert norm.item() == float("inf")
            else:
                assert abs(norm.item() - want) <= S.NORM_ERROR * want + 2.0 ** -149


@pytest.mark.parametrize("dst", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("n", [5, 9000, 300000])
@pytest.mark.parametrize("max_norm,scale", [(1e-2, 1.0), (1e-6, 0.25), (1.0, 2.0 ** -20), (2.0 ** 100, 2.0 ** -110)])
def test_factors_below_the_normal_numbers(max_norm, scale, n, shift, dst):
    """Gradients of a diverged step: max_norm / norm, or its product with scale, is subnormal, the
    clipped gradients are not.  (Those that are: half of TINY for each of two roundings.)"""
    H.device()
    g = torch.randn(n, generator=gen(1))
    g[::max(n // 4, 1)] *= 5e37
    src, out = Placed(1, n, F32, 0, shift, g[None]), Placed(1, n, dst, 0, 8)
    norm = torch.empty(1, device="cuda")
    want, clipped = S.clip([g], scale, max_norm)
    with dpr.dpr_grad_plan_create([src.view[0]], [out.view[0]]) as plan:
        for call in (dpr.dpr_grad_norm_clip, dpr.dpr_grad_clip):
            out.view.fill_(9)
            call(plan, norm, max_norm, scale=scale)
            assert abs(norm.item() - want) <= S.NORM_ERROR * want
            R.check(out.view[0], clipped[0], S.clip_bound(clipped[0], dst) + 2.0 ** -149, "out")
            out.check_guards("out")
    with dpr.dpr_grad_plan_create([src.view[0]]) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, max_norm, scale=scale)
        R.check(src.view[0], clipped[0], S.clip_bound(clipped[0], F32) + 2.0 ** -149, "in place")


@pytest.mark.parametrize("n", [100, 300000])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, 2.0 ** 100])
@pytest.mark.parametrize("scale", [2.0 ** -70, 1.0, 2.0 ** 100])
def test_an_infinite_norm_clips_to_zero_at_any_scale(scale, max_norm, n):
    H.device()
    g = torch.randn(n, generator=gen(1))
    g[3] = float("inf")
    norm, out = torch.empty(1, device="cuda"), torch.full((n,), 9.0, device="cuda")
    with dpr.dpr_grad_plan_create([g.cuda()], [out]) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, max_norm, scale=scale)
        assert norm.item() == float("inf") and bool(out[3].isnan())
        assert int((out == 0).sum()) == n - 1


@pytest.mark.parametrize("n", [1000, 50000])
def test_infinities_and_nan_show(n):
    H.device()
    g = torch.randn(n, generator=gen(1))
    norm, out = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
    g[n // 2] = float("inf")
    with dpr.dpr_grad_plan_create([g.cuda()], [out]) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, 1.0)
        assert norm.item() == float("inf") and bool(out[n // 2].isnan())
        assert int((out == 0).sum()) == n - 1
    g[0] = float("nan")
    t = g.cuda()
    with dpr.dpr_grad_plan_create([t]) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, float("inf"))
        assert bool(norm.isnan()) and bool(t.isnan().all())
    zeros = torch.zeros(n, device="cuda")
    with dpr.dpr_grad_plan_create([zeros], [out]) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, 0.0)
        assert norm.item() == 0 and not out.any()


def test_empty_lists():
    H.device()
    norm = torch.full((1,), 5.0, device="cuda")
    for grads in ([], [torch.empty(0, device="cuda")]):
        with dpr.dpr_grad_plan_create(grads) as plan:
            dpr.dpr_grad_clip(plan, norm, 1.0)
            assert norm.item() == 5
            dpr.dpr_grad_norm_clip(plan, norm, 1.0)
            assert norm.item() == 0
            norm.fill_(5)


def test_more_than_32_bits_of_elements():
    H.device()
    g = torch.zeros((1 << 32) + 4096, dtype=BF, device="cuda")
    g[-5:] = 3.0
    norm = torch.empty(1, device="cuda")
    with dpr.dpr_grad_plan_create([g]) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, 1.0)
    want = 45.0 ** 0.5
    assert abs(norm.item() - want) <= S.NORM_ERROR * want
    R.check(g[-5:], torch.full((5,), 3 / want, dtype=torch.float64),
            S.clip_bound(torch.full((5,), 3 / want), BF), "last elements")
    assert not g[:-5].any()


def test_a_list_of_more_elements_than_one_tensor_may_have():
    H.device()
    gs = [torch.zeros((1 << 33) + 16, dtype=BF, device="cuda") for _ in range(2)]
    for g in gs:
        g[-5:] = 3.0
    norm = torch.empty(1, device="cuda")
    with dpr.dpr_grad_plan_create(gs) as plan:
        dpr.dpr_grad_norm_clip(plan, norm, 1.0)
    want = 90.0 ** 0.5
    assert abs(norm.item() - want) <= S.NORM_ERROR * want
    one = torch.full((5,), 3 / want, dtype=torch.float64)
    for g in gs:
        R.check(g[-5:], one, S.clip_bound(one, BF), "last elements")
        assert not g[:64].any() and not g[-69:-5].any()


def test_refusals():
    H.device()
    g, norm = torch.ones(100000, device="cuda"), torch.empty(1, device="cuda")
    out = torch.empty(100000, device="cuda")
    plan = dpr.dpr_grad_plan_create([g], [out])
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(dpr.DprError):
            dpr.dpr_grad_norm(plan, norm, scale=bad)
    for bad in (-1.0, float("nan")):
        with pytest.raises(dpr.DprError):
            dpr.dpr_grad_norm_clip(plan, norm, bad)
        with pytest.raises(dpr.DprError):
            dpr.dpr_grad_clip(plan, norm, bad)
    for bad in (g[5:6], out[7:8]):
        with pytest.raises(dpr.DprError):
            dpr.dpr_grad_norm(plan, bad)
    with pytest.raises(dpr.DprError):
        dpr.dpr_grad_clip(plan, out[7:8], 1.0)
    # a list of more tiles than one launch takes needs a workspace
    large, result = torch.ones(1 << 20, device="cuda"), torch.empty(1 << 20, device="cuda")
    needs = dpr.dpr_grad_plan_create([large], [result])
    assert plan.workspace_bytes == 0 and 0 < needs.workspace_bytes <= 1 << 16
    for bad in (large, result):
        with pytest.raises(dpr.DprError):
            dpr.dpr_grad_norm(needs, norm, workspace=bad)
    with pytest.raises(ValueError):
        dpr.dpr_grad_norm(needs, norm, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    for bad in (norm.double(), torch.empty(2, device="cuda"), torch.empty(1)):
        with pytest.raises(ValueError):
            dpr.dpr_grad_norm(plan, bad)
    for bad in ([g[::2]], [g.half()], [torch.ones(4)]):
        with pytest.raises(ValueError):
            dpr.dpr_grad_plan_create(bad)
    for bad in ([out[:5]], [out, out]):
        with pytest.raises(ValueError):
            dpr.dpr_grad_plan_create([g], bad)
    for grads, outs in (([g, g], None), ([g], [g[1:].new_empty(0)]), ([g[:50], g[50:100]], [out[:50], out[49:99]]),
                        ([g[:50], g[50:100]], [g[50:100], out[:50]])):
        with pytest.raises((dpr.DprError, ValueError)):
            dpr.dpr_grad_plan_create(grads, outs)


def test_norm_on_another_device_than_the_plan():
    H.device()
    plan = dpr.dpr_grad_plan_create([torch.ones(8, device="cuda")])
    norm = torch.empty(1, device="cuda")
    plan.device += 1                 # as of a plan made there
    for call in (lambda: dpr.dpr_grad_norm(plan, norm), lambda: dpr.dpr_grad_clip(plan, norm, 1.0),
                 lambda: dpr.dpr_grad_norm_clip(plan, norm, 1.0)):
        with pytest.raises(ValueError, match="cuda"):
            call()
