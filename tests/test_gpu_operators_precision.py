"""The weight gradient's summation error, by bounds that follow how it sums: an
accumulator of the tensor core, which truncates, takes at most 1024 tokens; those
are added rounded (tests/operators_reference.py, weight_grad_chunk_bound)."""
import pytest
import torch

import gradient_reduction_gb300 as dpr
from tests import gpu_helpers as H
from tests import operators_reference as R

pytestmark = pytest.mark.gpu


def _sum(dy, saved, dweight):
    """(|gradient - exact|, exact, sum of magnitudes) in 64 bits."""
    step = torch.exp2(saved.steps.double() - 127).repeat_interleave(32, 1)[:, :saved.codes.shape[1]]
    x = saved.codes.double() * step
    want = dy.double().t() @ x
    return (dweight.double() - want).abs(), want, dy.double().abs().t() @ x.abs()


@pytest.mark.parametrize("rows", [8192, 16384])
def test_sums_of_one_sign(rows):
    """Truncation is a bias here: every addition loses.  76 tiles, one for each pair of CTAs, so no
    tile's tokens are dealt out and every sum runs over all of them.  tests/test_operators_abi.py
    shows that an accumulator over all tokens is out of this bound."""
    H.device()
    g = torch.Generator(device="cuda").manual_seed(rows)
    o, i = 1000, 4864
    dy = (1e-2 * torch.randn(rows, o, generator=g, device="cuda").abs()).bfloat16()
    x = torch.randn(rows, i, generator=g, device="cuda").abs()
    saved = dpr.dpr_checkpoint_empty(rows, i)
    dpr.dpr_checkpoint_save(x, saved)
    dw = torch.empty(o, i, device="cuda")
    dpr.dpr_linear_weight_grad(dy, saved, dw)
    err, want, magnitudes = _sum(dy, saved, dw)
    assert torch.equal(want, magnitudes)
    worst = float((err / want).max())
    assert worst <= R.weight_grad_chunk_bound(rows, 1), worst


@pytest.mark.parametrize("rows,o,i", [(4096, 256, 384), (16384, 64, 64), (2048, 1024, 1152),
                                      (1100, 2310, 2305), (333, 257, 511)])
def test_sums_of_both_signs(rows, o, i):
    """Bounds tight enough that a token left out or taken twice shows: it is 1 / rows of the
    magnitudes, 6e-5 of them at 16384 tokens, against some 1e-5."""
    H.device()
    g = torch.Generator(device="cuda").manual_seed(rows + o)
    dy = (1e-2 * torch.randn(rows, o, generator=g, device="cuda")).bfloat16()
    x = torch.randn(rows, i, generator=g, device="cuda")
    saved = dpr.dpr_checkpoint_empty(rows, i)
    dpr.dpr_checkpoint_save(x, saved)
    dw = torch.empty(o, i, device="cuda")
    dpr.dpr_linear_weight_grad(dy, saved, dw)
    err, _, magnitudes = _sum(dy, saved, dw)
    worst = float((err / magnitudes).max())
    assert worst <= R.weight_grad_chunk_bound(rows, 76), worst
