"""Layouts of the backward pass with two CTAs to a row: every matrix with a row stride and a start
of its own."""
import pytest
import torch

import gradient_reduction_gb300 as dpr
from tests import gpu_helpers as H
from tests import operators_reference as R
from tests.test_gpu_operators import BF, EPS, F32, Placed, activation, gen

pytestmark = pytest.mark.gpu

# elements between rows and before the first: x, dy, dx, codes, steps
LAYOUTS = {
    "32-byte rows": ((32, 0), (16, 16), (48, 32), (16, 0), (16, 0)),
    "16-byte rows": ((8, 8), (24, 0), (40, 8), (48, 16), (5, 3)),
    "8-byte codes": ((8, 8), (24, 0), (40, 8), (8, 8), (1, 1)),
    "odd rows": ((3, 0), (1, 0), (5, 0), (7, 0), (0, 1)),
    "odd starts": ((0, 1), (0, 3), (0, 5), (0, 1), (2, 7)),
}


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,width", [(2048, 4608), (2050, 4104), (200, 11008), (157, 12288),
                                        (90, 16376)])
def test_rows_of_two_blocks_at_any_stride(rows, width, dtype, layout):
    H.device()
    strides = LAYOUTS[layout]
    x = activation(rows, width, rows + width, dtype)
    dy = (1e-2 * torch.randn(rows, width, generator=gen(11))).to(dtype)
    w = (1 + 0.2 * torch.randn(width, generator=gen(12))).to(dtype)
    _, mean, rstd = R.norm_forward(x, w, w, EPS)
    mean, rstd = mean.float(), rstd.float()
    c, s = R.encode(x.double())
    px, pd = (Placed(rows, width, dtype, *at, fill=t) for at, t in zip(strides, (x, dy)))
    pc = Placed(rows, width, torch.int8, strides[3][0] + -width % 16, strides[3][1], fill=c)
    blocks = s.shape[1]
    ps = Placed(rows, blocks, torch.uint8, strides[4][0], strides[4][1], fill=s)
    for source, xx in ((px.view, x.double()), (dpr.Checkpoint(pc.view, ps.view), R.decode(c, s))):
        po = Placed(rows, width, dtype, *strides[2])
        pw, pb = Placed(1, width, F32), Placed(1, width, F32)
        dpr.dpr_layernorm_backward(pd.view, source, w.cuda(), mean.cuda(), rstd.cuda(), po.view,
                                   pw.view[0], pb.view[0])
        want = R.norm_backward(dy, xx, w, mean, rstd)
        bound = R.norm_backward_bounds(dy, xx, w, mean, rstd, dtype, F32)
        for got, v, b, what in zip((po.view, pw.view[0], pb.view[0]), want, bound,
                                   ("dx", "dweight", "dbias")):
            R.check(got, v, b, what)
        for p, what in ((px, "x"), (pd, "dy"), (po, "dx"), (pw, "dweight"), (pb, "dbias"),
                        (pc, "codes"), (ps, "steps")):
            p.check_guards(what)
