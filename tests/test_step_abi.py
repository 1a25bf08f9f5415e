"""C ABI of the training step's operators (include/dpr_step.h), without a GPU: every declared
function is exported, the header is plain C, bad arguments are refused on the host before anything
reaches CUDA (fake device addresses, never dereferenced), the binding refuses tensors that are not
on the GPU, and the kernels' sources take no buffer as unchanging."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from tests import step_cases as C
from tests import step_reference as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dpr_step.h")
OK, INVALID, ALIGN, UNSUP, CUDA, ALIAS = range(6)
BF16, FP32 = 0, 1
BASE, GB = 0x7F0000000000, 1 << 30
X, RES, H, Y, W, RSTD, DX, DW, WS, CODES, STEPS, OFFS = (BASE + i * 16 * GB for i in range(12))


class Ckpt(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("code_stride", ctypes.c_int64),
                ("steps", ctypes.c_void_p), ("step_stride", ctypes.c_int64)]


@pytest.fixture(scope="module")
def L():
    from gradient_reduction_gb300 import build
    build.build()
    import gradient_reduction_gb300 as g
    return g.lib()


def _ckpt(**kw):
    v = dict(codes=CODES, code_stride=64, steps=STEPS, step_stride=16)
    v.update(kw)
    return ctypes.byref(Ckpt(v["codes"], v["code_stride"], v["steps"], v["step_stride"]))


def test_exports_every_declared_function(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dpr_[a-z0-9_]+)\s*\(", src)))
    assert len(names) == 15
    import gradient_reduction_gb300 as dpr
    for n in names:
        assert hasattr(L, n), n
        assert n.endswith("_workspace") or hasattr(dpr, n), n


def test_header_is_plain_c(tmp_path):
    c = tmp_path / "t.c"
    c.write_text('#include "dpr_step.h"\nint main(void){dpr_grad_plan* p = 0; return p != 0;}\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), str(c)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_rms_forward_refusals(L):
    def call(**kw):
        v = dict(x=X, xs=64, r=RES, rs=64, rows=8, width=64, d=BF16, w=W, pd=BF16, eps=1e-6, h=H,
                 hs=64, y=Y, ys=64, rstd=RSTD, hc=None, yc=None)
        v.update(kw)
        return L.dpr_rmsnorm_forward(v["x"], v["xs"], v["r"], v["rs"], v["rows"], v["width"], v["d"],
                                     v["w"], v["pd"], v["eps"], v["h"], v["hs"], v["y"], v["ys"],
                                     v["rstd"], v["hc"], v["yc"], None)
    assert call(rows=-1) == INVALID and call(width=0) == INVALID
    assert call(rows=1 << 31) == UNSUP and call(width=1 << 21) == UNSUP
    assert call(xs=1 << 31) == UNSUP and call(rs=1 << 31) == UNSUP
    assert call(d=2) == INVALID and call(pd=-1) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(x=None) == INVALID
    assert call(y=None) == INVALID                              # nothing to give
    assert call(r=None) == INVALID                              # h without a sum
    assert call(xs=-1) == INVALID and call(rs=-1) == INVALID
    assert call(hs=63) == INVALID and call(ys=0) == INVALID
    assert call(x=X + 1) == ALIGN and call(r=RES + 1) == ALIGN and call(h=H + 1) == ALIGN
    assert call(d=FP32, y=Y + 2) == ALIGN and call(pd=FP32, w=W + 2) == ALIGN
    assert call(rstd=RSTD + 2) == ALIGN
    assert call(h=X + 64) == ALIAS and call(h=X, hs=128) == ALIAS
    assert call(y=RES + 64) == ALIAS and call(y=RES, ys=128) == ALIAS
    assert call(y=H) == ALIAS and call(h=X, y=X) == ALIAS
    assert call(rstd=Y + 16) == ALIAS and call(rstd=X) == ALIAS and call(rstd=RES + 4) == ALIAS
    assert call(w=Y) == ALIAS and call(w=H + 64) == ALIAS
    assert call(hc=_ckpt(codes=None)) == INVALID and call(hc=_ckpt(code_stride=63)) == INVALID
    assert call(yc=_ckpt(step_stride=1)) == INVALID
    assert call(yc=_ckpt(codes=H)) == ALIAS and call(hc=_ckpt(), yc=_ckpt()) == ALIAS
    assert call(rows=0, x=None, r=RES) == OK


def test_rms_backward_refusals(L):
    def call(**kw):
        need = ctypes.c_int64()
        v = dict(dy=X, ds=64, dh=RES, dhs=64, h=H, hs=64, hc=None, rows=8, width=64, d=BF16, w=W,
                 pd=BF16, rstd=RSTD, dx=DX, dxs=64, dw=DW, gd=FP32, acc=0, ws=WS, n=None)
        v.update(kw)
        if v["n"] is None:
            st = L.dpr_rmsnorm_backward_workspace(max(v["rows"], 0), max(v["width"], 1),
                                                  ctypes.byref(need))
            v["n"] = need.value if st == OK else 0
        return L.dpr_rmsnorm_backward(v["dy"], v["ds"], v["dh"], v["dhs"], v["h"], v["hs"], v["hc"],
                                      v["rows"], v["width"], v["d"], v["w"], v["pd"], v["rstd"],
                                      v["dx"], v["dxs"], v["dw"], v["gd"], v["acc"], v["ws"], v["n"],
                                      None)
    n = ctypes.c_int64(5)
    assert L.dpr_rmsnorm_backward_workspace(-1, 64, ctypes.byref(n)) == INVALID and n.value == 0
    assert L.dpr_rmsnorm_backward_workspace(8, 64, None) == INVALID
    assert call(rows=-1) == INVALID and call(width=0) == INVALID and call(width=1 << 21) == UNSUP
    assert call(d=3) == INVALID and call(gd=3) == INVALID and call(pd=3) == INVALID
    for missing in ("dy", "h", "rstd", "dx", "ws"):
        assert call(**{missing: None}) == INVALID, missing
    assert call(n=16) == INVALID and call(dxs=32) == INVALID
    assert call(hc=_ckpt(step_stride=1)) == INVALID
    assert call(ws=WS + 8) == ALIGN and call(dw=DW + 2) == ALIGN and call(dy=X + 1) == ALIGN
    assert call(dh=RES + 1) == ALIGN
    assert call(dx=X + 64) == ALIAS and call(dx=H, dxs=128) == ALIAS and call(dx=RES + 2) == ALIAS
    assert call(dw=DX) == ALIAS and call(dw=W) == ALIAS and call(ws=X) == ALIAS
    assert call(ws=RES) == ALIAS and call(dw=RSTD) == ALIAS
    assert call(hc=_ckpt(codes=DX)) == ALIAS
    assert call(rows=0, dy=None, dx=None, h=None, ws=None, dw=None, dh=None) == OK


def _product(L, name, **kw):
    n = ctypes.c_int64()
    v = dict(x=X, xs=128, rows=64, offs=OFFS, e=4, w=W, ws=128, es=128 * 128, o=128, i=128, y=Y,
             ys=128, d=BF16, work=WS, n=None)
    v.update(kw)
    st = getattr(L, name + "_workspace")(v["x"], v["xs"], v["rows"], v["e"], v["w"], v["ws"], v["es"],
                                         v["o"], v["i"], ctypes.byref(n))
    if st != OK:
        return st
    return getattr(L, name)(v["x"], v["xs"], v["rows"], v["offs"], v["e"], v["w"], v["ws"], v["es"],
                            v["o"], v["i"], v["y"], v["ys"], v["d"], v["work"],
                            n.value if v["n"] is None else v["n"], None)


@pytest.mark.parametrize("name", ["dpr_grouped_linear", "dpr_grouped_linear_input_grad"])
def test_product_refusals(L, name):
    def call(**kw):
        return _product(L, name, **kw)
    assert call(rows=-1) == INVALID and call(o=0) == INVALID and call(i=0) == INVALID
    assert call(e=0) == INVALID and call(e=1025) == UNSUP
    assert call(o=1 << 21) == UNSUP and call(rows=(1 << 22) + 1) == UNSUP
    assert call(e=1024, o=1 << 20, i=1 << 20) == UNSUP           # tiles beyond 31 bits
    assert call(d=5) == INVALID
    for missing in ("x", "offs", "w", "y"):
        assert call(**{missing: None}) == INVALID, missing
    assert call(ys=127) == INVALID and call(xs=-128) == INVALID and call(es=-1) == INVALID
    assert call(ws=1 << 31) == UNSUP and call(es=1 << 40) == UNSUP
    assert call(x=X + 1) == ALIGN and call(d=FP32, y=Y + 2) == ALIGN and call(offs=OFFS + 2) == ALIGN
    assert call(y=X) == ALIAS and call(y=W + 64) == ALIAS and call(y=OFFS) == ALIAS
    # aligned operands need no memory, others are copied
    n = ctypes.c_int64()
    size = getattr(L, name + "_workspace")
    assert size(X, 128, 64, 4, W, 128, 128 * 128, 128, 128, ctypes.byref(n)) == OK and n.value == 0
    assert size(X, 128, 64, 4, W, 128, 128 * 128, 128, 128, None) == INVALID
    assert size(X + 2, 128, 64, 4, W, 128, 128 * 128, 128, 128, ctypes.byref(n)) == OK
    assert n.value == 64 * 128 * 2
    assert size(X, 128, 64, 4, W, 129, 129 * 129, 128, 128, ctypes.byref(n)) == OK
    assert n.value == 4 * 128 * 128 * 2
    # but not weights that few tokens read, whose rows follow one another through all experts
    assert size(X, 128, 64, 4, W, 129, 128 * 129, 128, 128, ctypes.byref(n)) == OK and n.value == 0
    assert size(X, 128, 64, 4, W + 2, 128, 128 * 128, 128, 128, ctypes.byref(n)) == OK and n.value == 0
    assert size(X, 128, 1 << 16, 4, W, 129, 128 * 129, 128, 128, ctypes.byref(n)) == OK
    assert n.value == 4 * 128 * 128 * 2
    assert call(xs=129, work=None) == INVALID and call(xs=129, n=16) == INVALID
    assert call(xs=129, work=WS + 4) == ALIGN and call(xs=129, work=X) == ALIAS
    assert call(rows=0, x=None, y=None, w=None, offs=None) == OK


def test_weight_gradient_refusals(L):
    n = ctypes.c_int64()

    def call(**kw):
        v = dict(dy=X, ds=128, x=H, xs=64, c=None, rows=64, offs=OFFS, e=4, o=128, i=64, dw=DW,
                 dws=64, es=64 * 128, d=BF16, acc=0, ws=WS)
        v.update(kw)
        st = L.dpr_grouped_linear_weight_grad_workspace(v["dy"], v["ds"], v["x"], v["xs"], v["c"],
                                                        v["rows"], v["e"], v["o"], v["i"],
                                                        ctypes.byref(n))
        if st != OK:
            return st
        return L.dpr_grouped_linear_weight_grad(v["dy"], v["ds"], v["x"], v["xs"], v["c"], v["rows"],
                                                v["offs"], v["e"], v["o"], v["i"], v["dw"], v["dws"],
                                                v["es"], v["d"], v["acc"], v["ws"], n.value, None)
    assert call(rows=-1) == INVALID and call(o=0) == INVALID and call(i=0) == INVALID
    assert call(e=0) == INVALID and call(e=1025) == UNSUP and call(rows=(1 << 22) + 1) == UNSUP
    assert call(d=5) == INVALID
    for missing in ("dy", "x", "offs", "dw"):
        assert call(**{missing: None}) == INVALID, missing
    assert call(dws=63) == INVALID and call(es=64 * 127) == INVALID     # matrices on top of each other
    assert call(c=_ckpt(code_stride=63)) == INVALID and call(c=_ckpt(steps=None)) == INVALID
    assert call(dy=X + 1) == ALIGN and call(d=FP32, dw=DW + 2) == ALIGN and call(offs=OFFS + 1) == ALIGN
    assert call(dw=X) == ALIAS and call(dw=H) == ALIAS and call(c=_ckpt(codes=DW)) == ALIAS
    assert call(offs=DW + 4) == ALIAS
    assert call(ds=129, ws=None) == INVALID and call(ds=129, ws=X) == ALIAS
    assert call(rows=0, dy=None, x=None, ws=None, acc=1) == OK
    assert L.dpr_grouped_linear_weight_grad_workspace(X, 128, H, 64, None, 64, 4, 128, 64, None) == INVALID


@pytest.mark.parametrize("name", ["dpr_grouped_linear", "dpr_grouped_linear_input_grad"])
def test_which_products_are_dealt_out(L, name):
    """Aligned operands, and unaligned weights that few tokens read, need memory for parts alone."""
    for cases, parts in ((C.PRODUCTS_IN_PARTS, True), (C.ODD_PRODUCTS_IN_PARTS, True), (C.PRODUCTS_WHOLE, False)):
        for counts, along, to in cases:
            o, i = (along, to) if name.endswith("input_grad") else (to, along)
            stride = i if parts else -(-i // 8) * 8
            n = ctypes.c_int64()
            assert getattr(L, name + "_workspace")(X, -(-along // 8) * 8, sum(counts), len(counts), W, stride, o * stride,
                                                   o, i, ctypes.byref(n)) == OK
            assert (n.value > 0) == parts, (counts, o, i)


@pytest.mark.parametrize("saved", [False, True], ids=["stored", "saved"])
def test_which_weight_gradients_are_dealt_out(L, saved):
    for cases, parts in ((C.GRADS_IN_PARTS, True), (C.GRADS_WHOLE, False)):
        for counts, o, i in cases:
            n = ctypes.c_int64()
            aligned = [-(-v // 16) * 16 for v in (o, i)]
            c = _ckpt(code_stride=aligned[1], step_stride=-(-i // 512) * 16) if saved else None
            assert L.dpr_grouped_linear_weight_grad_workspace(X, aligned[0], H, aligned[1], c, sum(counts), len(counts),
                                                              o, i, ctypes.byref(n)) == OK
            assert (n.value > 0) == parts, (counts, o, i)


def _plan(L, tensors, outs=None):
    """Status of a plan of (address, type, elements) tensors; never CUDA's part of it."""
    n = len(tensors)
    arr = lambda v, t: (t * max(len(v), 1))(*v)
    p = ctypes.c_void_p()
    src = arr([t[0] for t in tensors], ctypes.c_void_p)
    dt = arr([t[1] for t in tensors], ctypes.c_int)
    num = arr([t[2] for t in tensors], ctypes.c_int64)
    dst = od = None
    if outs is not None:
        dst = arr([t[0] for t in outs], ctypes.c_void_p)
        od = arr([t[1] for t in outs], ctypes.c_int)
    st = L.dpr_grad_plan_create(ctypes.byref(p), n, src, dt, dst, od, num, None)
    assert p.value is None
    return st


def test_plan_refusals(L):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses would make a plan where there is a device")
    assert L.dpr_grad_plan_create(None, 0, None, None, None, None, None, None) == INVALID
    p = ctypes.c_void_p()
    assert L.dpr_grad_plan_create(ctypes.byref(p), -1, None, None, None, None, None, None) == INVALID
    assert L.dpr_grad_plan_create(ctypes.byref(p), 1, None, None, None, None, None, None) == INVALID
    assert L.dpr_grad_plan_create(ctypes.byref(p), (1 << 20) + 1, None, None, None, None, None,
                                  None) == INVALID
    assert _plan(L, [(X, 2, 8)]) == INVALID and _plan(L, [(X, BF16, -1)]) == INVALID
    assert _plan(L, [(None, BF16, 8)]) == INVALID
    assert _plan(L, [(X, BF16, (1 << 34) + 1)]) == UNSUP
    assert _plan(L, [(X + 1, BF16, 8)]) == ALIGN and _plan(L, [(X + 2, FP32, 8)]) == ALIGN
    assert _plan(L, [(X, BF16, 8)], [(Y + 2, FP32)]) == ALIGN
    assert _plan(L, [(X, BF16, 8), (X + 14, BF16, 8)]) == ALIAS              # in place, overlapping
    assert _plan(L, [(X, BF16, 8), (X + 64, BF16, 8)], [(Y, FP32), (Y + 16, FP32)]) == ALIAS
    assert _plan(L, [(X, BF16, 8)], [(X, FP32)]) == ALIAS                    # in place, another type
    assert _plan(L, [(X, BF16, 8), (Y, BF16, 8)], [(Y, BF16), (H, BF16)]) == ALIAS
    # what is left is CUDA's: one input twice, in place beside others, empty tensors anywhere
    assert _plan(L, [(X, BF16, 8), (X, BF16, 8)], [(Y, FP32), (H, FP32)]) == CUDA
    assert _plan(L, [(X, BF16, 8), (None, BF16, 0)]) == CUDA
    assert L.dpr_grad_plan_destroy(None) == OK
    n = ctypes.c_int64()
    assert L.dpr_grad_norm_workspace(None, ctypes.byref(n)) == INVALID
    assert L.dpr_grad_norm(None, 1.0, Y, WS, 1 << 20, None) == INVALID
    assert L.dpr_grad_clip(None, 1.0, 1.0, Y, None) == INVALID
    assert L.dpr_grad_norm_clip(None, 1.0, 1.0, Y, WS, 1 << 20, None) == INVALID


def test_plan_of_a_long_list(L):
    """Lists of more elements than one tensor may have, up to 2^38."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses would make a plan where there is a device")
    apart = [BASE + i * 64 * GB for i in range(17)]
    assert _plan(L, [(p, FP32, (1 << 33) + 8) for p in apart[:2]]) == CUDA
    assert _plan(L, [(p, BF16, 1 << 34) for p in apart]) == UNSUP


def test_binding_refuses_what_is_not_on_the_gpu():
    import gradient_reduction_gb300 as dpr
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    offs = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: dpr.dpr_rmsnorm_forward(x, None, 1e-6, x),
                 lambda: dpr.dpr_rmsnorm_backward(x, x, None, torch.zeros(4), x),
                 lambda: dpr.dpr_grouped_linear(x, offs, w, x),
                 lambda: dpr.dpr_grouped_linear_input_grad(x, offs, w, x),
                 lambda: dpr.dpr_grouped_linear_weight_grad(x, offs, x, w),
                 lambda: dpr.dpr_grad_plan_create([x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_names_a_tensor_that_is_missing():
    from gradient_reduction_gb300 import _step
    plan = _step.GradPlan(1, 0, 0, ())
    try:
        for call, what in ((lambda: _step._offsets(None, 2, 0), "offsets"), (lambda: _step._experts(None, "dweight", 0), "dweight"),
                           (lambda: _step._norm(plan, None), "norm")):
            with pytest.raises(ValueError, match=f"{what}: a tensor is needed"):
                call()
    finally:
        plan.handle = None               # made up


def test_no_kernel_takes_a_buffer_as_unchanging():
    """Programmatic launches are resident while the grid before them still writes what they will
    read: nothing may go through the non-coherent path."""
    csrc = os.path.join(ROOT, "gradient_reduction_gb300", "csrc")
    for name in ("rmsnorm.cu", "rmsnorm_backward.cu", "grouped.cu", "grad_clip.cu"):
        code = re.sub(r"//.*", "", open(os.path.join(csrc, name)).read())
        for word in ("__restrict__", "__ldg", "global.nc", "ld_nc_", "load_words<"):
            assert word not in code, f"{name}: {word}"


def test_reference_by_hand():
    """Definitions against numbers worked out by hand."""
    h = torch.tensor([[3.0, 4.0, 0.0, 0.0]])                    # mean square 25 / 4
    y, rstd = S.rms_forward(h, torch.ones(4), 0.0)
    assert rstd.item() == pytest.approx(0.4) and y[0, :2].tolist() == pytest.approx([1.2, 1.6])
    # a gradient along h is removed: y does not change with h's length
    dx, dw = S.rms_backward(h, h, torch.ones(4), rstd)
    assert dx.abs().max() < 1e-15 and dw.tolist() == pytest.approx([3.6, 6.4, 0, 0])
    assert S.spans([-5, 3, 2, 100], 10) == [(0, 3), (3, 3), (3, 10)]
    x = torch.eye(2)
    w = torch.tensor([[[1.0, 2.0], [3.0, 4.0]], [[5.0, 6.0], [7.0, 8.0]]])
    out, _ = S.product(x, [0, 1, 2], w, False)
    assert out.tolist() == [[1, 3], [6, 8]]                     # a column of each weight
    out, _ = S.product(x, [0, 1, 2], w, True)
    assert out.tolist() == [[1, 2], [7, 8]]
    dw, _ = S.weight_grads(x, [0, 1, 2], torch.tensor([[1.0, 2.0], [3.0, 4.0]]))
    assert dw.tolist() == [[[1, 2], [0, 0]], [[0, 0], [3, 4]]]
    norm, out = S.clip([torch.tensor([3.0]), torch.tensor([4.0])], 2.0, 5.0)
    assert norm == 10 and [t.item() for t in out] == [3.0, 4.0]
