"""C ABI of the backward-pass operators, without a GPU: every declared function
is exported, the header is plain C, bad arguments are refused on the host
before anything reaches CUDA (fake device addresses, never dereferenced), the
binding refuses tensors that are not on the GPU, and the reference's 8-bit
format agrees with hand-worked blocks."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from tests import operators_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dpr_ops.h")
OK, INVALID, ALIGN, UNSUP, CUDA, ALIAS = range(6)
BF16, FP32 = 0, 1
BASE = 0x7F0000000000
GB = 1 << 30


class Ckpt(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("code_stride", ctypes.c_int64),
                ("steps", ctypes.c_void_p), ("step_stride", ctypes.c_int64)]


@pytest.fixture(scope="module")
def L():
    from gradient_reduction_gb300 import build
    build.build()
    import gradient_reduction_gb300 as g
    return g.lib()


def test_exports_every_declared_function(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dpr_[a-z0-9_]+)\s*\(", src)))
    assert len(names) == 8
    for n in names:
        assert hasattr(L, n), n


def test_header_is_plain_c(tmp_path):
    c = tmp_path / "t.c"
    c.write_text('#include "dpr_ops.h"\nint main(void){dpr_checkpoint c = {0}; return c.codes != 0;}\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), str(c)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


X, Y, W, B, MEAN, RSTD, DX, DW, DB, WS, CODES, STEPS = (BASE + i * 16 * GB for i in range(12))


def _ckpt(**kw):
    v = dict(codes=CODES, code_stride=64, steps=STEPS, step_stride=16)
    v.update(kw)
    return ctypes.byref(Ckpt(v["codes"], v["code_stride"], v["steps"], v["step_stride"]))


def _forward(L, **kw):
    v = dict(x=X, xs=64, rows=8, width=64, dtype=BF16, w=W, b=B, pd=BF16, eps=1e-5, y=Y, ys=64,
             mean=MEAN, rstd=RSTD, xc=None, yc=None)
    v.update(kw)
    return L.dpr_layernorm_forward(v["x"], v["xs"], v["rows"], v["width"], v["dtype"], v["w"],
                                   v["b"], v["pd"], v["eps"], v["y"], v["ys"], v["mean"], v["rstd"],
                                   v["xc"], v["yc"], None)


def test_forward_refusals(L):
    assert _forward(L, rows=-1) == INVALID
    assert _forward(L, width=0) == INVALID
    assert _forward(L, rows=1 << 31) == UNSUP
    assert _forward(L, width=1 << 21, xs=1 << 21, ys=1 << 21) == UNSUP
    assert _forward(L, xs=1 << 31) == UNSUP
    assert _forward(L, dtype=2) == INVALID
    assert _forward(L, pd=-1) == INVALID
    assert _forward(L, eps=-1.0) == INVALID
    assert _forward(L, eps=float("nan")) == INVALID
    assert _forward(L, x=None) == INVALID
    assert _forward(L, y=None) == INVALID
    assert _forward(L, xs=-1) == INVALID
    assert _forward(L, ys=63) == INVALID
    assert _forward(L, ys=0) == INVALID                       # rows written on top of each other
    assert _forward(L, x=X + 1) == ALIGN
    assert _forward(L, dtype=FP32, y=Y + 2) == ALIGN
    assert _forward(L, pd=FP32, w=W + 2) == ALIGN
    assert _forward(L, mean=MEAN + 2) == ALIGN
    assert _forward(L, y=X + 64) == ALIAS                     # half over x
    assert _forward(L, y=X, ys=128) == ALIAS                  # x with another stride
    assert _forward(L, mean=Y + 16) == ALIAS
    assert _forward(L, rstd=MEAN) == ALIAS
    assert _forward(L, w=Y) == ALIAS
    assert _forward(L, mean=X) == ALIAS
    assert _forward(L, xc=_ckpt(codes=None)) == INVALID
    assert _forward(L, xc=_ckpt(code_stride=63)) == INVALID
    assert _forward(L, yc=_ckpt(step_stride=1)) == INVALID
    assert _forward(L, yc=_ckpt(codes=Y)) == ALIAS
    assert _forward(L, xc=_ckpt(), yc=_ckpt()) == ALIAS       # one buffer for both
    assert _forward(L, xc=_ckpt(codes=X)) == ALIAS
    assert _forward(L, rows=0, x=None, y=None) == OK


def _backward(L, **kw):
    need = ctypes.c_int64()
    v = dict(dy=X, ds=64, x=Y, xs=64, xc=None, rows=8, width=64, dtype=BF16, w=W, pd=BF16,
             mean=MEAN, rstd=RSTD, dx=DX, dxs=64, dw=DW, db=DB, gd=FP32, acc=0, ws=WS, n=None)
    v.update(kw)
    if v["n"] is None:
        st = L.dpr_layernorm_backward_workspace(max(v["rows"], 0), max(v["width"], 1),
                                                ctypes.byref(need))
        v["n"] = need.value if st == OK else 0
    return L.dpr_layernorm_backward(v["dy"], v["ds"], v["x"], v["xs"], v["xc"], v["rows"],
                                    v["width"], v["dtype"], v["w"], v["pd"], v["mean"], v["rstd"],
                                    v["dx"], v["dxs"], v["dw"], v["db"], v["gd"], v["acc"], v["ws"],
                                    v["n"], None)


def test_backward_refusals(L):
    n = ctypes.c_int64(5)
    assert L.dpr_layernorm_backward_workspace(-1, 64, ctypes.byref(n)) == INVALID and n.value == 0
    assert L.dpr_layernorm_backward_workspace(8, 64, None) == INVALID
    assert _backward(L, rows=-1) == INVALID
    assert _backward(L, width=0) == INVALID
    assert _backward(L, width=1 << 21) == UNSUP
    assert _backward(L, dtype=3) == INVALID
    assert _backward(L, gd=3) == INVALID
    assert _backward(L, dy=None) == INVALID
    assert _backward(L, x=None) == INVALID                    # neither x nor a checkpoint
    assert _backward(L, mean=None) == INVALID
    assert _backward(L, rstd=None) == INVALID
    assert _backward(L, dx=None) == INVALID
    assert _backward(L, ws=None) == INVALID
    assert _backward(L, n=16) == INVALID
    assert _backward(L, dxs=32) == INVALID
    assert _backward(L, xc=_ckpt(step_stride=1)) == INVALID
    assert _backward(L, ws=WS + 8) == ALIGN
    assert _backward(L, dw=DW + 2) == ALIGN
    assert _backward(L, dy=X + 1) == ALIGN
    assert _backward(L, dx=X + 64) == ALIAS
    assert _backward(L, dx=Y, dxs=128) == ALIAS
    assert _backward(L, dw=DX) == ALIAS
    assert _backward(L, db=DW) == ALIAS
    assert _backward(L, dw=W) == ALIAS
    assert _backward(L, ws=X) == ALIAS
    assert _backward(L, db=MEAN) == ALIAS
    assert _backward(L, xc=_ckpt(codes=DX)) == ALIAS
    assert _backward(L, rows=0, dy=None, dx=None, x=None, ws=None, dw=None, db=None) == OK


def test_checkpoint_refusals(L):
    save = lambda x=X, s=64, r=8, w=64, d=BF16, c=None: L.dpr_checkpoint_save(
        x, s, r, w, d, c or _ckpt(), None)
    load = lambda c=None, r=8, w=64, o=Y, s=64, d=BF16: L.dpr_checkpoint_load(
        c or _ckpt(), r, w, o, s, d, None)
    assert save(r=-1) == INVALID and load(r=-1) == INVALID
    assert save(w=0) == INVALID and load(w=0) == INVALID
    assert save(d=7) == INVALID and load(d=7) == INVALID
    assert save(x=None) == INVALID and load(o=None) == INVALID
    assert L.dpr_checkpoint_save(X, 64, 8, 64, BF16, None, None) == INVALID
    assert load(s=63) == INVALID and load(s=0) == INVALID
    assert save(c=_ckpt(code_stride=32)) == INVALID
    assert save(c=_ckpt(steps=None)) == INVALID
    assert save(x=X + 1) == ALIGN and load(d=FP32, o=Y + 2) == ALIGN
    assert save(c=_ckpt(codes=X + 64)) == ALIAS
    assert save(c=_ckpt(steps=CODES + 8)) == ALIAS
    assert load(o=STEPS) == ALIAS
    assert save(r=1 << 30, w=1 << 20, s=1 << 20, c=_ckpt(code_stride=1 << 20, step_stride=1 << 15)) in (
        UNSUP, ALIAS)
    assert save(r=0) == OK and load(r=0) == OK


def test_weight_grad_refusals(L):
    n = ctypes.c_int64()

    def call(dy=X, ds=128, c=None, rows=64, o=128, i=64, dw=DW, dws=64, d=BF16, ws=WS, none=False):
        x = None if none else (c or _ckpt())
        st = L.dpr_linear_weight_grad_workspace(dy, ds, x, rows, o, i, ctypes.byref(n))
        if st != OK:
            return st
        return L.dpr_linear_weight_grad(dy, ds, x, rows, o, i, dw, dws, d, 0, ws, n.value, None)
    assert call(rows=-1) == INVALID
    assert call(o=0) == INVALID and call(i=0) == INVALID
    assert call(o=1 << 21) == UNSUP and call(rows=1 << 31) == UNSUP
    assert call(d=5) == INVALID
    assert call(dy=None) == INVALID and call(none=True) == INVALID and call(dw=None) == INVALID
    assert call(dws=63) == INVALID and call(ds=-128) == INVALID
    assert call(c=_ckpt(code_stride=63)) == INVALID
    assert call(dy=X + 1) == ALIGN and call(d=FP32, dw=DW + 2) == ALIGN
    assert call(dw=X) == ALIAS and call(dw=CODES) == ALIAS and call(dw=STEPS) == ALIAS
    assert call(rows=(1 << 22) + 1) == UNSUP
    assert L.dpr_linear_weight_grad_workspace(X, 64, _ckpt(), 1, 1, 1, None) == INVALID
    # aligned inputs whose tiles are summed whole need none; odd rows are copied
    assert L.dpr_linear_weight_grad_workspace(X, 64, _ckpt(), 64, 64, 64, ctypes.byref(n)) == OK
    assert n.value == 0
    assert L.dpr_linear_weight_grad_workspace(X, 65, _ckpt(), 64, 65, 64, ctypes.byref(n)) == OK
    assert n.value == 64 * 72 * 2
    assert call(dy=X, ds=129, ws=None) == INVALID and call(ds=129, ws=WS + 4) == ALIGN
    assert call(ds=129, ws=X) == ALIAS


def test_binding_refuses_what_is_not_on_the_gpu():
    import gradient_reduction_gb300 as dpr
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dpr.dpr_layernorm_forward(x, None, None, 1e-5, x)
    c = dpr.dpr_checkpoint_empty(4, 64, device="cpu")
    assert c.codes.stride(0) % 16 == 0 and c.steps.stride(0) % 16 == 0
    assert c.nbytes == 4 * (64 + 2)
    with pytest.raises(ValueError, match="CUDA"):
        dpr.dpr_checkpoint_save(x, c)
    with pytest.raises(ValueError, match="CUDA"):
        dpr.dpr_checkpoint_load(c, x)
    with pytest.raises(ValueError, match="CUDA"):
        dpr.dpr_linear_weight_grad(x.bfloat16(), c, x)


def test_format_by_hand():
    """Blocks whose steps follow from the definition without computing: a peak of 127 takes step 1,
    127.5 takes step 2, 64 keeps step 1/2 (64 / 0.5 = 128 would not fit: step 1), 63 takes 1/2."""
    for peak, step in ((127.0, 1.0), (127.5, 2.0), (127.25, 1.0), (64.0, 1.0), (63.0, 0.5),
                       (1.0, 2.0 ** -6), (255.0, 4.0), (254.0, 2.0)):
        x = torch.zeros(1, 32, dtype=torch.float64)
        x[0, 3] = -peak
        codes, steps = R.encode(x)
        assert 2.0 ** (int(steps[0, 0]) - 127) == step, peak
        assert abs(int(codes[0, 3])) * step == pytest.approx(peak, abs=step / 2)
    x = torch.tensor([[0.5, 1.5, 2.5, -0.5, -1.5, 100.0] + [0.0] * 26], dtype=torch.float64)
    codes, steps = R.encode(x)                     # step 1: ties to even
    assert int(steps[0, 0]) == 127 and codes[0, :6].tolist() == [0, 2, 2, 0, -2, 100]
    x[0, 7] = float("inf")
    codes, steps = R.encode(x)
    assert int(steps[0, 0]) == 255 and not codes.any()
    assert R.decode(codes, steps).isnan().all()


def test_no_kernel_takes_a_buffer_as_unchanging():
    """The kernels are programmatic launches: they are resident while the grid before them still
    writes what they will read, so no buffer may be read through the non-coherent path, which
    __restrict__ on a source, __ldg and ld.global.nc allow or ask for."""
    csrc = os.path.join(ROOT, "gradient_reduction_gb300", "csrc")
    for name in ("checkpoint.cu", "layernorm.cu", "layernorm_backward.cu", "ops_device.cuh",
                 "ops_host.cu", "tensor_core.cuh", "weight_grad.cu"):
        code = re.sub(r"//.*", "", open(os.path.join(csrc, name)).read())
        for word in ("__restrict__", "__ldg", "global.nc", "ld_nc_", "load_words<"):
            assert word not in code, f"{name}: {word}"


def test_chunk_bound_separates_one_accumulator_from_many():
    """The summation the weight gradient's precision rests on, in 64 bits on the CPU: 16 exact terms
    of one sign at a time into an accumulator that truncates to 24 bits.  Emptied every 1024 tokens
    it stays within half of weight_grad_chunk_bound; run over all of them every sum is out of it."""
    def truncate(v):
        m, e = torch.frexp(v)
        return torch.ldexp(torch.floor(m * 2 ** 24) * 2.0 ** -24, e)

    def total(terms, chunk):
        out = torch.zeros(terms.shape[1], dtype=torch.float32)
        for t0 in range(0, terms.shape[0], chunk):
            acc = torch.zeros(terms.shape[1], dtype=torch.float64)
            for t in range(t0, min(t0 + chunk, terms.shape[0]), 16):
                acc = truncate(acc + terms[t:t + 16].sum(0))
            out = (out.double() + acc).float()
        return out.double()

    g = torch.Generator().manual_seed(1)
    for rows in (8192, 16384):
        dy = (1e-2 * torch.randn(rows, 64, generator=g).abs()).bfloat16().double()
        codes, steps = R.encode(torch.randn(rows, 64, generator=g).abs().double())
        terms = dy * R.decode(codes, steps)
        want = terms.sum(0)
        bound = R.weight_grad_chunk_bound(rows, 1)
        error = {c: (total(terms, c) - want).abs() / want for c in (1024, 2048, 4096, rows)}
        assert bool((error[1024] <= bound / 2).all())
        assert bool((error[rows] > bound).all())
        assert float(error[1024].mean()) < float(error[2048].mean()) < float(error[4096].mean())
        # a term left out or taken twice
        assert bool(((terms.max(0).values / want) > bound).all())
