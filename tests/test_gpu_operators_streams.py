"""The operators on streams other than PyTorch's current one: where their scratch
memory belongs, and what the count of run-out waits waits for."""
import pytest
import torch

import gradient_reduction_gb300 as dpr
from gradient_reduction_gb300 import _operators
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu


def _owner(t: torch.Tensor) -> int:
    """The stream in whose order the allocator hands out this tensor's memory again."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("memory that is not the allocator's")


@pytest.mark.parametrize("which", ["default", "legacy", "side object", "side handle", "current"])
def test_scratch_memory_belongs_to_the_stream_of_the_call(which):
    """Memory freed at the call's end must not be handed out in another stream's order while the
    kernels still use it; 0 and 1 (cudaStreamLegacy) are handles of the default stream."""
    H.device()
    side = torch.cuda.Stream()
    stream, owner = {"default": (0, 0), "legacy": (1, 0), "side object": (side, side.cuda_stream),
                     "side handle": (side.cuda_stream, side.cuda_stream), "current": (None, 0)}[which]
    # more than the allocator keeps in its small blocks, and than is kept between calls
    nbytes = _operators._KEEP_BYTES + (1 << 20)
    t = _operators._workspace(None, nbytes, stream, 0, torch.cuda.current_device())
    assert _owner(t) == owner


@pytest.mark.parametrize("handle", [0, 1])
def test_calls_on_the_default_stream_by_its_handle(handle):
    H.device()
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(70, 97, generator=g).bfloat16().cuda() for _ in range(2))
    saved = dpr.dpr_checkpoint_empty(70, 97)

    def call(stream):
        mean, rstd = torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dw, db, lin = (torch.empty(*s, device="cuda") for s in ((97,), (97,), (97, 97)))
        torch.cuda.synchronize()
        dpr.dpr_layernorm_forward(x, None, None, 1e-5, y, mean, rstd, saved, stream=stream)
        dpr.dpr_layernorm_backward(dy, saved, None, mean, rstd, dx, dw, db, stream=stream)
        dpr.dpr_linear_weight_grad(dx, saved, lin, stream=stream)
        torch.cuda.synchronize()
        return y, dx, dw, db, lin

    for got, want in zip(call(handle), call(None)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("programmatic", [True, False])
def test_unaligned_inputs_rewritten_before_every_weight_gradient(programmatic):
    """dy, codes and steps of odd strides, which are first copied to aligned rows, rewritten by the
    call just before (dx and the checkpoints of a layer norm, other values each time) on a side
    stream without waits: every weight gradient is of the values it was called with."""
    H.device()
    rows, o, i, turns = 300, 100, 97, 8
    old = dpr.dpr_set_programmatic_launch(programmatic)
    try:
        g = torch.Generator().manual_seed(3)
        xs = [torch.randn(rows, i, generator=g).bfloat16().cuda() for _ in range(turns)]
        dys = [torch.randn(rows, o, generator=g).bfloat16().cuda() for _ in range(turns)]
        mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        codes = torch.zeros(rows, i + 2, dtype=torch.int8, device="cuda")
        steps = torch.zeros(rows, 4 + 3, dtype=torch.uint8, device="cuda")
        saved = dpr.Checkpoint(codes[:, :i], steps[:, :4])
        dx = torch.zeros(rows, o + 1, dtype=torch.bfloat16, device="cuda")[:, :o]

        def step(k, out, stream):
            dpr.dpr_checkpoint_save(xs[k], saved, stream=stream)
            dpr.dpr_layernorm_backward(dys[k], dys[k], None, mean, rstd, dx, stream=stream)
            dpr.dpr_linear_weight_grad(dx, saved, out, stream=stream)

        want = []
        for k in range(turns):
            out = torch.full((o, i), float("nan"), device="cuda")
            step(k, out, None)
            torch.cuda.synchronize()
            want.append(out)
        side = torch.cuda.Stream()
        got = [torch.full((o, i), float("nan"), device="cuda") for _ in range(turns)]
        torch.cuda.synchronize()
        for k in range(turns):
            step(k, got[k], side)
        torch.cuda.synchronize()
        for k in range(turns):
            assert torch.equal(got[k], want[k]), k
            assert k == 0 or not torch.equal(got[k], got[k - 1])
    finally:
        dpr.dpr_set_programmatic_launch(old)


def test_the_count_of_failed_waits_waits_for_side_streams():
    """The count is read after work on a non-blocking stream has ended, not beside it: some 60 ms of
    passes over 1 GiB."""
    H.device()
    big = torch.zeros(1 << 28, device="cuda")
    assert dpr.dpr_device_wait_failures() == 0       # the first call also loads the counters
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):
            big.add_(1)
    pending = not side.query()
    assert dpr.dpr_device_wait_failures() == 0
    assert pending and side.query()
