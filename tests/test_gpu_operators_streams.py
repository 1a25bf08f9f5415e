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


# --- chains of calls whose buffers hold something else before every call -----

EPS = 1e-5


def _buffers(rows, width):
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")
    return (e(rows, width), e(rows, dtype=torch.float32), e(rows, dtype=torch.float32),
            dpr.dpr_checkpoint_empty(rows, width), dpr.dpr_checkpoint_empty(rows, width),
            e(rows, width), e(width), e(width), e(width, width))


def _flat(buffers):
    out = []
    for t in buffers:
        out += [t.codes, t.steps] if isinstance(t, dpr.Checkpoint) else [t]
    return out


def _poison(buffers):
    """0x5A in every byte: 1.5e16 as bf16 and fp32, 90 as a code, a step of 2^-37."""
    for t in _flat(buffers):
        if t.is_contiguous():
            t.view(torch.uint8).fill_(0x5A)
        else:
            t.fill_(0x5A)


def _chain(stream, inputs, buffers):
    x, dy, w, b = inputs
    y, mean, rstd, xs, ys, dx, dw, db, lin = buffers
    dpr.dpr_layernorm_forward(x, w, b, EPS, y, mean, rstd, xs, ys, stream=stream)
    dpr.dpr_layernorm_backward(dy, xs, w, mean, rstd, dx, dw, db, stream=stream)
    dpr.dpr_linear_weight_grad(dx, ys, lin, stream=stream)


def _inputs(rows, width, seed):
    g = torch.Generator().manual_seed(seed)
    t = [torch.randn(rows, width, generator=g) for _ in range(2)]
    t += [torch.randn(width, generator=g) for _ in range(2)]
    return [a.bfloat16().cuda() for a in t]


def _same(got, want, what):
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), f"{what}: tensor {i}"


# staged, single-element, two CTAs a row, three reads a row and two passes
@pytest.mark.parametrize("rows,width", [(300, 1056), (77, 100), (64, 97), (20, 8208), (2, 24592)])
@pytest.mark.parametrize("programmatic", [True, False])
@pytest.mark.parametrize("handle", ["object", "number"])
def test_chains_over_spoilt_buffers(rows, width, programmatic, handle):
    """Each repeat starts from buffers that hold neither its results nor an earlier repeat's, and
    takes other inputs than the one before; nothing waits between the calls.  A call that ran on
    another stream, not at all, or before the one it reads from had written would show."""
    H.device()
    old = dpr.dpr_set_programmatic_launch(programmatic)
    try:
        inputs = [_inputs(rows, width, 50 + k) for k in range(2)]
        buffers = _buffers(rows, width)
        want = []
        for k in range(2):
            _poison(buffers)
            torch.cuda.synchronize()
            _chain(None, inputs[k], buffers)
            torch.cuda.synchronize()
            want.append([t.clone() for t in _flat(buffers)])
        for a, b in zip(*want):
            assert not torch.equal(a, b)
        side = torch.cuda.Stream()
        results = []
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for k in range(6):
                _poison(buffers)
                _chain(side if handle == "object" else side.cuda_stream, inputs[k & 1], buffers)
                results.append([t.clone() for t in _flat(buffers)])
        torch.cuda.synchronize()
        for k, got in enumerate(results):
            _same(got, want[k & 1], f"repeat {k}")
    finally:
        dpr.dpr_set_programmatic_launch(old)


@pytest.mark.parametrize("rows,width", [(77, 1056), (64, 97), (20, 8208)])
def test_graph_replays_over_spoilt_buffers(rows, width):
    """Replays read the inputs and write the outputs of the time they run."""
    H.device()
    inputs = [_inputs(rows, width, 60 + k) for k in range(2)]
    given = [t.clone() for t in inputs[0]]
    buffers = _buffers(rows, width)
    want = []
    for k in range(2):
        _chain(None, inputs[k], buffers)
        torch.cuda.synchronize()
        want.append([t.clone() for t in _flat(buffers)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _chain(None, given, buffers)
    for k in range(4):
        for t, v in zip(given, inputs[k & 1]):
            t.copy_(v)
        _poison(buffers)
        graph.replay()
        torch.cuda.synchronize()
        _same(_flat(buffers), want[k & 1], f"replay {k}")


def test_kept_scratch_memory_over_spoilt_outputs():
    """Calls of several sizes with the kept scratch memory, on two streams at once and inside a
    capture, against separate workspaces; every output holds something else before each call."""
    H.device()
    sizes = [(40, 1056), (3, 8192), (700, 512), (40, 1056), (64, 4096)]
    calls, want = [], []
    for k, (rows, width) in enumerate(sizes):
        g = torch.Generator().manual_seed(70 + k)
        x, dy = (torch.randn(rows, width, generator=g).cuda() for _ in range(2))
        mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        out = [torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")]
        calls.append(((dy, x, None, mean, rstd, *out), out))
        _poison(out)
        dpr.dpr_layernorm_backward(*calls[-1][0],
                                   workspace=torch.empty(16 << 20, dtype=torch.uint8, device="cuda"))
        want.append([t.clone() for t in out])
    side = torch.cuda.Stream()
    for _ in range(3):
        for _, out in calls:
            _poison(out)
        torch.cuda.synchronize()
        for args, _ in calls[:3]:
            dpr.dpr_layernorm_backward(*args)
        with torch.cuda.stream(side):
            for args, _ in calls[3:]:
                dpr.dpr_layernorm_backward(*args)
        torch.cuda.synchronize()
        for (_, out), w in zip(calls, want):
            _same(out, w, "kept")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for args, _ in calls:
            dpr.dpr_layernorm_backward(*args)
    for _ in range(2):
        for _, out in calls:
            _poison(out)
        for args, _ in calls:
            dpr.dpr_layernorm_backward(*args)
        for _, out in calls:
            _poison(out)
        graph.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(calls, want):
            _same(out, w, "captured")
