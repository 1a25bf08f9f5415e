"""Waits inside the operators' kernels: they end by themselves, and one that runs out is counted.
Small programs compiled against the kernels' sources."""
import os
import subprocess

import pytest

from gradient_reduction_gb300 import build
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))


def _run(tmp_path, name):
    H.device()
    exe = str(tmp_path / name)
    cmd = [build._nvcc(), *build.ARCH, *build.FLAGS, os.path.join(TESTS, name + ".cu"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, f"exit code {r.returncode}: {r.stdout}{r.stderr}"
    return [line.split() for line in r.stdout.splitlines()]


def test_a_wait_ends_by_itself(tmp_path):
    """2^19 tries of at least 20 ns and at most 7800 cycles: 10 ms to 2.0 s at the GPU's highest
    clock of 2.07 GHz, 4 s at half of it."""
    lines = _run(tmp_path, "bounded_wait")
    assert [line[:3] for line in lines] == [["0", "1", "1"], ["0", "0", "0"], ["1", "1", "1"], ["1", "0", "0"]]
    for _, late, _, ms in lines:
        assert float(ms) < (1000 if late == "1" else 4500), lines
        assert late == "1" or float(ms) > 5, lines


def test_a_wait_that_runs_out_in_any_thread_is_counted(tmp_path):
    """The block of the thread counts it once; where the first thread of two CTAs' row gives up, the
    other CTA gets no more sums and counts too.  The next call is as if nothing had been."""
    lines = dict(_run(tmp_path, "staged_waits"))
    assert lines == {"none": "0", "thread": "1", "first-thread": "1", "pair-load": "1",
                     "pair-sums": "1", "first-thread-of-many": "1",
                     "first-thread-of-many-pairs": "2"}
