"""The bounded waits of orthogonalize_update's steps kernel, made to run out from the host
(tests/host/orthogonalize_gives_up.cu: the library's source with a limit of 50 ms a wait).

A count that units wait for is set far below what it can reach before the kernel starts.  The kernel
must end on its own and leave EWG_ERR_TIMEOUT, and the same workspace must serve the next call.
Nothing here faults, traps or hangs the GPU: every wait gives up after its limit."""
import os
import subprocess

import pytest

import embedding_weight_grad_gb300 as ewg
from embedding_weight_grad_gb300 import build as cuda_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("device") / "gives_up")
    subprocess.run([cuda_build.nvcc(), *cuda_build.ARCH, "-O3", "-std=c++17", "-I" + os.path.join(cuda_build.ROOT, "include"),
                    "-I" + cuda_build.CSRC, "-o", exe, os.path.join(HERE, "host", "orthogonalize_gives_up.cu")],
                   check=True, capture_output=True)
    return exe


# counts: [matrix][phase: X X^T, A A, update][block row] of units done, then the parts of a split product
CASES = [(1, 300, 300, 0), (1, 300, 300, 1), (1, 300, 300, 2), (1, 300, 300, 3), (1, 300, 300, 4), (1, 300, 300, 5),
         (1, 100, 100, 1), (1, 100, 100, 2), (5, 300, 700, 20), (1, 1000, 5000, 3), (1, 64, 90000, 3), (1, 64, 90000, 9),
         (1, 1000, 5000, 12 + 40), (24, 700, 700, 3 * 3 * 11 + 5)]


@pytest.mark.parametrize("batch,rows,cols,index", CASES)
def test_steps_wait_runs_out(program, batch, rows, cols, index):
    r = subprocess.run([program], input=f"{batch} {rows} {cols} {index}\n", capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r
    status, ms, after, differing = r.stdout.split()
    assert int(status) == ewg.ERR_TIMEOUT
    assert 45 < float(ms) < 2000, ms
    assert int(after) == ewg.OK and int(differing) == 0
