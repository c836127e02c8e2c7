"""The host side of orthogonalize_update's launches on made-up devices (no GPU): the library's own
source, compiled with the runtime's answers in place (tests/host/orthogonalize_launches.cu)."""
import os
import subprocess

import pytest

import embedding_weight_grad_gb300 as ewg
from embedding_weight_grad_gb300 import build as cuda_build

HERE = os.path.dirname(os.path.abspath(__file__))


def compile_host(exe, *sources):
    """A program of `sources` that runs without a GPU; device code only as far as the host code
    around it needs it."""
    subprocess.run([cuda_build.nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-cudart", "none", "-std=c++17",
                    "-I" + os.path.join(cuda_build.ROOT, "include"), "-I" + cuda_build.CSRC, "-o", exe, *sources,
                    os.path.join(HERE, "host", "no_runtime.cpp"), "-ldl"], check=True, capture_output=True)
    return exe


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    exe = compile_host(str(tmp_path_factory.mktemp("host") / "launches"),
                       os.path.join(HERE, "host", "orthogonalize_launches.cu"))

    def run(cases):
        r = subprocess.run([exe], input="".join("%d %d %d %d\n" % c for c in cases), capture_output=True, text=True)
        assert r.returncode == 0, r
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


SHAPES = [(1, 64, 4096), (1, 64, 76800), (1, 64, 90000), (1, 256, 1 << 20), (1, 300, 1 << 20), (1, 1001, 4097),
          (1, 2048, 7168), (3, 100, 50000), (9, 200, 9000), (24, 1024, 1024), (38, 256, 8192), (1, 49, 49)]


def test_split_parts_run_at_the_same_time(launches):
    """The parts of a split product wait for one another, so its units may not outnumber the pairs
    that run, whatever the device holds; and no part is empty."""
    cases = [(pairs, *s) for pairs in (1, 2, 10, 37, 66, 74, 75, 76, 148) for s in SHAPES]
    for (pairs, batch, rows, cols), (code, blocks, parts, units, room) in zip(cases, launches(cases)):
        at = (pairs, batch, rows, cols)
        assert code == 0 and 2 <= blocks <= 2 * pairs and blocks % 2 == 0, at
        assert 1 <= parts <= room, at
        if parts > 1:
            assert units <= blocks // 2, at
            inner = -(-max(rows, cols) // 64)
            assert (parts - 1) * -(-inner // parts) < inner, at
        if pairs >= 76:
            assert parts == room, at             # what the workspace is laid out for


def test_a_device_without_room_is_an_error(launches):
    """Where no pair of CTAs fits, the call returns an error (and does not divide by the pairs)."""
    for shape in SHAPES:
        ((code, blocks, *_),) = launches([(0, *shape)])
        assert code != 0 and blocks == 0


def test_its_set_up_concerns_no_other_call(tmp_path):
    """Where the set-up of the steps kernel fails, the calls that do without it work all the same, and a
    call that needs it reports the error and tries anew the next time."""
    exe = compile_host(str(tmp_path / "set_up"), os.path.join(HERE, "host", "set_up.cu"),
                       os.path.join(cuda_build.CSRC, "ewg_api.cu"), os.path.join(cuda_build.CSRC, "ewg_ops_api.cu"))
    codes = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    can, accumulate, logprobs, small, large, again = map(int, codes)
    assert (can, accumulate, logprobs, small) == (1, ewg.OK, ewg.OK, ewg.OK)
    assert (large, again) == (ewg.ERR_CUDA, ewg.OK)
