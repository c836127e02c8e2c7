"""The host side of layer norm's and AdamW's calls on made-up devices (no GPU): the library's own source, with
the runtime's answers in place."""
import os
import subprocess

import pytest

import embedding_weight_grad_gb300 as ewg
from embedding_weight_grad_gb300 import build as cuda_build
from test_orthogonalize_host import HERE, compile_host


def test_scalars_that_a_step_would_write(tmp_path):
    """A step's number, lr or grad_scale on the device may not lie in what the step writes; in gradients, and beside
    anything, it may."""
    exe = compile_host(str(tmp_path / "scalars"), os.path.join(HERE, "host", "adamw_scalars.cu"),
                       os.path.join(cuda_build.CSRC, "ewg_api.cu"), os.path.join(cuda_build.CSRC, "ewg_train_api.cu"))
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    assert len(lines) == 2 * 26
    for line in lines:
        bits, array, where, code = map(int, line.split())
        inside = where < 2 and array != 1 and (array != 4 or bits == 8)
        assert code == (ewg.ERR_UNSUPPORTED if inside else ewg.OK), line


@pytest.fixture(scope="module")
def norm_grad(tmp_path_factory):
    exe = compile_host(str(tmp_path_factory.mktemp("host") / "norm_grad"), os.path.join(HERE, "host", "norm_grad_launches.cu"))

    def run(cases):
        r = subprocess.run([exe], input="".join("%d %d %d %d %d\n" % c for c in cases), capture_output=True, text=True)
        assert r.returncode == 0, r
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


def test_a_gradient_fits_its_device(norm_grad):
    """A block of layer norm's gradient takes an SM's shared memory: there are no more of them than SMs, whatever the
    workspace has room for, so that none waits for another to end; and every block's share is joined."""
    cases = [(sms, n, H, bf16, lead) for sms in (8, 40, 76, 148, 152, 160) for n, H in ((1, 64), (100, 1024), (5000, 1001), (70000, 7168))
             for bf16 in (0, 1) for lead in (0, 1)]
    cases += [(sms, n, 16384, 1, 0) for sms in (8, 40, 76, 152) for n in (1, 5000)]
    results = []
    for i in range(0, len(cases), 60):                               # (devices are numbered below 64)
        results += norm_grad(cases[i:i + 60])
    assert len(results) == len(cases)
    for case, (code, blocks, parts, room) in zip(cases, results):
        sms, n, H = case[:3]
        assert code == 0 and 1 <= blocks <= sms, (case, blocks)
        cluster = 2 if H > 8192 else 1
        assert blocks // cluster <= room and parts == (blocks // cluster if blocks > cluster else 0), (case, blocks, parts, room)
        if n >= 70000:
            assert blocks == min(sms, room), (case, blocks)          # ... and none is left idle
