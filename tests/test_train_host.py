"""The host side of layer norm's and AdamW's calls on made-up devices (no GPU): the library's own source, with
the runtime's answers in place."""
import os
import subprocess

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
