"""Host-only checks of the token log probability and orthogonalisation entry points (no GPU)."""
import os
import re

import pytest
import torch

import embedding_weight_grad_gb300 as ewg
from embedding_weight_grad_gb300 import build as cuda_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ewg.lib()


def test_constants_match_the_header():
    src = open(os.path.join(ROOT, "include", "ewg.h")).read()
    assert re.search(r"#define EWG_MAX_TOP (\d+)", src).group(1) == str(ewg.MAX_TOP)
    ops = open(os.path.join(ROOT, "embedding_weight_grad_gb300", "csrc", "ewg_ops.cuh")).read()
    assert re.search(r"constexpr int kMaxTop = (\d+)", ops).group(1) == str(ewg.MAX_TOP)


def test_public_names():
    for name in ("token_logprobs", "token_logprobs_backward", "TokenLogprobs", "status_workspace",
                 "orthogonalize_update", "orthogonalize_workspace"):
        assert name in ewg.__all__ and callable(getattr(ewg, name))


def test_orthogonalize_workspace_bytes(lib):
    f = lib.ewg_orthogonalize_workspace_bytes
    for batch, rows, cols in [(0, 5, 5), (1, 0, 5), (1, 5, 0), (1, 16385, 16385), (1, 5, (1 << 20) + 1),
                              (65536, 1, 1), (-1, 5, 5), (60000, 16384, 1 << 20)]:
        assert f(batch, rows, cols) == 0
    assert f(1, 16384, 16384) > 0 and f(1, 3, 1 << 20) > 0 and f(65535, 1, 1) > 0
    # X^T twice and its rest, two A and B, of 2 bytes each; either orientation needs the same
    for batch, r, c in [(1, 256, 256), (24, 1024, 1024), (1, 1001, 4097), (1, 2048, 7168), (1, 64, 100000)]:
        need = f(batch, r, c)
        assert need == f(batch, c, r) and need % 256 == 0
        assert need >= batch * 6 * r * (r + c)
        assert f(batch, r, c + 16) > need


def test_refusals_that_need_no_gpu():
    z, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA device"):
        ewg.token_logprobs(z, t)
    with pytest.raises(ValueError, match="CUDA device"):
        ewg.token_logprobs_backward(z, t, z[:, 0], z[:, 0], z[:, 0])
    with pytest.raises(ValueError, match="CUDA device"):
        ewg.orthogonalize_update(z)


def test_every_device_helper_has_a_caller():
    """Instruction wrappers that no kernel uses are left over."""
    csrc = cuda_build.CSRC
    helpers = re.findall(r"__forceinline__ \w+ (\w+)\(", open(os.path.join(csrc, "ewg_ptx.cuh")).read())
    assert len(helpers) > 40
    text = "\n".join(open(os.path.join(csrc, f)).read() for f in sorted(os.listdir(csrc)))
    unused = [h for h in helpers if len(re.findall(r"\b%s(?:<[^>]*>)?\(" % h, text)) < 2]
    assert not unused, unused
