"""Host-only checks of the layer norm and AdamW entry points (no GPU)."""
import ctypes
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


def test_public_names():
    for name in ("LayerNorm", "layer_norm", "layer_norm_backward", "layer_norm_workspace", "AdamWPlan", "adamw_plan",
                 "adamw_step"):
        assert name in ewg.__all__ and callable(getattr(ewg, name))


def test_the_structure_matches_the_header():
    src = open(os.path.join(ROOT, "include", "ewg.h")).read()
    body = re.search(r"typedef struct ewg_adamw_tensor \{(.*?)\} ewg_adamw_tensor;", src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = re.findall(r"(\w+);", body)
    assert names == [f[0] for f in ewg._AdamWTensor._fields_]
    kinds = [re.sub(r"\s*\w+;", "", line).strip() for line in body.strip().splitlines()]
    sizes = {"void*": 8, "const void*": 8, "float*": 8, "int64_t": 8, "double": 8, "int": 4}
    assert sum(sizes[k.replace(" *", "*")] for k in kinds) == ctypes.sizeof(ewg._AdamWTensor)
    assert int(re.search(r"#define EWG_ADAMW_BLOCK (\d+)", src).group(1)) == ewg.ADAMW_BLOCK
    train = open(os.path.join(cuda_build.CSRC, "ewg_train.cuh")).read()
    assert int(re.search(r"constexpr int kAdamwBlock = (\d+)", train).group(1)) == ewg.ADAMW_BLOCK


def test_workspace_and_plan_bytes(lib):
    f = lib.ewg_layer_norm_workspace_bytes
    for rows, hidden in [(-1, 8), (1, 0), (1 << 31, 8), (8, (1 << 24) + 1)]:
        assert f(rows, hidden) == 0
    for rows, hidden in [(0, 1), (1, 1), (8192, 7168), (131072, 8192), ((1 << 31) - 1, 1), (1, 1 << 24)]:
        assert f(rows, hidden) > 0 and f(rows, hidden) % 256 == 0
    g = lib.ewg_adamw_plan_bytes
    assert g(-1) == 0 and g((1 << 20) + 1) == 0
    assert 0 < g(0) < g(1) < g(400) < g(1 << 20)


def test_refusals_that_need_no_gpu():
    x, v = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA device"):
        ewg.layer_norm(x, v, v)
    with pytest.raises(ValueError, match="CUDA device"):
        ewg.layer_norm_backward(x, x, x[:, 0], x[:, 0], v)
    with pytest.raises(ValueError, match="CUDA device"):
        ewg.adamw_plan([x], [x.clone()])
    with pytest.raises(ValueError, match="state_bits"):
        ewg.adamw_plan([x], [x.clone()], state_bits=4)


def test_an_empty_plan_needs_no_gpu():
    ewg.adamw_step(ewg.adamw_plan([], []), 1, lr=1e-3)


def test_a_launch_fits_its_argument():
    """A kernel's arguments are at most 32764 bytes."""
    train = open(os.path.join(cuda_build.CSRC, "ewg_train.cuh")).read()
    entries = int(re.search(r"constexpr int kAdamwEntries = (\d+)", train).group(1))
    entry = ewg.lib().ewg_adamw_plan_bytes(1) - ewg.lib().ewg_adamw_plan_bytes(0)
    assert entries * entry + 256 <= 32764
