"""The training example: its first gradients against autograd, and that it learns."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tied_embedding_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tied_embedding_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_gradients_match_autograd(example):
    """Within the bf16 roundings of the activations and their gradients (about six, each 2^-9)."""
    model = example.TiedModel(1000, 256)
    ids, targets = example.batch(1000, 4096, seed=5)
    loss = model.forward_backward(ids, targets)
    E = model.E.bfloat16().double().requires_grad_()
    W = model.W.bfloat16().double().requires_grad_()
    want = torch.nn.functional.cross_entropy(E[ids] @ W.T @ E.T, targets, ignore_index=-100)
    want.backward()
    assert abs(loss.item() - want.item()) < 2e-3 * want.item()
    for got, ref in ((model.E_grad, E.grad), (model.W_grad, W.grad)):
        assert (got.double() - ref).norm() < 2e-2 * ref.norm()


def test_it_learns(example):
    model, losses = example.train(steps=30)
    assert losses[-1] < 0.7 * losses[0], losses
    assert len(model.likely_next(7)) == 5
