"""The training example with layer norms and AdamW: its gradients against autograd in 64 bits, that its
steps run, and a whole step captured."""
import importlib.util
import os

import pytest
import torch

import embedding_weight_grad_gb300 as ewg

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prenorm_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("prenorm_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_gradients_match_autograd(example):
    """Each gradient is a sum of products of activations and gradients that went through at most eight
    roundings to bf16 (2^-8 each), independent ones: within 8^0.5 2^-8 < 1.2e-2 of the exact
    one in the 2-norm, and the loss within as much of itself."""
    model = example.PrenormModel(1000, 256)
    for v in model.norms:
        v.add_(0.3 * torch.randn(v.shape, device=v.device))
    ids, targets = example.batch(1000, 4096, seed=5)
    loss = model.forward_backward(ids, targets)
    E, W = model.E16.double().requires_grad_(), model.W.bfloat16().double().requires_grad_()
    w1, b1, w2, b2 = norms = [v.double().requires_grad_() for v in model.norms]

    def norm(x, w, b):
        d = x - x.mean(-1, keepdim=True)
        return d * (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w + b
    x = E[ids]
    h = x + norm(x, w1, b1) @ W.T
    want = torch.nn.functional.cross_entropy(norm(h, w2, b2) @ E.T, targets, ignore_index=-100)
    want.backward()
    assert abs(loss.item() - want.item()) < 1.2e-2 * want.item()
    for got, ref in zip((model.E_grad, model.W_grad, *model.norm_grads), (E, W, *norms)):
        assert (got.double() - ref.grad).norm() < 1.2e-2 * ref.grad.norm()


def test_it_runs(example):
    model, losses = example.train(steps=12)
    assert all(x == x and x < 20 for x in losses)
    assert model.table.exp_avg[0].dtype == torch.float8_e4m3fn and bool(model.E.isfinite().all())
    assert torch.equal(model.E16, model.E.bfloat16())


def test_a_captured_step_follows_the_schedule(example):
    """Forward, backward and AdamW captured once, with the step and the learning rate on the
    device: replayed, they leave the bits that the same calls one by one leave."""
    def run(model, ids, targets, step, lr):
        loss = model.forward_backward(ids, targets)
        for plan in (model.table, model.vectors):
            ewg.adamw_step(plan, step, lr=lr)
        for g in (model.E_grad, *model.norm_grads):
            g.zero_()
        return loss
    one, other = example.PrenormModel(1000, 256), example.PrenormModel(1000, 256)
    step, lr = torch.zeros((), dtype=torch.int64, device="cuda"), torch.zeros((), device="cuda")
    ids, targets = example.batch(1000, 4096, seed=0)
    lr.fill_(1e-3)
    losses = [run(one, ids, targets, 1, lr).item()]
    step.fill_(1)
    run(other, ids, targets, step, lr)                       # the first calls belong outside a capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        loss = run(other, ids, targets, step, lr)
    for t in (2, 3, 4):
        lr.fill_(1e-3 / t)
        graph.replay()
        losses.append(run(one, ids, targets, t, lr).item())
        assert loss.item() == losses[-1]
    for a, b in zip((one.E, one.E16, *one.norms, *one.table.exp_avg, *one.table.exp_avg_sq, *one.table.scales),
                    (other.E, other.E16, *other.norms, *other.table.exp_avg, *other.table.exp_avg_sq, *other.table.scales)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
