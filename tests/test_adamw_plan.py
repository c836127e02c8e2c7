"""What adamw_step asks of its plan's tensors before it launches anything, on tensors of the CPU (no GPU)."""
import pytest
import torch

import embedding_weight_grad_gb300 as ewg

GROUPS = ["params", "grads", "copies", "exp_avg", "exp_avg_sq", "scales"]


@pytest.fixture
def plan(monkeypatch):
    """A plan of two tensors; its steps are recorded in place of being enqueued."""
    n, blocks = 300, 2
    tensors = {k: [torch.zeros(n, dtype=d) for _ in range(2)]
               for k, d in zip(GROUPS, (torch.float32, torch.bfloat16, torch.bfloat16, torch.float8_e4m3fn, torch.float8_e4m3fn))}
    tensors["scales"] = [torch.zeros(blocks, 2) for _ in range(2)]
    plan = ewg.AdamWPlan(*[tensors[k] for k in ("params", "grads", "copies", "exp_avg", "exp_avg_sq", "scales")], 8, -1)
    plan.steps = []
    monkeypatch.setattr(ewg, "_enqueue", lambda *a: plan.steps.append(a))
    return plan


@pytest.mark.parametrize("group", GROUPS)
def test_memory_that_was_given_back(group, plan):
    """A storage that was resized to nothing, as sharded training and offloaders do, and resized again."""
    t = getattr(plan, group)[1]
    address, storage = t.data_ptr(), t.untyped_storage()
    nbytes = storage.nbytes()
    ewg.adamw_step(plan, 1, lr=1e-3)
    storage.resize_(0)
    with pytest.raises(ValueError, match="moved"):
        ewg.adamw_step(plan, 2, lr=1e-3)
    storage.resize_(nbytes)
    if t.data_ptr() != address:
        with pytest.raises(ValueError, match="moved"):
            ewg.adamw_step(plan, 2, lr=1e-3)
    assert len(plan.steps) == 1


@pytest.mark.parametrize("group", GROUPS)
def test_tensors_that_were_replaced(group, plan):
    t = getattr(plan, group)[0]
    kept = t.data
    t.data = torch.zeros_like(kept)
    with pytest.raises(ValueError, match="moved"):
        ewg.adamw_step(plan, 1, lr=1e-3)
    t.data = kept
    ewg.adamw_step(plan, 1, lr=1e-3)
    assert len(plan.steps) == 1


@pytest.mark.parametrize("group", GROUPS)
def test_a_replaced_tensor_at_the_old_address(group, plan, monkeypatch):
    """Where the old memory is gone and another tensor has come to lie there, which may be smaller."""
    before = dict(zip(map(id, plan._all), map(torch.Tensor.data_ptr, plan._all)))
    t = getattr(plan, group)[0]
    storage = t.untyped_storage()
    t.data = torch.zeros(10, dtype=t.dtype)
    storage.resize_(0)
    monkeypatch.setattr(ewg, "_data_ptr", lambda x: before[id(x)])
    with pytest.raises(ValueError, match="moved"):
        ewg.adamw_step(plan, 1, lr=1e-3)
    assert not plan.steps


def test_tensors_of_one_bucket(monkeypatch):
    """Views of one storage: it is looked at once, and any of them shows that it is gone."""
    bucket = torch.zeros(1200)
    plan = ewg.AdamWPlan([bucket[:300]], [bucket[300:600]], [None], [bucket[600:900]], [bucket[900:]], None, 32, -1)
    steps = []
    monkeypatch.setattr(ewg, "_enqueue", lambda *a: steps.append(a))
    assert len(plan._storages) == 1
    ewg.adamw_step(plan, 1, lr=1e-3)
    bucket.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="moved"):
        ewg.adamw_step(plan, 2, lr=1e-3)
    assert len(steps) == 1


def test_autograd_is_told_of_all_that_is_written(plan):
    """Of params, copies and states; gradients are only read."""
    versions = {k: [t._version for t in getattr(plan, k)] for k in GROUPS}
    ewg.adamw_step(plan, 1, lr=1e-3)
    for k in GROUPS:
        assert [t._version for t in getattr(plan, k)] == [v + (k != "grads") for v in versions[k]], k


def test_a_graph_that_saved_an_average(monkeypatch):
    """Its backward pass raises instead of using what the step left there."""
    p, g, m, v = (torch.ones(8) for _ in range(4))
    monkeypatch.setattr(ewg, "_enqueue", lambda *a: None)
    plan = ewg.AdamWPlan([p], [g], [None], [m], [v], None, 32, -1)
    w = torch.ones(8, requires_grad=True)
    loss = (w * m).sum()
    ewg.adamw_step(plan, 1, lr=1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
